"""Decode step over a paged KV cache: the library's public, per-step API.

``DecodeStep`` keeps a workload's req_to_token table, pools and step buffers
resident on one GPU and runs one decode layer step as a sequence of libpkv
calls on the current stream:

    pkv_build_indices   req_to_token -> kv_indptr / kv_indices (or the -1 padded table)
    pkv_store           this step's new K/V rows -> their pool slots
    pkv_decode          attention of every request's new token over its pages

With ``alloc=True`` the new token's slot is not taken from the workload but
allocated on the device first, as a serving loop would:

    pkv_alloc_extend        each request grows by one position: the slot after
                            its last one, or a fresh page from the free list
    pkv_write_req_to_token  that slot into the request's row of req_to_token

(the free list is restored before every step, so steps stay idempotent).

With ``fused=True`` (GQA) the decode call reads its pages straight from
req_to_token (PKV_LAYOUT_REQ_TO_TOKEN: no pkv_build_indices launch, no page list
in between) and, for the problem that stores, writes the new token's K/V into
the pool itself before attending (the fused store): a step is then one decode
launch (+ its merge) per problem.

For an encoder-decoder workload the cross-attention over the encoder region
runs either through its own page list ("paged": the page-aligned encoder of
"Approach 1") or through pkv_ragged_gather into a contiguous varlen buffer
followed by a varlen decode ("gather": "Approach 2").

With ``quant=True`` (GQA) the K/V pool is held in 4 bits (see pkv_quant_store): the
given bf16 pools are quantised once and not kept (k_pool and v_pool are None then), and the
step's calls are their 4-bit forms (pkv_quant_store, pkv_quant_decode or pkv_quant_extend,
and pkv_quant_gather before a contiguous cross-attention).  ``scales`` are the heads' fp32
(k_scale, v_scale), by default each head's largest finite magnitude in the pools / 2688.
With ``quant=8`` it is held in 8 bits, with a scale per tile and head (see pkv_byte_store), which
takes no ``scales``.

``BudgetedDecode`` is a serving loop of its own: prefills and decode steps over an 8-bit pool,
which count what each key receives, and evictions that keep every request within a budget.

No attention, quantisation, allocation or eviction is computed here: that runs in libpkv's kernels.
``BudgetedDecode`` keeps its requests' lengths with a few torch operators per call.
"""
from __future__ import annotations

from typing import Dict, Optional

import numpy as np
import torch

from . import _binding as B
from .workloads import Workload, fill_pool, make_values

__all__ = ["DecodeStep", "ExtendStep", "BudgetedDecode"]


class _ProblemBuffers:
    pass


def _pack(owners, device):
    """Moves tensors into consecutive 256-byte aligned slices of one new device buffer.

    ``owners`` lists (object, attribute) pairs; each attribute is replaced by a view of
    the buffer holding the same values, so one copy of the buffer fills them all (the
    per-step inputs come from the host in a single transfer, the outputs go back in one).
    Returns the buffer.
    """
    sizes = [getattr(o, a).numel() * getattr(o, a).element_size() for o, a in owners]
    offs, total = [], 0
    for nb in sizes:
        offs.append(total)
        total += (nb + 255) // 256 * 256
    buf = torch.empty(max(total, 256), dtype=torch.uint8, device=device)
    for (o, a), off, nb in zip(owners, offs, sizes):
        t = getattr(o, a)
        v = buf[off:off + nb].view(t.dtype).view(t.shape)
        v.copy_(t)
        setattr(o, a, v)
    return buf


class _QuantPool:
    """A 4-bit pool with its head scales, filled from bf16 pools [slots, Hkv, D]."""

    def __init__(self, k_pool, v_pool, page_size, err, scales=None):
        slots, hkv, d = k_pool.shape
        tile = min(page_size, 64)
        if slots % tile:
            raise ValueError("the pool's slots must be whole pages")
        dev = k_pool.device
        step = 1 << 20
        if scales is None:
            # the largest code (6) x the largest block scale (448) is the head's largest magnitude
            # (of its finite values: a block that holds another is NaN whatever the scale)
            tops = [torch.stack([p[i:i + step].abs().nan_to_num_(0.0, 0.0, 0.0).amax(dim=(0, 2)) for i in range(0, slots, step)])
                    for p in (k_pool, v_pool)]
            scales = [(t.amax(0).float() / 2688.0).clamp_(min=1e-30) for t in tops]
        self.page_size = page_size
        self.k_scale, self.v_scale = (x.to(dev) for x in scales)
        self.pool = torch.zeros((slots // tile, hkv, B.pkv_quant_tile_bytes(page_size, d)), dtype=torch.uint8, device=dev)
        for i in range(0, slots, step):
            n = min(step, slots - i)
            self.store(k_pool[i:i + n], v_pool[i:i + n], torch.arange(i, i + n, dtype=torch.int32, device=dev), err)

    def store(self, k_new, v_new, slot_mapping, err):
        B.pkv_quant_store(self.pool, k_new, v_new, slot_mapping, err, page_size=self.page_size, k_scale=self.k_scale,
                          v_scale=self.v_scale)

    def args(self, layout, q, out, **kw):
        return B.make_quant_args(layout, q, self.pool, out, page_size=self.page_size, k_scale=self.k_scale,
                                 v_scale=self.v_scale, **kw)

    def gather(self, r2t, req_pool_idx, seq_lens, max_len, k_out, v_out, cu, err, kv_start):
        B.pkv_quant_gather(self.pool, r2t, req_pool_idx, seq_lens, max_len, k_out, v_out, cu, err, page_size=self.page_size,
                           k_scale=self.k_scale, v_scale=self.v_scale, kv_start=kv_start)

    decode_size, extend_size = staticmethod(B.pkv_quant_decode_workspace_size), staticmethod(B.pkv_quant_extend_workspace_size)
    decode, extend = staticmethod(B.pkv_quant_decode), staticmethod(B.pkv_quant_extend)

    @staticmethod
    def store_launches(n):
        return 1


class _BytePool:
    """An 8-bit pool of `slots` slots, empty or filled from bf16 pools [slots, Hkv, D]."""

    def __init__(self, slots, hkv, d, page_size, device):
        tile = min(page_size, 64)
        if slots % tile:
            raise ValueError("the pool's slots must be whole pages")
        self.page_size, self.kv_heads = page_size, hkv
        self.pool = torch.zeros((slots // tile, B.pkv_byte_tile_bytes(page_size, d, hkv)), dtype=torch.uint8, device=device)
        self.workspace = torch.empty(B.pkv_byte_store_workspace_size(slots // tile, page_size), dtype=torch.uint8, device=device)

    @classmethod
    def of(cls, k_pool, v_pool, page_size, err, scales=None):
        if scales is not None:
            raise ValueError("an 8-bit pool has its own scales")
        slots, hkv, d = k_pool.shape
        self = cls(slots, hkv, d, page_size, k_pool.device)
        step = 1 << 20                                # (whole pages)
        for i in range(0, slots, step):
            n = min(step, slots - i)
            self.store(k_pool[i:i + n], v_pool[i:i + n], torch.arange(i, i + n, dtype=torch.int32, device=k_pool.device), err)
        return self

    def store(self, k_new, v_new, slot_mapping, err):
        B.pkv_byte_store(self.pool, k_new, v_new, slot_mapping, self.workspace, err, page_size=self.page_size)

    def args(self, layout, q, out, **kw):
        return B.make_byte_args(layout, q, self.pool, out, page_size=self.page_size, num_kv_heads=self.kv_heads, **kw)

    def gather(self, r2t, req_pool_idx, seq_lens, max_len, k_out, v_out, cu, err, kv_start):
        B.pkv_byte_gather(self.pool, r2t, req_pool_idx, seq_lens, max_len, k_out, v_out, cu, err, page_size=self.page_size,
                          kv_start=kv_start)

    decode_size, extend_size = staticmethod(B.pkv_byte_decode_workspace_size), staticmethod(B.pkv_byte_extend_workspace_size)
    decode, extend = staticmethod(B.pkv_byte_decode), staticmethod(B.pkv_byte_extend)

    @staticmethod
    def store_launches(n):
        return 1 if n <= 256 else 2


def _quantised(quant, k_pool, v_pool, page_size, err, scales):
    """The pool that ``quant`` names, filled from the bf16 ones: None, 4 bits (True or 4) or 8."""
    if quant not in (False, True, 4, 8):
        raise ValueError("quant must be False, True, 4 or 8")
    if not quant:
        return None
    return (_BytePool.of if quant == 8 else _QuantPool)(k_pool, v_pool, page_size, err, scales)


class DecodeStep:
    def __init__(self, wl: Workload, device="cuda", cross_mode: str = "paged", kv_chunk: int = 0,
                 pools=None, values: Optional[Dict[str, torch.Tensor]] = None, seed: Optional[int] = None,
                 alloc: bool = False, fused: bool = False, quant=False, scales=None):
        if cross_mode not in ("paged", "gather"):
            raise ValueError(cross_mode)
        if fused and wl.kind != "gqa":
            raise ValueError("the token-table layout and the fused store are GQA only")
        if quant and wl.kind != "gqa":
            raise ValueError("a quantised pool is GQA only")
        self.fused = bool(fused)
        self.wl = wl
        self.device = torch.device(device)
        self.cross_mode = cross_mode
        self.kv_chunk = int(kv_chunk)
        dev = self.device
        ps = wl.page_size
        self.r2t = wl.req_to_token.to(dev)
        self.req_pool_idx = wl.req_pool_idx.to(dev)
        if pools is None:
            pools = fill_pool(wl, device=dev, seed=seed)
        self.k_pool, self.v_pool = pools
        vals = make_values(wl, seed=seed) if values is None else values
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        self.quant = _quantised(quant, self.k_pool, self.v_pool, ps, self.err, scales)
        if quant:
            del pools
            self.k_pool = self.v_pool = None   # nothing reads the bf16 rows again
        Bn = wl.batch
        self.k_new = vals["k_new"].to(dev)
        self.v_new = vals["v_new"].to(dev) if vals["v_new"] is not None else None
        self.problems: Dict[str, _ProblemBuffers] = {}
        for p in wl.problems:
            pb = _ProblemBuffers()
            pb.spec = p
            pb.seq_lens = p.seq_lens.to(dev)
            pb.kv_start = p.kv_start.to(dev)
            pb.slot_mapping = p.slot_mapping.to(dev) if p.stores else None
            pb.max_len = int(p.seq_lens.max()) if Bn else 0
            pb.q = vals["q_" + p.name].to(dev)
            pb.out = torch.empty((Bn, wl.num_q_heads, wl.head_dim_v), dtype=torch.bfloat16, device=dev)
            pb.lse = torch.empty((Bn, wl.num_q_heads), dtype=torch.float32, device=dev)
            pb.gather = (p.name == "cross" and cross_mode == "gather")
            self.problems[p.name] = pb
        self.alloc = bool(alloc)
        if self.alloc:
            self._setup_alloc(seed)
        # the step's host inputs and its outputs each live in one buffer (one copy per direction)
        ins = [(self, "k_new"), (self, "req_pool_idx")] + ([(self, "v_new")] if self.v_new is not None else [])
        for name, pb in self.problems.items():
            ins += [(pb, "q"), (pb, "seq_lens")]
            if pb.slot_mapping is not None and not (self.alloc and name == self.alloc_problem):
                ins.append((pb, "slot_mapping"))
        if self.alloc:
            ins += [(self, "prefix_lens"), (self, "last_loc")]
        self.in_buf = _pack(ins, dev)
        self.out_buf = _pack([(pb, "out") for pb in self.problems.values()], dev)
        for pb in self.problems.values():
            p = pb.spec
            max_pages = -(-pb.max_len // ps) if pb.max_len else 0
            if pb.gather:
                rows = int(p.seq_lens.sum())
                pb.k_rag = torch.empty((max(rows, 1),) + tuple(self.k_new.shape[1:]), dtype=torch.bfloat16, device=dev)
                pb.v_rag = torch.empty_like(pb.k_rag)
                pb.cu = torch.empty(Bn + 1, dtype=torch.int32, device=dev)
                layout = B.PKV_LAYOUT_VARLEN
                pb.args = B.make_decode_args(B.PKV_KIND_GQA, layout, pb.q, pb.k_rag, pb.v_rag, pb.out,
                                             sm_scale=wl.sm_scale, max_seq_len=pb.max_len,
                                             cu_seqlens=pb.cu, lse=pb.lse, kv_chunk=self.kv_chunk)
            elif self.quant is not None:
                kw = dict(sm_scale=wl.sm_scale, max_seq_len=pb.max_len, lse=pb.lse, kv_chunk=self.kv_chunk,
                          total_kv=int(p.seq_lens.sum()))
                if self.fused:
                    pb.args = self.quant.args(B.PKV_LAYOUT_REQ_TO_TOKEN, pb.q, pb.out, seq_lens=pb.seq_lens,
                                              req_to_token=self.r2t, req_pool_idx=self.req_pool_idx,
                                              kv_start=pb.kv_start, **kw)
                else:
                    self._page_lists(pb, max_pages)
                    pb.args = self.quant.args(B.PKV_LAYOUT_CSR, pb.q, pb.out, kv_indptr=pb.kv_indptr,
                                              kv_indices=pb.kv_indices, kv_last_page_len=pb.kv_last, **kw)
            elif self.fused:
                # pages straight from req_to_token; the problem that stores writes its new rows itself
                kn, vn = (self.k_new, self.v_new) if p.stores else (None, None)
                pb.args = B.make_decode_args(B.PKV_KIND_GQA, B.PKV_LAYOUT_REQ_TO_TOKEN, pb.q, self.k_pool,
                                             self.v_pool, pb.out, page_size=ps, sm_scale=wl.sm_scale,
                                             max_seq_len=pb.max_len, seq_lens=pb.seq_lens, lse=pb.lse,
                                             kv_chunk=self.kv_chunk, req_to_token=self.r2t,
                                             req_pool_idx=self.req_pool_idx, kv_start=pb.kv_start,
                                             k_new=kn, v_new=vn)
            elif wl.kind == "mla":
                pb.block_table = torch.empty((Bn, max(max_pages, 1)), dtype=torch.int32, device=dev)
                pb.args = B.make_decode_args(B.PKV_KIND_MLA, B.PKV_LAYOUT_BLOCK_TABLE, pb.q, self.k_pool, None,
                                             pb.out, page_size=ps, sm_scale=wl.sm_scale, max_seq_len=pb.max_len,
                                             head_dim_v=wl.head_dim_v, block_table=pb.block_table,
                                             seq_lens=pb.seq_lens, lse=pb.lse, kv_chunk=self.kv_chunk)
            else:
                self._page_lists(pb, max_pages)
                pb.args = B.make_decode_args(B.PKV_KIND_GQA, B.PKV_LAYOUT_CSR, pb.q, self.k_pool, self.v_pool,
                                             pb.out, page_size=ps, sm_scale=wl.sm_scale, max_seq_len=pb.max_len,
                                             kv_indptr=pb.kv_indptr, kv_indices=pb.kv_indices,
                                             kv_last_page_len=pb.kv_last, lse=pb.lse, kv_chunk=self.kv_chunk)
            pb.quant = isinstance(pb.args, (B.QuantArgs, B.ByteArgs))
            nbytes = (self.quant.decode_size if pb.quant else B.pkv_decode_workspace_size)(pb.args)
            pb.ws_bytes = nbytes
            pb.workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)

    def _page_lists(self, pb, max_pages):
        """Buffers of a problem's CSR page lists."""
        dev, Bn = self.device, self.wl.batch
        pb.kv_indptr = torch.empty(Bn + 1, dtype=torch.int32, device=dev)
        pb.kv_indices = torch.empty(max(Bn * max_pages, 1), dtype=torch.int32, device=dev)
        pb.kv_last = torch.empty(Bn, dtype=torch.int32, device=dev)

    def _setup_alloc(self, seed):
        """Free list = the pool pages no cached position uses (page 0 is padding), in a
        seeded order; each request grows from its cached length by one position."""
        wl = self.wl
        ps = wl.page_size
        r2t = wl.req_to_token.numpy()
        rpi = wl.req_pool_idx.numpy().astype(np.int64)
        names = [n for n, pb in self.problems.items() if pb.spec.stores]
        if len(names) != 1:
            raise ValueError("device allocation needs exactly one problem that stores new tokens")
        self.alloc_problem = names[0]
        used = [np.zeros(1, dtype=np.int64)]
        for pb in self.problems.values():
            lens = pb.spec.seq_lens.numpy().astype(np.int64)
            starts = pb.spec.kv_start.numpy().astype(np.int64)
            cached = lens - 1 if pb.spec.stores else lens
            for b in range(wl.batch):
                used.append(r2t[rpi[b], starts[b]:starts[b] + cached[b]].astype(np.int64) // ps)
        used_pages = np.unique(np.concatenate(used))
        free = np.setdiff1d(np.arange(wl.num_pool_pages, dtype=np.int64), used_pages)
        free = np.random.default_rng(0 if seed is None else seed).permutation(free).astype(np.int32)
        spec = self.problems[self.alloc_problem].spec
        lens = spec.seq_lens.numpy().astype(np.int64)
        starts = spec.kv_start.numpy().astype(np.int64)
        prefix = lens - 1
        last = np.array([r2t[rpi[b], starts[b] + prefix[b] - 1] if prefix[b] > 0 else -1
                         for b in range(wl.batch)], dtype=np.int32)
        dev = self.device
        self.free_pages = torch.from_numpy(free).to(dev)
        self.free_state0 = torch.tensor([0, len(free)], dtype=torch.int32, device=dev)
        self.free_state = self.free_state0.clone()
        self.prefix_lens = torch.from_numpy(prefix.astype(np.int32)).to(dev)
        self.last_loc = torch.from_numpy(last).to(dev)
        self.out_cache_loc = torch.empty(wl.batch, dtype=torch.int32, device=dev)
        self.problems[self.alloc_problem].slot_mapping = self.out_cache_loc

    def allocate(self):
        """This step's slots on the device: one position per request, then into the rows."""
        wl = self.wl
        pb = self.problems[self.alloc_problem]
        self.free_state.copy_(self.free_state0, non_blocking=True)
        B.pkv_alloc_extend(self.prefix_lens, pb.seq_lens, self.last_loc, wl.page_size, wl.num_pool_pages,
                           self.free_pages, self.free_state, self.out_cache_loc, self.err)
        B.pkv_write_req_to_token(self.r2t, self.req_pool_idx, self.prefix_lens, pb.seq_lens, self.out_cache_loc,
                                 self.err, kv_start=pb.kv_start)

    # ------------------------------------------------------------------ steps
    def build_indices(self, name: str):
        pb = self.problems[name]
        wl = self.wl
        if pb.gather or self.fused:
            return
        if wl.kind == "mla":
            B.pkv_build_indices(self.r2t, self.req_pool_idx, pb.seq_lens, wl.page_size, wl.num_pool_pages,
                                self.err, kv_start=pb.kv_start, block_table=pb.block_table)
        else:
            B.pkv_build_indices(self.r2t, self.req_pool_idx, pb.seq_lens, wl.page_size, wl.num_pool_pages,
                                self.err, kv_start=pb.kv_start, kv_indptr=pb.kv_indptr, kv_indices=pb.kv_indices,
                                kv_last_page_len=pb.kv_last)

    def store(self, name: str = "self"):
        pb = self.problems[name]
        if self.quant is not None:
            self.quant.store(self.k_new, self.v_new, pb.slot_mapping, self.err)
            return
        if self.fused and not pb.gather:
            return                                   # the decode call stores the new rows itself
        B.pkv_store(self.k_pool, self.v_pool, self.k_new, self.v_new, pb.slot_mapping, self.err)

    def gather(self, name: str):
        pb = self.problems[name]
        if self.quant is not None:
            self.quant.gather(self.r2t, self.req_pool_idx, pb.seq_lens, pb.max_len, pb.k_rag, pb.v_rag, pb.cu, self.err,
                              pb.kv_start)
            return
        B.pkv_ragged_gather(self.k_pool, self.v_pool, self.r2t, self.req_pool_idx, pb.seq_lens, pb.max_len,
                            pb.k_rag, pb.v_rag, pb.cu, self.err, kv_start=pb.kv_start)

    def decode(self, name: str):
        pb = self.problems[name]
        (self.quant.decode if pb.quant else B.pkv_decode)(pb.args, pb.workspace, self.err)

    def run(self):
        """One decode step: (allocation), then for each problem page lists, (store), (gather), attention."""
        if self.alloc:
            self.allocate()
        for name, pb in self.problems.items():
            if pb.gather:
                self.gather(name)
            else:
                self.build_indices(name)
            if pb.spec.stores:
                self.store(name)
            self.decode(name)

    def launches_per_step(self) -> int:
        """libpkv kernel launches one ``run()`` issues."""
        n = 2 if self.alloc else 0                  # alloc_extend + write_req_to_token
        for pb in self.problems.values():
            if not self.fused or pb.gather:
                n += 1                               # gather or build_indices
            if not self.fused or pb.gather or self.quant is not None:
                n += (1 if self.quant is None else self.quant.store_launches(self.wl.batch)) if pb.spec.stores else 0
            # attention (+ merge when requests can split; a call over a quantised pool without one takes the least workspace)
            n += 1 + (1 if pb.ws_bytes > (256 if pb.quant else 0) else 0)
            n += 1 if pb.quant and self.wl.batch > 1024 else 0   # (the tile table of a large batch)
        return n

    def check_errors(self) -> int:
        """Synchronises and returns the device error bits raised so far."""
        return int(self.err.item())

    # ------------------------------------------------------------------ host I/O
    def host_step_tensors(self):
        """Pinned host copies of the step's packed inputs and outputs (for end-to-end timing)."""
        return {"inputs": self.in_buf.cpu().pin_memory()}, {"outputs": torch.empty_like(self.out_buf, device="cpu").pin_memory()}

    def run_from_host(self, h_in, h_out):
        """One host-to-device copy of the step's inputs (new K/V rows, q, lengths, slots, row
        indices: packed in one buffer), the step, one device-to-host copy of the outputs."""
        self.in_buf.copy_(h_in["inputs"], non_blocking=True)
        self.run()
        h_out["outputs"].copy_(self.out_buf, non_blocking=True)

    @staticmethod
    def bytes_of(tensors) -> int:
        return int(sum(t.numel() * t.element_size() for t in tensors.values()))


class ExtendStep:
    """One multi-query step over a paged KV cache (extend / target-verify / span rows):

        pkv_build_indices   req_to_token -> kv_indptr / kv_indices
        pkv_store           this step's new tokens' K/V -> their pool slots
        pkv_span_plan       (rows with segments) segment lists -> query rows and key bounds
        pkv_extend          attention of every query row over its visible keys

    With ``token_table=True`` pkv_extend reads the pages straight from req_to_token
    (PKV_LAYOUT_REQ_TO_TOKEN) and the step has no pkv_build_indices launch.  With
    ``quant=True`` the pool is held in 4 bits (pkv_quant_store, pkv_quant_extend), with
    ``quant=8`` in 8 (pkv_byte_store, pkv_byte_extend).
    """

    def __init__(self, ew, device="cuda", kv_chunk: int = 0, seed: Optional[int] = None, token_table: bool = False,
                 quant=False, scales=None):
        self.token_table = bool(token_table)
        self.ew = ew
        dev = self.device = torch.device(device)
        seed = ew.seed if seed is None else seed
        B_ = ew.batch
        self.r2t = ew.req_to_token.to(dev)
        self.req_pool_idx = ew.req_pool_idx.to(dev)
        self.seq_lens = ew.seq_lens.to(dev)
        self.slot_mapping = ew.slot_mapping.to(dev)
        gen = torch.Generator(device=dev)
        gen.manual_seed(4_000_037 + seed)
        shape = (ew.num_slots, ew.num_kv_heads, ew.head_dim)
        self.k_pool = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        self.v_pool = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        for t in (self.k_pool, self.v_pool):
            flat = t.view(-1)
            for i in range(0, flat.numel(), 1 << 28):
                flat[i:i + (1 << 28)].normal_(generator=gen)
        cgen = torch.Generator().manual_seed(5_000_011 + seed)
        total_q = int(ew.qo_lens.sum())
        n_new = int(ew.new_lens.sum())
        self.q = torch.randn((total_q, ew.num_q_heads, ew.head_dim), generator=cgen).to(torch.bfloat16).to(dev)
        self.k_new = torch.randn((n_new, ew.num_kv_heads, ew.head_dim), generator=cgen).to(torch.bfloat16).to(dev)
        self.v_new = torch.randn((n_new, ew.num_kv_heads, ew.head_dim), generator=cgen).to(torch.bfloat16).to(dev)
        qo = np.concatenate([[0], np.cumsum(ew.qo_lens.numpy())]).astype(np.int32)
        self.qo_indptr = torch.from_numpy(qo).to(dev)
        self.kv_end = None
        if ew.segments is not None:
            ind, kinds, starts, ends = [0], [], [], []
            for segs in ew.segments:
                for kd, a, e in segs:
                    kinds.append(kd)
                    starts.append(a)
                    ends.append(e)
                ind.append(len(kinds))
            self.seg = [torch.tensor(x, dtype=torch.int32, device=dev) for x in (ind, kinds, starts, ends)]
            self.plan_qo = torch.empty(B_ + 1, dtype=torch.int32, device=dev)
            self.q_pos = torch.empty(total_q, dtype=torch.int32, device=dev)
            self.kv_end = torch.empty(total_q, dtype=torch.int32, device=dev)
        ps = ew.page_size
        pages = int((-(-ew.seq_lens.numpy().astype(np.int64) // ps)).sum())
        self.kv_indptr = torch.empty(B_ + 1, dtype=torch.int32, device=dev)
        self.kv_indices = torch.empty(max(pages, 1), dtype=torch.int32, device=dev)
        self.kv_last = torch.empty(B_, dtype=torch.int32, device=dev)
        self.out = torch.empty((total_q, ew.num_q_heads, ew.head_dim), dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty((total_q, ew.num_q_heads), dtype=torch.float32, device=dev)
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        # the step's host inputs in one buffer (one copy per step)
        ins = [(self, "q"), (self, "k_new"), (self, "v_new"), (self, "seq_lens"), (self, "slot_mapping"),
               (self, "qo_indptr"), (self, "req_pool_idx")]
        if self.kv_end is not None:
            self._seg_holder = _ProblemBuffers()
            for i, t in enumerate(self.seg):
                setattr(self._seg_holder, "s%d" % i, t)
            ins += [(self._seg_holder, "s%d" % i) for i in range(len(self.seg))]
        self.in_buf = _pack(ins, dev)
        if self.kv_end is not None:
            self.seg = [getattr(self._seg_holder, "s%d" % i) for i in range(len(self.seg))]
        self.quant = _quantised(quant, self.k_pool, self.v_pool, ps, self.err, scales)
        if self.quant is not None:
            self.k_pool = self.v_pool = None   # nothing reads the bf16 rows again
            kw = dict(sm_scale=ew.sm_scale, max_seq_len=int(ew.seq_lens.max()), kv_end=self.kv_end, lse=self.lse,
                      qo_indptr=self.qo_indptr, kv_chunk=kv_chunk, total_kv=int(ew.seq_lens.sum()),
                      max_q_len=int(ew.qo_lens.max()))
            if self.token_table:
                self.args = self.quant.args(B.PKV_LAYOUT_REQ_TO_TOKEN, self.q, self.out, seq_lens=self.seq_lens,
                                            req_to_token=self.r2t, req_pool_idx=self.req_pool_idx, **kw)
            else:
                self.args = self.quant.args(B.PKV_LAYOUT_CSR, self.q, self.out, kv_indptr=self.kv_indptr,
                                            kv_indices=self.kv_indices, kv_last_page_len=self.kv_last, **kw)
        elif self.token_table:
            self.args = B.make_extend_args(B.PKV_LAYOUT_REQ_TO_TOKEN, self.q, self.k_pool, self.v_pool, self.out,
                                           self.qo_indptr, page_size=ps, sm_scale=ew.sm_scale,
                                           max_seq_len=int(ew.seq_lens.max()), kv_end=self.kv_end,
                                           seq_lens=self.seq_lens, req_to_token=self.r2t,
                                           req_pool_idx=self.req_pool_idx, lse=self.lse, kv_chunk=kv_chunk)
        else:
            self.args = B.make_extend_args(B.PKV_LAYOUT_CSR, self.q, self.k_pool, self.v_pool, self.out, self.qo_indptr,
                                           page_size=ps, sm_scale=ew.sm_scale, max_seq_len=int(ew.seq_lens.max()),
                                           kv_end=self.kv_end, kv_indptr=self.kv_indptr, kv_indices=self.kv_indices,
                                           kv_last_page_len=self.kv_last, lse=self.lse, kv_chunk=kv_chunk)
        self.ws_bytes = (self.quant.extend_size if quant else B.pkv_extend_workspace_size)(self.args)
        self.workspace = torch.empty(max(self.ws_bytes, 256), dtype=torch.uint8, device=dev)

    def build_indices(self):
        if self.token_table:
            return                                   # pkv_extend reads req_to_token itself
        ew = self.ew
        B.pkv_build_indices(self.r2t, self.req_pool_idx, self.seq_lens, ew.page_size, ew.num_pool_pages, self.err,
                            kv_indptr=self.kv_indptr, kv_indices=self.kv_indices, kv_last_page_len=self.kv_last)

    def store(self):
        if self.quant is not None:
            self.quant.store(self.k_new, self.v_new, self.slot_mapping, self.err)
            return
        B.pkv_store(self.k_pool, self.v_pool, self.k_new, self.v_new, self.slot_mapping, self.err)

    def plan(self):
        if self.kv_end is not None:
            B.pkv_span_plan(*self.seg, self.plan_qo, self.q_pos, self.kv_end, self.err)

    def attend(self):
        (B.pkv_extend if self.quant is None else self.quant.extend)(self.args, self.workspace, self.err)

    def run(self):
        self.build_indices()
        self.store()
        self.plan()
        self.attend()

    def launches_per_step(self) -> int:
        if self.quant is not None:
            # spans and their merge (small calls: one launch and the least workspace); with many rows the copy out of the pool and its attention besides
            # (alone for one request), not counting the join of the latter's pieces where it splits keys
            held = int(self.ew.qo_lens.max()) * (self.ew.num_q_heads // self.ew.num_kv_heads) > 128
            n = (2 if self.ws_bytes > 256 else 1) if not held or self.ew.batch > 1 else 0
            n += 2 if held else 0
            return n + self.quant.store_launches(int(self.ew.qo_lens.sum())) + (0 if self.token_table else 1) + (1 if self.kv_end is not None else 0)
        return (2 if self.token_table else 3) + (1 if self.kv_end is not None else 0) + (1 if self.ws_bytes > 0 else 0)

    def check_errors(self) -> int:
        return int(self.err.item())

    def host_step_tensors(self):
        """Pinned host copies of the step's packed inputs and of its output (for end-to-end timing)."""
        return {"inputs": self.in_buf.cpu().pin_memory()}, {"out": torch.empty_like(self.out, device="cpu").pin_memory()}

    def run_from_host(self, h_in, h_out):
        """One host-to-device copy of the step's inputs (q, new K/V rows, lengths, slots, query
        offsets, segments: packed in one buffer), the step, one copy of the output back."""
        self.in_buf.copy_(h_in["inputs"], non_blocking=True)
        self.run()
        h_out["out"].copy_(self.out, non_blocking=True)


class BudgetedDecode:
    """A batch's serving loop over an 8-bit pool, each request within a budget of tokens:

        prefill()  pkv_alloc_extend, pkv_write_req_to_token, pkv_byte_store, pkv_byte_extend, and
                   pkv_byte_weights of each request's last ``window`` rows
        step()     the same for one token per request, with pkv_byte_decode, which adds up what
                   each key receives
        evict()    pkv_evict: requests above the budget lose the pages that received least, but
                   none of the first ``keep_first`` and last ``keep_last`` tokens

    Request b has row b of the table ``r2t`` and of ``acc`` (what its keys received so far).  Pages
    come from one free list and go back to it.  ``width`` bounds a request's tokens between two
    evictions; positions that are rotated into q and k are the caller's to count, as an eviction
    makes ``seq_lens`` smaller.  Every buffer stays where it is, so step() and evict() can be captured.

    A prefill() or step() for which the free list has too few pages raises PKV_DEVERR_CAPACITY in ``err``,
    one that would take a request past ``width`` PKV_DEVERR_RANGE.  It changes nothing else: lengths, table,
    weights, free list and pool stay as they were, and the output is zeros (lse -inf).  After an
    eviction the same call may be made again.
    """

    def __init__(self, batch, num_q_heads, num_kv_heads, head_dim, page_size, num_pages, width, budget, keep_first=4,
                 keep_last=64, window=32, sm_scale=None, device="cuda"):
        dev = self.device = torch.device(device)
        i32 = lambda v: torch.full((batch,), v, dtype=torch.int32, device=dev)  # noqa: E731
        self.batch, self.num_q_heads, self.head_dim = batch, num_q_heads, head_dim
        self.page_size, self.num_pages, self.width, self.window = page_size, num_pages, width, window
        self.sm_scale = head_dim ** -0.5 if sm_scale is None else sm_scale
        self.pool = _BytePool(num_pages * page_size, num_kv_heads, head_dim, page_size, dev)
        self.r2t = torch.zeros((batch, width), dtype=torch.int32, device=dev)
        self.acc = torch.zeros((batch, width), dtype=torch.float32, device=dev)
        self.rows = torch.arange(batch, dtype=torch.int32, device=dev)
        self.last_loc = i32(0)
        self.lens = torch.zeros((2, batch), dtype=torch.int32, device=dev)    # each request's keys; those that attention sees
        self.start = torch.zeros((3, batch), dtype=torch.int32, device=dev)   # both as a refused call leaves them; new slots
        self.seq_lens, self.seen_lens = self.lens
        self.prefix_lens, _, self.new_loc = self.start
        self.start_is = torch.tensor([[0], [0], [-1]], dtype=torch.int32, device=dev)
        self.start_keys = torch.tensor([[True], [False], [False]], device=dev)
        self.before_row = self.rows.long() * width - 1     # index of the column before each row's first
        self.budget, self.keep_first, self.keep_last = i32(budget), i32(keep_first), i32(keep_last)
        self.free_pages = torch.arange(num_pages, dtype=torch.int32, device=dev)
        self.free_state = torch.tensor([0, num_pages], dtype=torch.int32, device=dev)
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        self.q = torch.zeros((batch, num_q_heads, head_dim), dtype=torch.bfloat16, device=dev)
        self.k_new = torch.zeros((batch, num_kv_heads, head_dim), dtype=torch.bfloat16, device=dev)
        self.v_new = torch.zeros_like(self.k_new)
        self.out = torch.zeros_like(self.q)
        self.lse = torch.zeros((batch, num_q_heads), dtype=torch.float32, device=dev)
        self.args = self._args(self.q, self.out, self.lse, acc_in=self.acc, acc_out=self.acc)
        self.workspace = torch.empty(B.pkv_byte_decode_workspace_size(self.args), dtype=torch.uint8, device=dev)
        self.evict_workspace = torch.empty(B.pkv_evict_workspace_size(batch, width, page_size), dtype=torch.uint8, device=dev)

    def _args(self, q, out, lse, **kw):
        kw.setdefault("max_seq_len", self.width)
        return self.pool.args(B.PKV_LAYOUT_REQ_TO_TOKEN, q, out, sm_scale=self.sm_scale, lse=lse, seq_lens=self.seen_lens,
                              req_to_token=self.r2t, req_pool_idx=self.rows, **kw)

    def _grow(self, new_lens, new_loc, k_new, v_new):
        """Each request by new_lens [B] tokens, at slots new_loc (-1 all of them): slots, table columns, rows -> whether
        there was room (bool [1], on the device).  A refused allocation writes no slot, and rows of slot -1 are not stored."""
        torch.where(self.start_keys, self.seq_lens, self.start_is, out=self.start)
        lens = self.prefix_lens + new_lens
        lens.masked_fill_(lens > self.width, -1)       # past the table: no length, so the allocation refuses the call
        torch.take(self.r2t, (self.before_row + self.prefix_lens).clamp_(0, self.r2t.numel() - 1), out=self.last_loc)
        B.pkv_alloc_extend(self.prefix_lens, lens, self.last_loc, self.page_size, self.num_pages, self.free_pages,
                           self.free_state, new_loc, self.err)
        room = new_loc[:1] >= 0
        torch.where(room, lens, self.start[:2], out=self.lens)
        B.pkv_write_req_to_token(self.r2t, self.rows, self.prefix_lens, self.seq_lens, new_loc, self.err)
        self.pool.store(k_new, v_new, new_loc, self.err)
        return room

    def prefill(self, q, k_new, v_new, new_lens):
        """new_lens: each request's new tokens (host integers), whose rows q, k_new, v_new hold in order -> out."""
        total = sum(new_lens)
        if len(new_lens) != self.batch or min(new_lens) < 0 or q.shape[0] != total:
            raise ValueError("new_lens must count q's rows, request by request")
        out = torch.zeros_like(q)
        if total == 0:
            return out
        at = np.concatenate([[0], np.cumsum(new_lens)]).astype(np.int32)
        up = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(self.device)  # noqa: E731
        # what the requests will hold, from the device: the workspaces are sized by it, not by the table
        # (the uploads below wait for the stream too)
        keys = [n + m for n, m in zip(self.seq_lens.tolist(), new_lens)]
        bounds = dict(max_seq_len=min(self.width, max(keys)), total_kv=sum(keys))
        room = self._grow(up(np.asarray(new_lens, dtype=np.int32)), torch.full((total,), -1, dtype=torch.int32, device=self.device),
                          k_new, v_new)
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=self.device)
        args = self._args(q, out, lse, qo_indptr=up(at) * room, max_q_len=max(new_lens), **bounds)
        B.pkv_byte_extend(args, torch.empty(B.pkv_byte_extend_workspace_size(args), dtype=torch.uint8, device=self.device), self.err)
        seen = [min(n, self.window) for n in new_lens]
        if not sum(seen):
            return out
        rows = up(np.concatenate([np.arange(e - n, e) for e, n in zip(at[1:], seen)]))
        first = up(np.concatenate([[0], np.cumsum(seen)]).astype(np.int32)) * room
        args = self._args(q[rows], None, lse[rows], qo_indptr=first, max_q_len=max(seen), acc_in=self.acc, acc_out=self.acc, **bounds)
        B.pkv_byte_weights(args, torch.empty(B.pkv_byte_weights_workspace_size(args), dtype=torch.uint8, device=self.device), self.err)
        return out

    def step(self):
        """One token per request, of q, k_new and v_new -> out."""
        self._grow(1, self.new_loc, self.k_new, self.v_new)
        B.pkv_byte_decode(self.args, self.workspace, self.err)
        return self.out

    def evict(self):
        B.pkv_evict(self.r2t, self.rows, self.seq_lens, self.acc, self.budget, self.free_pages, self.free_state,
                    self.evict_workspace, self.err, page_size=self.page_size, num_pool_pages=self.num_pages,
                    max_seq_len=self.width, keep_first=self.keep_first, keep_last=self.keep_last)

    def check_errors(self) -> int:
        return int(self.err.item())
