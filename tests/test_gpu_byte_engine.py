"""The engine over an 8-bit pool: decode and extend steps, and the loop that prefills, decodes, counts
and evicts, against the plain references applied one after the other."""
import numpy as np
import pytest
import torch

import _byte_ref as R
from test_gpu_byte import host, to_bf16, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from paged_kv_cache_req_gb300 import build
    build.build()
    from paged_kv_cache_req_gb300 import _binding
    return _binding


def on_host(quant, D):
    """The pool's tiles on the host."""
    return R.Pool(quant.pool.cpu().numpy(), quant.page_size, D, quant.kv_heads)


@pytest.mark.parametrize("name,batch,fused,cross", [("tiny_gqa", None, False, "paged"), ("tiny_gqa", None, True, "paged"),
                                                    ("whisper_encdec", 3, False, "paged"), ("whisper_encdec", 3, True, "gather")])
def test_decode_step(B, name, batch, fused, cross):
    from paged_kv_cache_req_gb300.engine import DecodeStep
    from paged_kv_cache_req_gb300.workloads import make_workload
    wl = make_workload(name, batch=batch)
    step = DecodeStep(wl, fused=fused, cross_mode=cross, quant=8)
    assert step.k_pool is None
    for _ in range(2):           # a step stores the same rows again: nothing changes
        step.run()
        assert step.check_errors() == 0
    pool = on_host(step.quant, wl.head_dim_v)
    r2t, rpi = step.r2t.cpu().numpy(), wl.req_pool_idx.numpy()
    for pname, pb in step.problems.items():
        lens, starts = pb.spec.seq_lens.numpy(), pb.spec.kv_start.numpy()
        for b in range(wl.batch):
            slots = r2t[rpi[b], starts[b]:starts[b] + lens[b]]
            k, v = pool.read(slots, 0), pool.read(slots, 1)
            if pb.spec.stores:   # the new row went in
                new = host(step.k_new)[b]
                assert (np.abs(k[-1] - new) <= 2.0 ** -4 * np.abs(new) + 2.0 ** -10 * pool.largest(slots)[:, None] * 64).all()
            # (rows read back as bf16 are exact; the bf16 decode rounds its weights to bf16)
            o, l, _, tol, lt, _ = R.attention(host(pb.q)[b:b + 1].astype(np.float64), k, v, [lens[b]], wl.sm_scale,
                                              pool.largest(slots) if lens[b] else np.ones(wl.num_kv_heads), held=pb.gather)
            R.assert_within(host(pb.out)[b:b + 1], o, tol, "%s %d" % (pname, b))
            R.assert_within(host(pb.lse)[b:b + 1], l, lt, "%s %d lse" % (pname, b))


@pytest.mark.parametrize("name,batch,token_table,held", [("qwen3_0p6b_prefill", 2, False, True), ("qwen3_0p6b_prefill", 1, True, True),
                                                         ("llama3_8b_verify", 3, True, False)])
def test_extend_step(B, name, batch, token_table, held):
    from paged_kv_cache_req_gb300.engine import ExtendStep
    from paged_kv_cache_req_gb300.workloads import make_extend_workload
    ew = make_extend_workload(name, batch=batch)
    step = ExtendStep(ew, token_table=token_table, quant=8)
    step.run()
    assert step.check_errors() == 0
    pool = on_host(step.quant, ew.head_dim)
    r2t, rpi, lens = step.r2t.cpu().numpy(), ew.req_pool_idx.numpy(), ew.seq_lens.numpy()
    at = np.concatenate([[0], np.cumsum(ew.qo_lens.numpy())])
    for b in range(ew.batch):
        slots = r2t[rpi[b], :lens[b]]
        n = at[b + 1] - at[b]
        rows = at[b] + np.unique([0, n // 3, n - 1])
        ends = lens[b] - n + 1 + rows - at[b]
        o, l, _, tol, lt, _ = R.attention(host(step.q[rows]).astype(np.float64), pool.read(slots, 0), pool.read(slots, 1),
                                          ends, ew.sm_scale, pool.largest(slots), held=held)
        R.assert_within(host(step.out[rows]), o, tol, "request %d" % b)
        R.assert_within(host(step.lse[rows]), l, lt, "request %d lse" % b)


def test_refusals(B):
    from paged_kv_cache_req_gb300.engine import DecodeStep
    from paged_kv_cache_req_gb300.workloads import make_workload
    wl = make_workload("tiny_gqa")
    with pytest.raises(ValueError):
        DecodeStep(wl, quant=5)
    with pytest.raises(ValueError):
        DecodeStep(wl, quant=8, scales=(torch.ones(2), torch.ones(2)))


class Mirror:
    """The loop's state on the host, from the definitions."""

    def __init__(self, loop, H):
        self.loop, self.H = loop, H
        self.pool = R.Pool(loop.pool.pool.cpu().numpy(), loop.page_size, loop.head_dim, H)
        self.free, self.state = loop.free_pages.cpu().numpy(), loop.free_state.tolist()
        self.r2t, self.acc = loop.r2t.cpu().numpy(), loop.acc.cpu().numpy().astype(np.float64)
        self.lens = np.zeros(loop.batch, dtype=np.int64)

    def grow(self, k, v, new):
        ps, at, slots = self.loop.page_size, 0, []
        for b, n in enumerate(new):
            for _ in range(n):
                L = self.lens[b]
                if L % ps == 0:
                    first = self.free[self.state[0]] * ps
                    self.state = [self.state[0] + 1, self.state[1] - 1]
                    slot = first
                else:
                    slot = self.r2t[b, L - 1] + 1
                self.r2t[b, L] = slot
                slots.append(slot)
                self.lens[b] += 1
        self.pool.store(host(k), host(v), slots)

    def same(self, what):
        L = self.loop
        assert L.check_errors() == 0
        assert (L.seq_lens.cpu().numpy() == self.lens).all() and L.free_state.tolist() == self.state, what
        assert (L.free_pages.cpu().numpy() == self.free).all(), what
        r2t = L.r2t.cpu().numpy()
        for b, n in enumerate(self.lens):
            assert (r2t[b, :n] == self.r2t[b, :n]).all(), what
        assert (L.pool.pool.cpu().numpy() == self.pool.data).all(), what

    def attend(self, b, q, ends, what, out, lse, held):
        slots = self.r2t[b, :self.lens[b]]
        o, l, w, tol, lt, wt = R.attention(host(q).astype(np.float64), self.pool.read(slots, 0), self.pool.read(slots, 1), ends,
                                           self.loop.sm_scale, self.pool.largest(slots), held)
        R.assert_within(host(out), o, tol, what + " out")
        if lse is not None:
            R.assert_within(host(lse), l, lt, what + " lse")
        return w, wt


@pytest.mark.parametrize("ps,D,H,g,graph", [(1, 64, 2, 4, False), (16, 128, 2, 2, False), (16, 64, 1, 8, True), (4, 128, 1, 3, True)])
def test_loop(B, ps, D, H, g, graph):
    """Prefill, decode past the budget, evict, decode on over what is left, evict again."""
    from paged_kv_cache_req_gb300.engine import BudgetedDecode
    rng = np.random.default_rng(ps + D)
    batch, width, budget, window = 3, 256, 96, 8
    loop = BudgetedDecode(batch, H * g, H, D, ps, 3 * 256 // ps, width, budget, keep_first=3, keep_last=17, window=window)
    m = Mirror(loop, H)
    new = [150, 40, 97]
    total = sum(new)
    q, k, v = (to_bf16(values(rng, (total, h, D), s)) for h, s in ((H * g, 1.0), (H, 1.0), (H, 0.3)))
    out = loop.prefill(q, k, v, new)
    m.grow(k, v, new)
    m.same("prefill")
    at = np.concatenate([[0], np.cumsum(new)])
    bound = np.zeros_like(m.acc)
    for b, n in enumerate(new):
        w, wt = m.attend(b, q[at[b]:at[b + 1]], np.arange(1, n + 1), "prefill %d" % b, out[at[b]:at[b + 1]], None, True)
        m.acc[b, :n] += w[-window:].sum((0, 1))
        bound[b, :n] += wt[-window:].sum((0, 1)) + (window * H * g + 1) * 2.0 ** -23 * m.acc[b, :n]
    R.assert_within(host(loop.acc), m.acc, bound, "weights of the prefill")

    def evict():
        # the kernel's own sums decide (they were held to their bound)
        acc = loop.acc.cpu().numpy()
        want = R.evict(m.r2t, acc, range(batch), [0] * batch, m.lens, [budget] * batch, [3] * batch, [17] * batch, ps, m.free, m.state)
        loop.evict()
        m.r2t, m.lens, m.free, m.state = want[0], want[2].astype(np.int64), want[3], want[4]
        m.same("evict")
        for b in range(batch):
            assert (loop.acc.cpu().numpy()[b] == want[1][b]).all()
        assert (m.lens <= budget).all()

    evict()
    captured = None
    for i in range(40):
        for t, h, s in ((loop.q, H * g, 1.0), (loop.k_new, H, 1.0 + i % 5), (loop.v_new, H, 0.3)):
            t.copy_(to_bf16(values(rng, (batch, h, D), s)))
        before = loop.acc.cpu().numpy().astype(np.float64)
        if graph and i == 1:
            torch.cuda.synchronize()
            state = [x.clone() for x in (loop.seq_lens, loop.r2t, loop.free_state, loop.acc, loop.pool.pool, loop.prefix_lens, loop.last_loc)]
            captured = torch.cuda.CUDAGraph()
            with torch.cuda.graph(captured):
                loop.step()
            for x, y in zip(state, (loop.seq_lens, loop.r2t, loop.free_state, loop.acc, loop.pool.pool, loop.prefix_lens, loop.last_loc)):
                assert torch.equal(x, y)          # capturing ran nothing
        captured.replay() if captured is not None else loop.step()
        m.grow(loop.k_new, loop.v_new, [1] * batch)
        m.same("step %d" % i)
        for b in range(batch):
            w, wt = m.attend(b, loop.q[b:b + 1], [m.lens[b]], "step %d request %d" % (i, b), loop.out[b:b + 1], loop.lse[b:b + 1], False)
            n = m.lens[b]
            want = before[b, :n] + w.sum((0, 1))
            assert before[b, n - 1] == 0           # a new token starts with none
            R.assert_within(host(loop.acc)[b, :n], want, wt.sum((0, 1)) + (H * g + 1) * 2.0 ** -23 * want, "step %d weights" % i)
        if i in (17, 39):
            evict()
