"""The loop within a budget when it cannot grow: a free list that has run out, a table that is too narrow.
A refused call changes nothing but the error word, and after an eviction the same call goes on."""
import numpy as np
import pytest
import torch

import _byte_ref as R
from test_gpu_byte import B, host, to_bf16, values  # noqa: F401
from test_gpu_byte_engine import Mirror

pytestmark = pytest.mark.gpu


class Run:
    """A loop and its state on the host, from the definitions."""

    def __init__(self, B, seed, ps, D, H, g, pages, width, budget=64):
        from paged_kv_cache_req_gb300.engine import BudgetedDecode
        self.B, self.rng, self.ps, self.D, self.H, self.g, self.budget = B, np.random.default_rng(seed), ps, D, H, g, budget
        self.loop = BudgetedDecode(3, H * g, H, D, ps, pages, width, budget, keep_first=3, keep_last=17, window=8)
        self.loop.pool.pool.fill_(0xEE)
        self.m = Mirror(self.loop, H)

    def rows(self, n):
        return [to_bf16(values(self.rng, (n, h, self.D), s)) for h, s in ((self.H * self.g, 1.0), (self.H, 1.0), (self.H, 0.3))]

    def prefill(self, new):
        q, k, v = self.rows(sum(new))
        out = self.loop.prefill(q, k, v, new)
        self.m.grow(k, v, new)
        self.m.same("prefill %s" % new)
        at = np.concatenate([[0], np.cumsum(new)])
        for b, n in enumerate(new):
            L = self.m.lens[b]
            self.m.attend(b, q[at[b]:at[b + 1]], np.arange(L - n + 1, L + 1), "prefill %d" % b, out[at[b]:at[b + 1]], None, True)

    def next_rows(self):
        for t, x in zip((self.loop.q, self.loop.k_new, self.loop.v_new), self.rows(3)):
            t.copy_(x)

    def grown(self, before, what):
        """The step that ran was right."""
        loop, m = self.loop, self.m
        m.grow(loop.k_new, loop.v_new, [1] * 3)
        m.same(what)
        for b in range(3):
            n = m.lens[b]
            w, wt = m.attend(b, loop.q[b:b + 1], [n], what, loop.out[b:b + 1], loop.lse[b:b + 1], False)
            want = before[b, :n] + w.sum((0, 1))
            R.assert_within(host(loop.acc)[b, :n], want, wt.sum((0, 1)) + (self.H * self.g + 1) * 2.0 ** -23 * want, what + " weights")

    def state(self):
        loop = self.loop
        return [x.clone() for x in (loop.seq_lens, loop.r2t, loop.acc, loop.free_pages, loop.free_state, loop.pool.pool)]

    def refused(self, call, flag, what):
        """The call raises the flag and leaves everything as it was."""
        before = self.state()
        call()
        assert self.loop.check_errors() == flag, what
        for x, y, name in zip(before, self.state(), ("seq_lens", "r2t", "acc", "free_pages", "free_state", "pool")):
            assert torch.equal(x, y), "%s: %s changed" % (what, name)
        self.loop.err.zero_()

    def evict(self):
        m, loop = self.m, self.loop
        want = R.evict(m.r2t, loop.acc.cpu().numpy(), range(3), [0] * 3, m.lens, [self.budget] * 3, [3] * 3, [17] * 3, self.ps, m.free, m.state)
        loop.evict()
        m.r2t, m.lens, m.free, m.state = want[0], want[2].astype(np.int64), want[3], want[4]
        m.same("evict")


def captured(loop):
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loop.step()
    return graph.replay


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("ps,pages,steps", [(16, 20, 6), (64, 6, 14), (1, 295, 1)])
def test_a_full_pool(B, ps, pages, steps, graph):
    """Steps until no page is left, one more and a prefill that are refused, an eviction, and the step again."""
    r = Run(B, 80 + ps, ps, 64, 2, 2, pages, 256)
    r.prefill([200, 42, 50])
    step = r.loop.step
    for i in range(steps):
        before = host(r.loop.acc).astype(np.float64)
        r.next_rows()
        if graph and i == 0:
            step = captured(r.loop)
        step()
        r.grown(before, "step %d" % i)
    r.next_rows()
    for i in range(2):
        r.refused(step, B.PKV_DEVERR_CAPACITY, "step without a page")
        assert not r.loop.out.any() and torch.isneginf(r.loop.lse).all()
    q, k, v = r.rows(70)
    out = []
    r.refused(lambda: out.append(r.loop.prefill(q, k, v, [0, 70, 0])), B.PKV_DEVERR_CAPACITY, "prefill without pages")
    assert not out[0].any()
    r.evict()
    before = host(r.loop.acc).astype(np.float64)
    r.next_rows()
    step()
    r.grown(before, "step after the eviction")
    r.prefill([3, 0, 1])


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("ps,width", [(16, 205), (64, 256), (1, 203)])
def test_a_request_as_long_as_its_row(B, ps, width, graph):
    """Steps up to the table's width, further ones and a prefill that are refused, an eviction, and the step again."""
    r = Run(B, 90 + ps, ps, 64, 2, 2, 3 * -(-width // ps), width)
    r.prefill([30, width - 3, 50])
    step = r.loop.step
    for i in range(3):
        before = host(r.loop.acc).astype(np.float64)
        r.next_rows()
        if graph and i == 0:
            step = captured(r.loop)
        step()
        r.grown(before, "step %d" % i)
    assert r.m.lens.max() == width
    r.next_rows()
    for i in range(3):
        r.refused(step, B.PKV_DEVERR_RANGE, "step past the width")
        assert not r.loop.out.any() and torch.isneginf(r.loop.lse).all()
    q, k, v = r.rows(width)
    r.refused(lambda: r.loop.prefill(q, k, v, [width, 0, 0]), B.PKV_DEVERR_RANGE, "prefill past the width")
    r.evict()
    before = host(r.loop.acc).astype(np.float64)
    r.next_rows()
    step()
    r.grown(before, "step after the eviction")


@pytest.mark.parametrize("new", [[300, 2] + [0] * 30, [5] * 32, [0] * 31 + [1]])
def test_prefill_workspaces_follow_the_keys(B, new):
    """32 rows of 16384 columns, nearly all of them empty: what a prefill takes is by its keys, not by the table."""
    from paged_kv_cache_req_gb300.engine import BudgetedDecode
    rng, H, D = np.random.default_rng(100), 2, 64
    loop = BudgetedDecode(32, 2 * H, H, D, 16, 200, 16384, 1024, window=8)
    for turn in range(2):
        q, k, v = (to_bf16(values(rng, (sum(new), h, D))) for h in (2 * H, H, H))
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        out = loop.prefill(q, k, v, new)
        assert loop.check_errors() == 0 and torch.isfinite(out).all()
        # K and V of 32 x 16384 keys in bf16 are 256 MB
        assert torch.cuda.max_memory_allocated() - before < 64 << 20
