"""pkv_evict on the GPU against the definition: every output is moved or whole, and compared for equality."""
import numpy as np
import pytest
import torch

import _byte_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def B():
    from paged_kv_cache_req_gb300 import build
    build.build()
    from paged_kv_cache_req_gb300 import _binding
    return _binding


def up(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


class Case:
    def __init__(self, rng, lens, ps, starts=None, ties=False):
        B_ = len(lens)
        self.ps, self.lens = ps, np.array(lens, dtype=np.int32)
        self.starts = np.zeros(B_, np.int32) if starts is None else np.array(starts, dtype=np.int32)
        npg = -(-self.lens // ps)
        self.pages = int(npg.sum()) + 5
        width = int((self.starts + self.lens).max(initial=0)) + 7
        self.rows = rng.permutation(B_ + 2)[:B_].astype(np.int32)
        self.table = rng.integers(0, 1 << 20, (B_ + 2, width)).astype(np.int32)     # columns of nobody hold anything
        order = rng.permutation(self.pages)
        at = 0
        for b in range(B_):
            p = order[at:at + npg[b]]
            at += npg[b]
            self.table[self.rows[b], self.starts[b]:self.starts[b] + self.lens[b]] = (p[:, None] * ps + np.arange(ps)).reshape(-1)[:self.lens[b]]
        self.acc = np.exp(2 * rng.standard_normal(self.table.shape)).astype(np.float32)
        if ties:
            self.acc = rng.integers(0, 3, self.table.shape).astype(np.float32)
        self.free = rng.permutation(self.pages + 9).astype(np.int32)
        self.state = [int(npg.sum()) + 2, 4]

    def run(self, B, budget, first=None, last=None, elsewhere=False, max_len=None, num_pages=None, **over):
        v = dict(table=self.table, acc=self.acc, rows=self.rows, lens=self.lens, starts=self.starts, free=self.free,
                 state=np.array(self.state, dtype=np.int32))
        v.update({k: np.asarray(x, dtype=v[k].dtype) for k, x in over.items()})
        d = {k: up(x) for k, x in v.items()}
        n = len(self.lens)
        vec = lambda x: None if x is None else up(np.broadcast_to(np.asarray(x, np.int32), (n,)).copy())  # noqa: E731
        outs = dict(req_to_token_out=torch.full_like(d["table"], -9), acc_out=torch.full_like(d["acc"], -9.0),
                    seq_lens_out=torch.full_like(d["lens"], -9), free_state_out=torch.full_like(d["state"], -9)) if elsewhere else {}
        max_len = int(self.lens.max(initial=0)) if max_len is None else max_len
        ws = torch.full((B.pkv_evict_workspace_size(n, max_len, self.ps),), 0xFF, dtype=torch.uint8, device=DEV)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        B.pkv_evict(d["table"], d["rows"], d["lens"], d["acc"], vec(budget), d["free"], d["state"], ws, err, page_size=self.ps,
                    num_pool_pages=self.pages if num_pages is None else num_pages, max_seq_len=max_len, kv_start=d["starts"],
                    keep_first=vec(first), keep_last=vec(last), **outs)
        o = (outs["req_to_token_out"], outs["acc_out"], outs["seq_lens_out"], d["free"], outs["free_state_out"]) if elsewhere else \
            (d["table"], d["acc"], d["lens"], d["free"], d["state"])
        if elsewhere:
            for k in ("table", "acc", "lens", "state"):
                assert np.array_equal(d[k].cpu().numpy(), v[k], equal_nan=k == "acc"), k
        return [x.cpu().numpy() for x in o], err.item()

    def want(self, budget, first=None, last=None):
        n = len(self.lens)
        vec = lambda x: np.broadcast_to(np.asarray(0 if x is None else x), (n,))  # noqa: E731
        return R.evict(self.table, self.acc, self.rows, self.starts, self.lens, vec(budget), vec(first), vec(last), self.ps,
                       self.free, self.state)

    def check(self, B, budget, first=None, last=None, **kw):
        want = self.want(budget, first, last)
        got, e = self.run(B, budget, first, last, **kw)
        assert e == 0
        for g, w, name in zip(got, want, ("table", "acc", "lens", "free", "state")):
            assert np.array_equal(g, np.asarray(w, dtype=g.dtype), equal_nan=name == "acc"), name
        got, e = self.run(B, budget, first, last, elsewhere=True, **kw)
        assert e == 0
        mine = np.zeros(self.table.shape, bool)
        kept = mine.copy()
        for b, L in enumerate(self.lens):
            mine[self.rows[b], self.starts[b]:self.starts[b] + L] = True
            kept[self.rows[b], self.starts[b]:self.starts[b] + want[2][b]] = True
        assert (got[0][kept] == want[0][kept]).all() and (got[0][~kept] == -9).all()
        assert np.array_equal(got[1][mine], want[1][mine], equal_nan=True) and (got[1][~mine] == -9).all()
        for i in (2, 3, 4):
            assert (got[i] == np.asarray(want[i])).all()


CASES = [  # lens, ps, budget, first, last
    ([1, 2, 3, 30, 31, 32, 33, 100], 1, 20, 2, 5),
    ([1000, 17, 16, 15, 0, 300], 16, 100, 20, 33),
    ([640, 641, 639], 64, 200, 0, 0),
    ([500], 2, 100, None, None),
    ([700, 600], 4, [1, 0], [0, 9], [0, 0]),
    ([3000, 100], 8, 500, [3000, 0], 64),                # the first keeps all
    ([5000], 1, 4999, 0, 1),
    ([2500, 9, 4000], 32, 1000, 100, 500),
    ([300] * 40, 1, 100, 4, 16),
    ([20000], 1, 777, 4, 100),                           # several blocks to a request
    ([140001], 1, 70000, 4, 100),                        # keys beyond shared memory
    ([30000, 25000], 16, 4096, 4, 100),
    ([9000, 4], 1024, 3000, 1, 1),
    ([0, 0], 16, 5, 0, 0),
]


@pytest.mark.parametrize("lens,ps,budget,first,last", CASES)
@pytest.mark.parametrize("ties", [False, True])
def test_evict(B, lens, ps, budget, first, last, ties):
    rng = np.random.default_rng(sum(lens) + ps)
    Case(rng, lens, ps, starts=[(b % 3) * ps for b in range(len(lens))], ties=ties).check(B, budget, first, last)


def test_special_scores(B):
    """NaN counts most, then infinity; -0 equals 0; negative ones go first."""
    rng = np.random.default_rng(1)
    c = Case(rng, [64, 64], 1)
    x = np.array([0.0, -0.0, 1.0, -1.0, np.inf, -np.inf, np.nan, 3e38, 1e-45, -1e-45], dtype=np.float32)
    c.acc[:] = x[rng.integers(0, len(x), c.acc.shape)]
    for budget in range(1, 64, 5):
        c.check(B, budget)
    # sums that differ by less than fp32 tells: the order of the pages decides
    c = Case(rng, [64], 4)
    c.acc[:] = 1.0
    c.acc[c.rows[0], 8] = np.float32(2.0 ** -30)
    c.acc[c.rows[0], 12] = np.float32(2.0 ** -31)
    c.check(B, 32)


def test_all_the_same(B):
    rng = np.random.default_rng(2)
    c = Case(rng, [3000, 2999], 1)
    c.acc[:] = 0.25
    c.check(B, 1000, 10, 10)


def test_many_requests(B):
    rng = np.random.default_rng(3)
    c = Case(rng, [int(x) for x in rng.integers(0, 60, 1500)], 4)
    c.check(B, rng.integers(0, 50, 1500), rng.integers(0, 9, 1500), rng.integers(0, 9, 1500))


def test_flags_leave_a_request_alone(B):
    rng = np.random.default_rng(4)
    lens = [100, 200, 90]
    c = Case(rng, lens, 16, starts=[0, 16, 0])
    good, _ = c.run(B, 48)
    alone = np.delete(np.arange(3), 1)

    def spared(bit, **kw):
        got, e = c.run(B, kw.pop("budget", 48), **kw)
        assert e == bit, kw
        assert got[2][1] == kw.get("lens", lens)[1]
        for b in alone:
            assert (got[0][c.rows[b]] == good[0][c.rows[b]]).all() and (got[1][c.rows[b]] == good[1][c.rows[b]]).all()
            assert got[2][b] == good[2][b]
        if "table" not in kw:
            assert (got[0][c.rows[1]] == c.table[c.rows[1]]).all() and (got[1][c.rows[1]] == c.acc[c.rows[1]]).all()
        lost = int(sum(lens[b] - good[2][b] for b in alone)) // 16
        assert got[4].tolist() == [c.state[0] - lost, c.state[1] + lost]

    spared(1, starts=[0, 8, 0])
    spared(1, lens=[100, 20000, 90])
    spared(1, lens=[100, -3, 90])
    spared(1, budget=[48, -1, 48])
    spared(1, first=[0, -1, 0])
    spared(1, last=[0, -1, 0])
    spared(1, rows=[c.rows[0], 77, c.rows[2]])
    spared(4, max_len=150)
    bad = c.table.copy()
    bad[c.rows[1], 16 + 32] = c.pages * 16
    spared(1, table=bad)
    bad = c.table.copy()
    bad[c.rows[1], 16 + 32] += 1
    spared(2, table=bad)
    # two requests with one row: neither is touched
    got, e = c.run(B, 48, rows=[c.rows[0], c.rows[0], c.rows[2]], lens=[100, 100, 90], starts=[0, 0, 0])
    assert e == 1 and got[2].tolist()[:2] == [100, 100] and (got[0][c.rows[0]] == c.table[c.rows[0]]).all()
    # no room before the head of the free list: nobody is touched
    for state in ([3, 4], [-5, 4], [1 << 30, 0]):
        got, e = c.run(B, 48, state=state)
        assert e == 4 and got[2].tolist() == lens and got[4].tolist() == state
        assert (got[0] == c.table).all() and (got[1] == c.acc).all() and (got[3] == c.free).all()


def test_again_and_in_a_graph(B):
    """Evictions from a row that keeps growing, captured once and replayed."""
    rng = np.random.default_rng(5)
    c = Case(rng, [160, 96], 16)
    d = dict(table=up(c.table), acc=up(c.acc), lens=up(c.lens), free=up(c.free), state=up(np.array(c.state, dtype=np.int32)))
    rows, budget, zero = up(c.rows), up(np.array([64, 64], dtype=np.int32)), up(c.starts)
    ws = torch.empty(B.pkv_evict_workspace_size(2, 160, 16), dtype=torch.uint8, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def call():
        B.pkv_evict(d["table"], rows, d["lens"], d["acc"], budget, d["free"], d["state"], ws, err, page_size=16,
                    num_pool_pages=c.pages, max_seq_len=160, kv_start=zero)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for _ in range(3):
        want = c.want([64, 64])
        graph.replay()
        torch.cuda.synchronize()
        assert err.item() == 0
        for k, w in zip(("table", "acc", "lens", "free", "state"), want):
            assert (d[k].cpu().numpy() == np.asarray(w)).all(), k
        # the requests grow by the pages that were freed
        c.table, c.acc, c.lens, c.free, c.state = want
        for b in range(2):
            page = int(c.free[c.state[0]])
            c.state = [c.state[0] + 1, c.state[1] - 1]
            L = int(c.lens[b])
            c.table[c.rows[b], L:L + 16] = page * 16 + np.arange(16)
            c.acc[c.rows[b], L:L + 16] = rng.random(16).astype(np.float32)
            c.lens[b] = L + 16
        for k, x in (("table", c.table), ("acc", c.acc), ("lens", c.lens), ("free", c.free), ("state", np.array(c.state, dtype=np.int32))):
            d[k].copy_(up(np.asarray(x)))


def test_refusals(B):
    rng = np.random.default_rng(6)
    c = Case(rng, [64], 16)
    with pytest.raises(B.PkvError):
        c.ps = 12
        c.run(B, 16)
    c.ps = 16
    with pytest.raises(ValueError):
        c.acc = c.acc[:, :-1].copy()
        c.run(B, 16)
