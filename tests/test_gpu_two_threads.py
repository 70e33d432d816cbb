"""First calls of a process from two threads at once, where a launch needs more shared memory than
a kernel has from the start: the split merges of pkv_decode and pkv_alloc_extend."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FIRST_CALLS = """
import sys, threading
import torch
from paged_kv_cache_req_gb300 import _binding as B

dev = "cuda"
i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)
failed = []
barrier = threading.Barrier(2)


def attend(kind, D, Hq, splits):
    # one key; the upper bound on the lengths sizes the merge
    dv = 512 if kind == B.PKV_KIND_MLA else D
    pool = torch.zeros((64, 576) if kind == B.PKV_KIND_MLA else (64, 1, D), dtype=torch.bfloat16, device=dev)
    q = torch.ones((1, Hq, pool.shape[-1]), dtype=torch.bfloat16, device=dev)
    out = torch.empty((1, Hq, dv), dtype=torch.bfloat16, device=dev)
    a = B.make_decode_args(kind, B.PKV_LAYOUT_BLOCK_TABLE, q, pool, None if kind == B.PKV_KIND_MLA else pool, out, page_size=64,
                           sm_scale=1.0, max_seq_len=64 * splits, head_dim_v=dv, kv_chunk=64, block_table=i32(1, 1),
                           seq_lens=i32(1) + 1)
    ws = torch.empty(B.pkv_decode_workspace_size(a), dtype=torch.uint8, device=dev)
    err, s = i32(1), torch.cuda.Stream()
    return lambda: B.pkv_decode(a, ws, err, stream=s), err


def alloc(n):
    free = torch.arange(n, dtype=torch.int32, device=dev)
    state = torch.tensor([0, n], dtype=torch.int32, device=dev)
    args = (i32(n), i32(n) + 1, i32(n) - 1, 1, n, free, state, i32(n))
    err, s = i32(1), torch.cuda.Stream()

    def call():
        with torch.cuda.stream(s):
            state.copy_(start[n])
        B.pkv_alloc_extend(*args, err, stream=s)
    start[n] = state.clone()
    return call, err


def work(k):
    for call, _ in calls[k]:
        barrier.wait()
        for _ in range(3):
            try:
                call()
            except B.PkvError as e:
                failed.append("%d: %s" % (k, e))


start = {}
calls = [[attend(B.PKV_KIND_GQA, 128, 16, n), attend(B.PKV_KIND_GQA, 64, 16, n), attend(B.PKV_KIND_MLA, 576, 128, m), alloc(k)]
         for n, m, k in ((1000, 900, 3500), (3000, 1700, 8000))]
torch.cuda.synchronize()
threads = [threading.Thread(target=work, args=(k,)) for k in (0, 1)]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert all(err.item() == 0 for c in calls for _, err in c)
sys.exit("\\n".join(failed) if failed else 0)
"""


def test_first_calls_from_two_threads():
    from paged_kv_cache_req_gb300 import build
    build.build()
    for _ in range(4):
        r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=ROOT, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr
