"""The 4-bit attention calls at the ends of what they allow: many short segments per warp, weights
and scales far apart, first calls from several threads, large batches."""
import numpy as np
import pytest
import torch

import _quant_ref as R
from test_gpu_quant import DEV, Cache, check, decode, extend, host, to_bf16, up, values  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from paged_kv_cache_req_gb300 import build
    build.build()
    from paged_kv_cache_req_gb300 import _binding
    return _binding


@pytest.mark.parametrize("D,H,g", [(128, 8, 4), (64, 20, 1)])
def test_short_segments_follow_one_another(B, D, H, g):
    """Pages of 64 and requests of one to three tiles, several to a warp: each segment's query rows are
    fetched while the tile before it is worked on."""
    rng = np.random.default_rng(90 + D)
    lens = rng.integers(1, 190, 500).tolist()
    cache = Cache(rng, lens, 64, H, D)
    q = to_bf16(values(rng, (len(lens), H * g, D)))
    out, lse, e = decode(B, cache, q, kv_chunk=256)
    assert e == 0
    check(cache, q, out, lse, only=list(range(0, 500, 9)) + [499])
    for _ in range(10):
        o2, l2, e = decode(B, cache, q, kv_chunk=256)
        assert e == 0 and torch.equal(out, o2) and torch.equal(lse, l2)
