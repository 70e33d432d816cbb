"""A 4-bit step holds no bf16 pool."""
import gc

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def engine():
    from paged_kv_cache_req_gb300 import build
    build.build()
    from paged_kv_cache_req_gb300 import engine
    return engine


def _held(make):
    gc.collect()
    before = torch.cuda.memory_allocated()
    step = make()
    gc.collect()
    return step, torch.cuda.memory_allocated() - before


def test_the_bf16_pools_are_let_go(engine):
    from paged_kv_cache_req_gb300.workloads import make_extend_workload, make_workload
    for kw in ({}, dict(cross_mode="gather")):
        wl = make_workload("whisper_encdec", batch=5)
        plain, size = _held(lambda: engine.DecodeStep(wl, **kw))
        bf16 = plain.k_pool.nbytes + plain.v_pool.nbytes
        step, quant = _held(lambda: engine.DecodeStep(wl, quant=True, **kw))
        assert step.k_pool is None and step.v_pool is None
        # 9 / 32 of the pools, and workspaces that differ by some MB
        assert quant < size - bf16 * 23 // 32 + (32 << 20)
        step.run()
        assert step.check_errors() == 0
    ew = make_extend_workload("llama3_8b_verify", batch=16)
    plain, size = _held(lambda: engine.ExtendStep(ew, token_table=True))
    bf16 = plain.k_pool.nbytes + plain.v_pool.nbytes
    step, quant = _held(lambda: engine.ExtendStep(ew, token_table=True, quant=True))
    assert step.k_pool is None and quant < size - bf16 * 23 // 32 + (32 << 20)
    step.run()
    assert step.check_errors() == 0


def test_given_pools_stay_the_callers(engine):
    from paged_kv_cache_req_gb300.workloads import make_workload
    wl = make_workload("tiny_gqa", batch=4)
    pools = engine.fill_pool(wl, device="cuda")
    want = [p.clone() for p in pools]
    step = engine.DecodeStep(wl, pools=pools, quant=True)
    step.run()
    assert step.check_errors() == 0 and all(torch.equal(p, w) for p, w in zip(pools, want))
