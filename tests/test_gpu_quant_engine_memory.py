"""A 4-bit step and the bf16 pools it is made from: they are let go, and what is not a number in them
costs its own block alone."""
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


def test_a_value_that_is_no_number_leaves_the_head_its_scale(engine):
    from paged_kv_cache_req_gb300.workloads import make_workload
    wl = make_workload("tiny_gqa", batch=4)
    clean = engine.fill_pool(wl, device="cuda")
    want = engine.DecodeStep(wl, pools=clean, quant=True)
    pools = [p.clone() for p in clean]
    # (slot 0 is padding: no request reads it)
    pools[0][0, 0, 3], pools[1][0, 1, 5], pools[1][0, 0, 40] = float("inf"), float("nan"), float("-inf")
    step = engine.DecodeStep(wl, pools=pools, quant=True)
    assert step.check_errors() == 0
    assert torch.equal(step.quant.k_scale, want.quant.k_scale) and torch.equal(step.quant.v_scale, want.quant.v_scale)
    want.run()
    step.run()
    assert step.check_errors() == 0
    for name, pb in step.problems.items():
        assert torch.equal(pb.out, want.problems[name].out)
