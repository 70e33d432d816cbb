"""The 4-bit attention calls' sizes and refusals on the host, at the ends of what they allow."""
import pytest

from test_quant_host import B, _args  # noqa: F401


@pytest.mark.parametrize("kw", [
    dict(batch=2, total_q=32768, max_seq_len=1 << 20),
    dict(batch=2, total_q=32768, max_seq_len=1 << 20, total_kv=1100000, max_q_len=32000),
    dict(batch=8, total_q=262144, max_seq_len=131072, total_kv=400000),
    dict(batch=8, total_q=262144, max_seq_len=131072, total_kv=400000, kv_chunk=4096)])
def test_many_long_rows_are_planned(B, kw):
    """Requests of many rows take the copied keys: their rows do not count against the span kernel's limit."""
    kw = dict(kw, qo_indptr=256, num_q_heads=32, num_kv_heads=8, q_row_stride=32 * 128, tile_stride=8 * 2304)
    size = B.pkv_quant_extend_workspace_size(_args(B, **kw))
    # the copies of the keys and values, and no more partials than the few rows' spans and the split blocks have
    copies = 2 * kw.get("total_kv", kw["batch"] * kw["max_seq_len"]) * 8 * 128 * 2
    assert size > copies
    if "kv_chunk" not in kw:
        assert size < copies + (1 << 28)
