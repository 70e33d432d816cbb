"""The 4-bit attention calls' sizes and refusals on the host, at the ends of what they allow."""
import pytest
import torch

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


def test_attention_refuses_wrong_workspaces_and_flags(B, monkeypatch):
    """A workspace with holes (fewer bytes in reach than it counts) and flags that are no int32 words do
    not reach the C call."""
    monkeypatch.setattr(B, "_device", lambda: -1)      # (host tensors stand in for the device's)
    calls = []

    def fn(args, ws, nbytes, err, stream):
        calls.append((ws, nbytes, err))
        return B.PKV_OK

    class Stream:
        cuda_stream = 0
    a = B.QuantArgs()
    a._dev = -1
    ws, err = torch.zeros(1024, dtype=torch.uint8), torch.zeros(1, dtype=torch.int32)
    for bad in (dict(workspace=ws[::2]), dict(workspace=ws.view(32, 32).T), dict(err_flags=err.long()),
                dict(err_flags=err.float()), dict(err_flags=torch.zeros((2, 2), dtype=torch.int32)[:, 0])):
        with pytest.raises(ValueError):
            B._quant_attend(fn, "pkv_quant_decode", a, **dict(dict(workspace=ws, err_flags=err, stream=Stream), **bad))
    assert not calls
    B._quant_attend(fn, "pkv_quant_decode", a, ws[256:], err, Stream)
    assert calls == [(ws.data_ptr() + 256, 768, err.data_ptr())]
