"""The binding of the calls on shared pages: errors that come up at a launch end the call."""
import ctypes
import types

import pytest
import torch

import gemm_rtn_sym_gb300 as w4
from tests.kv_cases import DEV, gpu, paged

CALLS = {"w4_kv_pages_held": lambda t: w4.w4_kv_pages(t, t, t, t, t, 16, 4, holders=t),
         "w4_kv_fork": lambda t: w4.w4_kv_fork(t, t, t, t, t, t, t, 16),
         "w4_kv_compact": lambda t: w4.w4_kv_compact(t, t, t, t, 16),
         "w4_kv_copy": lambda t: w4.w4_kv_copy(t, t, t),
         "w4_kv_append_norm": lambda t: w4.w4_kv_append_norm(t, t, t, t, t, t, t, t, t, t, t),
         "w4_attn_decode_shared": lambda t: w4.w4_attn_decode_shared(t, t, t, t, t, t, t, t)}


@pytest.mark.parametrize("status", [w4.W4_ERR_CUDA, w4.W4_ERR_TIMEOUT])
@pytest.mark.parametrize("name", CALLS)
def test_an_error_at_a_launch_is_raised_and_the_call_is_not_made_again(monkeypatch, name, status):
    """A call of several kernels has changed something where a later one cannot be launched: made again, it would count
    holders down twice."""
    made = []
    fake = {n: lambda *a: status for n in ("kv_pages_held", "kv_fork", "kv_compact", "kv_copy", "kv_append_norm", "attn_decode_shared")}
    monkeypatch.setattr(w4, "_compiled", lambda: types.SimpleNamespace(**fake))
    monkeypatch.setattr(w4, "_call", lambda *a: made.append(a))
    with pytest.raises(w4.W4Error) as e:
        CALLS[name](torch.zeros(2, 2))
    assert e.value.status == status and name in str(e.value) and made == []


@pytest.mark.gpu
def test_a_launch_that_cuda_refuses(cuda_lib, monkeypatch):
    """Launches into a capture that has become invalid (a synchronisation of its stream) are refused on the host."""
    made, call = [], w4._call
    monkeypatch.setattr(w4, "_call", lambda *a: (made.append(a[0]), call(*a)))
    cudart = ctypes.CDLL("libcudart.so.13")
    k, v = paged(4, 16, 2, 64, "token", 1.0, 0)
    copies, side = gpu([[0], [1], [16]]), torch.cuda.Stream()
    table, ring, holders, lens = gpu([[-1, -1]] * 3), gpu([2, 0, 3, 1]), gpu([0] * 4), gpu([0] * 3)
    outs = dict(new_lens=gpu([0] * 3), starts=gpu([0] * 4), slots=gpu([0] * 5, torch.int64), positions=gpu([0] * 5),
                free_range_out=gpu([0, 0], torch.int64))
    free, target = gpu([0, 4], torch.int64), gpu([5, 0, 0])
    w4.w4_kv_copy(k, v, copies)
    torch.cuda.synchronize()
    stream, graph = ctypes.c_void_p(side.cuda_stream), ctypes.c_void_p()
    assert cudart.cudaStreamBeginCapture(stream, 2) == 0  # (no limits for other calls)
    try:
        assert cudart.cudaStreamSynchronize(stream) != 0
        with torch.cuda.stream(side):
            for f in (lambda: w4.w4_kv_copy(k, v, copies),
                      lambda: w4.w4_kv_pages(lens, target, table, ring, free, 16, 5, holders=holders, **outs)):
                with pytest.raises(w4.W4Error) as e:
                    f()
                assert e.value.status == w4.W4_ERR_CUDA
    finally:
        assert cudart.cudaStreamEndCapture(stream, ctypes.byref(graph)) != 0
        cudart.cudaGetLastError()
    assert made == []
    with torch.cuda.stream(side):  # the stream is as good as before
        got = w4.w4_kv_pages(lens, target, table, ring, free, 16, 5, holders=holders, **outs)
    torch.cuda.synchronize()
    assert got[0].tolist() == [5, 0, 0] and holders.tolist() == [0, 0, 1, 0] and w4.w4_last_device_status() == 0
