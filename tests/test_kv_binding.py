"""The binding of the paged cache's calls, on the host: what it does around a library call (which is replaced here)."""
import types
import weakref

import pytest
import torch

import gemm_rtn_sym_gb300 as w4

SIZE = 5000


@pytest.mark.parametrize("without_raw_alloc", [True, False])
def test_the_workspace_lives_as_long_as_the_call(monkeypatch, without_raw_alloc):
    """Where the workspace is a tensor (another device than the current one, or no raw allocation), it is there until
    the library has been called: its memory may be another's as soon as it is gone."""
    bf16 = dict(dtype=torch.bfloat16)
    q, k, v = torch.zeros(2, 4, 16, **bf16), torch.zeros(3, 8, 2, 16, **bf16), torch.zeros(3, 8, 2, 16, **bf16)
    table, lens = torch.zeros(2, 2, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    made, empty = [], torch.empty

    def kept_track_of(*args, **kwargs):
        t = empty(*args, **kwargs)
        made.append((weakref.ref(t), t.data_ptr()))
        return t

    called = []

    def library(name, index, *args):
        scratch, size = args[-2:]
        called.append(name)
        assert size == SIZE
        alive = [ref() for ref, address in made if address == scratch]
        assert any(t is not None and t.numel() == SIZE for t in alive)

    # tensors on the host have device index −1
    monkeypatch.setattr(w4, "_device_index", lambda t, name: -1)
    monkeypatch.setattr(w4, "_current_device", lambda: 5)
    monkeypatch.setattr(w4, "_lib", types.SimpleNamespace(w4_attn_decode_workspace_bytes=lambda *a: SIZE))
    monkeypatch.setattr(w4, "_call", library)
    if without_raw_alloc:
        monkeypatch.setattr(w4, "_raw_alloc", None)
    monkeypatch.setattr(torch, "empty", kept_track_of)
    w4.w4_attn_decode(q, k, v, table, lens)
    assert called == ["w4_attn_decode"]


@pytest.mark.gpu
def test_a_workspace_that_is_a_tensor_gives_the_same_bits(cuda_lib, monkeypatch):
    from tests.kv_cases import AttentionCase

    case = AttentionCase([700, 33], [1, 2], 8, 2, 128, 16, seed=41)
    first = case.run(w4)
    monkeypatch.setattr(w4, "_raw_alloc", None)
    for _ in range(3):
        assert torch.equal(first.view(torch.int16), case.run(w4).view(torch.int16))
    case.check(first)
