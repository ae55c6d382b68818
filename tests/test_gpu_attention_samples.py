"""The attention layer with shared prompts, norms and a pool that is moved together: each step against the same layer
computed from the cache's own contents in 64 bits, and the command."""
import numpy as np
import pytest
import torch

import gemm_rtn_sym_gb300 as w4
from gemm_rtn_sym_gb300 import attention_block, workloads as wl
from oracle import kv_oracle as KO
from oracle import kv_share_oracle as SO
from oracle import w4_oracle as O
from tests.kv_cases import DEV, gpu, values

pytestmark = pytest.mark.gpu


def dequantised(w):
    packed, scales = w4.w4_quantize_rtn(w)
    return np.asarray(O.dequantize_fp64(packed.cpu().numpy(), wl.bits(scales), packed.shape[1] * 2), np.float64)


@pytest.mark.parametrize("format", [16, 8])
def test_samples_of_prompts(cuda_lib, format):
    """Two prompts, the first with five samples and the second with two; samples grow, drop drafts, end and begin anew."""
    hidden, Hq, H, D, P = 512, 8, 2, 128, 16
    block = attention_block.AttentionBlock(hidden, Hq, H, D, 120, P, 9, 400, format=format, seed=3, norms=True, shared=True)
    w_out = dequantised(wl.random_bf16((hidden, Hq * D), wl.W_STD, seed=4, device=DEV))
    groups = (gpu([0, 6, 9]), torch.tensor([0, 6], device=DEV), gpu([230, 33]))
    weights = [values(w) for w in block.norms]
    lens = np.zeros(9, np.int64)

    def cached(name):
        x = values(getattr(block, name))
        return x * values(block.scales[name + "_scales"]).transpose(0, 2, 1)[..., None] if block.scales else x

    def step(target, seed, shared):
        nonlocal lens
        target = np.array(target)
        fresh = np.maximum(target - lens, 0)
        x = wl.random_bf16((int(fresh.sum()), hidden), 1.0, seed=seed, device=DEV)
        y = block.step(x, gpu(target), groups if shared else None)
        torch.cuda.synchronize()
        assert w4.w4_last_device_status() == 0 and block.lens.tolist() == target.tolist()
        position = np.concatenate([np.arange(a, max(a, b)) for a, b in zip(lens, target)])
        lens = target
        if not len(position):
            return
        # The step's own queries, normalised and turned, from the projection that the layer computes; attention and the
        # projection back in 64 bits.  Errors: a rounding of the queries, the attention's and the projection's bounds.
        qkv = values(w4.w4_gemm(x, *block.qkv))
        T = len(position)
        q = SO.norm(qkv[:, :Hq * D].reshape(T, Hq, D), weights[0], np.float64(np.float32(1e-6)), False)
        q = KO.rotate(q, np.tile(position, (3, 1)), block.cos.cpu().numpy(), block.sin.cpu().numpy(), block.sections)
        q = KO.bf16(q.astype(np.float32)).astype(np.float64)
        tokens = SO.token_rows(block.table.cpu().numpy(), lens, P)
        starts = np.concatenate([[0], np.cumsum(fresh)])
        k, v = (cached(n).reshape(-1, 1, H, D) for n in ("k", "v"))
        ref, spread, largest = KO.attention(q, k, v, tokens, lens, starts, D ** -0.5)
        # A query on the border of two bf16 values may have gone the other way: one step of each of a score's terms.
        moved = 2 * 2.0 ** -8 * largest
        off = KO.attention_bound(ref, spread, largest, D, int(lens.max()), format) + np.expm1(moved) * spread
        want = ref.reshape(T, -1) @ w_out.T
        bound = off.reshape(T, -1) @ np.abs(w_out).T + 4e-3 * (np.abs(ref).reshape(T, -1) @ np.abs(w_out).T) + 2.0 ** -8 * np.abs(want) + 1e-6
        assert (np.abs(values(y) - want) <= bound).all()
        # and the keys of the step's last token, normalised and turned
        at = tokens[fresh.nonzero()[0][-1], position[-1]]
        key = SO.norm(qkv[-1:, Hq * D:(Hq + H) * D].reshape(1, H, D), weights[1], 1e-6, False)
        key = KO.rotate(key, np.full((3, 1), position[-1]), block.cos.cpu().numpy(), block.sin.cpu().numpy(), block.sections)
        step_of = np.abs(key).max(-1, keepdims=True) * (2.0 ** -8 + (0.51 / 127 if format == 8 else 0))
        assert (np.abs(k[at] - key) <= step_of + 1e-5).all()

    def fork(source, keep):
        nonlocal lens
        block.fork(gpu(source), gpu(keep))
        torch.cuda.synchronize()
        lens = np.where(np.array(source) >= 0, keep, lens)
        assert w4.w4_last_device_status() == 0 and block.lens.tolist() == lens.tolist()

    step([230, 0, 0, 0, 0, 0, 33, 0, 0], 1, False)
    fork([-1, 0, 0, 0, 0, 0, -1, 6, 6], [0, 230, 230, 230, 230, 230, 0, 33, 33])
    step([230, 231, 231, 231, 231, 231, 33, 34, 34], 2, True)      # a token each
    step([230, 236, 236, 232, 236, 236, 33, 39, 39], 3, True)      # verify passes
    step([230, 233, 236, 232, 234, 0, 33, 36, 39], 4, True)        # rejected drafts; a sample ends
    fork([-1, -1, -1, -1, -1, 2, -1, -1, -1], [0, 0, 0, 0, 0, 235, 0, 0, 0])  # and begins anew, from another one
    block.compact()
    step([230, 246, 249, 245, 247, 248, 33, 49, 52], 5, True)      # 13 rows each
    step([230, 0, 250, 246, 0, 249, 33, 50, 0], 6, True)
    held = block.holders.cpu().numpy()
    assert (held > 0).sum() < sum(-(-int(n) // P) for n in lens) and held.max() == 4
    step([0] * 9, 7, True)
    assert int(block.free_range[1] - block.free_range[0]) == 120 and int(block.holders.sum()) == 0


def test_command(cuda_lib):
    assert attention_block.main(["--requests", "3", "--drafts", "3", "--steps", "2", "--samples", "4"]) == 0
    assert attention_block.main(["--requests", "2", "--drafts", "5", "--steps", "2", "--samples", "9", "--norms", "--format", "8"]) == 0
    assert attention_block.main(["--requests", "3", "--steps", "1", "--norms"]) == 0
