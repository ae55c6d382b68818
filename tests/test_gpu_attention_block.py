"""The attention layer built from the 4-bit projections and the paged cache: each step against the same layer computed
from the cache's own contents in 64 bits, through prompts, verify passes, dropped drafts and ended requests."""
import numpy as np
import pytest
import torch

import gemm_rtn_sym_gb300 as w4
from gemm_rtn_sym_gb300 import attention_block, workloads as wl
from oracle import kv_oracle as KO
from tests.kv_cases import DEV, gpu, values

pytestmark = pytest.mark.gpu


def cached(block, name):
    """Keys or values [pages, page_size, heads, dim] that the cache stands for."""
    x = values(getattr(block, name))
    if block.scales:
        x = x * values(block.scales[name + "_scales"]).transpose(0, 2, 1)[..., None]
    return x


@pytest.mark.parametrize("format", [16, 8])
def test_steps(cuda_lib, format):
    hidden, Hq, H, D = 512, 8, 2, 128
    block = attention_block.AttentionBlock(hidden, Hq, H, D, 60, 16, 3, 300, format=format, seed=3)
    dense = [wl.random_bf16(s, wl.W_STD, seed=3 + i, device=DEV) for i, s in enumerate((((Hq + 2 * H) * D, hidden), (hidden, Hq * D)))]
    history = [[], [], []]
    lens = [0, 0, 0]
    for i, target in enumerate([[40, 3, 200], [45, 8, 205], [42, 4, 201], [43, 5, 202], [0, 6, 203], [17, 7, 190], [18, 8, 191]]):
        T = sum(max(0, b - a) for a, b in zip(lens, target))
        x = wl.random_bf16((T, hidden), 1.0, seed=100 + i, device=DEV)
        y = block.step(x, gpu(target))
        torch.cuda.synchronize()
        assert w4.w4_last_device_status() == 0 and block.lens.tolist() == target
        at = 0
        for b in range(3):
            history[b] = history[b][:target[b]]
            for row in values(x)[at:at + max(0, target[b] - lens[b])]:
                history[b].append(row)
            at += max(0, target[b] - lens[b])
        # Keys in the cache: the projection of each token's own input, turned by its position.  Errors: the 4-bit
        # weights are exact here (the same codes), the projection's bound 4e-3·Σ|ŵx|, two roundings to bf16 and, in
        # 8 bits, half a step of the row's largest value / 127.
        w_hat = [dequantised(*w4.w4_quantize_rtn(w)) for w in dense]
        k_all, v_all = cached(block, "k"), cached(block, "v")
        table = block.table.cpu().numpy()
        for b in range(3):
            for p in {0, target[b] // 2, target[b] - 1} & set(range(target[b])):
                inner = w_hat[0][Hq * D:(Hq + H) * D] @ history[b][p]
                size = np.abs(w_hat[0][Hq * D:(Hq + H) * D]) @ np.abs(history[b][p])
                turned = KO.rotate(inner.reshape(1, H, D), np.full((3, 1), p), block.cos.cpu().numpy(), block.sin.cpu().numpy(), block.sections)[0]
                got = k_all[table[b, p // 16], p % 16]
                bound = 2 * 4e-3 * size.max() + 2.0 ** -7 * np.abs(turned).max() + (np.abs(turned).max() / 127 if format == 8 else 0)
                assert np.abs(got - turned).max() <= bound
        if T:
            # The layer's output, from the cache's contents: attention in 64 bits of the step's own queries.
            qkv = w4.w4_gemm(x, *block.qkv)
            starts = np.concatenate([[0], np.cumsum([max(0, b - a) for a, b in zip(lens, target)])])
            position = np.concatenate([np.arange(a, max(a, b)) for a, b in zip(lens, target)])
            q = KO.rotate(values(qkv)[:, :Hq * D].reshape(T, Hq, D), np.tile(position, (3, 1)), block.cos.cpu().numpy(),
                          block.sin.cpu().numpy(), block.sections)
            q = KO.bf16(q.astype(np.float32)).astype(np.float64)
            ref, spread, largest = KO.attention(q, k_all, v_all, table, target, starts, D ** -0.5)
            off = KO.attention_bound(ref, spread, largest, D, max(target), format) + 2.0 ** -8 * spread  # and a rounding of q
            out = values(y)
            want = ref.reshape(T, -1) @ w_hat[1].T
            size = np.abs(ref).reshape(T, -1) @ np.abs(w_hat[1]).T
            bound = off.reshape(T, -1) @ np.abs(w_hat[1]).T + 4e-3 * size + 2.0 ** -8 * np.abs(want) + 1e-6
            assert (np.abs(out - want) <= bound).all()
        lens = target


def dequantised(packed, scales):
    from oracle import w4_oracle as O

    return np.asarray(O.dequantize_fp64(packed.cpu().numpy(), wl.bits(scales), packed.shape[1] * 2), np.float64)


def test_command(cuda_lib):
    assert attention_block.main(["--requests", "4", "--drafts", "3", "--steps", "2"]) == 0
    assert attention_block.main(["--requests", "3", "--drafts", "12", "--steps", "1", "--format", "8"]) == 0


def test_a_request_fills_its_last_page(cuda_lib):
    """`longest` need not be a multiple of the page: every position that the pages hold has its cosines and sines."""
    block = attention_block.AttentionBlock(512, 8, 2, 128, 60, 16, 2, 300, seed=3)
    block.step(wl.random_bf16((303, 512), 1.0, seed=1, device=DEV), gpu([303, 0]))
    x = wl.random_bf16((1, 512), 1.0, seed=2, device=DEV)
    block.step(x, gpu([304, 0]))
    torch.cuda.synchronize()
    assert w4.w4_last_device_status() == 0 and block.lens.tolist() == [304, 0]
    # the key of position 303, turned by its angles
    key = values(w4.w4_gemm(x, *block.qkv))[:, 8 * 128:10 * 128].reshape(1, 2, 128)
    frequency = 1e6 ** (-np.arange(64) * 2 / 128)
    angle = np.arange(304)[:, None] * frequency
    turned = KO.rotate(key, np.full((3, 1), 303), np.cos(angle), np.sin(angle), block.sections)[0]
    got = values(block.k)[int(block.table[0, 18]), 303 % 16]
    # one rounding to bf16, and the fp32 angles' cosines and sines (2⁻²⁴ of each) and products
    assert (np.abs(got - turned) <= 2.0 ** -8 * np.abs(turned) + 2.0 ** -21 * np.abs(key).max()).all()
