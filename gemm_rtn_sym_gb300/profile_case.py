"""Run one small, self-checking case of a single kernel, for a profiler.

    python -m gemm_rtn_sym_gb300.profile_case quantize --workload outlier
    python -m gemm_rtn_sym_gb300.profile_case quantize_scaled --workload outlier
    python -m gemm_rtn_sym_gb300.profile_case gemm --workload outlier --M 8
    python -m gemm_rtn_sym_gb300.profile_case gemm --workload layer70b --matrix 2 --M 208
    python -m gemm_rtn_sym_gb300.profile_case grouped --workload layer27b --M 1
    python -m gemm_rtn_sym_gb300.profile_case grouped --workload layer27b --M 1 --group 128 --asym
    python -m gemm_rtn_sym_gb300.profile_case quantize --workload outlier --group 32 --asym
    python -m gemm_rtn_sym_gb300.profile_case gemm --workload outlier --M 8 --group 32 --asym
    python -m gemm_rtn_sym_gb300.profile_case gptq --workload ffn
    python -m gemm_rtn_sym_gb300.profile_case attention --heads 64,8,128 --requests 16 --length 4096 --M 13
    python -m gemm_rtn_sym_gb300.profile_case attention --heads 40,8,128 --requests 16 --length 8192 --M 1 --bits 8
    python -m gemm_rtn_sym_gb300.profile_case append --heads 40,8,128 --M 16001
    python -m gemm_rtn_sym_gb300.profile_case append --heads 40,8,128 --M 16001 --norms
    python -m gemm_rtn_sym_gb300.profile_case shared --heads 40,8,128 --requests 64 --length 16385 --M 1
    python -m gemm_rtn_sym_gb300.profile_case copy --heads 40,8,128 --M 2000

The inputs are the seeded synthetic matrices of ``workloads``.  For ``gemm`` the
weights are quantised first (one quantiser launch), then the matmul runs
``--launches`` times on the same inputs.  ``grouped`` quantises every matrix
of the workload and runs one grouped plan over all of them.  ``--group`` and
``--asym`` select the affine formats (w4_quantize_rtn / w4_quantize_rtn_asym at
that group size, w4_gemm_affine).  ``gptq`` factors a seeded synthetic
calibration statistic once and runs the GPTQ quantiser ``--launches`` times.
``attention`` runs w4_attn_decode for ``--requests`` requests of ``--length`` tokens, ``--M`` of them new, over a
paged cache of standard normal values; ``append`` turns and stores the rows of ``--M`` tokens (``--norms``: normalised
before).  ``shared`` runs w4_attn_decode_shared for ``--requests`` requests of 100 tokens of their own, ``--M`` of them
new, behind one prefix of ``--length`` tokens; ``copy`` copies ``--M`` pages.  The case checks the device status
word at the end and exits non-zero if any wait timed out.  It times nothing:
numbers taken under a profiler are not benchmark results.
"""
from __future__ import annotations

import argparse
import sys

import torch

from . import W4_PATH_AUTO, W4_PATH_SMALL_M, W4_PATH_TENSOR
from . import load, w4_gemm_ex, w4_gemm_grouped, w4_grouped_plan, w4_last_device_status, w4_quantize_rtn
from . import w4_attn_decode, w4_attn_decode_shared, w4_kv_append, w4_kv_append_norm, w4_kv_copy
from . import w4_gemm_affine, w4_gptq_factor, w4_gptq_quantize, w4_quantize_rtn_asym, w4_quantize_rtn_scaled
from . import workloads as wl

PATHS = {"auto": W4_PATH_AUTO, "small": W4_PATH_SMALL_M, "tensor": W4_PATH_TENSOR}


def cache_case(a, dev) -> str:
    """Runs a call on the paged cache; says what ran."""
    q_heads, kv_heads, dim = (int(x) for x in a.heads.split(","))
    page = 16
    each = -(-a.length // page) if a.kernel == "attention" else 0
    pages = a.requests * each if a.kernel == "attention" else -(-a.M // page)
    own = 100
    if a.kernel == "shared":
        each = -(-a.length // page)
        pages = each + a.requests * (-(-own // page) + 1)
    if a.kernel == "copy":
        pages = 2 * a.M
    g = torch.Generator(device=dev)
    g.manual_seed(1)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(torch.bfloat16)
    shape, k_scales, v_scales = (pages, page, kv_heads, dim), None, None
    if a.bits == 8:
        k, v = (torch.randint(-127, 128, shape, generator=g, device=dev, dtype=torch.int8) for _ in range(2))
        k_scales, v_scales = (torch.full((pages, kv_heads, page), 0.02, dtype=torch.bfloat16, device=dev) for _ in range(2))
    elif a.kernel != "append":
        k, v = normal(*shape), normal(*shape)
    else:
        k, v = (torch.zeros(shape, dtype=torch.bfloat16, device=dev) for _ in range(2))
    if a.kernel == "attention":
        q = normal(a.requests * a.M, q_heads, dim)
        table = torch.randperm(pages, generator=g, device=dev).to(torch.int32).view(a.requests, each)
        lens = torch.full((a.requests,), a.length, dtype=torch.int32, device=dev)
        for _ in range(a.launches):
            w4_attn_decode(q, k, v, table, lens, k_scales=k_scales, v_scales=v_scales)
        return f"attention {a.heads} {a.requests} requests of {a.length} tokens, {a.M} new, {a.bits} bits"
    if a.kernel == "shared":
        q = normal(a.requests * a.M, q_heads, dim)
        ids = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        first = a.length // page  # of a request's own pages, in its row of the table
        mine = ids[each:].view(a.requests, -1)
        table = torch.cat([ids[:first].expand(a.requests, first), mine], 1).contiguous()
        lens = torch.full((a.requests,), a.length + own, dtype=torch.int32, device=dev)
        groups = torch.tensor([0, a.requests], dtype=torch.int32, device=dev)
        prefix = torch.tensor([a.length], dtype=torch.int32, device=dev)
        for _ in range(a.launches):
            w4_attn_decode_shared(q, k, v, table, lens, groups, ids[None, :each], prefix, k_scales=k_scales, v_scales=v_scales)
        return f"shared {a.heads} {a.requests} requests behind {a.length} tokens, {a.M} new, {a.bits} bits"
    if a.kernel == "copy":
        ids = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        copies = torch.stack([ids[:a.M], ids[a.M:], torch.full_like(ids[:a.M], page)]).contiguous()
        for _ in range(a.launches):
            w4_kv_copy(k, v, copies, k_scales=k_scales, v_scales=v_scales)
        return f"copy {a.heads} {a.M} pages, {a.bits} bits"
    new_q, new_k, new_v = normal(a.M, q_heads, dim), normal(a.M, kv_heads, dim), normal(a.M, kv_heads, dim)
    angles = torch.outer(torch.arange(a.M, device=dev, dtype=torch.float32), 10000.0 ** (-torch.arange(dim // 2, device=dev) / (dim // 2)))
    positions = torch.arange(a.M, dtype=torch.int32, device=dev)
    slots = torch.arange(a.M, dtype=torch.int64, device=dev)
    if a.norms:
        weights = 1 + 0.1 * normal(2, dim)
        for _ in range(a.launches):
            w4_kv_append_norm(new_q, new_k, new_v, weights[0], weights[1], positions, angles.cos(), angles.sin(), k, v, slots,
                              k_scales=k_scales, v_scales=v_scales)
        return f"append {a.heads} {a.M} tokens with norms, {a.bits} bits"
    for _ in range(a.launches):
        w4_kv_append(new_q, new_k, new_v, positions, angles.cos(), angles.sin(), k, v, slots, k_scales=k_scales, v_scales=v_scales)
    return f"append {a.heads} {a.M} tokens, {a.bits} bits"


def main(argv=None) -> int:
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("kernel", choices=["quantize", "quantize_scaled", "gemm", "grouped", "gptq", "attention", "append", "shared", "copy"])
    p.add_argument("--workload", default="outlier", choices=sorted(wl.SHAPES))
    p.add_argument("--matrix", type=int, default=0, help="index into the workload's matrices")
    p.add_argument("--M", type=int, default=8, help="token rows of x (gemm), new tokens (of each request, attention)")
    p.add_argument("--heads", default="40,8,128", help="query heads, key-value heads, head_dim (attention, append)")
    p.add_argument("--requests", type=int, default=16)
    p.add_argument("--length", type=int, default=4096, help="tokens of each request in the cache")
    p.add_argument("--bits", type=int, default=16, choices=[8, 16])
    p.add_argument("--path", default="auto", choices=sorted(PATHS))
    p.add_argument("--launches", type=int, default=3)
    p.add_argument("--group", type=int, default=128, choices=[32, 64, 128])
    p.add_argument("--norms", action="store_true", help="append: queries and keys normalised before")
    p.add_argument("--asym", action="store_true", help="asymmetric codes with zero points")
    a = p.parse_args(argv)

    load()
    dev = torch.device("cuda", 0)
    torch.cuda.set_device(dev)
    if a.kernel in ("attention", "append", "shared", "copy"):
        what = cache_case(a, dev)
        torch.cuda.synchronize()
        status = w4_last_device_status(dev)
        print(f"{what}: {a.launches} launches, device status {status}")
        return 0 if status == 0 else 1
    if a.kernel == "grouped":
        problems, zeros = [], []
        for i, (N, K) in enumerate(wl.SHAPES[a.workload]):
            W = wl.weight(a.workload, i, device=dev)
            if a.asym:
                packed, scales, z = w4_quantize_rtn_asym(W, a.group)
                zeros.append(z)
            else:
                packed, scales = w4_quantize_rtn(W, a.group)
            del W
            x = wl.activations(a.workload, a.M, K, i, device=dev)
            problems.append((x, packed, scales, torch.empty((a.M, N), dtype=torch.bfloat16, device=dev)))
        plan = w4_grouped_plan(problems, group=a.group, zeros=zeros if a.asym else None)
        for _ in range(a.launches):
            w4_gemm_grouped(plan)
        torch.cuda.synchronize()
        status = w4_last_device_status(dev)
        print(f"grouped {a.workload} M={a.M}: {len(problems)} problems, {plan.items} items, "
              f"{a.launches} launches, device status {status}")
        return 0 if status == 0 else 1
    N, K = wl.SHAPES[a.workload][a.matrix]
    W = wl.weight(a.workload, a.matrix, device=dev)
    packed = torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((N, K // a.group), dtype=torch.bfloat16, device=dev)
    zeros = torch.empty((N, K // a.group), dtype=torch.int8, device=dev) if a.asym else None
    affine = a.asym or a.group != 128
    fmt = f" g{a.group} {'asym' if a.asym else 'sym'}"

    def quantize():
        if a.asym:
            w4_quantize_rtn_asym(W, a.group, packed=packed, scales=scales, zeros=zeros)
        else:
            w4_quantize_rtn(W, a.group, packed=packed, scales=scales)
    if a.kernel == "quantize":
        for _ in range(a.launches):
            quantize()
        what = f"quantize {a.workload}[{a.matrix}] {N}x{K}{fmt}"
    elif a.kernel == "gptq":
        H = wl.calibration_hessian(K, 4096, seed=wl.seed_for(a.workload, a.matrix, 4), device=dev)
        U = w4_gptq_factor(H)
        for _ in range(a.launches):
            w4_gptq_quantize(W, U, a.group, packed=packed, scales=scales)
        what = f"gptq {a.workload}[{a.matrix}] {N}x{K} g{a.group}"
    elif a.kernel == "quantize_scaled":
        s = wl.workload_channel_scales(a.workload, a.matrix, device=dev)
        for _ in range(a.launches):
            w4_quantize_rtn_scaled(W, s, packed=packed, scales=scales)
        what = f"quantize_scaled {a.workload}[{a.matrix}] {N}x{K}"
    else:
        quantize()
        del W
        x = wl.activations(a.workload, a.M, K, a.matrix, device=dev)
        y = torch.empty((a.M, N), dtype=torch.bfloat16, device=dev)
        for _ in range(a.launches):
            if affine:
                w4_gemm_affine(x, packed, scales, zeros, group=a.group, out=y, path=PATHS[a.path])
            else:
                w4_gemm_ex(x, packed, scales, out=y, path=PATHS[a.path])
        what = f"gemm {a.workload}[{a.matrix}] M={a.M} N={N} K={K} path={a.path}{fmt}"
    torch.cuda.synchronize()
    status = w4_last_device_status(dev)
    print(f"{what}: {a.launches} launches, device status {status}")
    return 0 if status == 0 else 1


if __name__ == "__main__":
    sys.exit(main())
