"""One attention layer of a decode server: 4-bit projections around the paged key-value cache.

    python -m gemm_rtn_sym_gb300.attention_block
    python -m gemm_rtn_sym_gb300.attention_block --format 8 --requests 16 --drafts 12

A step moves every request from its length to a target (``w4_kv_pages``), projects the new tokens with the fused 4-bit
qkv weights (``w4_gemm``), turns queries and keys and stores keys and values (``w4_kv_append``), attends over the pages
(``w4_attn_decode``) and projects back (``w4_gemm``).  The command runs prompts, decode steps and speculative-verify
passes whose rejected drafts are dropped, on seeded synthetic weights of the 7168×5120 layer class (40 query and 8
key-value heads of 128), and ends requests until every page is free again.  It times nothing.
"""
from __future__ import annotations

import argparse

import torch

from . import w4_attn_decode, w4_gemm, w4_kv_append, w4_kv_pages, w4_last_device_status, w4_quantize_rtn
from . import workloads as wl


class AttentionBlock:
    """The layer's weights, its cache of `pages` pages and the state of `requests` requests (all of length 0)."""

    def __init__(self, hidden: int, q_heads: int, kv_heads: int, head_dim: int, pages: int, page_size: int, requests: int,
                 longest: int, sections=(16, 24, 24), format: int = 16, device="cuda", seed: int = 1):
        self.heads = (q_heads, kv_heads, head_dim)
        self.page_size = page_size
        device = torch.device(device)
        qkv = wl.random_bf16(((q_heads + 2 * kv_heads) * head_dim, hidden), wl.W_STD, seed=seed, device=device)
        out = wl.random_bf16((hidden, q_heads * head_dim), wl.W_STD, seed=seed + 1, device=device)
        self.qkv, self.out = w4_quantize_rtn(qkv), w4_quantize_rtn(out)
        shape = (pages, page_size, kv_heads, head_dim)
        dtype = torch.bfloat16 if format == 16 else torch.int8
        self.k, self.v = (torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))
        self.scales = {}
        if format == 8:
            self.scales = {n: torch.zeros((pages, kv_heads, page_size), dtype=torch.bfloat16, device=device)
                           for n in ("k_scales", "v_scales")}
        self.table = torch.full((requests, -(-longest // page_size)), -1, dtype=torch.int32, device=device)
        self.free_pages = torch.arange(pages, dtype=torch.int32, device=device)
        self.free_range = torch.tensor([0, pages], dtype=torch.int64, device=device)
        self.lens = torch.zeros(requests, dtype=torch.int32, device=device)
        self.sections = sections
        rotary = 2 * sum(sections)
        frequency = 1e6 ** (-torch.arange(rotary // 2, dtype=torch.float64, device=device) * 2 / rotary)
        # A row for every position that the table's pages hold: a request may fill its last page.
        held = self.table.shape[1] * page_size
        angle = torch.arange(held, dtype=torch.float64, device=device)[:, None] * frequency
        self.cos, self.sin = angle.cos().float(), angle.sin().float()

    def step(self, x: torch.Tensor, target: torch.Tensor) -> torch.Tensor:
        """x bf16 [new tokens, hidden], request after request; target int32 [requests].  Returns bf16 [new tokens,
        hidden].  Requests may also shrink (rejected drafts) or end (target 0); those have no rows in x.  A request whose
        pages the pool does not have keeps its length (self.lens then differs from target), and its rows of the result
        mean nothing."""
        T = x.shape[0]
        self.lens, starts, slots, positions, self.free_range = w4_kv_pages(
            self.lens, target, self.table, self.free_pages, self.free_range, self.page_size, T)
        if T == 0:
            return x
        Hq, H, D = self.heads
        qkv = w4_gemm(x, *self.qkv)
        q, k, v = (qkv[:, a * D:b * D].unflatten(1, (b - a, D)) for a, b in ((0, Hq), (Hq, Hq + H), (Hq + H, Hq + 2 * H)))
        # Text: every axis has the token's own position.
        w4_kv_append(q, k, v, positions, self.cos, self.sin, self.k, self.v, slots, sections=self.sections, q_out=q,
                     **self.scales)
        attended = w4_attn_decode(q, self.k, self.v, self.table, self.lens, starts=starts, **self.scales)
        return w4_gemm(attended.flatten(1), *self.out)


def main(argv=None) -> int:
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--requests", type=int, default=8)
    p.add_argument("--drafts", type=int, default=6)
    p.add_argument("--steps", type=int, default=4)
    p.add_argument("--format", type=int, default=16, choices=[16, 8])
    a = p.parse_args(argv)
    torch.cuda.set_device(0)
    hidden, B, pages = 5120, a.requests, 64 * a.requests
    block = AttentionBlock(hidden, 40, 8, 128, pages, 16, B, 1024, format=a.format)
    lens = torch.tensor([17 + 31 * i % 400 for i in range(B)], dtype=torch.int32)
    dev = block.lens.device

    def step(what: str, target: torch.Tensor, rows: int, seed: int) -> None:
        y = block.step(wl.random_bf16((rows, hidden), 1.0, seed=seed, device=dev), target.to(dev))
        print(f"{what:8s} {rows:5d} rows -> {tuple(y.shape)}, lengths {block.lens.tolist()}, "
              f"free pages {int(block.free_range[1] - block.free_range[0])}")

    step("prompts", lens, int(lens.sum()), 1)
    for i in range(a.steps):
        lens = lens + a.drafts + 1
        step("verify", lens, B * (a.drafts + 1), 10 + i)
        lens = lens - torch.arange(B, dtype=torch.int32) % (a.drafts + 1)  # rejected drafts
        step("reject", lens, 0, 0)
        lens = lens + 1
        step("decode", lens, B, 20 + i)
    step("end", torch.zeros_like(lens), 0, 0)
    status = w4_last_device_status()
    if status != 0 or int(block.free_range[1] - block.free_range[0]) != pages:
        print(f"failed: device status {status}, free pages {block.free_range.tolist()} of {pages}")
        return 1
    print("ok: every page is free again")
    return 0


if __name__ == "__main__":
    raise SystemExit(main())
