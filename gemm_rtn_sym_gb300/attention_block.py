"""One attention layer of a decode server: 4-bit projections around the paged key-value cache.

    python -m gemm_rtn_sym_gb300.attention_block
    python -m gemm_rtn_sym_gb300.attention_block --format 8 --requests 16 --drafts 12
    python -m gemm_rtn_sym_gb300.attention_block --samples 7 --norms

A step moves every request from its length to a target (``w4_kv_pages``), projects the new tokens with the fused 4-bit
qkv weights (``w4_gemm``), turns queries and keys and stores keys and values (``w4_kv_append``), attends over the pages
(``w4_attn_decode``) and projects back (``w4_gemm``).  The command runs prompts, decode steps and speculative-verify
passes whose rejected drafts are dropped, on seeded synthetic weights of the 7168×5120 layer class (40 query and 8
key-value heads of 128), and ends requests until every page is free again.  It times nothing.

With ``--samples`` every prompt is continued by several requests that share its pages (``w4_kv_fork``, ``w4_kv_copy``,
pages with holders), attention reads a prompt's keys and values once for all of them (``w4_attn_decode_shared``), and the
pool is moved together in between (``w4_kv_compact``).  With ``--norms`` queries and keys are normalised head by head on
their way into the cache (``w4_kv_append_norm``).
"""
from __future__ import annotations

import argparse

import torch

from . import w4_attn_decode, w4_attn_decode_shared, w4_gemm, w4_kv_append, w4_kv_append_norm, w4_kv_compact, w4_kv_copy
from . import w4_kv_fork, w4_kv_pages, w4_last_device_status, w4_quantize_rtn
from . import workloads as wl


class AttentionBlock:
    """The layer's weights, its cache of `pages` pages and the state of `requests` requests (all of length 0).  norms: queries
    and keys are normalised head by head.  shared: requests may share pages."""

    def __init__(self, hidden: int, q_heads: int, kv_heads: int, head_dim: int, pages: int, page_size: int, requests: int,
                 longest: int, sections=(16, 24, 24), format: int = 16, device="cuda", seed: int = 1, norms: bool = False,
                 shared: bool = False):
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
        self.holders = torch.zeros(pages, dtype=torch.int32, device=device) if shared else None
        self.norms = tuple(1 + wl.random_bf16((head_dim,), 0.1, seed=seed + 2 + i, device=device) for i in range(2)) if norms else None
        self.sections = sections
        rotary = 2 * sum(sections)
        frequency = 1e6 ** (-torch.arange(rotary // 2, dtype=torch.float64, device=device) * 2 / rotary)
        # A row for every position that the table's pages hold: a request may fill its last page.
        held = self.table.shape[1] * page_size
        angle = torch.arange(held, dtype=torch.float64, device=device)[:, None] * frequency
        self.cos, self.sin = angle.cos().float(), angle.sin().float()

    def fork(self, source: torch.Tensor, keep: torch.Tensor) -> None:
        """Requests of length 0 begin as the first keep[b] tokens of request source[b] (int32 [requests]; −1: none)."""
        self.lens, copies, self.free_range = w4_kv_fork(self.lens, source, keep, self.table, self.holders, self.free_pages,
                                                        self.free_range, self.page_size)
        w4_kv_copy(self.k, self.v, copies, **self.scales)

    def compact(self) -> None:
        """Moves the pages in use to the lowest ids."""
        self.table, self.holders, self.free_pages, self.free_range, copies = w4_kv_compact(
            self.lens, self.table, self.holders, self.free_range, self.page_size)
        w4_kv_copy(self.k, self.v, copies, **self.scales)

    def step(self, x: torch.Tensor, target: torch.Tensor, groups=None) -> torch.Tensor:
        """x bf16 [new tokens, hidden], request after request; target int32 [requests].  Returns bf16 [new tokens,
        hidden].  Requests may also shrink (rejected drafts) or end (target 0); those have no rows in x.  A request whose
        pages the pool does not have keeps its length (self.lens then differs from target), and its rows of the result
        mean nothing.  groups: (group_starts, requests whose pages are the groups' prefixes, prefix_lens) of requests that
        share prefixes."""
        T = x.shape[0]
        self.lens, starts, slots, positions, self.free_range = w4_kv_pages(
            self.lens, target, self.table, self.free_pages, self.free_range, self.page_size, T, holders=self.holders)
        if T == 0:
            return x
        Hq, H, D = self.heads
        qkv = w4_gemm(x, *self.qkv)
        q, k, v = (qkv[:, a * D:b * D].unflatten(1, (b - a, D)) for a, b in ((0, Hq), (Hq, Hq + H), (Hq + H, Hq + 2 * H)))
        # Text: every axis has the token's own position.
        if self.norms is None:
            w4_kv_append(q, k, v, positions, self.cos, self.sin, self.k, self.v, slots, sections=self.sections, q_out=q,
                         **self.scales)
        else:
            w4_kv_append_norm(q, k, v, *self.norms, positions, self.cos, self.sin, self.k, self.v, slots,
                              sections=self.sections, q_out=q, **self.scales)
        if groups is None:
            attended = w4_attn_decode(q, self.k, self.v, self.table, self.lens, starts=starts, **self.scales)
        else:
            group_starts, owners, prefix_lens = groups
            attended = w4_attn_decode_shared(q, self.k, self.v, self.table, self.lens, group_starts, self.table[owners],
                                             prefix_lens, starts=starts, **self.scales)
        return w4_gemm(attended.flatten(1), *self.out)


def main(argv=None) -> int:
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--requests", type=int, default=8)
    p.add_argument("--drafts", type=int, default=6)
    p.add_argument("--steps", type=int, default=4)
    p.add_argument("--format", type=int, default=16, choices=[16, 8])
    p.add_argument("--samples", type=int, default=0, help="requests that continue each prompt, over its pages")
    p.add_argument("--norms", action="store_true", help="normalise queries and keys head by head")
    a = p.parse_args(argv)
    torch.cuda.set_device(0)
    each = 1 + a.samples  # a prompt's request, which keeps its pages, and those that continue it
    hidden, B, pages = 5120, a.requests * each, 64 * a.requests * each
    block = AttentionBlock(hidden, 40, 8, 128, pages, 16, B, 1024, format=a.format, norms=a.norms, shared=a.samples > 0)
    lens = torch.tensor([17 + 31 * (i // each) % 400 if i % each == 0 else 0 for i in range(B)], dtype=torch.int32)
    dev = block.lens.device
    groups = None
    grows = torch.tensor([a.samples == 0 or i % each > 0 for i in range(B)], dtype=torch.int32)

    def step(what: str, target: torch.Tensor, rows: int, seed: int) -> None:
        y = block.step(wl.random_bf16((rows, hidden), 1.0, seed=seed, device=dev), target.to(dev), groups)
        print(f"{what:8s} {rows:5d} rows -> {tuple(y.shape)}, lengths {block.lens.tolist()}, "
              f"free pages {int(block.free_range[1] - block.free_range[0])}")

    step("prompts", lens, int(lens.sum()), 1)
    if a.samples:
        owners = torch.arange(0, B, each)
        source = torch.where(grows > 0, torch.arange(B) // each * each, -1).to(torch.int32)
        lens = lens[owners].repeat_interleave(each)
        block.fork(source.to(dev), lens.to(dev))
        groups = (torch.arange(0, B + 1, each, dtype=torch.int32, device=dev), owners.to(dev), lens[owners].to(dev))
    rows = int(grows.sum())
    for i in range(a.steps):
        lens = lens + grows * (a.drafts + 1)
        step("verify", lens, rows * (a.drafts + 1), 10 + i)
        lens = lens - grows * (torch.arange(B, dtype=torch.int32) % (a.drafts + 1))  # rejected drafts
        step("reject", lens, 0, 0)
        if a.samples:
            block.compact()
        lens = lens + grows
        step("decode", lens, rows, 20 + i)
    groups = None
    step("end", torch.zeros_like(lens), 0, 0)
    status = w4_last_device_status()
    if status != 0 or int(block.free_range[1] - block.free_range[0]) != pages:
        print(f"failed: device status {status}, free pages {block.free_range.tolist()} of {pages}")
        return 1
    print("ok: every page is free again")
    return 0


if __name__ == "__main__":
    raise SystemExit(main())
