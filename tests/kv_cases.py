"""Inputs for the paged key-value cache's tests (host side only)."""
import numpy as np
import torch

from oracle import kv_oracle as KO

DEV = "cuda"


def values(t):
    return t.detach().double().cpu().numpy()


def gpu(a, dtype=torch.int32):
    return torch.tensor(np.asarray(a), dtype=dtype, device=DEV)


def bf16_tensor(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16)


def paged(pages, page_size, heads, dim, order, fill, seed):
    """Cache memory [pages, page_size, heads, dim] on the GPU, in pages of tokens
    ("token"), of heads ("head"), or keys and values side by side ("pair")."""
    def view(base):
        return base if order != "head" else base.transpose(1, 2)
    shape = (pages, page_size, heads, dim) if order != "head" else (pages, heads, page_size, dim)
    if order == "pair":
        both = torch.empty((pages, 2) + shape[1:], dtype=torch.bfloat16, device=DEV)
        k, v = both[:, 0], both[:, 1]
    else:
        k, v = (view(torch.empty(shape, dtype=torch.bfloat16, device=DEV)) for _ in range(2))
    if fill is None:
        k.copy_(bf16_tensor(k.shape, seed))
        v.copy_(bf16_tensor(v.shape, seed + 1))
    else:
        k.fill_(fill)
        v.fill_(fill)
    return k, v


def block_tables(lens, page_size, seed, spare=3, extra_columns=2):
    """(table int32 [B, width] with −1 where unused, number of pages)."""
    have = [-(-int(n) // page_size) for n in lens]
    pages = sum(have) + spare
    ids = np.random.default_rng(seed).permutation(pages)
    table = np.full((len(lens), max(have, default=0) + extra_columns), -1, np.int32)
    at = 0
    for b, h in enumerate(have):
        table[b, :h] = ids[at:at + h]
        at += h
    return table, pages


class AttentionCase:
    """A cache with NaN in every place no request owns, its queries and tables."""

    def __init__(self, lens, fresh, Hq, H, D, page_size, order="token", format=16, seed=0, std=1.0, garbage=float("nan")):
        self.lens, self.fresh, self.page_size, self.format = list(lens), list(fresh), page_size, format
        self.starts = np.concatenate([[0], np.cumsum(fresh)]).astype(np.int32)
        T = int(self.starts[-1])
        self.table, pages = block_tables(lens, page_size, seed)
        kd, vd = bf16_tensor((pages, page_size, H, D), seed + 1, std), bf16_tensor((pages, page_size, H, D), seed + 2)
        owned = np.zeros((pages, page_size), bool)
        for b, n in enumerate(self.lens):
            for p in range(int(n)):
                owned[self.table[b, p // page_size], p % page_size] = True
        free = ~torch.tensor(owned)
        self.q = bf16_tensor((T, Hq, D), seed + 3, 1.5)
        self.k_scales = self.v_scales = None
        self.k, self.v = paged(pages, page_size, H, D, order, 0.0, 0)
        if format == 16:
            kd[free], vd[free] = garbage, garbage
            self.k.copy_(kd)
            self.v.copy_(vd)
            self.kv, self.vv = values(kd), values(vd)
        else:
            out = []
            for x in (kd, vd):
                codes, scale = KO.rtn8(values(x))
                scale[~owned] = garbage
                scales = torch.tensor(scale, dtype=torch.bfloat16).transpose(1, 2).contiguous().to(DEV)
                out.append((torch.tensor(codes), scales, codes * scale[..., None]))
            shape = self.k.shape
            strides = self.k.stride()
            self.k = torch.empty_strided(shape, strides, dtype=torch.int8, device=DEV).copy_(out[0][0])
            self.v = torch.empty_strided(shape, strides, dtype=torch.int8, device=DEV).copy_(out[1][0])
            self.k_scales, self.v_scales = out[0][1], out[1][1]
            self.kv, self.vv = out[0][2], out[1][2]

    def run(self, w4, window=0, scale=None, uniform=False, table=None, lens=None, starts=None, **more):
        starts = None if uniform else gpu(self.starts if starts is None else starts)
        return w4.w4_attn_decode(self.q.to(DEV), self.k, self.v, gpu(self.table if table is None else table),
                                 gpu(self.lens if lens is None else lens), starts=starts, k_scales=self.k_scales,
                                 v_scales=self.v_scales, window=window, scale=scale, **more)

    def check(self, out, window=0, scale=None, rows=slice(None), columns=slice(None)):
        """The rows (and columns) of `out` against the reference, within its bound."""
        D = self.q.shape[2]
        ref, spread, largest = KO.attention(values(self.q), self.kv, self.vv, self.table, self.lens, self.starts,
                                            D ** -0.5 if scale is None else scale, window)
        bound = KO.attention_bound(ref, spread, largest, D, max(self.lens, default=1), self.format)
        got, ref, bound = (x[rows][..., columns] for x in (values(out), ref, bound))
        assert np.isfinite(got).all(), f"{np.count_nonzero(~np.isfinite(got))} values are not finite"
        worst = (np.abs(got - ref) / np.maximum(bound, 1e-300)).max() if got.size else 0.0
        assert worst <= 1.0, f"largest error is {worst:.3g} of the bound"
