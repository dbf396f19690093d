"""8-bit latent pages in plain 64-bit form: the quantiser, pages built and taken apart by their layout.

A page of P tokens: codes [P][dl] (e4m3), rope keys [P][64] (bf16), scales [P] (fp32); a value is
its code or rope entry times its token's scale, a power of two."""
from __future__ import annotations

import math

import torch

ROPE = 64


def e4m3(y):
    """fp64 values to the nearest of e4m3 (|y| <= 448), ties to even: steps of 2^-9 below 2^-6, then an eighth of the power of two below."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def quantise(x, dl):
    """Rows x [n, dl + 64] -> (codes [n, dl] as the fp64 values of e4m3, rope [n, 64] as fp64 bf16 values, scale [n])."""
    y = x.double().cpu()
    size = torch.where(torch.isfinite(y), y.abs(), torch.zeros_like(y))
    top = torch.maximum(size[:, :dl].amax(1) / 448, size[:, dl:].amax(1) / 2.0 ** 64).clamp(min=2.0 ** -64)
    scale = torch.exp2(torch.ceil(torch.log2(top)))
    scale = torch.where(top <= scale / 2, scale / 2, scale)  # the logarithm of a power of two may round up
    c = y[:, :dl] / scale[:, None]
    codes = torch.where(torch.isfinite(c), e4m3(torch.where(torch.isfinite(c), c, torch.zeros_like(c))), torch.full_like(c, math.nan))
    return codes, (y[:, dl:] / scale[:, None]).to(torch.bfloat16).double(), scale


def parts(cache, dl):
    """Views (codes uint8 [N, P, dl], rope bf16 [N, P, 64], scales fp32 [N, P]) of pages [N, 1, P, dl + 132] (any page stride)."""
    N, _, P, _ = cache.shape
    flat = cache.as_strided((N, P * (dl + 132)), (cache.stride(0), 1), cache.storage_offset())
    rope = flat[:, P * dl:P * (dl + 128)].view(torch.bfloat16)
    scales = flat[:, P * (dl + 128):].view(torch.float32)
    return (flat[:, :P * dl].as_strided((N, P, dl), (cache.stride(0), dl, 1)),
            rope.as_strided((N, P, ROPE), (rope.stride(0), ROPE, 1)), scales)


def poisoned_pages(N, page, dl, gap=0, device="cuda"):
    """A view [N, 1, page, dl + 132] whose pages lie `gap` bytes apart; every code, rope entry and scale is NaN, gaps hold 0x7f."""
    size = page * (dl + 132)
    back = torch.full((N, size + gap), 0x7F, dtype=torch.uint8, device=device)
    cache = back.as_strided((N, 1, page, dl + 132), (size + gap, size, dl + 132, 1))
    parts(cache, dl)[2].fill_(math.nan)
    parts(cache, dl)[1].fill_(math.nan)
    return cache


def put(cache, dl, page, slots, x):
    """The quantised rows x into slots (a slice) of one page; the rows that the page then stands for, fp64 on the CPU."""
    codes, rope, scale = quantise(x, dl)
    c, r, s = parts(cache, dl)
    c[page, slots] = codes.float().to(torch.float8_e4m3fn).view(torch.uint8).to(cache.device)
    r[page, slots] = rope.to(torch.bfloat16).to(cache.device)
    s[page, slots] = scale.float().to(cache.device)
    return torch.cat([codes, rope], 1) * scale[:, None]


def values(cache, dl):
    """All rows [N, P, dl + 64] that the pages stand for, fp64 on the CPU."""
    c, r, s = parts(cache, dl)
    c = c.contiguous().view(torch.float8_e4m3fn).double().cpu()
    return torch.cat([c, r.double().cpu()], -1) * s.double().cpu()[..., None]


def paged8(lens, page, dl, seed, gap=0, spare=3, width_extra=0, sizes=None, device="cuda"):
    """Latents of the given lengths in random pages of a poisoned cache; (cache, block table, seq_lens, rows in fp64).
    sizes: factor of each token (default: powers of two from 1/4 to 2, a few tokens 0)."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    N = sum(need) + spare
    cache = poisoned_pages(N, page, dl, gap, device)
    perm = torch.randperm(N, generator=g).tolist()
    table = torch.full((len(lens), max(1, max(need)) + width_extra), -1, dtype=torch.int32)
    rows, at = [], 0
    for r, n in enumerate(lens):
        x = torch.randn(n, dl + ROPE, generator=g)
        f = torch.exp2(torch.randint(-2, 2, (n, 1), generator=g).float()) if sizes is None else sizes(n)
        if sizes is None and n > 20:
            f[torch.randint(0, n, (2,), generator=g)] = 0
        x = x * f
        rows.append(torch.empty(n, dl + ROPE, dtype=torch.float64))
        for j in range(need[r]):
            table[r, j] = perm[at]
            k = x[j * page:(j + 1) * page]
            rows[r][j * page:(j + 1) * page] = put(cache, dl, perm[at], slice(0, k.shape[0]), k)
            at += 1
    return cache, table.to(device), torch.tensor(lens, dtype=torch.int32, device=device), rows
