"""Rows of a shared batch whose own limit is not the prefix's (kda_latent_decode_shared): members that are shorter than what their group has
in common, empty entries among them, and what the decision to share makes of those."""
import math

import pytest
import torch

import kimi_delta_attention_varlen_gb300 as kda
from tests.latent_helpers import assert_attention, decode_reference
from tests.test_gpu_latent import paged_latents, poisoned, queries
from tests.test_gpu_latent_shared import run_both, run_shared, with_ballast

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
SCALE = 192 ** -0.5
I32 = dict(dtype=torch.int32, device=DEV)


def run_plain(q, cache, table, sl, dl, scale=SCALE, req=None):
    R, L, H, D = q.shape
    out, lse = poisoned(R, L, H, dl), torch.full((R, L, H), math.nan, device=DEV)
    ws = torch.empty(kda.kda_latent_decode_workspace_size(R, L, H, dl, D - dl), dtype=torch.uint8, device=DEV)
    kda.kda_latent_decode(q, cache, table, sl, out, ws, latent_dim=dl, scale=scale, req=req, lse=lse)
    torch.cuda.synchronize()
    assert kda.kda_prefill_workspace_status(ws) == 0
    return out, lse


def same_bits(a, b):
    return torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


def three_bf16(x):
    """A number as a sum of three bf16 values (its 24 leading bits)."""
    parts = []
    for _ in range(3):
        parts.append(float(torch.tensor(x).to(BF)))
        x -= parts[-1]
    return parts


# Rows that see at most 64 tokens take what the rounding of their weights leaves off, in whichever kernel.  Two tokens hold the weight: z = 0 and
# ln w with w next to (1 + 2^-8) / 2, halfway between two bf16 values, and latents a and -2 a, so that the output is about 2^-8.6 of a.  The
# output's rounding is then 2^-8 of that.  Weights in two parts are off by 2^-16 of themselves, the scores (fp32, below 1) and the approximate
# exponential by less: 2^-13 sum p |x| covers them eightfold.  A weight rounded once is off by 2^-8, the output by 2^-9 sum p |x|.
@pytest.mark.parametrize("dl", [512, 256])
@pytest.mark.parametrize("L,heads,lens", [(1, 16, [645, 2, 640, 3, 61, 64, 2, 1]), (31, 1, [94, 80, 33, 65]), (2, 16, [300, 65, 66, 3])])
def test_rows_that_see_few_tokens_of_a_long_prefix(L, heads, lens, dl):
    page, longest = 16, max(lens)
    cache, table, _, rows = paged_latents([longest], page, dl, seed=L)
    x = rows[0].clone()
    x[:, dl:] = 0
    x[2:, dl + 63] = -20.0
    x[1, :dl] = -2 * x[0, :dl]
    for h in range(heads):
        w = (1 + 2.0 ** -8) / 2 * (1 + (-1) ** h * (h + 1) * 2.0 ** -13)
        x[1, dl + 3 * h:dl + 3 * h + 3] = torch.tensor(three_bf16(math.log(w)), device=DEV)
    for j in range(-(-longest // page)):
        part = x[j * page:(j + 1) * page]
        cache[table[0, j].long(), 0, :part.shape[0]] = part
    q = torch.zeros(len(lens), L, heads, dl + 64, dtype=BF, device=DEV)
    q[..., dl + 63] = 1
    for h in range(heads):
        q[:, :, h, dl + 3 * h:dl + 3 * h + 3] = 1
    tables = table.expand(len(lens), -1).contiguous()
    ref = decode_reference(q, lambda r, n: x[:n], lens, 1.0, dl)
    few = torch.tensor([[1 < n - (L - 1 - t) <= 64 for t in range(L)] for n in lens])
    assert few.sum() >= 3
    for k, (out, lse) in enumerate(run_both(q, cache, tables, torch.tensor(lens, **I32), torch.tensor([0, len(lens)], **I32),
                                            torch.tensor([10 ** 6], **I32), dl, scale=1.0)):
        assert_attention(out, lse, ref, f"L {L} {'with ballast' if k else 'alone'}")
        want, mag = ref[0][few], ref[1][few]
        over = (out.double().cpu()[few] - want).abs() - (2.0 ** -8 * want.abs() + 2.0 ** -13 * mag)
        assert over.max() <= 0, f"{'with ballast' if k else 'alone'}: {float(over.max()):.3e} over its tolerance"


@pytest.mark.parametrize("dl", [512, 256])
@pytest.mark.parametrize("others", ["invalid", "empty", "short"])
def test_members_that_save_nothing_do_not_make_a_group_share(others, dl):
    """One member on 32,768 tokens among 63 that see 64 tokens or none: there is nothing to compute together, and the call is the plain one's bit
    for bit.  (With 64 such members it is not: the next test.)"""
    R, n, page, H = 64, 32768, 64, 32
    cache, table, _, rows = paged_latents([n], page, dl, seed=40)
    tables = table.expand(R, -1).contiguous()
    lens, pick = [n] + [64] * (R - 1), list(range(R))
    if others == "empty":
        lens[1:] = [0] * (R - 1)
    elif others == "invalid":
        pick[1:] = [-1] * (R - 1)
    q = queries(R, 1, H, dl + 64, seed=40)
    sl, req = torch.tensor(lens, **I32), torch.tensor(pick, **I32)
    got = run_shared(q, cache, tables, sl, torch.tensor([0, R], **I32), torch.tensor([n], **I32), dl, req=req)
    assert same_bits(got, run_plain(q, cache, tables, sl, dl, req=req))
    seen = [m if p >= 0 else 0 for m, p in zip(lens, pick)]
    some = [0, 1, 63]
    ref = decode_reference(q[some], lambda i, m: rows[0][:m], [seen[i] for i in some], SCALE, dl)
    assert_attention(got[0][some], got[1][some], ref, others)


@pytest.mark.parametrize("heads,shares", [(1, True), (32, True), (48, True), (64, False), (128, False)])
def test_which_kernels_take_a_batch_that_sharing_pays_for(heads, shares):
    """Compared with the plain call on the same batch, whose items are cut alike: bit for bit the same where entries have 64 rows and more, summed
    in another order where they have fewer."""
    R, n, page, dl = (600 if heads == 1 else 64), 32768, 64, 512
    cache, table, _, rows = paged_latents([n], page, dl, seed=41)
    tables, sl = table.expand(R, -1).contiguous(), torch.full((R,), n, **I32)
    q = queries(R, 1, heads, dl + 64, seed=41)
    got = run_shared(q, cache, tables, sl, torch.tensor([0, R], **I32), torch.tensor([n], **I32), dl)
    assert same_bits(got, run_plain(q, cache, tables, sl, dl)) != shares
    some = [0, R - 1]
    assert_attention(got[0][some], got[1][some], decode_reference(q[some], lambda i, m: rows[0][:m], [n, n], SCALE, dl))


@pytest.mark.parametrize("dl,heads,R,prefix,shares", [(512, 16, 4, 32768, False), (512, 8, 8, 16384, False), (512, 4, 4, 32768, False), (512, 16, 64, 8192, True),
                                                      (256, 8, 256, 512, True), (256, 32, 256, 1024, True), (256, 16, 4, 4096, False), (256, 4, 64, 4096, True)])
def test_sharing_follows_what_was_measured(dl, heads, R, prefix, shares):
    """Entries of few rows and latents of 256, on the side of the decision where they were measured to be faster: the plain call bit for bit, or
    summed in another order."""
    page = 64
    cache, table, _, rows = paged_latents([prefix + 37], page, dl, seed=42)
    tables, sl = table.expand(R, -1).contiguous(), torch.full((R,), prefix + 37, **I32)
    q = queries(R, 1, heads, dl + 64, seed=42)
    got = run_shared(q, cache, tables, sl, torch.tensor([0, R], **I32), torch.tensor([prefix], **I32), dl)
    assert same_bits(got, run_plain(q, cache, tables, sl, dl)) != shares
    some = [0, R - 1]
    assert_attention(got[0][some], got[1][some], decode_reference(q[some], lambda i, m: rows[0][:m], [prefix + 37] * 2, SCALE, dl))


@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_values_of_a_long_prefix_that_a_short_member_does_not_see(bad):
    """Sixty-three entries on 3.2 million tokens (the same 50 pages over and over) with a value that is not finite in every fiftieth page, and one of
    40 tokens before the first of them: its output stays finite, and no wait runs out over the others'."""
    page, pages, times, H, dl, R = 64, 50, 1000, 32, 512, 64
    cache, table, _, rows = paged_latents([page * pages], page, dl, seed=53)
    cache[table[0, 20].long(), 0, 5, [9, 300]] = bad
    tables = table[:, :pages].repeat(R, times).contiguous()
    n = [page * pages * times] * R
    n[17] = 40
    q = queries(R, 1, H, dl + 64, seed=53)
    out, lse = run_shared(q, cache, tables, torch.tensor(n, **I32), torch.tensor([0, R], **I32), torch.tensor([n[0]], **I32), dl)
    others = [r for r in range(R) if r != 17]
    assert not torch.isfinite(out[others][..., [9, 300]]).any()
    assert_attention(out[[17]], lse[[17]], decode_reference(q[[17]], lambda r, m: rows[0][:m], [40], SCALE, dl))


@pytest.mark.parametrize("groups", [[9000], [8000, 1000], [1] * 300 + [8500]])
def test_batches_of_many_thousand_entries(groups):
    """More entries than the plan keeps lengths of, of many lengths, in batches that sharing pays for."""
    page, dl, R = 64, 256, sum(groups)
    cache, table, _, rows = paged_latents([1000], page, dl, seed=43)
    tables = table.expand(R, -1).contiguous()
    lens = [(r * 37) % 1001 if r % 11 else 0 for r in range(R)]
    cu = torch.tensor([0] + groups, **I32).cumsum(0, dtype=torch.int32)
    q, sl = queries(R, 1, 1, dl + 64, seed=43), torch.tensor(lens, **I32)
    got = run_shared(q, cache, tables, sl, cu, torch.full((len(groups),), 700, **I32), dl)
    assert not same_bits(got, run_plain(q, cache, tables, sl, dl))
    some = list(range(40)) + list(range(8180, 8204)) + list(range(R - 40, R))
    assert_attention(got[0][some], got[1][some], decode_reference(q[some], lambda i, m: rows[0][:m], [lens[i] for i in some], SCALE, dl))
    assert (got[0][sl == 0] == 0).all() and (got[1][sl == 0] == -math.inf).all()
