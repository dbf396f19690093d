"""8-bit latent pages on the GPU: written (quantised bit for bit as the plain 64-bit form does), read back, attended to
(tests/latent_helpers.py: formulas and tolerances).  Whatever lies outside a request's tokens holds NaN throughout."""
import math

import pytest
import torch

import kimi_delta_attention_varlen_gb300 as kda
from kimi_delta_attention_varlen_gb300 import workloads as wl
from tests import latent8_helpers as h8
from tests.latent_helpers import LSE_ABS, OUT_REL, Z_REL, assert_attention, decode_reference
from tests.test_gpu_latent import paged_latents, poisoned, queries

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
SCALE = 192 ** -0.5


def same(a, b):
    """Equal, NaN where NaN."""
    return bool(((a == b) | (torch.isnan(a) & torch.isnan(b))).all())


# ---------------------------------------------------------------- append --

def tables(lens, page, spare, seed, width_extra=0):
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    N = sum(need) + spare
    perm = torch.randperm(N, generator=g).tolist()
    table = torch.full((len(lens), max(1, max(need)) + width_extra), -1, dtype=torch.int32)
    at = 0
    for r, k in enumerate(need):
        table[r, :k] = torch.tensor(perm[at:at + k], dtype=torch.int32)
        at += k
    return table, N


def run_append(x, cu, req, table, lens, cache, dl, page, itype=torch.int32, stream=None):
    t, sl = table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    pt = kda.page_table_descriptor(t, sl, torch.ones(cache.shape[0], dtype=torch.int32, device=DEV), page)
    kda.kda_latent_append8(x, torch.tensor(cu, dtype=torch.int32, device=DEV), torch.tensor(req, dtype=itype, device=DEV), pt, cache,
                           latent_dim=dl, stream=stream)
    torch.cuda.synchronize()


def check_append(x, cu, req, table, lens, page, dl, gap=0, itype=torch.int32):
    N = int(table.max()) + 3
    cache = h8.poisoned_pages(N, page, dl, gap)
    want = h8.poisoned_pages(N, page, dl, gap, "cpu")
    for i, r in enumerate(req):
        if not 0 <= r < len(lens):
            continue
        n = cu[i + 1] - cu[i]
        for e in range(n):
            pos, tok = lens[r] - n + e, cu[i] + e
            if pos < 0 or tok >= x.shape[0]:
                continue
            p = int(table[r, pos // page]) if pos // page < table.shape[1] else -1
            if 0 <= p < N:
                h8.put(want, dl, p, slice(pos % page, pos % page + 1), x[tok:tok + 1].cpu())
    run_append(x, cu, req, table, lens, cache, dl, page, itype)
    size = page * (dl + 132)
    got = cache.as_strided((N, size + gap), (size + gap, 1)).cpu()
    ref = want.as_strided((N, size + gap), (size + gap, 1))
    assert torch.equal(got[:, size:], ref[:, size:]), "gaps"
    gc, gr, gs = h8.parts(cache, dl)
    wc, wr, ws = h8.parts(want, dl)
    assert same(gc.contiguous().view(torch.float8_e4m3fn).float().cpu(), wc.contiguous().view(torch.float8_e4m3fn).float())
    assert same(gr.float().cpu(), wr.float()) and same(gs.cpu(), ws)


@pytest.mark.parametrize("dl", [512, 256])
@pytest.mark.parametrize("page", [8, 48, 64, 200])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_append_prompts_and_single_tokens(dl, page, dtype):
    lens = [1, 70, 333, 0, 64, 200]
    new = [1, 70, 1, 0, 3, 129]
    table, N = tables(lens, page, 2, seed=page + dl)
    g = wl.generator(page, DEV)
    T = sum(new)
    x = torch.randn(T, dl + 64, generator=g, device=DEV) * torch.exp2(torch.randint(-30, 30, (T, 1), generator=g, device=DEV).float())
    order = [4, 0, 5, 2, 3, 1]
    cu = [0]
    for r in order:
        cu.append(cu[-1] + new[r])
    check_append(x.to(dtype), cu, order, table, lens, page, dl, gap=32 if page == 48 else 0, itype=torch.int64 if page == 8 else torch.int32)


@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_append_values_at_the_edges(dtype):
    """Ties, the largest of a unit, subnormal codes, zeros, huge and tiny values, NaN and infinities, rope keys that set the unit."""
    dl = 256
    x = torch.zeros(16, dl + 64)
    x[0, :8] = torch.tensor([448.0, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, -2.0 ** -9, 0.0, 464.0 / 2])
    x[1, :3] = torch.tensor([450.0, 1.0, -1.0])
    x[2, 0], x[2, 300] = 1e-30, 3.0
    x[3, 0], x[3, 300] = 1.0, 2.0 ** 70
    x[4, 0], x[4, 300] = 1.0, 1.5 * 2.0 ** 64
    x[5, :4] = torch.tensor([math.nan, math.inf, -math.inf, 2.0])
    x[6, 256:260] = torch.tensor([math.nan, math.inf, -math.inf, 2.0])
    x[7, 0] = 3e38
    x[8, 0], x[8, 1] = 2.0 ** 127, 1.0
    x[9, 0] = 1e-38
    x[10, :] = -0.0
    x[11, :] = torch.linspace(-1, 1, dl + 64)
    x[12, :] = torch.exp2(torch.linspace(-40, 8, dl + 64))
    x[13, 0] = 1.75 * 2.0 ** -56  # exactly 448 units of 2^-64
    x[14, 0] = 1.875 * 2.0 ** -56
    x[15, 256] = 2.0 ** 64
    table, _ = tables([16], 8, 1, seed=1)
    check_append(x.to(dtype).to(DEV), [0, 16], [0], table, [16], 8, dl)


def test_append_ignores_what_it_must():
    """Invalid requests, negative positions, pages outside the pool, offsets beyond the rows and rows outside all entries."""
    dl, page, lens = 512, 16, [20, 5, 40]
    table, N = tables(lens, page, 2, seed=3)
    table[2, 1] = N + 100
    x = torch.randn(60, dl + 64, generator=wl.generator(4, DEV), device=DEV).to(BF)
    # entry 0 invalid; entry 1 has more rows than its request tokens; entry 3 ends behind the rows given
    check_append(x, [2, 6, 14, 44, 70], [-1, 1, 2, 7], table, lens, page, dl)
    check_append(x, [0, 10, 70], [3, 0], table, lens, page, dl)


@pytest.mark.parametrize("stride", [584, 1152, 2112])
def test_append_takes_a_slice_of_a_projection(stride):
    x = torch.randn(37, stride, generator=wl.generator(stride, DEV), device=DEV).to(BF)[:, 8:584]
    table, _ = tables([37], 64, 2, seed=5)
    check_append(x, [0, 37], [0], table, [37], 64, 512)


# ------------------------------------------------------------------- read --

def read_back(cache, table, lens, page, dl, cu, req, first, total, itype=torch.int32, gap=0, stream=None):
    t = table.to(DEV)
    pt = kda.page_table_descriptor(t, torch.tensor(lens, dtype=torch.int32, device=DEV),
                                   torch.ones(cache.shape[0], dtype=torch.int32, device=DEV), page)
    back = torch.full((total + 2, dl + 64 + gap), 7.0, dtype=BF, device=DEV)
    out = back[1:total + 1, :dl + 64]
    f = None if first is None else torch.tensor(first, dtype=torch.int32, device=DEV)
    kda.kda_latent_read(cache, torch.tensor(cu, dtype=torch.int32, device=DEV), torch.tensor(req, dtype=itype, device=DEV), pt, out,
                        latent_dim=dl, first=f, stream=stream)
    torch.cuda.synchronize()
    assert (back[0] == 7).all() and (back[-1] == 7).all() and (back[:, dl + 64:] == 7).all()
    return out


@pytest.mark.parametrize("dl", [512, 256])
@pytest.mark.parametrize("page", [8, 48, 64, 200])
@pytest.mark.parametrize("eight", [True, False])
def test_read_rows(dl, page, eight):
    lens = [1, 70, 333, 0, 64, 200]
    if eight:
        cache, table, _, rows = h8.paged8(lens, page, dl, seed=page, gap=16)
    else:
        cache, table, _, rows = paged_latents(lens, page, dl, seed=page, gap=24)
        rows = [r.double().cpu() for r in rows]
    # whole requests, parts, one request twice, tokens behind the end, before the first, invalid requests, an empty entry
    req, first, n = [2, 0, 5, 5, 1, 4, 9, -1, 3, 2], [0, 0, 100, 50, 60, -3, 0, 0, 0, 332], [333, 1, 100, 7, 30, 9, 4, 3, 2, 0]
    cu = [5]
    for k in n:
        cu.append(cu[-1] + k)
    total = cu[-1] + 6
    out = read_back(cache, table, lens, page, dl, cu, req, first, total, torch.int64 if page == 8 else torch.int32, gap=8)
    want = torch.zeros(total, dl + 64, dtype=torch.float64)
    want[:5], want[cu[-1]:] = 7, 7
    for i, (r, f) in enumerate(zip(req, first)):
        for e in range(n[i]):
            if 0 <= r < len(lens) and 0 <= f + e < lens[r]:
                want[cu[i] + e] = rows[r][f + e]
    assert torch.equal(out.double().cpu(), want)  # every 8-bit value is a bf16 number
    out = read_back(cache, table, lens, page, dl, [0, 333, 340], [2, 4], None, 338)  # the last entry ends behind the rows
    assert torch.equal(out[:333].double().cpu(), rows[2]) and torch.equal(out[333:].double().cpu(), rows[4][:5])


def test_read_zeros_where_a_page_is_invalid_and_passes_nan_on():
    dl, page = 256, 16
    cache, table, _, rows = h8.paged8([50], page, dl, seed=9)
    h8.parts(cache, dl)[0][int(table[0, 0]), 3, 7] = 0x7F
    table = table.cpu()
    table[0, 1], table[0, 2] = cache.shape[0], -5
    out = read_back(cache, table, [50], page, dl, [0, 50], [0], None, 50)
    assert (out[16:48] == 0).all() and torch.isnan(out[3, 7]) and int(torch.isnan(out).sum()) == 1
    assert torch.equal(out[48:].double().cpu(), rows[0][48:])


def test_written_rows_come_back_within_their_rounding():
    """|x - back| <= half a step: 2^-4 of the value, or half of 2^-9 units; the rope key half a bf16 step."""
    dl, page, lens = 512, 64, [777]
    table, N = tables(lens, page, 1, seed=2)
    x = torch.randn(777, dl + 64, generator=wl.generator(8, DEV), device=DEV).to(BF)
    cache = h8.poisoned_pages(N, page, dl)
    run_append(x, [0, 777], [0], table, lens, cache, dl, page)
    out = read_back(cache, table, lens, page, dl, [0, 777], [0], None, 777)
    unit = h8.quantise(x, dl)[2].to(DEV)[:, None]
    d = (out.double() - x.double()).abs()
    assert (d[:, :dl] <= torch.maximum(2.0 ** -4 * x[:, :dl].double().abs(), 2.0 ** -10 * unit)).all()
    assert torch.equal(out[:, dl:], x[:, dl:])  # a power of two away: the same bf16 digits


@pytest.mark.parametrize("rows", [1, 3, 40])
def test_lists_of_which_most_entries_have_no_rows(rows):
    """5,000 entries, of which a few have rows: a step of a server that lists all of its requests."""
    dl, page, R = 256, 16, 5000
    g = torch.Generator().manual_seed(rows)
    has = sorted(torch.randperm(R, generator=g)[:60].tolist())
    lens = [0] * R
    for r in has:
        lens[r] = rows
    cache, table, sl, data = h8.paged8(lens, page, dl, seed=3)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    out = read_back(cache, table, lens, page, dl, cu, list(range(R)), None, cu[-1])
    assert torch.equal(out.double().cpu(), torch.cat([data[r] for r in has]))
    x = torch.randn(cu[-1], dl + 64, generator=wl.generator(rows, DEV), device=DEV).to(BF)
    run_append(x, cu, list(range(R)), table, lens, cache, dl, page)
    c, rope, scale = h8.quantise(x, dl)
    out = read_back(cache, table, lens, page, dl, cu, list(range(R)), None, cu[-1])
    assert torch.equal(out.double().cpu(), torch.cat([c, rope], 1) * scale[:, None])


# ----------------------------------------------------------------- decode --

def run_decode8(q, cache, table, lens, dl, scale, req=None, stream=None, lse=True):
    R, L, H, _ = q.shape
    out = poisoned(R, L, H, dl)
    ls = torch.full((R, L, H), math.nan, device=DEV) if lse else None
    ws = torch.empty(kda.kda_latent_decode8_workspace_size(R, L, H, dl, 64), dtype=torch.uint8, device=DEV)
    ws.fill_(0xA5)
    torch.cuda.synchronize()
    kda.kda_latent_decode8(q, cache, table, lens, out, ws, latent_dim=dl, scale=scale, req=req, lse=ls, stream=stream)
    torch.cuda.synchronize()
    assert kda.kda_prefill_workspace_status(ws) == 0
    return out, ls


def check_decode8(lens, page, dl, heads, L=1, seed=0, scale=SCALE, **kw):
    cache, table, sl, rows = h8.paged8(lens, page, dl, seed=seed, **kw)
    q = queries(len(lens), L, heads, dl + 64, seed=seed)
    out, lse = run_decode8(q, cache, table, sl, dl, scale)
    assert_attention(out, lse, decode_reference(q, lambda r, n: rows[r][:n], lens, scale, dl), f"page {page} dl {dl} heads {heads} L {L}")


@pytest.mark.parametrize("dl", [512, 256])
@pytest.mark.parametrize("page", [8, 16, 48, 64, 128, 200])
def test_decode_lengths_and_pages(page, dl):
    check_decode8([0, 1, 2, 63, 64, 65, 127, 128, 129, 191, 193, 500, 1000, page, page + 1, 3 * page - 1], page, dl, 32, seed=page + dl)


@pytest.mark.parametrize("heads", [1, 2, 5, 8, 16, 17, 31, 32, 33, 48, 64, 100, 128, 192])
def test_decode_heads(heads):
    check_decode8([1, 70, 333], 32, 512, heads, seed=heads, gap=48)
    check_decode8([200, 65], 16, 256, heads, seed=heads)


@pytest.mark.parametrize("L,heads", [(2, 32), (3, 16), (4, 128), (5, 8), (7, 1), (70, 2)])
def test_decode_draft_tokens_are_causal(L, heads):
    check_decode8([0, 1, L - 1, L, L + 1, 64 + L, 129, 700], 16, 512, heads, L=L, seed=L, width_extra=3)


@pytest.mark.parametrize("n,L", [(40, 3), (130, 5), (66, 4), (20000, 6), (64, 70), (131, 70)])
def test_decode_nan_reaches_only_draft_tokens_that_see_it(n, L):
    cache, table, sl, rows = h8.paged8([n], 16, 512, seed=n + L)
    q = queries(1, L, 8, 576, seed=L)
    tok = n - 2  # the query tokens from L - 2 on see it
    ref = decode_reference(q, lambda r, k: rows[r][:k], [n], SCALE, 512)
    h8.parts(cache, 512)[0][int(table[0, tok // 16]), tok % 16, [9, 300, 511]] = 0x7F
    out, lse = run_decode8(q, cache, table, sl, 512, SCALE)
    assert torch.isnan(out[0, L - 2:]).all() and torch.isnan(lse[0, L - 2:]).all()
    assert_attention(out[:, :L - 2], lse[:, :L - 2], [x[:, :L - 2] for x in ref], f"n {n} L {L}")


@pytest.mark.parametrize("lens,heads", [([40000], 32), ([9999, 3, 25000], 16), ([6400] * 5, 64), ([20000, 1], 128)])
def test_decode_long_contexts(lens, heads):
    check_decode8(lens, 64, 512, heads, seed=heads)


def test_decode_many_requests_of_all_lengths():
    g = torch.Generator().manual_seed(5)
    check_decode8(torch.randint(0, 400, (700,), generator=g).tolist(), 16, 256, 8, seed=5)


@pytest.mark.parametrize("itype", [torch.int32, torch.int64])
def test_decode_picks_requests_and_leaves_invalid_ones_empty(itype):
    lens = [100, 0, 65, 900, 5]
    cache, table, sl, rows = h8.paged8(lens, 64, 512, seed=11)
    req = [3, -1, 0, 5, 3, 2]
    q = queries(6, 2, 16, 576, seed=3)
    out, lse = run_decode8(q, cache, table, sl, 512, SCALE, req=torch.tensor(req, dtype=itype, device=DEV))
    n = [lens[r] if 0 <= r < 5 else 0 for r in req]
    assert_attention(out, lse, decode_reference(q, lambda i, k: rows[req[i]][:k] if n[i] else rows[0][:0], n, SCALE, 512))
    assert (out[1] == 0).all() and (lse[3] == -math.inf).all()


def test_decode_invalid_pages_read_as_zero_rows():
    lens = [200, 130]
    cache, table, sl, rows = h8.paged8(lens, 32, 512, seed=21)
    table[0, 2], table[1, 0] = cache.shape[0], -7
    rows[0][64:96], rows[1][:32] = 0, 0
    q = queries(2, 1, 32, 576, seed=4)
    out, lse = run_decode8(q, cache, table, sl, 512, SCALE)
    assert_attention(out, lse, decode_reference(q, lambda r, n: rows[r][:n], lens, SCALE, 512))


@pytest.mark.parametrize("sizes", [-20, 0, 30])
@pytest.mark.parametrize("scale", [1e-6, SCALE, 3.0])
def test_decode_scales_and_sizes_of_latents(sizes, scale):
    """Units from 2^-40 to 2^50, of both kinds in one request: the weights of tokens with large values and with small ones."""
    g = torch.Generator().manual_seed(6)
    cache, table, sl, rows = h8.paged8([300, 900], 64, 512, seed=13,
                                       sizes=lambda n: torch.exp2(torch.randint(sizes - 6, sizes + 3, (n, 1), generator=g).float()))
    q = (queries(2, 1, 32, 576, seed=9).float() * 2.0 ** -sizes).to(BF)
    out, lse = run_decode8(q, cache, table, sl, 512, scale)
    assert_attention(out, lse, decode_reference(q, lambda r, n: rows[r][:n], [300, 900], scale, 512))


def test_decode_a_token_of_tiny_values_that_holds_the_weight():
    """Half of the weight on a token whose unit is 2^-60 of the others': its share of the sum is not lost with its values."""
    dl = 256
    x = torch.randn(100, dl + 64, generator=torch.Generator().manual_seed(1))
    x[:, dl:] = 0
    x[7, :dl] = 0
    x[7, 0] = 2.0 ** -40
    cache = h8.poisoned_pages(3, 64, dl)
    rows = torch.cat([h8.put(cache, dl, 1, slice(0, 64), x[:64]), h8.put(cache, dl, 0, slice(0, 36), x[64:])])
    table, sl = torch.tensor([[1, 0]], dtype=torch.int32, device=DEV), torch.tensor([100], dtype=torch.int32, device=DEV)
    q = torch.zeros(1, 1, 8, dl + 64, device=DEV, dtype=BF)  # all scores 0: token 7 has 1 / 100
    q[0, 0, 4:, 0] = 1.0
    out, lse = run_decode8(q, cache, table, sl, dl, 1.0)
    assert_attention(out, lse, decode_reference(q, lambda r, n: rows[:n], [100], 1.0, dl))


def test_decode_sink_and_a_long_flat_rest():
    """One token with half of the weight, 60,000 that share the other half: none of the small weights is lost."""
    dl, n = 256, 60000
    x = torch.zeros(n, dl + 64)
    x[:, 0] = 1.0
    x[:, 1] = torch.randint(0, 2, (n,), generator=torch.Generator().manual_seed(2)) * 0.5 + 0.5
    x[0, :] = 0
    x[0, dl] = math.log(n) * 8
    x[0, 5] = 1.0
    cache = h8.poisoned_pages(-(-n // 64), 64, dl)
    rows = torch.cat([h8.put(cache, dl, j, slice(0, min(64, n - 64 * j)), x[64 * j:64 * j + 64]) for j in range(cache.shape[0])])
    table, sl = torch.arange(cache.shape[0], dtype=torch.int32, device=DEV)[None], torch.tensor([n], dtype=torch.int32, device=DEV)
    q = torch.zeros(1, 1, 4, dl + 64, device=DEV, dtype=BF)
    q[..., dl] = 0.125
    out, lse = run_decode8(q, cache, table, sl, dl, 1.0)
    assert_attention(out, lse, decode_reference(q, lambda r, k: rows[:k], [n], 1.0, dl))


@pytest.mark.parametrize("dl", [512, 256])
def test_decode_millions_of_tokens(dl):
    """One request of 3.2 million tokens, whose table lists the same 50 pages over and over: 20,000 tokens and more to a CTA, so that
    the accumulator is set aside.  Each row's weight counts as often as it is listed."""
    page, pages, times = 64, 50, 1000
    cache, table, _, rows = h8.paged8([page * pages], page, dl, seed=51)
    n = page * pages * times - 17
    table = table[:, :pages].repeat(1, times).contiguous()
    q = queries(1, 1, 32, dl + 64, seed=51)
    out, lse = run_decode8(q, cache, table, torch.tensor([n], dtype=torch.int32, device=DEV), dl, SCALE)
    x = rows[0]
    count = torch.full((page * pages,), float(times), dtype=torch.float64)
    count[-17:] -= 1
    z = q[0, 0].double().cpu() @ x.T * SCALE + count.log()
    want_lse = torch.logsumexp(z, -1)
    p = torch.softmax(z, -1)
    bound = (q[0, 0].double().cpu().abs() @ x.abs().T * SCALE).amax(-1)
    assert_attention(out[0, 0], lse[0, 0], (p @ x[:, :dl], p @ x[:, :dl].abs(), want_lse, bound))


@pytest.mark.parametrize("heads,fall", [(4, False), (32, False), (32, True)])
def test_decode_scores_that_rise_or_fall_over_millions_of_tokens(heads, fall):
    """Scores 40 apart over 4.2 million tokens of two units, 27,000 tokens to a CTA: both maxima move again and again, and what was set
    aside is brought to the new ones."""
    dl, page, N = 256, 64, 65536
    n = N * page - 5
    cache = torch.empty(N, 1, page, dl + 132, dtype=torch.uint8, device=DEV)
    g = wl.generator(61, DEV)
    codes, rope, scales = h8.parts(cache, dl)
    one = torch.randn(97, dl, generator=g, device=DEV).clamp(-448, 448).to(torch.float8_e4m3fn)  # tokens' codes, in turn
    t = torch.arange(N * page, device=DEV)
    codes.copy_(one.view(torch.uint8)[t % 97].view(N, page, dl))
    unit = torch.where(t % 3 == 0, 2.0 ** -7, 1.0)
    rope.zero_()
    level = 40.0 * t / n
    rope[..., 0] = ((40 - level if fall else level) / unit).to(BF).view(N, page)  # (rounded: the score is what the page holds)
    scales.copy_(unit.view(N, page))
    table = torch.arange(N, dtype=torch.int32, device=DEV)[None]
    q = torch.zeros(1, 1, heads, dl + 64, dtype=BF, device=DEV)
    q[..., dl] = 1
    q[0, 0, 1:, 3] = 0.25
    out, lse = run_decode8(q, cache, table, torch.tensor([n], dtype=torch.int32, device=DEV), dl, 1.0)
    u = unit[:n].double()
    r0 = rope[..., 0].reshape(-1)[:n].double() * u
    c3 = one[:, 3].double()[t[:n] % 97] * u
    want, mag, want_lse, bound = [], [], [], []
    for h in (0, 1):
        z = r0 + (0.25 * c3 if h else 0)
        p = torch.softmax(z, 0)
        by = torch.zeros(97, dtype=torch.float64, device=DEV).index_add_(0, t[:n] % 97, p * u)
        want.append(by @ one.double())
        mag.append(by @ one.double().abs())
        want_lse.append(torch.logsumexp(z, 0))
        bound.append((r0.abs() + 0.25 * c3.abs()).max())
    ref = [torch.stack(x).cpu() for x in (want, mag, want_lse, bound)]
    assert_attention(out[0, 0, :2], lse[0, 0, :2], ref, f"heads {heads} fall {fall}")
    assert torch.equal(out[0, 0, 1].expand(heads - 1, -1), out[0, 0, 1:]) and torch.equal(lse[0, 0, 1].expand(heads - 1), lse[0, 0, 1:])


def test_decode_queries_that_are_not_finite_stay_in_their_rows():
    lens = [70, 300]
    cache, table, sl, rows = h8.paged8(lens, 64, 512, seed=2)
    q = queries(2, 1, 32, 576, seed=5)
    ref = decode_reference(q, lambda r, n: rows[r][:n], lens, SCALE, 512)
    q[0, 0, 3, 17], q[1, 0, 9, 540], q[1, 0, 30, 0] = math.nan, math.inf, -math.inf
    out, lse = run_decode8(q, cache, table, sl, 512, SCALE)
    bad = torch.zeros(2, 1, 32, dtype=torch.bool)
    bad[0, 0, 3] = bad[1, 0, 9] = bad[1, 0, 30] = True
    assert torch.isnan(out.cpu()[bad]).all() and torch.isnan(lse.cpu()[bad]).all()
    want, mag, want_lse, bound = ref
    good = ~bad
    assert_attention(out.cpu()[good], lse.cpu()[good], (want[good], mag[good], want_lse[good], bound[good]))


def test_decode_queries_of_all_sizes():
    """Rows whose values span 2^20, rows of tiny and of huge values, rows whose rope part outweighs the latent part and the reverse."""
    lens = [500]
    cache, table, sl, rows = h8.paged8(lens, 64, 512, seed=31, sizes=lambda n: torch.ones(n, 1))
    q = queries(1, 1, 12, 576, seed=31).float()
    q[0, 0, 0] *= 1e-30
    q[0, 0, 1] = 0
    q[0, 0, 2, :512] = 0
    q[0, 0, 3, 512:] = 0
    q[0, 0, 4, :512] *= 1e-12
    q[0, 0, 5, 512:] *= 1e-12
    q[0, 0, 6] *= torch.exp2(-20 * torch.rand(576, device=DEV, generator=wl.generator(1, DEV)))
    q[0, 0, 7, 1:512] *= 1e-3
    q = q.to(BF)
    out, lse = run_decode8(q, cache, table, sl, 512, SCALE)
    assert_attention(out, lse, decode_reference(q, lambda r, n: rows[r][:n], lens, SCALE, 512))


def test_decode_is_repeatable_and_follows_the_stream():
    lens = [3000, 17, 900, 0, 12345]
    cache, table, sl, rows = h8.paged8(lens, 64, 512, seed=41)
    q = queries(5, 1, 32, 576, seed=6)
    a, la = run_decode8(q, cache, table, sl, 512, SCALE)
    stream = torch.cuda.Stream()
    b, lb = run_decode8(q, cache, table, sl, 512, SCALE, stream=stream)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16)) and torch.equal(la, lb)
    c, _ = run_decode8(q, cache, table, sl, 512, SCALE, lse=False)
    assert torch.equal(a.view(torch.int16), c.view(torch.int16))


def test_write_read_and_attend_captured_in_a_graph():
    """A serving step in one graph: reserve, quantised append, decode, read back; replayed with other lengths and rows."""
    dl, page, R, H = 512, 16, 3, 32
    lens0 = [0, 0, 0]
    table = torch.full((R, 40), -1, dtype=torch.int32, device=DEV)
    sl, ref = torch.zeros(R, dtype=torch.int32, device=DEV), torch.zeros(100, dtype=torch.int32, device=DEV)
    pt = kda.page_table_descriptor(table, sl, ref, page)
    cache = h8.poisoned_pages(100, page, dl)
    i32 = dict(dtype=torch.int32, device=DEV)
    req, new, cu = torch.arange(R, **i32), torch.zeros(R, **i32), torch.zeros(R + 1, **i32)
    src, dst, info = torch.empty(R, **i32), torch.empty(R, **i32), torch.empty(4, **i32)
    pws = torch.empty(kda.kda_pages_workspace_size(100, R), dtype=torch.uint8, device=DEV)
    ws = torch.empty(kda.kda_latent_decode8_workspace_size(R, 1, H, dl, 64), dtype=torch.uint8, device=DEV)
    x, q = torch.zeros(256, 576, dtype=BF, device=DEV), torch.zeros(R, 1, H, 576, dtype=BF, device=DEV)
    out, lse, back = torch.empty(R, 1, H, dl, dtype=BF, device=DEV), torch.empty(R, 1, H, device=DEV), torch.empty(256, 576, dtype=BF, device=DEV)

    def step():
        kda.kda_pages_reserve(pt, req, new, src, dst, info, pws)
        kda.kda_pages_copy(cache, src, dst)
        kda.kda_latent_append8(x, cu, req, pt, cache, latent_dim=dl)
        kda.kda_latent_decode8(q, cache, table, sl, out, ws, latent_dim=dl, scale=SCALE, lse=lse)
        kda.kda_latent_read(cache, cu, req, pt, back, latent_dim=dl)

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
    history = [torch.zeros(0, 576, dtype=torch.float64) for _ in range(R)]
    for k, n in enumerate(([37, 1, 100], [1, 1, 1], [5, 130, 0], [1, 2, 1])):
        new.copy_(torch.tensor(n))
        cu.copy_(torch.tensor([0, n[0], n[0] + n[1], sum(n)]))
        g = wl.generator(50 + k, DEV)
        x.copy_(torch.randn(256, 576, generator=g, device=DEV))
        q.copy_(torch.randn(R, 1, H, 576, generator=g, device=DEV))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        at = 0
        for r in range(R):
            c, rope, scale = h8.quantise(x[at:at + n[r]], dl) if n[r] else (torch.zeros(0, dl).double(), torch.zeros(0, 64).double(), torch.zeros(0).double())
            history[r] = torch.cat([history[r], torch.cat([c, rope], 1) * scale[:, None]])
            at += n[r]
        lens0 = [h.shape[0] for h in history]
        assert sl.tolist() == lens0 and info[0] == 0
        assert_attention(out, lse, decode_reference(q, lambda r, m: history[r][:m], lens0, SCALE, dl), f"step {k}")
        at = 0
        for r in range(R):
            assert torch.equal(back[at:at + n[r]].double().cpu(), history[r][:n[r]])
            at += n[r]


def strided(table):
    """The same block table as a slice of a wider one, rows 5 entries further apart, whose other entries are no pages."""
    wide = torch.full((table.shape[0], table.shape[1] + 5), 1 << 30, dtype=torch.int32, device=table.device)
    wide[:, 2:2 + table.shape[1]] = table
    return wide[:, 2:2 + table.shape[1]]


def test_strided_block_tables():
    dl, page, lens = 256, 16, [40, 0, 333]
    cache, table, sl, rows = h8.paged8(lens, page, dl, seed=71)
    q = queries(3, 2, 16, dl + 64, seed=71)
    out, lse = run_decode8(q, cache, strided(table), sl, dl, SCALE)
    assert_attention(out, lse, decode_reference(q, lambda r, n: rows[r][:n], lens, SCALE, dl))
    got = read_back(cache, strided(table), lens, page, dl, [0, 40, 373], [0, 2], None, 373)
    assert torch.equal(got.double().cpu(), torch.cat([rows[0], rows[2]]))
    x = torch.randn(7, dl + 64, generator=wl.generator(72, DEV), device=DEV).to(BF)
    run_append(x, [0, 7], [2], strided(table), lens, cache, dl, page)
    c, rope, scale = h8.quantise(x, dl)
    got = read_back(cache, table, lens, page, dl, [0, 333], [2], None, 333)
    assert torch.equal(got.double().cpu(), torch.cat([rows[2][:326], torch.cat([c, rope], 1) * scale[:, None]]))


def test_calls_on_two_streams_at_once():
    """Two decodes, each on a stream and a workspace of its own, again and again; and writes and reads of other requests between them."""
    dl, sets = 512, []
    for k in range(2):
        lens = [3000 + 500 * k, 17, 900, 64]
        cache, table, sl, rows = h8.paged8(lens, 64, dl, seed=80 + k)
        q = queries(4, 1, 32, 576, seed=80 + k)
        ws = torch.empty(kda.kda_latent_decode8_workspace_size(4, 1, 32, dl, 64), dtype=torch.uint8, device=DEV)
        pt = kda.page_table_descriptor(table, sl, torch.ones(cache.shape[0], dtype=torch.int32, device=DEV), 64)
        sets.append((lens, cache, table, sl, rows, q, ws, pt, torch.empty(4, 1, 32, dl, dtype=BF, device=DEV),
                     torch.empty(900, 576, dtype=BF, device=DEV), torch.cuda.Stream()))
    cu, req = torch.tensor([0, 900], dtype=torch.int32, device=DEV), torch.tensor([2], dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    for _ in range(10):
        for lens, cache, table, sl, rows, q, ws, pt, out, back, st in sets:
            kda.kda_latent_decode8(q, cache, table, sl, out, ws, latent_dim=dl, scale=SCALE, stream=st)
            kda.kda_latent_read(cache, cu, req, pt, back, latent_dim=dl, stream=st)
    torch.cuda.synchronize()
    for lens, cache, table, sl, rows, q, ws, pt, out, back, st in sets:
        assert kda.kda_prefill_workspace_status(ws) == 0
        assert_attention(out, None, decode_reference(q, lambda r, n: rows[r][:n], lens, SCALE, dl))
        assert torch.equal(back.double().cpu(), rows[2])


def test_pages_of_bytes_are_copied():
    for page, gap in ((16, 0), (8, 32), (8, 5)):  # the last: pages that are not 16-byte aligned
        size = page * 644
        cache = torch.zeros(9, size + gap, dtype=torch.uint8, device=DEV).as_strided((9, 1, page, 644), (size + gap, size, 644, 1))
        cache.copy_(torch.randint(0, 255, cache.shape, dtype=torch.uint8, device=DEV))
        want = cache.clone()
        src, dst = torch.tensor([3, 0, -1, 8], dtype=torch.int32, device=DEV), torch.tensor([5, 1, 2, 20], dtype=torch.int32, device=DEV)
        kda.kda_pages_copy(cache, src, dst)
        torch.cuda.synchronize()
        want[5], want[1] = want[3], want[0]
        assert torch.equal(cache, want)


def test_decode_rows_far_apart():
    """Pages beyond 4 GiB of the cache's start."""
    dl, page = 512, 64
    size = page * 644
    pitch = 1 << 20
    N = 4200
    back = torch.full((N * pitch,), 0x7F, dtype=torch.uint8, device=DEV)
    cache = back.as_strided((N, 1, page, 644), (pitch, size, 644, 1))
    x = torch.randn(100, 576, generator=torch.Generator().manual_seed(3))
    rows = torch.cat([h8.put(cache, dl, N - 1, slice(0, 64), x[:64]), h8.put(cache, dl, N - 2, slice(0, 36), x[64:])])
    table, sl = torch.tensor([[N - 1, N - 2]], dtype=torch.int32, device=DEV), torch.tensor([100], dtype=torch.int32, device=DEV)
    q = queries(1, 1, 8, 576, seed=1)
    out, lse = run_decode8(q, cache, table, sl, dl, SCALE)
    assert_attention(out, lse, decode_reference(q, lambda r, n: rows[:n], [100], SCALE, dl))
    got = read_back(cache, table, [100], page, dl, [0, 100], [0], None, 100)
    assert torch.equal(got.double().cpu(), rows)
    y = torch.randn(2, 576, generator=wl.generator(3, DEV), device=DEV).to(BF)
    run_append(y, [0, 2], [0], table, [100], cache, dl, page)
    assert torch.equal(read_back(cache, table, [100], page, dl, [0, 2], [0], [98], 2)[:, 512:], y[:, 512:])


def test_tolerances_are_those_of_bf16_outputs():
    assert OUT_REL == 1.25 * 2.0 ** -8 and Z_REL == 2.0 ** -17 and LSE_ABS == 1e-5
