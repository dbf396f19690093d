"""Latent attention on the GPU, the absorbed form over paged latents and the expanded form over
varlen batches, against plain 64-bit forms (tests/latent_helpers.py: formulas and tolerances).
Whatever lies outside a request's tokens holds NaN and infinities throughout."""
import math

import pytest
import torch

import kimi_delta_attention_varlen_gb300 as kda
from kimi_delta_attention_varlen_gb300 import workloads as wl
from tests.latent_helpers import LSE_ABS, OUT_REL, Z_REL, assert_attention, decode_reference, prefill_reference

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def poisoned(*shape):
    """NaN, +inf and -inf in turn."""
    t = torch.empty(*shape, dtype=BF, device=DEV)
    flat = t.view(-1)
    flat[0::3], flat[1::3], flat[2::3] = math.nan, math.inf, -math.inf
    return t


def paged_latents(lens, page, dl, seed, gap=0, spare=3, width_extra=0):
    """Random latents of the given lengths in random pages of a poisoned cache whose rows lie
    `gap` elements apart; (cache view, block table, seq_lens, per-request rows)."""
    g = wl.generator(seed, DEV)
    D = dl + 64
    need = [-(-n // page) for n in lens]
    N = sum(need) + spare
    back = poisoned(N, page * D + gap)
    cache = back.as_strided((N, 1, page, D), (page * D + gap, page * D, D, 1))
    perm = torch.randperm(N, generator=g, device=DEV).tolist()
    W = max(1, max(need)) + width_extra
    table = torch.full((len(lens), W), -1, dtype=torch.int32)
    rows, at = [], 0
    for r, n in enumerate(lens):
        x = torch.randn(n, D, generator=g, device=DEV).to(BF)
        rows.append(x)
        for j in range(need[r]):
            p = perm[at]
            at += 1
            table[r, j] = p
            part = x[j * page:(j + 1) * page]
            cache[p, 0, :part.shape[0]] = part
    return cache, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), rows


def run_decode(q, cache, table, lens, dl, scale, req=None, stream=None, lse=True):
    R, L, H, D = q.shape
    out = poisoned(R, L, H, dl)
    ls = torch.full((R, L, H), math.nan, device=DEV) if lse else None
    ws = torch.empty(kda.kda_latent_decode_workspace_size(R, L, H, dl, D - dl), dtype=torch.uint8, device=DEV)
    ws.fill_(0xA5)
    torch.cuda.synchronize()
    kda.kda_latent_decode(q, cache, table, lens, out, ws, latent_dim=dl, scale=scale, req=req, lse=ls, stream=stream)
    torch.cuda.synchronize()
    assert kda.kda_prefill_workspace_status(ws) == 0
    return out, ls


def queries(R, L, H, D, seed):
    return torch.randn(R, L, H, D, generator=wl.generator(seed + 77, DEV), device=DEV).to(BF)


SCALE = 192 ** -0.5


@pytest.mark.parametrize("dl", [512, 256])
@pytest.mark.parametrize("page", [8, 16, 48, 64, 128, 200])
def test_decode_lengths_and_pages(page, dl):
    lens = [0, 1, 2, 63, 64, 65, 127, 128, 129, 191, 193, 500, 1000, page, page + 1, 3 * page - 1]
    cache, table, sl, rows = paged_latents(lens, page, dl, seed=page + dl)
    q = queries(len(lens), 1, 32, dl + 64, seed=page)
    out, lse = run_decode(q, cache, table, sl, dl, SCALE)
    assert_attention(out, lse, decode_reference(q, lambda r, n: rows[r][:n], lens, SCALE, dl), f"page {page} dl {dl}")


@pytest.mark.parametrize("heads", [1, 2, 5, 8, 16, 17, 32, 48, 64, 65, 100, 128, 192])
def test_decode_heads(heads):
    lens = [1, 70, 333]
    cache, table, sl, rows = paged_latents(lens, 32, 512, seed=heads, gap=24)
    q = queries(3, 1, heads, 576, seed=heads)
    out, lse = run_decode(q, cache, table, sl, 512, SCALE)
    assert_attention(out, lse, decode_reference(q, lambda r, n: rows[r][:n], lens, SCALE, 512), f"heads {heads}")


@pytest.mark.parametrize("L,heads", [(2, 32), (3, 16), (4, 128), (5, 8), (7, 1), (70, 2)])
def test_decode_draft_tokens_are_causal(L, heads):
    # lengths below L: the first query tokens see nothing
    lens = [0, 1, L - 1, L, L + 1, 64 + L, 129, 700]
    cache, table, sl, rows = paged_latents(lens, 16, 512, seed=L, width_extra=3)
    q = queries(len(lens), L, heads, 576, seed=L)
    out, lse = run_decode(q, cache, table, sl, 512, SCALE)
    assert_attention(out, lse, decode_reference(q, lambda r, n: rows[r][:n], lens, SCALE, 512), f"L {L} heads {heads}")


@pytest.mark.parametrize("n,L", [(40, 3), (130, 5), (66, 4), (20000, 6), (64, 70), (131, 70)])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_decode_draft_values_that_are_not_finite_reach_only_tokens_that_see_them(n, L, bad):
    cache, table, sl, rows = paged_latents([n], 16, 512, seed=n + L)
    q = queries(1, L, 8, 576, seed=L)
    tok = n - 2  # the last but one of the draft tokens' rows: the query tokens from L - 2 on see it
    dims = [9, 300, 511]
    q[..., dims] = 0
    ref = decode_reference(q, lambda r, k: rows[r][:k], [n], SCALE, 512)
    cache[table[0, tok // 16].long(), 0, tok % 16, dims] = bad  # in a latent, so in its key too: 0 * bad is no number
    out, lse = run_decode(q, cache, table, sl, 512, SCALE)
    assert torch.isnan(out[0, L - 2:]).all() and torch.isnan(lse[0, L - 2:]).all()
    assert_attention(out[:, :L - 2], lse[:, :L - 2], [x[:, :L - 2] for x in ref], f"n {n} L {L}")


@pytest.mark.parametrize("lens,heads", [([40000], 32), ([9999, 3, 25000], 16), ([6400] * 5, 64), ([20000, 1], 128)])
def test_decode_long_contexts(lens, heads):
    # few rows: the cache axis is split and the parts are joined
    cache, table, sl, rows = paged_latents(lens, 64, 512, seed=heads)
    q = queries(len(lens), 1, heads, 576, seed=heads)
    out, lse = run_decode(q, cache, table, sl, 512, SCALE)
    assert_attention(out, lse, decode_reference(q, lambda r, n: rows[r][:n], lens, SCALE, 512), "long")
    again, lse2 = run_decode(q, cache, table, sl, 512, SCALE)
    assert torch.equal(out, again) and torch.equal(lse, lse2)  # no result depends on the order of arrival


def test_decode_many_requests():
    g = wl.generator(5)
    lens = torch.randint(0, 400, (700,), generator=g).tolist()
    cache, table, sl, rows = paged_latents(lens, 16, 512, seed=9)
    q = queries(len(lens), 1, 4, 576, seed=3)
    out, lse = run_decode(q, cache, table, sl, 512, SCALE)
    assert_attention(out, lse, decode_reference(q, lambda r, n: rows[r][:n], lens, SCALE, 512), "many")


def test_decode_large_scores_and_growing_maxima():
    # scores rise by hundreds along the cache: every tile brings a new maximum
    n, dl = 1000, 512
    cache, table, sl, rows = paged_latents([n], 64, dl, seed=1)
    x = rows[0]
    u = torch.randn(576, generator=wl.generator(2, DEV), device=DEV)
    ramp = torch.linspace(-6, 6, n, device=DEV)[:, None]
    new = (x.float() * 0.1 + ramp * u / u.norm() * 4).to(BF)
    for j in range(table.shape[1]):
        part = new[j * 64:(j + 1) * 64]
        cache[table[0, j].long(), 0, :part.shape[0]] = part
    q = (u[None, None, None].expand(1, 1, 16, 576) * torch.tensor([1.0, -1.0] * 8, device=DEV)[None, None, :, None]).to(BF).contiguous()
    out, lse = run_decode(q, cache, table, sl, dl, 1.0)
    assert_attention(out, lse, decode_reference(q, lambda r, k: new[:k], [n], 1.0, dl), "ramp")


def test_decode_rows_by_request_index_and_invalid_rows():
    lens = [100, 0, 257, 64]
    cache, table, sl, rows = paged_latents(lens, 32, 512, seed=4)
    pick = [2, -1, 0, 4, 3, 2, 1 << 20]
    q = queries(len(pick), 1, 16, 576, seed=1)
    ok = [p if 0 <= p < 4 else None for p in pick]
    ref = decode_reference(q, lambda r, n: rows[ok[r]][:n] if n else rows[0][:0], [0 if p is None else lens[p] for p in ok], SCALE, 512)
    for dt in (torch.int32, torch.int64):
        out, lse = run_decode(q, cache, table, sl, 512, SCALE, req=torch.tensor(pick, dtype=dt, device=DEV))
        assert_attention(out, lse, ref, f"req {dt}")
    out64, _ = run_decode(q[1:2].contiguous(), cache, table, sl, 512, SCALE, req=torch.tensor([-1 - (1 << 40)], device=DEV), lse=False)
    assert (out64 == 0).all()


def test_decode_invalid_pages_read_as_zeros_and_lengths_are_clamped():
    lens = [150, 90]
    cache, table, sl, rows = paged_latents(lens, 16, 512, seed=6)
    table = table.clone()
    table[0, 2], table[0, 9], table[1, 0] = -1, cache.shape[0], 2 ** 31 - 1
    q = queries(2, 1, 32, 576, seed=2)
    for r, j in ((0, 2), (0, 9), (1, 0)):
        rows[r][16 * j:16 * j + 16] = 0
    out, lse = run_decode(q, cache, table, sl, 512, SCALE)
    assert_attention(out, lse, decode_reference(q, lambda r, n: rows[r][:n], lens, SCALE, 512), "invalid pages")
    # a length above the row's capacity is that capacity; a negative one is 0
    full = torch.randn(2 * 16, 576, device=DEV).to(BF)
    cache2 = full.view(2, 1, 16, 576)
    t2 = torch.tensor([[1, 0], [0, 1]], dtype=torch.int32, device=DEV)
    out, lse = run_decode(q, cache2, t2, torch.tensor([2 ** 31 - 1, -5], dtype=torch.int32, device=DEV), 512, SCALE)
    assert_attention(out, lse, decode_reference(q, lambda r, n: torch.cat([full[16:], full[:16]])[:n], [32, 0], SCALE, 512), "clamped")


def test_decode_shared_pages_strided_table_and_own_stream():
    lens = [130, 130, 70]
    cache, table, sl, rows = paged_latents(lens, 64, 512, seed=8, gap=8)
    table[1] = table[0]  # a fork shares its pages
    wide = torch.full((3, 11), 2 ** 30, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    q = queries(3, 1, 32, 576, seed=4)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out, lse = run_decode(q, cache, wide[:, :table.shape[1]], sl, 512, SCALE, stream=st)
    assert_attention(out, lse, decode_reference(q, lambda r, n: rows[0 if r == 1 else r][:n], lens, SCALE, 512), "shared")


def test_decode_pages_beyond_32_bit_offsets():
    page, D, N = 64, 576, 7
    stride = (1 << 30) + 8  # elements between pages: the last one starts beyond 2^32 elements
    back = torch.empty((N - 1) * stride + page * D, dtype=BF, device=DEV)
    cache = back.as_strided((N, 1, page, D), (stride, page * D, D, 1))
    x = torch.randn(3 * page, D, generator=wl.generator(1, DEV), device=DEV).to(BF)
    order = [6, 2, 5]
    for j, p in enumerate(order):
        cache[p, 0] = x[j * page:(j + 1) * page]
    q = queries(1, 1, 32, D, seed=11)
    n = 3 * page - 5
    out, lse = run_decode(q, cache, torch.tensor([order], dtype=torch.int32, device=DEV),
                          torch.tensor([n], dtype=torch.int32, device=DEV), 512, SCALE)
    assert_attention(out, lse, decode_reference(q, lambda r, k: x[:k], [n], SCALE, 512), "far pages")


def test_decode_in_a_graph_follows_new_lengths():
    lens = [200, 3000]
    cache, table, sl, rows = paged_latents(lens, 64, 512, seed=3)
    q = queries(2, 1, 32, 576, seed=5)
    out, lse = torch.empty(2, 1, 32, 512, dtype=BF, device=DEV), torch.empty(2, 1, 32, device=DEV)
    ws = torch.empty(kda.kda_latent_decode_workspace_size(2, 1, 32, 512, 64), dtype=torch.uint8, device=DEV)
    kda.kda_latent_decode(q, cache, table, sl, out, ws, latent_dim=512, scale=SCALE, lse=lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_latent_decode(q, cache, table, sl, out, ws, latent_dim=512, scale=SCALE, lse=lse)
    for now in ([200, 3000], [1, 2500], [0, 65]):
        sl.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert_attention(out, lse, decode_reference(q, lambda r, n: rows[r][:n], now, SCALE, 512), f"graph {now}")


# ---------------------------------------------------------------- prefill --

def prompt_batch(nq, nk, heads, seed, tail=5):
    """q, k_nope / v as slices of one projection, k_rope as the tail of latent rows; rows behind the last token are poisoned."""
    g = wl.generator(seed, DEV)
    Tq, Tk = sum(nq), sum(nk)
    kv, rows, q = poisoned(Tk + tail, heads, 256), poisoned(Tk + tail, 576), poisoned(Tq + tail, heads, 192)
    kv[:Tk] = torch.randn(Tk, heads, 256, generator=g, device=DEV).to(BF)
    rows[:Tk, 512:] = torch.randn(Tk, 64, generator=g, device=DEV).to(BF)
    q[:Tq] = torch.randn(Tq, heads, 192, generator=g, device=DEV).to(BF)
    cu = [[0], [0]]
    for a, b in zip(nq, nk):
        cu[0].append(cu[0][-1] + a)
        cu[1].append(cu[1][-1] + b)
    return q[:Tq], kv[:Tk, :, :128], rows[:Tk, 512:], kv[:Tk, :, 128:], cu[0], cu[1]


def run_prefill(q, kn, kr, v, cu_q, cu_k, scale=SCALE, stream=None):
    Tq, H, _ = q.shape
    guard = poisoned(Tq + 2, H, 128)
    out, lse = guard[1:-1], torch.full((Tq, H), math.nan, device=DEV)
    ws = torch.empty(kda.kda_latent_prefill_workspace_size(Tq, len(cu_q) - 1, H), dtype=torch.uint8, device=DEV)
    ws.fill_(0xA5)
    before = guard.view(torch.int16).clone()
    cq, ck = (torch.tensor(c, dtype=torch.int32, device=DEV) for c in (cu_q, cu_k))
    torch.cuda.synchronize()
    kda.kda_latent_prefill(q, kn, kr, v, cq, ck, out, ws, scale=scale, lse=lse, stream=stream)
    torch.cuda.synchronize()
    assert kda.kda_prefill_workspace_status(ws) == 0
    assert torch.equal(guard.view(torch.int16)[[0, -1]], before[[0, -1]])
    return out, lse


def check_prefill(nq, nk, heads, seed, **kw):
    q, kn, kr, v, cu_q, cu_k = prompt_batch(nq, nk, heads, seed)
    out, lse = run_prefill(q, kn, kr, v, cu_q, cu_k, **kw)
    assert_attention(out, lse, prefill_reference(q, kn, kr, v, cu_q, cu_k, kw.get("scale", SCALE)), f"{nq} {nk} heads {heads}")


@pytest.mark.parametrize("n", [1, 2, 31, 63, 64, 65, 127, 128, 129, 191, 255, 256, 257, 383, 385, 640])
def test_prefill_one_prompt(n):
    check_prefill([n], [n], 2, seed=n)


@pytest.mark.parametrize("heads", [1, 3, 8, 32])
def test_prefill_batch_with_empty_and_short_prompts(heads):
    nq = [64, 0, 100, 1, 37, 300, 0, 128, 129, 5]
    check_prefill(nq, nq, heads, seed=heads)


@pytest.mark.parametrize("nq,nk", [([1, 50, 200], [129, 50, 900]), ([256, 3, 17], [300, 1000, 17]), ([5, 1, 128], [2000, 1, 128 * 5]),
                                   ([130, 0, 2], [131, 40, 258])])
def test_prefill_on_prefixes(nq, nk):
    check_prefill(nq, nk, 4, seed=sum(nk))


def test_prefill_queries_that_see_nothing():
    # fewer keys than queries: the first queries of a sequence see no key
    check_prefill([10, 200, 300, 40], [4, 0, 131, 40], 3, seed=12)
    q, kn, kr, v, cu_q, cu_k = prompt_batch([7], [0], 2, seed=1)
    out, lse = run_prefill(q, kn, kr, v, cu_q, cu_k)
    assert (out == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("nq,nk,tok", [([300], [300], 100), ([300], [300], 260), ([200, 40], [1500, 40], 1400), ([256], [5000], 4800),
                                       ([70], [70], 69)])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_prefill_values_that_are_not_finite_reach_only_queries_that_see_them(nq, nk, tok, bad):
    q, kn, kr, v, cu_q, cu_k = prompt_batch(nq, nk, 2, seed=tok)
    ref = prefill_reference(q, kn, kr, v, cu_q, cu_k, SCALE)
    v[tok, 1, 5], v[tok, 1, 77] = bad, bad
    out, lse = run_prefill(q, kn, kr, v, cu_q, cu_k)
    sees = torch.zeros_like(out, dtype=torch.bool)
    first = max(0, tok - (nk[0] - nq[0]))  # the first query of the sequence that sees the token
    sees[first:nq[0], 1, 5] = sees[first:nq[0], 1, 77] = True
    hit = out[sees].float()
    assert (torch.isnan(hit) if math.isnan(bad) else hit == bad).all()
    assert_attention(torch.where(sees, ref[0].to(DEV).to(BF), out), lse, ref, "others")


def test_prefill_keys_that_are_not_numbers_reach_only_queries_that_see_them():
    for tok in (3, 130, 299):
        q, kn, kr, v, cu_q, cu_k = prompt_batch([300], [300], 2, seed=tok)
        ref = prefill_reference(q, kn, kr, v, cu_q, cu_k, SCALE)
        kn[tok, 1, 7] = math.nan
        out, lse = run_prefill(q, kn, kr, v, cu_q, cu_k)
        assert torch.isnan(out[tok:, 1]).all() and torch.isnan(lse[tok:, 1]).all()
        fine = torch.ones(300, 2, dtype=torch.bool, device=DEV)
        fine[tok:, 1] = False
        assert_attention(torch.where(fine[..., None], out, ref[0].to(DEV).to(BF)), torch.where(fine, lse, ref[2].to(DEV).float()), ref, "others")


def test_prefill_large_scores():
    check_prefill([300], [300], 2, seed=5, scale=3.0)


def test_prefill_longer_batch_is_repeatable():
    q, kn, kr, v, cu_q, cu_k = prompt_batch([1500, 700, 2100], [1500, 1100, 2100], 2, seed=2)
    out, lse = run_prefill(q, kn, kr, v, cu_q, cu_k)
    assert_attention(out, lse, prefill_reference(q, kn, kr, v, cu_q, cu_k, SCALE), "long")
    again, lse2 = run_prefill(q, kn, kr, v, cu_q, cu_k)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("heads", [3, 16])
def test_prefill_many_prompts(heads):
    # far more (block, head) pairs than SMs: whole pairs, longest first; the other tests' few pairs are cut into equal shares
    nq = [130, 128, 1, 0, 300, 64, 257] * 60
    nk = [n + (i % 5) * 77 for i, n in enumerate(nq)]
    check_prefill(nq, nk, heads, seed=heads)


@pytest.mark.parametrize("nq,nk,heads", [([256], [5000], 1), ([40, 600], [9000, 3000], 2), ([1, 1, 1], [20000, 1, 700], 4), ([513], [513], 1)])
def test_prefill_pairs_cut_over_many_shares(nq, nk, heads):
    check_prefill(nq, nk, heads, seed=len(nq) + heads)


def test_prefill_contiguous_and_head_major_inputs_agree_on_another_stream():
    q, kn, kr, v, cu_q, cu_k = prompt_batch([150, 61], [150, 200], 5, seed=3)
    out, lse = run_prefill(q, kn, kr, v, cu_q, cu_k)
    st = torch.cuda.Stream()
    head_major = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    out2, lse2 = run_prefill(q, kn.contiguous(), kr.contiguous(), head_major(v), cu_q, cu_k, stream=st)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_prefill_values_shared_by_all_heads():
    # head stride 0: one key and value head for all query heads
    q, kn, kr, v, cu_q, cu_k = prompt_batch([140], [140], 4, seed=9)
    kn1, v1 = kn[:, :1].expand(-1, 4, -1), v[:, :1].expand(-1, 4, -1)
    out, lse = run_prefill(q, kn1, kr, v1, cu_q, cu_k)
    assert_attention(out, lse, prefill_reference(q, kn1, kr, v1, cu_q, cu_k, SCALE), "shared heads")


def test_prefill_and_decode_are_the_same_attention():
    # the last token's output, expanded and absorbed: q W_k^T against the latents, W_v behind
    n, H = 333, 8
    g = wl.generator(21, DEV)
    c = torch.randn(n, 576, generator=g, device=DEV).to(BF)
    wk = (torch.randn(H, 512, 128, generator=g, device=DEV) / 512 ** 0.5).to(BF)
    wv = (torch.randn(H, 512, 128, generator=g, device=DEV) / 512 ** 0.5).to(BF)
    q = torch.randn(n, H, 192, generator=g, device=DEV).to(BF)
    kn, v = (torch.einsum("td,hde->the", c[:, :512].float(), w.float()).to(BF) for w in (wk, wv))
    out, _ = run_prefill(q, kn, c[:, 512:], v, [0, n], [0, n])
    qa = torch.cat([torch.einsum("he,hde->hd", q[-1, :, :128].float(), wk.float()), q[-1, :, 128:].float()], -1).to(BF)
    pad = poisoned(6, 1, 64, 576)
    pad.view(-1, 576)[:n] = c
    lat, _ = run_decode(qa[None, None].contiguous(), pad, torch.arange(6, dtype=torch.int32, device=DEV)[None],
                        torch.tensor([n], dtype=torch.int32, device=DEV), 512, SCALE)
    want = torch.einsum("hd,hde->he", lat[0, 0].double(), wv.double())
    # each side rounds its keys or queries, probabilities and outputs to bf16: a few 2^-9 of the values' size
    assert (out[-1].double() - want).abs().max() <= 6 * 2.0 ** -9 * v.double().abs().max()


@pytest.mark.parametrize("nq,nk", [([10] * 31, [10] * 31), ([10] * 32, [10] * 32), ([0, 9] * 14 + [300], [0, 9] * 14 + [9000]),
                                   ([40] * 39 + [500], [6000] + [40 + 130 * (i % 3) for i in range(38)] + [7000]),
                                   ([8192, 1], [8192, 3])])
@pytest.mark.parametrize("heads", [1, 4])
def test_prefill_lists_of_few_and_of_many_blocks(nq, nk, heads):
    """Batches around 32 blocks of queries, whole or cut, with empty sequences between."""
    check_prefill(nq, nk, heads, seed=len(nq) + heads)


# ------------------------------------------------------------ long sums --
# The tensor cores cut each product off at 2^-25 of the sum that it joins (a 26-bit window), so a sum of N products may
# lose N * 2^-25 of its size, all in one direction where the values have one sign.  Held to the tolerance of every other
# output, which leaves 2^-10: no more than 2^15 products in a row.

def long_rows(n, width, heavy, seed):
    """Rows of values in [1, 2) and one rope column: 1 in row 0 (`heavy`), else 0."""
    x = torch.empty(n, width, dtype=BF, device=DEV).uniform_(1, 2, generator=wl.generator(seed, DEV))
    x[:, -64:] = 0
    x[0, -64] = 1 if heavy else 0
    return x


def assert_long_sum(out, lse, x, z0, what):
    """Weights e^z0 of row 0 and 1 of the others."""
    n = x.shape[0]
    total = math.exp(z0) + n - 1
    want = (x.sum(0, dtype=torch.float64) + (math.exp(z0) - 1) * x[0].double()) / total
    over = (out.double() - want).abs() / want
    assert over.max() <= OUT_REL + 2 * Z_REL * z0, f"{what}: off by {float(over.max()):.2e}"
    assert (lse.double() - math.log(total)).abs().max() <= LSE_ABS + Z_REL * z0, what


@pytest.mark.parametrize("heavy", [False, True])
@pytest.mark.parametrize("dl,heads", [(512, 16), (512, 32), (512, 64), (256, 16)])
def test_decode_sums_of_a_million_values(dl, heads, heavy):
    # as many requests as SMs, all on the same pages: each is one CTA's
    R, n = torch.cuda.get_device_properties(0).multi_processor_count, 1 << 20
    x = long_rows(n, dl + 64, heavy, seed=dl)
    table = torch.arange(n // 64, dtype=torch.int32, device=DEV)[None].expand(R, -1).contiguous()
    q = torch.zeros(R, 1, heads, dl + 64, dtype=BF, device=DEV)
    q[..., dl] = 14 if heavy else 0  # e^14 is about a million: half of the weight is row 0's
    out, lse = run_decode(q, x.view(-1, 1, 64, dl + 64), table, torch.full((R,), n, dtype=torch.int32, device=DEV), dl, 1.0)
    assert_long_sum(out, lse, x[:, :dl], 14.0 if heavy else 0.0, f"dl {dl} heads {heads}")


@pytest.mark.parametrize("heavy", [False, True])
@pytest.mark.parametrize("nq", [1, 200])
def test_prefill_sums_of_a_million_values(nq, heavy):
    # a head a CTA, keys and values shared by the heads; the last query sees all rows, the others nearly
    H, n = torch.cuda.get_device_properties(0).multi_processor_count, 1 << 20
    x = long_rows(n, 192, heavy, seed=nq)
    v = x[:, None, :128].expand(-1, H, -1)
    q = torch.zeros(nq, H, 192, dtype=BF, device=DEV)
    q[..., 128] = 14 if heavy else 0
    out, lse = run_prefill(q, v, x[:, 128:], v, [0, nq], [0, n], scale=1.0)
    assert_long_sum(out[-1], lse[-1], x[:, :128], 14.0 if heavy else 0.0, f"{nq} queries")


@pytest.mark.parametrize("heavy", [False, True])
def test_decode_sums_of_parts_of_many_tiles(heavy):
    # one request over all CTAs, each part longer than the accumulator takes in a row; two groups of rows
    n = 1 << 22
    x = long_rows(n, 576, heavy, seed=7)
    q = torch.zeros(1, 2, 48, 576, dtype=BF, device=DEV)
    q[..., 512] = 14 if heavy else 0
    out, lse = run_decode(q, x.view(-1, 1, 64, 576), torch.arange(n // 64, dtype=torch.int32, device=DEV)[None],
                          torch.tensor([n], dtype=torch.int32, device=DEV), 512, 1.0)
    assert_long_sum(out[0, 1], lse[0, 1], x[:, :512], 14.0 if heavy else 0.0, "last token")
    assert_long_sum(out[0, 0], lse[0, 0], x[:-1, :512], 14.0 if heavy else 0.0, "first token")


@pytest.mark.parametrize("heavy", [False, True])
def test_prefill_sums_of_parts_of_many_tiles(heavy):
    n, nq = 1 << 22, 140
    x = long_rows(n, 192, heavy, seed=8)
    v = x[:, None, :128].expand(-1, 2, -1)
    q = torch.zeros(nq, 2, 192, dtype=BF, device=DEV)
    q[..., 128] = 14 if heavy else 0
    out, lse = run_prefill(q, v, x[:, 128:], v, [0, nq], [0, n], scale=1.0)
    for i in (0, 127, 128, nq - 1):
        assert_long_sum(out[i], lse[i], x[:n - nq + 1 + i, :128], 14.0 if heavy else 0.0, f"query {i}")


def test_decode_sums_set_aside_as_the_maximum_grows():
    # scores that rise by 40 over a million tokens: what was set aside is rescaled again and again
    R, n = torch.cuda.get_device_properties(0).multi_processor_count, 1 << 20
    x = long_rows(n, 576, False, seed=9)
    x[:, 512] = torch.linspace(0, 20, n, device=DEV).to(BF)
    x[:, 513] = torch.linspace(0, 0.05, n, device=DEV).to(BF)
    q = torch.zeros(R, 1, 16, 576, dtype=BF, device=DEV)
    q[..., 512:514] = 2
    out, lse = run_decode(q, x.view(-1, 1, 64, 576), torch.arange(n // 64, dtype=torch.int32, device=DEV)[None].expand(R, -1).contiguous(),
                          torch.full((R,), n, dtype=torch.int32, device=DEV), 512, 1.0)
    z = 2 * x[:, 512:514].double().sum(-1)
    p = torch.softmax(z, 0)
    want = (p[:, None] * x[:, :512].double()).sum(0)
    assert ((out.double() - want).abs() / want).max() <= OUT_REL + 2 * Z_REL * 40
    assert (lse.double() - torch.logsumexp(z, 0)).abs().max() <= LSE_ABS + Z_REL * 41


def test_prefill_sums_set_aside_as_the_maximum_grows():
    H, n = torch.cuda.get_device_properties(0).multi_processor_count, 1 << 20
    x = long_rows(n, 192, False, seed=10)
    x[:, 128] = torch.linspace(0, 20, n, device=DEV).to(BF)
    x[:, 129] = torch.linspace(0, 0.05, n, device=DEV).to(BF)
    v = x[:, None, :128].expand(-1, H, -1)
    q = torch.zeros(3, H, 192, dtype=BF, device=DEV)
    q[..., 128:130] = 2
    out, lse = run_prefill(q, v, x[:, 128:], v, [0, 3], [0, n], scale=1.0)
    z = 2 * x[:, 128:130].double().sum(-1)
    p = torch.softmax(z, 0)
    want = (p[:, None] * x[:, :128].double()).sum(0)
    assert ((out[-1].double() - want).abs() / want).max() <= OUT_REL + 2 * Z_REL * 40
    assert (lse[-1].double() - torch.logsumexp(z, 0)).abs().max() <= LSE_ABS + Z_REL * 41


def test_prefill_pairs_that_take_longer_than_a_second():
    """Three sequences of one query, the first on 200 million keys, with a head a CTA: while its pair runs, the warps that
    are done with it wait to be handed the third one."""
    H = torch.cuda.get_device_properties(0).multi_processor_count
    n = 200_000_000
    ones = torch.ones(n + 2, 128, dtype=BF, device=DEV)  # keys and values in one, shared by all heads
    k = ones[:, None].expand(-1, H, -1)
    q = torch.randn(3, H, 192, generator=wl.generator(3, DEV), device=DEV).to(BF)
    out, lse = run_prefill(q, k, ones[:, :64], k, [0, 1, 2, 3], [0, n, n + 1, n + 2], scale=1.0)
    assert (out == 1).all()  # ones, whatever their weights
    want = q.double().sum(-1) + torch.tensor([math.log(n), 0, 0], device=DEV)[:, None]
    # a score: 192 products with 1, each addition within 2^-23 of the magnitudes added (12 partial sums of 16); the weights
    # are 1 and their sums, in steps of 64, exact up to 2^30
    assert ((lse.double() - want).abs() <= 12 * 2.0 ** -23 * q.double().abs().sum(-1) + 1e-5).all()


# -------------------------------------------- few keys in a tile of many --
# Two to four weights do not average their rounding to bf16 away: rows that see few keys take what it leaves off, also
# where other rows of their tile see more than one key tile.

@pytest.mark.parametrize("nq", [128, 256, 300])
def test_prefill_rows_of_few_keys_before_rows_of_many(nq):
    prefixes = [1, 2, 3, 4, 20, 64]
    check_prefill([nq] * len(prefixes), [nq + n for n in prefixes], 64, seed=nq)


@pytest.mark.parametrize("dl", [256, 512])
@pytest.mark.parametrize("L", [65, 70, 90])
def test_decode_draft_tokens_that_see_few_tokens(L, dl):
    lens = [L, L + 1, L + 2, L + 3, L + 30, L + 62, L + 63, L + 64]
    cache, table, sl, rows = paged_latents(lens, 16, dl, seed=L)
    q = queries(len(lens), L, 32, dl + 64, seed=L)
    out, lse = run_decode(q, cache, table, sl, dl, SCALE)
    assert_attention(out, lse, decode_reference(q, lambda r, n: rows[r][:n], lens, SCALE, dl), f"L {L}")


# ------------------------------------------------------- schedules, widths --

@pytest.mark.parametrize("nq,nk,heads", [([777, 435, 600, 512, 700], [9000, 5000, 8000, 7111, 6500], 16),
                                         ([200 - 3 * (i % 4) for i in range(36)], [5000 - 37 * i for i in range(36)], 6)])
def test_prefill_last_round_cut_behind_whole_rounds(nq, nk, heads):
    # more pairs than CTAs, fewer than eight a CTA, and long ones in the last round: each CTA takes whole pairs, then a
    # stretch of the rest that makes up for their length; lists of at most 32 blocks, and of more
    check_prefill(nq, nk, heads, seed=heads)


@pytest.mark.parametrize("nq,nk", [([1024, 0, 1100, 2049, 1500, 3, 1300, 1800, 1, 769], None),
                                   ([1025, 768, 1536, 1, 2500, 900, 1700, 1300], [1400, 768, 2000, 700, 2500, 1000, 1650, 1300])])
def test_prefill_pairs_in_turn_with_short_blocks_last(nq, nk):
    # at least eight pairs a CTA, and sequences long enough that the first quarter of their blocks comes in a second pass
    heads = 32
    nk = nk or nq
    assert sum(-(-n // 256) for n in nq) * heads >= 8 * torch.cuda.get_device_properties(0).multi_processor_count
    check_prefill(nq, nk, heads, seed=len(nq))


@pytest.mark.parametrize("heads", [1, 5, 16, 17, 48, 64, 65, 128])
def test_decode_heads_on_latents_of_256(heads):
    lens = [1, 70, 333, 0, 2000]
    cache, table, sl, rows = paged_latents(lens, 32, 256, seed=heads, gap=40)
    q = queries(len(lens), 1, heads, 320, seed=heads)
    out, lse = run_decode(q, cache, table, sl, 256, SCALE)
    assert_attention(out, lse, decode_reference(q, lambda r, n: rows[r][:n], lens, SCALE, 256), f"heads {heads}")


@pytest.mark.parametrize("L,heads", [(2, 32), (3, 16), (4, 128), (5, 8), (7, 1), (70, 2)])
def test_decode_draft_tokens_on_latents_of_256(L, heads):
    lens = [0, 1, L - 1, L, L + 1, 64 + L, 129, 700]
    cache, table, sl, rows = paged_latents(lens, 16, 256, seed=L, width_extra=3)
    q = queries(len(lens), L, heads, 320, seed=L)
    out, lse = run_decode(q, cache, table, sl, 256, SCALE)
    assert_attention(out, lse, decode_reference(q, lambda r, n: rows[r][:n], lens, SCALE, 256), f"L {L} heads {heads}")


@pytest.mark.parametrize("lens,heads", [([40000], 32), ([9999, 3, 25000], 16), ([6400] * 5, 64), ([20000, 1], 128)])
def test_decode_long_contexts_on_latents_of_256(lens, heads):
    cache, table, sl, rows = paged_latents(lens, 64, 256, seed=heads)
    q = queries(len(lens), 1, heads, 320, seed=heads)
    out, lse = run_decode(q, cache, table, sl, 256, SCALE)
    assert_attention(out, lse, decode_reference(q, lambda r, n: rows[r][:n], lens, SCALE, 256), "long")
    again, lse2 = run_decode(q, cache, table, sl, 256, SCALE)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("n,L,heads", [(40, 3, 8), (130, 5, 8), (66, 4, 16), (20000, 6, 32), (64, 70, 1), (300, 4, 64)])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_decode_values_that_are_not_finite_in_latents_of_256(n, L, heads, bad):
    cache, table, sl, rows = paged_latents([n], 16, 256, seed=n + L)
    q = queries(1, L, heads, 320, seed=L)
    tok, dims = n - 2, [9, 130, 255]
    q[..., dims] = 0
    ref = decode_reference(q, lambda r, k: rows[r][:k], [n], SCALE, 256)
    cache[table[0, tok // 16].long(), 0, tok % 16, dims] = bad
    out, lse = run_decode(q, cache, table, sl, 256, SCALE)
    assert torch.isnan(out[0, L - 2:]).all() and torch.isnan(lse[0, L - 2:]).all()
    assert_attention(out[:, :L - 2], lse[:, :L - 2], [x[:, :L - 2] for x in ref], f"n {n} L {L}")


def test_calls_in_a_row_on_one_workspace():
    """Appends, decode steps of other sizes and prompts queued without a wait: each kernel may come while the one before
    it runs out, and they share their workspaces."""
    g = wl.generator(31, DEV)
    page, N, R = 16, 600, 5
    bt, sl, ref = torch.full((R, 100), -1, dtype=torch.int32, device=DEV), torch.zeros(R, dtype=torch.int32, device=DEV), torch.zeros(N, dtype=torch.int32, device=DEV)
    pt = kda.page_table_descriptor(bt, sl, ref, page)
    cache = poisoned(N, 1, page, 576)
    ids = torch.arange(R, dtype=torch.int32, device=DEV)
    ms, md, info = (torch.empty(n, dtype=torch.int32, device=DEV) for n in (R, R, 4))
    pws = torch.empty(kda.kda_pages_workspace_size(N, R), dtype=torch.uint8, device=DEV)
    steps = [[1000, 3, 0, 64, 129], [1, 1, 1, 1, 1], [200, 61, 5, 3, 0], [1, 1, 1, 1, 1], [1, 2, 3, 4, 5]]
    forms = [(1, 32), (2, 8), (1, 128), (1, 16), (4, 64)]  # query tokens, heads
    dws = torch.empty(max(kda.kda_latent_decode_workspace_size(R, L, H, 512, 64) for L, H in forms), dtype=torch.uint8, device=DEV)
    prompts = [([300, 5], [300, 900], 4), ([1500], [1500], 1), ([60] * 40, [60] * 40, 3), ([1], [3000], 8), ([64, 200], [64, 200], 2)]
    batches = [prompt_batch(nq, nk, H, seed=i) for i, (nq, nk, H) in enumerate(prompts)]
    fws = torch.empty(max(kda.kda_latent_prefill_workspace_size(sum(nq), len(nq), H) for nq, _, H in prompts), dtype=torch.uint8, device=DEV)
    work = []
    for new, (L, H), (q, kn, kr, v, cu_q, cu_k) in zip(steps, forms, batches):
        work.append(dict(new=torch.tensor(new, dtype=torch.int32, device=DEV), cu=torch.tensor([0] + new, device=DEV).cumsum(0).int(),
                         rows=torch.randn(sum(new), 576, generator=g, device=DEV).to(BF), q=torch.randn(R, L, H, 576, generator=g, device=DEV).to(BF),
                         out=poisoned(R, L, H, 512), lse=torch.full((R, L, H), math.nan, device=DEV),
                         cq=torch.tensor(cu_q, dtype=torch.int32, device=DEV), ck=torch.tensor(cu_k, dtype=torch.int32, device=DEV),
                         po=poisoned(q.shape[0], q.shape[1], 128), pl=torch.full(q.shape[:2], math.nan, device=DEV)))
    torch.cuda.synchronize()
    for w, (q, kn, kr, v, _, _) in zip(work, batches):
        kda.kda_pages_reserve(pt, ids, w["new"], ms, md, info, pws)
        kda.kda_pages_copy(cache, ms, md)
        kda.kda_latent_append(w["rows"], w["cu"], ids, pt, cache)
        kda.kda_latent_decode(w["q"], cache, bt, sl, w["out"], dws, latent_dim=512, scale=SCALE, lse=w["lse"])
        kda.kda_latent_prefill(q, kn, kr, v, w["cq"], w["ck"], w["po"], fws, scale=SCALE, lse=w["pl"])
    torch.cuda.synchronize()
    assert int(info[0]) == 0 and kda.kda_prefill_workspace_status(dws) == 0 and kda.kda_prefill_workspace_status(fws) == 0
    held = [torch.empty(0, 576, dtype=BF, device=DEV) for _ in range(R)]
    for i, (w, new, (q, kn, kr, v, cu_q, cu_k)) in enumerate(zip(work, steps, batches)):
        at = 0
        for r, n in enumerate(new):
            held[r] = torch.cat([held[r], w["rows"][at:at + n]])
            at += n
        assert_attention(w["out"], w["lse"], decode_reference(w["q"], lambda r, n: held[r][:n], [h.shape[0] for h in held], SCALE, 512), f"step {i}")
        assert_attention(w["po"], w["pl"], prefill_reference(q, kn, kr, v, cu_q, cu_k, SCALE), f"prompts {i}")
