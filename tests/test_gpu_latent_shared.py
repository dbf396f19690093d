"""Attention of groups of requests that hold the same first pages (kda_latent_decode_shared) on the GPU, against the plain 64-bit
form of each request alone (tests/latent_helpers.py: formulas and tolerances).  Whatever lies outside a request's tokens holds NaN
and infinities."""
import math

import pytest
import torch

import kimi_delta_attention_varlen_gb300 as kda
from kimi_delta_attention_varlen_gb300 import workloads as wl
from tests.latent_helpers import assert_attention, decode_reference
from tests.test_gpu_latent import paged_latents, poisoned, queries

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
SCALE = 192 ** -0.5


def grouped(groups, page, dl, seed, gap=0, spare=3, width_extra=0):
    """groups: [(prefix, [suffix lengths])].  The whole pages of a prefix are held together, the page that it ends in is each
    member's own.  (cache, table, seq_lens, rows per request, cu_groups, shared) """
    lens, cu = [], [0]
    for prefix, suffixes in groups:
        lens += [prefix + s for s in suffixes]
        cu.append(len(lens))
    cache, table, sl, rows = paged_latents(lens, page, dl, seed, gap, spare, width_extra)
    for (prefix, suffixes), a in zip(groups, cu):
        if not suffixes:
            continue
        whole = prefix // page
        for r in range(a + 1, a + len(suffixes)):
            table[r, :whole] = table[a, :whole]
            rows[r][:prefix] = rows[a][:prefix]
            if prefix % page:  # the page that the prefix ends in
                cache[table[r, whole].long(), 0, :prefix % page] = rows[a][whole * page:prefix]
    i32 = dict(dtype=torch.int32, device=DEV)
    return cache, table, sl, rows, torch.tensor(cu, **i32), torch.tensor([p for p, _ in groups], **i32)


def with_ballast(cache, table, sl, cu, shared, q):
    """The same batch with one more group behind it, 300 entries that share 4,096 tokens: enough for sharing to pay, so that the groups
    in front of it are computed together however small they are (alone the call leaves them to the plain kernel).
    (cache, table, sl, cu, shared, q) with those entries; entries are picked by row, so req is not used with it."""
    M, page, D = 300, cache.shape[2], cache.shape[3]
    need = 4096 // page + 1
    N = cache.shape[0]
    g = wl.generator(N, DEV)
    more = torch.empty(N + need, 1, page, D, dtype=BF, device=DEV)
    more[:N] = cache
    more[N:] = torch.randn(need, 1, page, D, generator=g, device=DEV).to(BF)
    W = max(table.shape[1], need)
    wide = torch.full((table.shape[0] + M, W), -1, dtype=torch.int32, device=DEV)
    wide[:table.shape[0], :table.shape[1]] = table
    wide[wide == N] = N + need  # a number behind the pool stays one
    wide[table.shape[0]:, :need] = torch.arange(N, N + need, dtype=torch.int32, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    return (more, wide, torch.cat([sl, torch.full((M,), 4096, **i32)]), torch.cat([cu, cu[-1:] + M]), torch.cat([shared, torch.tensor([4096], **i32)]),
            torch.cat([q, torch.randn(M, *q.shape[1:], generator=g, device=DEV).to(BF)]))


def run_shared(q, cache, table, lens, cu, shared, dl, scale=SCALE, req=None, stream=None, lse=True):
    R, L, H, D = q.shape
    out = poisoned(R, L, H, dl)
    ls = torch.full((R, L, H), math.nan, device=DEV) if lse else None
    ws = torch.empty(kda.kda_latent_decode_shared_workspace_size(R, cu.numel() - 1, L, H, dl, D - dl), dtype=torch.uint8, device=DEV)
    ws.fill_(0xA5)
    torch.cuda.synchronize()
    kda.kda_latent_decode_shared(q, cache, table, lens, cu, shared, out, ws, latent_dim=dl, scale=scale, req=req, lse=ls, stream=stream)
    torch.cuda.synchronize()
    assert kda.kda_prefill_workspace_status(ws) == 0
    return out, ls


def run_both(q, cache, table, sl, cu, shared, dl, scale=SCALE):
    """The batch alone, and its entries out of the batch with ballast."""
    R = q.shape[0]
    yield run_shared(q, cache, table, sl, cu, shared, dl, scale)
    cache, table, sl, cu, shared, q = with_ballast(cache, table, sl, cu, shared, q)
    out, lse = run_shared(q, cache, table, sl, cu, shared, dl, scale)
    # of the ballast, whose entries all see the same tokens, two
    rows = cache[table[R, :4096 // cache.shape[2] + 1].long()].reshape(-1, cache.shape[3])[:4096]
    assert_attention(out[[R, -1]], lse[[R, -1]], decode_reference(q[[R, -1]], lambda r, n: rows[:n], [4096, 4096], scale, dl), "ballast")
    yield out[:R], lse[:R]


def check_shared(groups, page, dl, heads, L=1, seed=0, scale=SCALE, **kw):
    cache, table, sl, rows, cu, shared = grouped(groups, page, dl, seed, **kw)
    q = queries(sl.numel(), L, heads, dl + 64, seed=seed)
    lens = sl.tolist()
    ref = decode_reference(q, lambda r, n: rows[r][:n], lens, scale, dl)
    for k, (out, lse) in enumerate(run_both(q, cache, table, sl, cu, shared, dl, scale)):
        assert_attention(out, lse, ref, f"page {page} dl {dl} heads {heads} L {L} {'with ballast' if k else 'alone'}")


@pytest.mark.parametrize("dl", [512, 256])
@pytest.mark.parametrize("page", [8, 48, 64, 200])
def test_lengths_and_pages(page, dl):
    check_shared([(300, [1, 0, 64, 65]), (64, [5, 200]), (0, [70, 0]), (page, [1, 1, 1]), (3 * page - 1, [0, 2]), (1000, [33]), (129, [127, 128, 129])],
                 page, dl, 32, seed=page + dl)


@pytest.mark.parametrize("heads", [1, 2, 5, 8, 16, 17, 32, 48, 64, 100, 128, 192])
def test_heads(heads):
    check_shared([(200, [1, 70, 3]), (65, [9, 10])], 16, 512, heads, seed=heads, gap=24)


@pytest.mark.parametrize("prefix", [63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256, 257, 383, 384, 640])
def test_prefix_lengths(prefix):
    check_shared([(prefix, [3, 90, 1])], 8, 512, 16, seed=prefix)


@pytest.mark.parametrize("members", [1, 2, 3, 4, 5, 7, 8, 9, 16, 33])
def test_members(members):
    check_shared([(321, [(7 * i) % 50 for i in range(members)]), (100, [5] * (members + 1))], 32, 256, 32, seed=members)


@pytest.mark.parametrize("L,heads", [(2, 32), (3, 16), (4, 128), (7, 1), (70, 2)])
def test_draft_tokens_are_causal(L, heads):
    check_shared([(200, [L, L + 1, 64 + L]), (130, [L + 3, 2 * L])], 16, 512, heads, L=L, seed=L, width_extra=3)


@pytest.mark.parametrize("L", [1, 3, 7, 70])
def test_prefix_that_is_not_behind_all_query_tokens(L):
    """Requests that end inside the prefix or just behind it: the drafts' mask falls into the shared pages, members are shorter
    than what is called shared."""
    page, dl = 16, 256
    cache, table, sl, rows, cu, shared = grouped([(256, [0, 1, 2, 100]), (160, [0, 0])], page, dl, seed=L)
    lens = [256, 257, 140, 356, 160, 33]  # the third and the last are shorter than their prefix
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    q = queries(6, L, 8, dl + 64, seed=L)
    for told in ([256, 160], [10 ** 6, 10 ** 6]):
        if told[0] > 256:  # members that hold the same pages throughout
            table[:4] = table[3].clone()
            table[4:] = table[4].clone()
            for r in range(4):
                rows[r] = rows[3]
            rows[5] = rows[4]
        ref = decode_reference(q, lambda r, n: rows[r][:n], lens, SCALE, dl)
        for out, lse in run_both(q, cache, table, sl, cu, torch.tensor(told, dtype=torch.int32, device=DEV), dl):
            assert_attention(out, lse, ref, f"L {L} told {told}")


def test_nothing_shared_is_plain_decode():
    lens = [100, 0, 3000, 64]
    cache, table, sl, rows = paged_latents(lens, 64, 512, seed=3)
    q = queries(4, 1, 32, 576, seed=3)
    ref = decode_reference(q, lambda r, n: rows[r][:n], lens, SCALE, 512)
    i32 = dict(dtype=torch.int32, device=DEV)
    for cu, shared in (([0, 4], [0]), ([0, 4], [63]), ([0, 4], [-5]), ([0, 1, 2, 3, 4], [100, 0, 3000, 64]), ([0, 0, 4, 4], [9, 0, 9]), ([2, 3], [640])):
        for out, lse in run_both(q, cache, table, sl, torch.tensor(cu, **i32), torch.tensor(shared, **i32), 512) if cu[-1] == 4 else \
                [run_shared(q, cache, table, sl, torch.tensor(cu, **i32), torch.tensor(shared, **i32), 512)]:
            assert_attention(out, lse, ref, f"{cu} {shared}")


@pytest.mark.parametrize("itype", [torch.int32, torch.int64])
def test_requests_picked_by_index_and_invalid_ones(itype):
    cache, table, sl, rows, cu, shared = grouped([(300, [1, 40, 5]), (70, [1, 2])], 16, 512, seed=4)
    req = [2, -1, 0, 1, 9, 4, 3]
    cu = torch.tensor([0, 5, 7], dtype=torch.int32, device=DEV)
    q = queries(7, 2, 16, 576, seed=4)
    out, lse = run_shared(q, cache, table, sl, cu, shared, 512, req=torch.tensor(req, dtype=itype, device=DEV))
    n = [int(sl[r]) if 0 <= r < 5 else 0 for r in req]
    assert_attention(out, lse, decode_reference(q, lambda i, k: rows[req[i]][:k] if n[i] else rows[0][:0], n, SCALE, 512))
    assert (out[1] == 0).all() and (lse[4] == -math.inf).all()
    only_bad = torch.full((7,), -1, dtype=itype, device=DEV)
    out, lse = run_shared(q, cache, table, sl, cu, shared, 512, req=only_bad)
    assert (out == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("groups,heads", [([(40000, [100] * 4)], 32), ([(20000, [1] * 70)], 16), ([(9999, [3] * 9), (25000, [70] * 5)], 64), ([(17000, [500, 20000])], 128)])
def test_long_prefixes(groups, heads):
    check_shared(groups, 64, 512, heads, seed=heads)


@pytest.mark.parametrize("dl", [512, 256])
def test_a_prefix_of_millions_of_tokens(dl):
    """Four entries on 3.2 million tokens, the same 50 pages over and over: the accumulator of the prefix is set aside."""
    page, pages, times, H = 64, 50, 1000, 32
    cache, table, _, rows = paged_latents([page * pages] + [page + 5 + r for r in range(4)], page, dl, seed=52)
    listed = table[0, :pages].repeat(times)
    tables = torch.full((4, pages * times + 2), -1, dtype=torch.int32, device=DEV)
    tables[:, :pages * times] = listed
    tables[:, pages * times:] = table[1:, :2]
    n = [page * pages * times + page + 5 + r for r in range(4)]
    i32 = dict(dtype=torch.int32, device=DEV)
    q = queries(4, 1, H, dl + 64, seed=52)
    out, lse = run_shared(q, cache, tables, torch.tensor(n, **i32), torch.tensor([0, 4], **i32), torch.tensor([page * pages * times], **i32), dl)
    for r in range(4):
        x = torch.cat([rows[0], rows[1 + r]]).double().cpu()
        count = torch.ones(x.shape[0], dtype=torch.float64)
        count[:page * pages] = times
        qq = q[r, 0].double().cpu()
        z = qq @ x.T * SCALE + count.log()
        p = torch.softmax(z, -1)
        bound = (qq.abs() @ x.abs().T * SCALE).amax(-1)
        assert_attention(out[r, 0], lse[r, 0], (p @ x[:, :dl], p @ x[:, :dl].abs(), torch.logsumexp(z, -1), bound))


def test_many_groups():
    g = torch.Generator().manual_seed(8)
    groups = [(int(torch.randint(0, 400, (1,), generator=g)), torch.randint(0, 90, (int(torch.randint(0, 6, (1,), generator=g)),), generator=g).tolist())
              for _ in range(150)]
    check_shared(groups, 16, 256, 8, seed=8)


@pytest.mark.parametrize("scale", [1e-6, 0.3, 3.0])
def test_scales(scale):
    check_shared([(500, [30, 70]), (200, [100])], 32, 512, 32, seed=5, scale=scale)


@pytest.mark.parametrize("where", ["prefix", "suffix"])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_values_that_are_not_finite_reach_only_requests_that_see_them(where, bad):
    """A value of the prefix reaches all members of its group, one of a suffix its request alone."""
    page, dl = 16, 512
    cache, table, sl, rows, cu, shared = grouped([(200, [9, 70, 30]), (130, [20, 25])], page, dl, seed=6)
    q = queries(5, 1, 16, 576, seed=6)
    dims = [9, 300, 511]
    q[..., dims] = 0
    ref = decode_reference(q, lambda r, n: rows[r][:n], sl.tolist(), SCALE, dl)
    tok = 100 if where == "prefix" else 250
    cache[table[1, tok // page].long(), 0, tok % page, dims] = bad  # 0 * bad is no number: the score is one neither
    hit = [0, 1, 2] if where == "prefix" else [1]
    clean = [r for r in range(5) if r not in hit]
    for out, lse in run_both(q, cache, table, sl, cu, shared, dl):
        assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
        assert_attention(out[clean], lse[clean], [x[clean] for x in ref], where)


@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("tok", [125, 126, 60])
def test_values_of_the_prefix_that_some_query_tokens_do_not_see(bad, tok):
    """The requests end with the prefix: the first query tokens see none of its last tokens, nor what is not finite in them."""
    page, dl, L = 16, 256, 4
    cache, table, sl, rows, cu, shared = grouped([(128, [0, 0, 0])], page, dl, seed=7)
    lens = [128, 127, 126]
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    q = queries(3, L, 8, dl + 64, seed=7)
    q[..., 9] = 0
    ref = decode_reference(q, lambda r, n: rows[r][:n], lens, SCALE, dl)
    cache[table[0, tok // page].long(), 0, tok % page, 9] = bad
    sees = torch.tensor([[tok < n - (L - 1 - t) for t in range(L)] for n in lens])
    clean = ~sees
    for out, lse in run_both(q, cache, table, sl, cu, shared, dl):
        assert torch.isnan(out.cpu()[sees]).all() and torch.isnan(lse.cpu()[sees]).all()
        if clean.any():
            assert_attention(out.cpu()[clean], lse.cpu()[clean], [x[clean] for x in ref], f"token {tok}")


def test_queries_that_are_not_finite_stay_in_their_rows():
    cache, table, sl, rows, cu, shared = grouped([(200, [9, 70, 30])], 16, 512, seed=9)
    q = queries(3, 1, 32, 576, seed=9)
    ref = decode_reference(q, lambda r, n: rows[r][:n], sl.tolist(), SCALE, 512)
    q[0, 0, 3, 17], q[1, 0, 9, 540], q[2, 0, 30, 0] = math.nan, math.inf, -math.inf
    bad = torch.zeros(3, 1, 32, dtype=torch.bool)
    bad[0, 0, 3] = bad[1, 0, 9] = bad[2, 0, 30] = True
    for out, lse in run_both(q, cache, table, sl, cu, shared, 512):
        assert torch.isnan(out.cpu()[bad]).all() and torch.isnan(lse.cpu()[bad]).all()
        assert_attention(out.cpu()[~bad], lse.cpu()[~bad], [x[~bad] for x in ref])


def test_scores_that_differ_widely_between_prefix_and_suffix():
    """All the weight in the prefix, or all in the suffix: the join takes both maxima as they are."""
    page, dl = 16, 256
    cache, table, sl, rows, cu, shared = grouped([(160, [40, 30])], page, dl, seed=10)
    for f, r in ((1, 0), (0, 1)):
        for t in range(sl[r]):
            big = (t < 160) == bool(f)
            rows[r][t, 0] = 30.0 if big else -30.0
    for r in (0, 1):
        for j in range(-(-int(sl[r]) // page)):
            part = rows[r][j * page:(j + 1) * page]
            if j >= 10 or r == 0:
                cache[table[r, j].long(), 0, :part.shape[0]] = part
        rows[r][:160] = rows[0][:160]
    q = queries(2, 1, 4, dl + 64, seed=10)
    q[..., 0] = torch.tensor([20.0, -20.0, 200.0, -200.0], device=DEV)
    ref = decode_reference(q, lambda r, n: rows[r][:n], sl.tolist(), 1.0, dl)
    for out, lse in run_both(q, cache, table, sl, cu, shared, dl, scale=1.0):
        assert_attention(out, lse, ref)


def test_invalid_pages_read_as_zero_rows():
    cache, table, sl, rows, cu, shared = grouped([(96, [70, 100])], 32, 512, seed=11)
    table[:, 1], table[1, 4] = cache.shape[0], -7
    for r in (0, 1):
        rows[r][32:64] = 0
    rows[1][128:160] = 0
    q = queries(2, 1, 32, 576, seed=11)
    ref = decode_reference(q, lambda r, n: rows[r][:n], sl.tolist(), SCALE, 512)
    for out, lse in run_both(q, cache, table, sl, cu, shared, 512):
        assert_attention(out, lse, ref)


def test_forked_requests_share_what_the_fork_left_them():
    """kda_pages_fork, reserve with copy on write, append, then shared decode with the parent's length at the fork."""
    page, dl, n0 = 16, 512, 200
    i32 = dict(dtype=torch.int32, device=DEV)
    table, sl, ref = torch.full((6, 30), -1, **i32), torch.zeros(6, **i32), torch.zeros(120, **i32)
    pt = kda.page_table_descriptor(table, sl, ref, page)
    cache = poisoned(120, 1, page, 576)
    ws = torch.empty(kda.kda_pages_workspace_size(120, 6), dtype=torch.uint8, device=DEV)
    info = torch.empty(4, **i32)

    def grow(req, counts, x):
        src, dst = torch.empty(len(req), **i32), torch.empty(len(req), **i32)
        rq = torch.tensor(req, **i32)
        kda.kda_pages_reserve(pt, rq, torch.tensor(counts, **i32), src, dst, info, ws)
        kda.kda_pages_copy(cache, src, dst)
        kda.kda_latent_append(x, torch.tensor([0] + counts, **i32).cumsum(0, dtype=torch.int32), rq, pt, cache)

    g = wl.generator(12, DEV)
    x = torch.randn(n0, 576, generator=g, device=DEV).to(BF)
    grow([0], [n0], x)
    kda.kda_pages_fork(pt, torch.zeros(3, **i32), torch.tensor([2, 3, 5], **i32))
    req, history = [0, 2, 3, 5], {}
    counts = [1, 40, 7, 16]
    y = torch.randn(sum(counts), 576, generator=g, device=DEV).to(BF)
    grow(req, counts, y)
    at = 0
    for r, c in zip(req, counts):
        history[r] = torch.cat([x, y[at:at + c]])
        at += c
    q = queries(4, 1, 32, 576, seed=12)
    out, lse = run_shared(q, cache, table, sl, torch.tensor([0, 4], **i32), torch.tensor([n0], **i32), dl, req=torch.tensor(req, **i32))
    assert_attention(out, lse, decode_reference(q, lambda i, n: history[req[i]][:n], [n0 + c for c in counts], SCALE, dl))


def test_repeatable_on_any_stream_and_without_lse():
    cache, table, sl, rows, cu, shared = grouped([(3000, [17, 900, 0]), (500, [64] * 20), (0, [12345])], 64, 512, seed=13)
    q = queries(sl.numel(), 1, 32, 576, seed=13)
    a, la = run_shared(q, cache, table, sl, cu, shared, 512)
    b, lb = run_shared(q, cache, table, sl, cu, shared, 512, stream=torch.cuda.Stream())
    assert torch.equal(a.view(torch.int16), b.view(torch.int16)) and torch.equal(la, lb)
    c, _ = run_shared(q, cache, table, sl, cu, shared, 512, lse=False)
    assert torch.equal(a.view(torch.int16), c.view(torch.int16))


def test_captured_in_a_graph_and_replayed_with_other_groups():
    cache, table, sl, rows, cu, shared = grouped([(320, [17, 90, 1]), (128, [64, 5])], 64, 512, seed=14)
    q = queries(5, 1, 32, 576, seed=14)
    out, lse = torch.empty(5, 1, 32, 512, dtype=BF, device=DEV), torch.empty(5, 1, 32, device=DEV)
    ws = torch.empty(kda.kda_latent_decode_shared_workspace_size(5, 2, 1, 32, 512, 64), dtype=torch.uint8, device=DEV)

    def call():
        kda.kda_latent_decode_shared(q, cache, table, sl, cu, shared, out, ws, latent_dim=512, scale=SCALE, lse=lse)

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            call()
    for told_cu, told, lens in (([0, 3, 5], [320, 128], sl.tolist()), ([0, 3, 5], [64, 0], sl.tolist()), ([0, 3, 3], [256, 9], [330, 340, 320, 10, 0]),
                                ([0, 0, 5], [7, 0], [337, 1, 64, 192, 133])):
        cu.copy_(torch.tensor(told_cu))
        shared.copy_(torch.tensor(told))
        sl.copy_(torch.tensor(lens))
        out.fill_(math.nan)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert_attention(out, lse, decode_reference(q, lambda r, n: rows[r][:n], lens, SCALE, 512), f"{told_cu} {told}")


@pytest.mark.parametrize("itype", [torch.int32, torch.int64])
def test_a_shared_batch_with_padding(itype):
    """400 entries on one prefix, every fifth of them invalid or empty, in a batch that sharing pays for; twice, bit for bit."""
    page, dl, R = 64, 512, 400
    cache, table, sl, rows, _, _ = grouped([(4096, [0, 40, 700])], page, dl, seed=21)
    pick = [(0, 1, 2, 1, -1)[i % 5] for i in range(R - 2)] + [7, 1]
    q = queries(R, 1, 16, 576, seed=21)
    i32 = dict(dtype=torch.int32, device=DEV)
    args = (q, cache, table, sl, torch.tensor([0, R], **i32), torch.tensor([4110], **i32), dl)
    req = torch.tensor(pick, dtype=itype, device=DEV)
    out, lse = run_shared(*args, req=req)
    again, _ = run_shared(*args, req=req)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    bad = [i for i, p in enumerate(pick) if p not in (0, 1, 2)]
    assert (out[bad] == 0).all() and (lse[bad] == -math.inf).all()
    some = [0, 1, 2, 3, 200, 201, 202, 396, 397, 399]
    some = [i for i in some if pick[i] in (0, 1, 2)]
    ref = decode_reference(q[some], lambda i, n: rows[pick[some[i]]][:n], [int(sl[pick[i]]) for i in some], SCALE, dl)
    assert_attention(out[some], lse[some], ref)


def test_a_shared_batch_captured_and_replayed():
    cache, table, sl, rows, cu, shared = grouped([(320, [17, 90, 1]), (128, [64, 5])], 64, 512, seed=14)
    cache, table, sl, cu, shared, q = with_ballast(cache, table, sl, cu, shared, queries(5, 1, 32, 576, seed=14))
    R = q.shape[0]
    out, lse = torch.empty(R, 1, 32, 512, dtype=BF, device=DEV), torch.empty(R, 1, 32, device=DEV)
    ws = torch.empty(kda.kda_latent_decode_shared_workspace_size(R, 3, 1, 32, 512, 64), dtype=torch.uint8, device=DEV)

    def call():
        kda.kda_latent_decode_shared(q, cache, table, sl, cu, shared, out, ws, latent_dim=512, scale=SCALE, lse=lse)

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            call()
    for told, lens in (([320, 128, 4096], [337, 410, 321, 192, 133]), ([64, 0, 4096], [337, 410, 321, 192, 133]), ([320, 128, 0], [337, 410, 321, 192, 133]),
                       ([256, 128, 4000], [330, 340, 320, 10, 0])):
        shared.copy_(torch.tensor(told))
        sl[:5] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        out.fill_(math.nan)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert kda.kda_prefill_workspace_status(ws) == 0
        assert_attention(out[:5], lse[:5], decode_reference(q[:5], lambda r, n: rows[r][:n], lens, SCALE, 512), f"{told}")


def test_which_batches_share():
    """Alone, a small batch is the plain call's, bit for bit; in a batch that sharing pays for it is summed in another order; entries of
    64 rows are the plain call's in any batch."""
    for heads, same_in_ballast in ((32, False), (64, True)):
        cache, table, sl, rows, cu, shared = grouped([(1280, [17, 90, 1]), (640, [64, 5])], 64, 512, seed=30)
        q = queries(5, 1, heads, 576, seed=30)
        plain = torch.empty(5, 1, heads, 512, dtype=BF, device=DEV)
        ws = torch.empty(kda.kda_latent_decode_workspace_size(5, 1, heads, 512, 64), dtype=torch.uint8, device=DEV)
        kda.kda_latent_decode(q, cache, table, sl, plain, ws, latent_dim=512, scale=SCALE)
        (alone, _), (among, _) = run_both(q, cache, table, sl, cu, shared, 512)
        assert torch.equal(alone.view(torch.int16), plain.view(torch.int16))
        # (the same kernel may cut its items elsewhere in a larger batch: equality of bits says the most about the smaller difference)
        far = (among.float() - plain.float()).abs().max() / plain.float().abs().max()
        assert far <= 2.0 ** -6 and (same_in_ballast or not torch.equal(among.view(torch.int16), plain.view(torch.int16)))


def test_strided_block_tables_and_two_streams():
    sets = []
    for k in range(2):
        cache, table, sl, rows, cu, shared = grouped([(600, [17, 90, 1]), (128 + 64 * k, [64, 5])], 64, 512, seed=90 + k, gap=64)
        q = queries(5, 1, 32, 576, seed=90 + k)
        cache, table, sl, cu, shared, q = with_ballast(cache, table, sl, cu, shared, q)
        wide = torch.full((table.shape[0], table.shape[1] + 3), 1 << 30, dtype=torch.int32, device=DEV)
        wide[:, 1:-2] = table
        ws = torch.empty(kda.kda_latent_decode_shared_workspace_size(q.shape[0], 3, 1, 32, 512, 64), dtype=torch.uint8, device=DEV)
        sets.append((cache, wide[:, 1:-2], sl, rows, cu, shared, q, ws, torch.empty(*q.shape[:3], 512, dtype=BF, device=DEV), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(6):
        for cache, table, sl, rows, cu, shared, q, ws, out, st in sets:
            kda.kda_latent_decode_shared(q, cache, table, sl, cu, shared, out, ws, latent_dim=512, scale=SCALE, stream=st)
    torch.cuda.synchronize()
    for cache, table, sl, rows, cu, shared, q, ws, out, st in sets:
        assert kda.kda_prefill_workspace_status(ws) == 0
        assert_attention(out[:5], None, decode_reference(q[:5], lambda r, n: rows[r][:n], sl[:5].tolist(), SCALE, 512))


def test_two_calls_queued_on_two_workspaces():
    sets = [grouped([(600, [17, 90, 1]), (128, [64, 5])], 64, 512, seed=s) for s in (15, 16)]
    qs = [queries(5, 1, 32, 576, seed=s) for s in (15, 16)]
    outs, wss = [torch.empty(5, 1, 32, 512, dtype=BF, device=DEV) for _ in range(2)], []
    for _ in range(2):
        wss.append(torch.empty(kda.kda_latent_decode_shared_workspace_size(5, 2, 1, 32, 512, 64), dtype=torch.uint8, device=DEV))
    for _ in range(5):
        for k in range(2):
            cache, table, sl, rows, cu, shared = sets[k]
            kda.kda_latent_decode_shared(qs[k], cache, table, sl, cu, shared, outs[k], wss[k], latent_dim=512, scale=SCALE)
    torch.cuda.synchronize()
    for k in range(2):
        cache, table, sl, rows, cu, shared = sets[k]
        assert_attention(outs[k], None, decode_reference(qs[k], lambda r, n: rows[r][:n], sl.tolist(), SCALE, 512))
