"""The latent-attention and cache-page operators on real work: inputs, plain forms, sizes.

A hybrid decoder alternates recurrent (delta-rule) layers with attention layers whose keys and
values come from one shared latent vector a token.  Its server keeps, next to the recurrent
states, a paged cache of those latents: each token is one row [latent | rope] of a page, a page
holds `page` tokens, and a block table lists each request's pages.  Four operators are measured:

  decode    absorbed form: every head's query, already multiplied into the latent space, attends
            to the latents themselves; one token a request, or a few draft tokens (causal)
  prefill   expanded form: per-head keys (nope part per head, one shared rope part) and values,
            causal, over a batch of sequences of different lengths, with or without a prefix
  turnover  one serving step of page upkeep: fork requests, reserve room for the new tokens
            (copy-on-write of shared last pages), copy those pages, append the new latents,
            release the requests that ended
  compact   live pages move to the lowest page numbers: plan, table update, page copies

`run` computes them in elementary torch operations where `own` is false and calls the framework
where it is true.
"""
import math
import random

import torch

own = False
DEV = "cuda"
LATENT, ROPE = 512, 64          # generic latent width and shared rope width
NOPE, VDIM = 128, 128           # per-head sizes of the expanded form (the framework's head size)


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one request of a chat a thousand tokens long: a call where latency is all
        dict(name="decode one request", op="decode", requests=1, lo=1009, hi=1009, draft=1, heads=32, page=64),
        # a modest batch on small pages, few heads a GPU
        dict(name="decode 48 short, 16 heads", op="decode", requests=48, lo=1, hi=2047, draft=1, heads=16, page=16),
        # long-context requests: few rows, the cache axis has to be split over the SMs
        dict(name="decode 2 long contexts", op="decode", requests=2, lo=131072, hi=131072, draft=1, heads=32, page=64),
        # a loaded server's step: the lengths of the framework's batched workload, 512 requests
        dict(name="decode 512 requests", op="decode", requests=512, lo=512, hi=8192, draft=1, heads=32, page=64),
        # verification of 4 draft tokens, all 128 heads on one GPU
        dict(name="verify 4 drafts, 128 heads", op="decode", requests=33, lo=1500, hi=6001, draft=4, heads=128, page=48),
        # three short prompts (the framework's smallest batch)
        dict(name="prefill 3 short prompts", op="prefill", seqs=3, lo=37, hi=100, prefix=0, heads=32),
        # prompts continued on cached prefixes: few queries against many keys
        dict(name="prefill on long prefixes", op="prefill", seqs=5, lo=201, hi=777, prefix=9001, heads=16),
        # the framework's batched workload: 16 prompts of 512 to 8192 tokens
        dict(name="prefill 16 prompts", op="prefill", seqs=16, lo=512, hi=8192, prefix=0, heads=32),
        # a step of a small server: a few forks, one new token each
        dict(name="turnover 24 requests", op="turnover", requests=24, forks=6, ended=3, new=1, lo=1, hi=3000, pages=2048, page=64),
        # a loaded server that samples in parallel: half of the requests forked, a few draft tokens each
        dict(name="turnover 512 requests", op="turnover", requests=512, forks=256, ended=100, new=3, lo=512, hi=8192, pages=68000, page=64),
        # a small pool after a burst
        dict(name="compact 300 pages", op="compact", pages=301, live=0.4, page=16),
        # a pool that filled up and then lost half of its requests
        dict(name="compact 24000 pages", op="compact", pages=24001, live=0.5, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prefill", "prefill", "turnover", "compact"])
    if op == "decode":
        heads, draft = rng.choice([8, 16, 32, 64, 128]), rng.choice([1, 1, 1, 2, 3, 5])
        hi = _log(rng, 2, 131072)
        # at most 512 requests, at most the largest listed case's tokens x rows
        most = max(1, min(512, int(2.2e6 / hi), int(7.0e7 / (hi * heads * draft))))
        return dict(op=op, requests=_log(rng, 1, most) if most > 1 else 1, lo=max(1, int(hi * rng.choice([0.1, 0.5, 1.0]))),
                    hi=hi, draft=draft, heads=heads, page=rng.choice([8, 16, 32, 48, 64, 64, 128, 200]))
    if op == "prefill":
        heads = rng.choice([2, 4, 8, 16, 32, 32, 48])
        hi = _log(rng, 2, 8192)
        prefix = rng.choice([0, 0, _log(rng, 1, 16384)])
        most = max(1, min(16, int(1.3e10 / (hi * (hi + prefix) * heads))))
        return dict(op=op, seqs=rng.randint(1, most), lo=max(1, int(hi * rng.choice([0.1, 0.5, 1.0]))), hi=hi, prefix=prefix,
                    heads=heads)
    if op == "turnover":
        requests = _log(rng, 2, 512)
        hi, page = _log(rng, 8, 8192), rng.choice([16, 32, 64, 128])
        forks = rng.randint(0, requests)
        pages = 2 * (requests + forks) * (2 + hi // page)
        return dict(op=op, requests=requests, forks=forks, ended=rng.randint(0, requests // 2), new=rng.choice([1, 1, 2, 5, 130]),
                    lo=rng.choice([1, hi // 2 + 1, hi]), hi=hi, pages=max(64, min(pages + 400, 4000000 // page)), page=page)
    return dict(op=op, pages=_log(rng, 16, 24000), live=rng.choice([0.1, 0.3, 0.5, 0.8, 0.95]), page=rng.choice([16, 32, 64, 64]))


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _lengths(n, lo, hi, gen):
    x = torch.randint(lo, hi + 1, (n,), generator=gen, device=DEV)
    x[0] = hi  # the longest is always there
    return x.to(torch.int32)


def _prompt_lengths(case):
    """Query and key lengths of a prefill case: lo..hi (the longest there once) and half to all of the prefix before them."""
    rng = random.Random(case["hi"])
    nq = [case["hi"]] + [rng.randint(case["lo"], case["hi"]) for _ in range(case["seqs"] - 1)]
    return nq, [n + rng.randint(case["prefix"] // 2, case["prefix"]) for n in nq]


def _random_cache(pages, page, gen):
    c = torch.empty(pages, 1, page, LATENT + ROPE, dtype=torch.bfloat16, device=DEV)
    return c.normal_(generator=gen)


def _tables(lens, page, pages, width, rows, gen):
    """Block tables of requests that hold random pages of the pool, their refcounts, -1 where unused."""
    n = lens.numel()
    need = (lens.long() + page - 1) // page
    used = torch.arange(width, device=DEV)[None, :] < need[:, None]
    perm = torch.randperm(pages, generator=gen, device=DEV)
    table = torch.full((rows, width), -1, dtype=torch.int32, device=DEV)
    ids = torch.cumsum(used.reshape(-1).long(), 0).reshape(n, width) - 1
    table[:n] = torch.where(used, perm[ids.clamp(0, pages - 1)].to(torch.int32), -1)
    ref = torch.zeros(pages, dtype=torch.int32, device=DEV)
    ref[perm[:int(need.sum())]] = 1
    return table, ref


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "decode":
        R, L, H, P = case["requests"], case["draft"], case["heads"], case["page"]
        lens = _lengths(R, max(case["lo"], L), max(case["hi"], L), g)
        width = -(-int(lens.max()) // P)
        pages = int(((lens.long() + P - 1) // P).sum()) + 7
        s = dict(cache=_random_cache(pages, P, g), lens=lens, scale=(NOPE + ROPE) ** -0.5,
                 q=torch.randn(R, L, H, LATENT + ROPE, generator=g, device=DEV).to(torch.bfloat16),
                 out=torch.empty(R, L, H, LATENT, dtype=torch.bfloat16, device=DEV), lse=torch.empty(R, L, H, device=DEV))
        s["table"], _ = _tables(lens, P, pages, width, R, g)
        # scratch that a program allocates once (the plain form has none)
        if own:
            import kimi_delta_attention_varlen_gb300 as kda
            s["workspace"] = torch.empty(kda.kda_latent_decode_workspace_size(R, L, H, LATENT, ROPE), dtype=torch.uint8, device=DEV)
    elif case["op"] == "prefill":
        B, H = case["seqs"], case["heads"]
        # the case fixes the lengths, the seed their order: every seed's batch has as many tokens
        nq, nk = _prompt_lengths(case)
        order = torch.randperm(B, generator=g, device=DEV)
        nq, nk = (torch.tensor(n, dtype=torch.int32, device=DEV)[order] for n in (nq, nk))
        cu_q, cu_k = (torch.nn.functional.pad(torch.cumsum(n, 0), (1, 0)).to(torch.int32) for n in (nq, nk))
        Tq, Tk = int(cu_q[-1]), int(cu_k[-1])
        # the up-projection's result: per head [nope key | value]; the rope key is the tail of the latent rows
        kv = torch.empty(Tk, H, NOPE + VDIM, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
        rows = torch.empty(Tk, LATENT + ROPE, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
        s = dict(q=torch.empty(Tq, H, NOPE + ROPE, dtype=torch.bfloat16, device=DEV).normal_(generator=g), k_nope=kv[..., :NOPE],
                 v=kv[..., NOPE:], k_rope=rows[:, LATENT:], cu_q=cu_q, cu_k=cu_k, spans=list(zip(cu_q.tolist(), cu_k.tolist())),
                 scale=(NOPE + ROPE) ** -0.5, out=torch.empty(Tq, H, VDIM, dtype=torch.bfloat16, device=DEV),
                 lse=torch.empty(Tq, H, device=DEV))
        if own:
            import kimi_delta_attention_varlen_gb300 as kda
            s["workspace"] = torch.empty(kda.kda_latent_prefill_workspace_size(Tq, B, H), dtype=torch.uint8, device=DEV)
    elif case["op"] == "turnover":
        R, F, P, N = case["requests"], case["forks"], case["page"], case["pages"]
        lens = _lengths(R, case["lo"], case["hi"], g)
        # a pool that is too small for the drawn lengths holds shorter requests
        room = max(1, (N - 2 * (R + F) * (1 + case["new"] // P)) // R - 1) * P
        lens = lens.clamp(max=room)
        width = -(-(int(lens.max()) + case["new"]) // P)
        rows = R + F + 3
        table, ref = _tables(lens, P, N, width, rows, g)
        all_lens = torch.zeros(rows, dtype=torch.int32, device=DEV)
        all_lens[:R] = lens
        first = torch.cat([table.reshape(-1), all_lens, ref])  # the tables in one buffer, as a server allocates them
        work = first.clone()
        a, b = table.numel(), table.numel() + rows
        src = torch.randint(0, R, (F,), generator=g, device=DEV).to(torch.int32)  # a request may be forked several times
        n = R + F
        req = torch.randperm(n, generator=g, device=DEV).to(torch.int32)
        s = dict(first=first, work=work, table=work[:a].view(rows, width), lens=work[a:b], ref=work[b:], page=P, cache=_random_cache(N, P, g),
                 src=src, dst=torch.arange(R, n, device=DEV, dtype=torch.int32), req=req, new=torch.full((n,), case["new"], dtype=torch.int32, device=DEV),
                 cu=torch.arange(0, (n + 1) * case["new"], case["new"], device=DEV, dtype=torch.int32),
                 x=torch.empty(n * case["new"], LATENT + ROPE, dtype=torch.bfloat16, device=DEV).normal_(generator=g),
                 ended=req[:case["ended"]].clone(), move_src=torch.empty(n, dtype=torch.int32, device=DEV),
                 move_dst=torch.empty(n, dtype=torch.int32, device=DEV), info=torch.empty(4, dtype=torch.int32, device=DEV))
        if own:
            import kimi_delta_attention_varlen_gb300 as kda
            s["workspace"] = torch.empty(kda.kda_pages_workspace_size(N, n), dtype=torch.uint8, device=DEV)
    else:
        P, N = case["page"], case["pages"]
        # requests of 16 pages on average hold the live pages; every eighth request shares its pages with another
        live = max(1, int(N * case["live"]))
        width = 32
        need = torch.randint(1, width + 1, (-(-live // 16) + 1,), generator=g, device=DEV)
        need = torch.minimum(need, (live - torch.cumsum(need, 0) + need).clamp(min=0))
        n = need.numel()
        table, ref = _tables((need * P).to(torch.int32), P, N, width, n + n // 8, g)
        table[n:] = table[:n // 8]
        ref += torch.zeros_like(ref).index_add_(0, table[:n // 8].reshape(-1).clamp(min=0).long(), (table[:n // 8].reshape(-1) >= 0).to(torch.int32))
        lens = torch.cat([need, need[:n // 8]]).to(torch.int32) * P
        first = torch.cat([table.reshape(-1), lens, ref])
        work = first.clone()
        a, b = table.numel(), table.numel() + lens.numel()
        s = dict(first=first, work=work, table=work[:a].view(-1, width), lens=work[a:b], ref=work[b:], page=P, cache=_random_cache(N, P, g),
                 move_src=torch.empty(N // 2, dtype=torch.int32, device=DEV), move_dst=torch.empty(N // 2, dtype=torch.int32, device=DEV),
                 info=torch.empty(4, dtype=torch.int32, device=DEV))
        if own:
            import kimi_delta_attention_varlen_gb300 as kda
            s["workspace"] = torch.empty(kda.kda_pages_workspace_size(N, 0), dtype=torch.uint8, device=DEV)
    s["op"] = case["op"]
    return s


# ------------------------------------------------------------ plain forms --

def _softmax_rows(s, seen):
    """exp(s - max) over the seen places, its sum (0 where nothing is seen) and the log-sum-exp (-inf there)."""
    s.masked_fill_(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = s.sub_(m0).exp_()
    total = p.sum(-1, keepdim=True)
    return p, total, (m0 + total.log()).squeeze(-1)


def _plain_decode(s):
    q, lens = s["q"].float(), s["lens"].long()
    R, L, H, D = q.shape
    kv = s["cache"][s["table"].clamp(min=0).long()].reshape(R, -1, D).float()
    scores = torch.matmul(q.reshape(R, L * H, D), kv.transpose(1, 2)).mul_(s["scale"]).view(R, L, H, -1)
    limit = lens[:, None] - torch.arange(L - 1, -1, -1, device=DEV)[None, :]
    p, total, lse = _softmax_rows(scores, torch.arange(kv.shape[1], device=DEV) < limit[:, :, None, None])
    out = torch.matmul(p.view(R, L * H, -1), kv[..., :LATENT]).view(R, L, H, LATENT)
    s["out"].copy_(out / total.clamp(min=1e-30))
    s["lse"].copy_(lse)
    return {"out": s["out"], "lse": s["lse"]}


def _plain_prefill(s):
    # sequence by sequence: padded to the longest, the batch's scores would not fit
    for (q0, k0), (q1, k1) in zip(s["spans"], s["spans"][1:]):
        q = s["q"][q0:q1].float().transpose(0, 1)
        k = torch.cat([s["k_nope"][k0:k1].float(), s["k_rope"][k0:k1, None].float().expand(-1, q.shape[0], -1)], -1)
        scores = torch.matmul(q, k.permute(1, 2, 0)).mul_(s["scale"])
        seen = torch.arange(k1 - k0, device=DEV)[None, :] <= torch.arange(q1 - q0, device=DEV)[:, None] + (k1 - k0 - q1 + q0)
        p, total, lse = _softmax_rows(scores, seen)
        out = torch.matmul(p, s["v"][k0:k1].float().transpose(0, 1)) / total.clamp(min=1e-30)
        s["out"][q0:q1] = out.transpose(0, 1).to(torch.bfloat16)
        s["lse"][q0:q1] = lse.transpose(0, 1)
    return {"out": s["out"], "lse": s["lse"]}


def _pages_of(lens, page):
    return (lens.long() + page - 1) // page


def _plain_turnover(s):
    table, lens, ref, P = s["table"], s["lens"], s["ref"], s["page"]
    N, W = ref.numel(), table.shape[1]
    at = torch.arange(W, device=DEV)
    # fork: the child's row is the parent's, one more reference to each of its pages
    src, dst = s["src"].long(), s["dst"].long()
    held = at[None, :] < _pages_of(lens[src], P)[:, None]
    rows = torch.where(held, table[src], -1)
    table[dst] = rows
    lens[dst] = lens[src]
    ref.index_add_(0, rows.clamp(min=0).reshape(-1).long(), held.reshape(-1).to(torch.int32))
    # reserve: new pages in order of request and position, a shared unfinished last page among them
    req, new = s["req"].long(), s["new"].long()
    before = lens[req].long()
    have, need = _pages_of(before, P), _pages_of(before + new, P)
    last = table[req].gather(1, (have - 1).clamp(min=0)[:, None]).squeeze(1).long()
    cow = (new > 0) & (before % P != 0) & (ref[last.clamp(min=0)] > 1)
    first = have - cow.long()
    want = at[None, :].ge(first[:, None]) & at[None, :].lt(need[:, None])
    rank = torch.cumsum(want.reshape(-1).long(), 0).view_as(want) - 1
    free = torch.argsort((ref != 0).to(torch.int32), stable=True)  # free pages first, lowest numbers first
    free_count, demand = (ref == 0).sum(), want.sum()
    grown = torch.where(want, free[rank.clamp(0, N - 1)].to(torch.int32), table[req])
    table[req] = grown
    fresh = grown.gather(1, first.clamp(0, W - 1)[:, None]).squeeze(1)
    s["move_src"].copy_(torch.where(cow, last, -1))
    s["move_dst"].copy_(torch.where(cow, fresh.long(), -1))
    ref.index_add_(0, last.clamp(min=0), -cow.to(torch.int32))
    ref.index_add_(0, grown.clamp(min=0).reshape(-1).long(), want.reshape(-1).to(torch.int32))
    lens[req] = (before + new).to(torch.int32)
    s["info"].copy_(torch.stack([torch.zeros_like(demand), cow.sum(), demand, free_count]))
    # copy the shared pages, then append the new rows
    cache = s["cache"]
    moved = cow.nonzero().squeeze(1)
    cache[fresh[moved].long()] = cache[last[moved]]
    count = s["cu"][1:] - s["cu"][:-1]
    owner = torch.repeat_interleave(torch.arange(req.numel(), device=DEV), count.long(), output_size=s["x"].shape[0])
    pos = lens[req][owner].long() - count[owner].long() + torch.arange(s["x"].shape[0], device=DEV) - s["cu"][owner].long()
    cache[table[req[owner], pos // P].long(), 0, pos % P] = s["x"]
    # release the requests that ended
    ended = s["ended"].long()
    held = at[None, :] < _pages_of(lens[ended], P)[:, None]
    ref.index_add_(0, table[ended].clamp(min=0).reshape(-1).long(), -held.reshape(-1).to(torch.int32))
    table[ended] = -1
    lens[ended] = 0


def _plain_compact(s):
    table, ref = s["table"], s["ref"]
    N = ref.numel()
    used = ref != 0
    live, number = used.sum(), torch.arange(N, device=DEV)
    out_of_place, hole = used & (number >= live), ~used & (number < live)
    moves = out_of_place.sum()
    src = torch.argsort((~out_of_place).to(torch.int32), stable=True)[:N // 2]
    dst = torch.argsort((~hole).to(torch.int32), stable=True)[:N // 2]
    valid = torch.arange(N // 2, device=DEV) < moves
    s["move_src"].copy_(torch.where(valid, src, -1))
    s["move_dst"].copy_(torch.where(valid, dst, -1))
    k = valid.nonzero().squeeze(1)
    src, dst = src[k], dst[k]
    to = number.clone()
    to[src] = dst
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].to(torch.int32), table))
    ref[dst] = ref[src]
    ref[src] = 0
    s["info"].copy_(torch.stack([torch.zeros_like(moves), moves, live, N - live]))
    s["cache"][dst] = s["cache"][src]


# -------------------------------------------------------------------- run --

def run(s):
    op = s["op"]
    if not own:
        if op == "decode":
            return _plain_decode(s)
        if op == "prefill":
            return _plain_prefill(s)
        s["work"].copy_(s["first"])  # every pass starts from the same tables
        (_plain_turnover if op == "turnover" else _plain_compact)(s)
    else:
        import kimi_delta_attention_varlen_gb300 as kda
        if op == "decode":
            kda.kda_latent_decode(s["q"], s["cache"], s["table"], s["lens"], s["out"], s["workspace"], latent_dim=LATENT,
                                  scale=s["scale"], lse=s["lse"])
            return {"out": s["out"], "lse": s["lse"]}
        if op == "prefill":
            kda.kda_latent_prefill(s["q"], s["k_nope"], s["k_rope"], s["v"], s["cu_q"], s["cu_k"], s["out"], s["workspace"],
                                   scale=s["scale"], lse=s["lse"])
            return {"out": s["out"], "lse": s["lse"]}
        s["work"].copy_(s["first"])
        pt = kda.page_table_descriptor(s["table"], s["lens"], s["ref"], s["page"])
        if op == "turnover":
            kda.kda_pages_fork(pt, s["src"], s["dst"])
            kda.kda_pages_reserve(pt, s["req"], s["new"], s["move_src"], s["move_dst"], s["info"], s["workspace"])
            kda.kda_pages_copy(s["cache"], s["move_src"], s["move_dst"])
            kda.kda_latent_append(s["x"], s["cu"], s["req"], pt, s["cache"])
            kda.kda_pages_release(pt, s["ended"])
        else:
            kda.kda_pages_compact(pt, s["move_src"], s["move_dst"], s["info"], s["workspace"])
            kda.kda_pages_copy(s["cache"], s["move_src"], s["move_dst"])
    return {"table": s["table"], "lens": s["lens"], "ref": s["ref"], "move_src": s["move_src"], "move_dst": s["move_dst"],
            "info": s["info"], "cache": s["cache"]}


# ------------------------------------------------------------ work, exact --

def work(case):
    op = case["op"]
    row = (LATENT + ROPE) * 2
    if op == "decode":
        R, L, H = case["requests"], case["draft"], case["heads"]
        lo, hi = max(case["lo"], L), max(case["hi"], L)
        tokens = hi + (R - 1) * (lo + hi) / 2
        pairs = tokens * L - R * L * (L - 1) / 2
        return {"bytes": tokens * row + R * L * H * (row + LATENT * 2 + 4) + tokens / case["page"] * 4,
                "flops": 2 * H * pairs * (LATENT + ROPE + LATENT)}
    if op == "prefill":
        H, (lq, lk) = case["heads"], _prompt_lengths(case)
        nq, nk = sum(lq), sum(lk)
        pairs = sum(a * (b - a) + a * (a + 1) / 2 for a, b in zip(lq, lk))
        return {"bytes": 2 * H * (nq * (NOPE + ROPE + VDIM) + nk * (NOPE + VDIM)) + nk * ROPE * 2 + nq * H * 4,
                "flops": 2 * H * pairs * (NOPE + ROPE + VDIM)}
    P = case["page"]
    if op == "turnover":
        R, F, new = case["requests"], case["forks"], case["new"]
        # a forked request and its children each copy the shared last page, unless it is full
        parents = R * (1 - (1 - 1 / R) ** F)
        copies = (F + parents) * (P - 1) / P
        return {"bytes": copies * 2 * P * row + (R + F) * new * 2 * row + 4 * case["pages"] + 8 * (R + F) * ((case["lo"] + case["hi"]) / 2 / P),
                "flops": 0}
    N, live = case["pages"], case["live"]
    return {"bytes": N * live * (1 - live) * 2 * P * row + 4 * N * 2 + 8 * N * live, "flops": 0}


def exact(case, seed):
    """From the definition, in 64 bits, one (request or sequence, query) block at a time."""
    if case["op"] not in ("decode", "prefill"):
        return None  # whole numbers and copied bytes
    s = prepare(case, seed)
    if case["op"] == "decode":
        R, L, H, D = s["q"].shape
        P = case["page"]
        out = torch.zeros(R, L, H, LATENT, dtype=torch.float64, device=DEV)
        lse = torch.full((R, L, H), -math.inf, dtype=torch.float64, device=DEV)
        for r, n in enumerate(s["lens"].tolist()):
            pages = s["table"][r, :-(-n // P)].long()
            kv = s["cache"][pages].reshape(-1, D)[:n].double()
            for t in range(L):
                seen = kv[:n - (L - 1 - t)]
                if seen.shape[0]:
                    z = s["q"][r, t].double() @ seen.T * s["scale"]
                    lse[r, t] = torch.logsumexp(z, -1)
                    out[r, t] = torch.softmax(z, -1) @ seen[:, :LATENT]
        return {"out": out, "lse": lse}
    Tq, H = s["q"].shape[:2]
    out = torch.zeros(Tq, H, VDIM, dtype=torch.float64, device=DEV)
    lse = torch.full((Tq, H), -math.inf, dtype=torch.float64, device=DEV)
    for (q0, k0), (q1, k1) in zip(s["spans"], s["spans"][1:]):
        rope = s["k_rope"][k0:k1].double()
        for a in range(q0, q1, 2048):
            b = min(a + 2048, q1)
            last = torch.arange(a - q0, b - q0, device=DEV) + (k1 - k0) - (q1 - q0)  # the last key that each query sees
            n = int(last[-1]) + 1
            if n <= 0:
                continue
            hidden = torch.arange(n, device=DEV)[None, :] > last[:, None]
            for h in range(H):
                z = (s["q"][a:b, h, :NOPE].double() @ s["k_nope"][k0:k0 + n, h].double().T + s["q"][a:b, h, NOPE:].double() @ rope[:n].T) * s["scale"]
                z = z.masked_fill(hidden, -math.inf)
                lse[a:b, h] = torch.logsumexp(z, -1)
                out[a:b, h] = torch.nan_to_num(torch.softmax(z, -1)) @ s["v"][k0:k0 + n, h].double()
    return {"out": out, "lse": lse}
