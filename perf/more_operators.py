"""The latent cache in 8 bits and the attention of requests that share a prefix, on real work: inputs, plain forms, sizes.

A server that keeps a hybrid decoder's latents (one row [latent | rope] a token, in pages) runs out of
memory before it runs out of anything else, and many of its requests begin with the same tokens: samples of
one prompt, a system prompt, a document that many ask about.  Four operators are measured:

  write   latents quantised as they are written into 8-bit pages: e4m3 codes of the latent with one power
          of two a token as their scale, the rope key beside them in bf16, in units of the same scale
  read    rows of cached tokens, from 8-bit or bf16 pages, as dense bf16 (for the projections of a prompt
          that continues on a cached prefix)
  decode  absorbed attention over 8-bit pages: one token a request or a few draft tokens (causal)
  shared  absorbed attention over bf16 pages where groups of requests hold the same first pages

`run` computes them in elementary torch operations where `own` is false and calls the framework
where it is true.

An 8-bit page of P tokens is P * (dl + 2 * 64 + 4) bytes: the codes [P][dl], then the rope keys [P][64] in
bf16, then the scales [P] in fp32.  A value is its code (or rope entry) times its token's scale.
"""
import math
import random

import torch

own = False
DEV = "cuda"
ROPE = 64
SCALE = (128 + ROPE) ** -0.5  # per-head size of the expanded form and the rope


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one new token of each request of a small server
        dict(name="write 24 tokens", op="write", requests=24, new=1, lo=1, hi=3000, latent=512, page=64, dtype="bf16"),
        # the prompts of the framework's batched workload, written whole
        dict(name="write 16 prompts", op="write", requests=16, new=0, lo=512, hi=8192, latent=512, page=64, dtype="bf16"),
        # three short prefixes out of bf16 pages (the framework's smallest batch)
        dict(name="read 3 short prefixes", op="read", requests=3, first=0, lo=37, hi=100, latent=512, page=16, bits=16),
        # prefixes as long as the batched workload's prompts, out of 8-bit pages
        dict(name="read 16 prefixes", op="read", requests=16, first=0, lo=512, hi=8192, latent=512, page=64, bits=8),
        # one request of a chat a thousand tokens long: a call where latency is all
        dict(name="decode8 one request", op="decode", requests=1, lo=1009, hi=1009, draft=1, heads=32, latent=512, page=64),
        # long contexts, for which the cache was made small: few rows, the cache axis split over the SMs
        dict(name="decode8 2 long contexts", op="decode", requests=2, lo=131072, hi=131072, draft=1, heads=32, latent=512, page=64),
        # a loaded server's step: the lengths of the framework's batched workload, 512 requests
        dict(name="decode8 512 requests", op="decode", requests=512, lo=512, hi=8192, draft=1, heads=32, latent=512, page=64),
        # verification of 4 draft tokens, all 128 heads on one GPU
        dict(name="decode8 4 drafts 128 heads", op="decode", requests=33, lo=1500, hi=6001, draft=4, heads=128, latent=512, page=48),
        # a few parallel samples of one prompt
        dict(name="shared 8 samples", op="shared", groups=1, members=8, prefix=4133, lo=1, hi=257, draft=1, heads=32, latent=512, page=64),
        # many questions about one long document
        dict(name="shared 64 on a document", op="shared", groups=1, members=64, prefix=32768, lo=1, hi=1009, draft=1, heads=32, latent=512,
             page=64),
        # a loaded server whose requests begin with one of seven system prompts
        dict(name="shared 7 system prompts", op="shared", groups=7, members=96, prefix=6001, lo=64, hi=2048, draft=1, heads=32, latent=512,
             page=64),
        # samples of three prompts under verification, all 128 heads on one GPU
        dict(name="shared 4 drafts 128 heads", op="shared", groups=3, members=7, prefix=9001, lo=16, hi=500, draft=4, heads=128, latent=512,
             page=48),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "decode", "decode", "shared", "shared"])
    latent, page = rng.choice([512, 512, 256]), rng.choice([8, 16, 32, 48, 64, 64, 128, 200])
    if op in ("write", "read"):
        hi = _log(rng, 2, 8192)
        requests = _log(rng, 1, max(1, min(512, 131072 // hi)) + 1)
        lo = max(1, int(hi * rng.choice([0.1, 0.5, 1.0])))
        if op == "write":
            return dict(op=op, requests=requests, new=rng.choice([0, 0, 1, 3]), lo=lo, hi=hi, latent=latent, page=page,
                        dtype=rng.choice(["bf16", "bf16", "fp32"]))
        return dict(op=op, requests=requests, first=rng.choice([0, 0, rng.randint(1, 700)]), lo=lo, hi=hi, latent=latent, page=page,
                    bits=rng.choice([8, 16]))
    heads, draft = rng.choice([8, 16, 32, 64, 128]), rng.choice([1, 1, 1, 2, 3, 5])
    if op == "decode":
        hi = _log(rng, 2, 131072)
        # at most 512 requests, at most the largest listed case's tokens x rows
        most = max(1, min(512, int(2.2e6 / hi), int(7.0e7 / (hi * heads * draft))))
        return dict(op=op, requests=_log(rng, 1, most) if most > 1 else 1, lo=max(1, int(hi * rng.choice([0.1, 0.5, 1.0]))), hi=hi,
                    draft=draft, heads=heads, latent=latent, page=page)
    prefix, hi = _log(rng, 8, 32768), _log(rng, 2, 2048)
    most = max(1, min(512, int(2.0e6 / (prefix + hi)), int(6.5e7 / ((prefix + hi) * heads * draft))))
    groups = rng.randint(1, min(most, 9))
    return dict(op=op, groups=groups, members=_log(rng, 1, max(1, most // groups) + 0.49), prefix=prefix, lo=max(1, int(hi * rng.choice([0.1, 1.0]))),
                hi=hi, draft=draft, heads=heads, latent=latent, page=page)


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _lengths(case, n, lo, hi):
    """Lengths lo..hi, the longest once: fixed by the case, so that every seed's batch has as many tokens."""
    rng = random.Random(case["hi"] * 31 + n)
    return [hi] + [rng.randint(lo, hi) for _ in range(n - 1)]


def _shuffled(values, g):
    return torch.tensor(values, dtype=torch.int32, device=DEV)[torch.randperm(len(values), generator=g, device=DEV)]


def _offsets(n):
    return torch.nn.functional.pad(torch.cumsum(n, 0), (1, 0)).to(torch.int32)


def _groups(case):
    """Members and prefix lengths of a case's groups: half to all of the case's figures, the largest first."""
    rng = random.Random(case["prefix"] * 7 + case["members"])
    G, M, P = case["groups"], case["members"], case["prefix"]
    return [M] + [rng.randint((M + 1) // 2, M) for _ in range(G - 1)], [P] + [rng.randint((P + 1) // 2, P) for _ in range(G - 1)]


def _tables(lens, page, pages, width, g):
    """Block tables of requests that hold random pages of the pool, -1 where unused."""
    need = (lens.long() + page - 1) // page
    used = torch.arange(width, device=DEV)[None, :] < need[:, None]
    perm = torch.randperm(pages, generator=g, device=DEV)
    ids = torch.cumsum(used.reshape(-1).long(), 0).reshape(lens.numel(), width) - 1
    return torch.where(used, perm[ids.clamp(0, pages - 1)].to(torch.int32), -1)


def _random_pages16(pages, page, D, g):
    return torch.empty(pages, 1, page, D, dtype=torch.bfloat16, device=DEV).normal_(generator=g)


def _parts(cache, dl):
    """Codes [N, P, dl] (e4m3), rope keys [N, P, 64] (bf16) and scales [N, P] (fp32) of 8-bit pages, as views."""
    N, _, P, _ = cache.shape
    flat = cache.view(N, -1)
    return (flat[:, :P * dl].view(torch.float8_e4m3fn).view(N, P, dl), flat[:, P * dl:P * (dl + 128)].view(torch.bfloat16).view(N, P, ROPE),
            flat[:, P * (dl + 128):].view(torch.float32))


def _random_pages8(pages, page, dl, g):
    """8-bit pages of latents and rope keys of size 1."""
    cache = torch.empty(pages, 1, page, dl + 132, dtype=torch.uint8, device=DEV)
    codes, rope, scales = _parts(cache, dl)
    e = torch.randint(5, 8, (pages, page), generator=g, device=DEV)
    for a in range(0, pages, 4096):
        b = min(pages, a + 4096)
        codes[a:b] = (torch.randn(b - a, page, dl, generator=g, device=DEV) * 64).clamp(-448, 448).to(torch.float8_e4m3fn)
        rope[a:b] = (torch.randn(b - a, page, ROPE, generator=g, device=DEV) * torch.exp2(e[a:b, :, None].float())).to(torch.bfloat16)
    scales.copy_(torch.exp2(-e.float()))
    return cache


def prepare(case, seed):
    g = _gen(seed)
    op, dl, P = case["op"], case["latent"], case["page"]
    s = dict(op=op, latent=dl, page=P)
    if op in ("write", "read"):
        R = case["requests"]
        lens = _shuffled(_lengths(case, R, case["lo"], case["hi"]), g)
        width = -(-case["hi"] // P)
        pages = int(((lens.long() + P - 1) // P).sum()) + 5
        s.update(lens=lens, table=_tables(lens, P, pages, width, g), ref=torch.ones(pages, dtype=torch.int32, device=DEV),
                 req=torch.randperm(R, generator=g, device=DEV).to(torch.int32))
        here = lens[s["req"].long()]
        if op == "write":  # the last `new` tokens of each request (0: all of them)
            n = here if case["new"] == 0 else here.clamp(max=case["new"])
            s["cu"] = _offsets(n)
            x = torch.randn(int(s["cu"][-1]), dl + ROPE, generator=g, device=DEV) * (0.5 + torch.rand(1, generator=g, device=DEV))
            s.update(cache=_random_pages8(pages, P, dl, g), x=x.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32))
        else:  # the tokens from `first` on (from the last one where a request is shorter than that)
            s["first"] = torch.clamp(torch.full_like(here, case["first"]), max=here - 1)
            s["cu"] = _offsets(here - s["first"])
            s["cache"] = _random_pages8(pages, P, dl, g) if case["bits"] == 8 else _random_pages16(pages, P, dl + ROPE, g)
            s["out"] = torch.empty(int(s["cu"][-1]), dl + ROPE, dtype=torch.bfloat16, device=DEV)
        return s
    L, H = case["draft"], case["heads"]
    if op == "decode":
        R = case["requests"]
        lens = _shuffled(_lengths(case, R, max(case["lo"], L), max(case["hi"], L)), g)
        pages = int(((lens.long() + P - 1) // P).sum()) + 7
        table = _tables(lens, P, pages, -(-int(lens.max()) // P), g)
        s["cache"] = _random_pages8(pages, P, dl, g)
    else:
        members, prefix = _groups(case)
        R, G = sum(members), case["groups"]
        of = torch.repeat_interleave(torch.arange(G, device=DEV), torch.tensor(members, device=DEV), output_size=R)
        shared = torch.tensor(prefix, dtype=torch.int32, device=DEV)
        whole = shared.long() // P  # pages that the members hold together; the page that the prefix ends in is each one's own
        lens = shared[of] + _shuffled(_lengths(case, R, max(case["lo"], L), max(case["hi"], L)), g)
        need = (lens.long() + P - 1) // P
        width, total = int(need.max()), int(whole.sum())
        pages = total + int((need - whole[of]).sum()) + 3
        perm = torch.randperm(pages, generator=g, device=DEV)
        at = torch.arange(width, device=DEV)[None, :]
        mine = (at >= whole[of][:, None]) & (at < need[:, None])
        rank = torch.cumsum(mine.reshape(-1).long(), 0).view_as(mine) - 1 + total
        base = (torch.cumsum(whole, 0) - whole)[of][:, None] + at
        number = torch.where(mine, rank, base).clamp(0, pages - 1)
        table = torch.where(at < need[:, None], perm[number].to(torch.int32), -1)
        s.update(cache=_random_pages16(pages, P, dl + ROPE, g), shared=shared, cu_groups=_offsets(torch.tensor(members, device=DEV)))
    s.update(lens=lens, table=table.contiguous(), q=torch.randn(R, L, H, dl + ROPE, generator=g, device=DEV).to(torch.bfloat16),
             out=torch.empty(R, L, H, dl, dtype=torch.bfloat16, device=DEV), lse=torch.empty(R, L, H, device=DEV))
    if own:  # scratch that a program allocates once (the plain forms have none)
        import kimi_delta_attention_varlen_gb300 as kda
        need = kda.kda_latent_decode8_workspace_size(R, L, H, dl, ROPE) if op == "decode" else \
            kda.kda_latent_decode_shared_workspace_size(R, s["shared"].numel(), L, H, dl, ROPE)
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------ plain forms --

def _owners(cu, total):
    """Of each row: the list entry that it belongs to, and its place there."""
    n = (cu[1:] - cu[:-1]).long()
    i = torch.repeat_interleave(torch.arange(n.numel(), device=DEV), n, output_size=total)
    return i, torch.arange(total, device=DEV) - cu[:-1].long()[i]


def _plain_write(s):
    dl, P, x = s["latent"], s["page"], s["x"].float()
    i, e = _owners(s["cu"], x.shape[0])
    r = s["req"].long()[i]
    pos = s["lens"][r].long() - (s["cu"][1:] - s["cu"][:-1]).long()[i] + e
    # the smallest power of two, from 2^-64 on, that brings the latent into e4m3's +-448 and the rope key below 2^64
    fits = lambda most, top: torch.frexp(most / top)  # noqa: E731  (m 2^k with 1/2 <= m < 1)
    (m, k), (mr, kr) = fits(x[:, :dl].abs().amax(1), 448.0), fits(x[:, dl:].abs().amax(1), 2.0 ** 64)
    k = torch.where(m == 0.5, k - 1, k).masked_fill(m == 0, -64)
    kr = torch.where(mr == 0.5, kr - 1, kr).masked_fill(mr == 0, -64)
    k = torch.maximum(torch.maximum(k, kr), torch.full_like(k, -64))
    unit = torch.ldexp(torch.ones_like(m), -k)[:, None]
    codes, rope, scales = _parts(s["cache"], dl)
    page, slot = s["table"][r, pos // P].long(), pos % P
    codes.view(torch.uint8)[page, slot] = (x[:, :dl] * unit).to(torch.float8_e4m3fn).view(torch.uint8)
    rope[page, slot] = (x[:, dl:] * unit).to(torch.bfloat16)
    scales[page, slot] = torch.ldexp(torch.ones_like(m), k)


def _rows8(parts, index):
    """Values of 8-bit tokens in 32 bits (each is exact), rows chosen by `index`."""
    codes, rope, scales = parts
    return torch.cat([codes.view(torch.uint8)[index].view(torch.float8_e4m3fn).float(), rope[index].float()], -1) * scales[index][..., None]


def _plain_read(s):
    P = s["page"]
    i, e = _owners(s["cu"], s["out"].shape[0])
    r, pos = s["req"].long()[i], s["first"].long()[i] + e
    at = (s["table"][r, pos // P].long(), pos % P)
    if s["cache"].dtype == torch.uint8:
        s["out"].copy_(_rows8(_parts(s["cache"], s["latent"]), at))
    else:
        s["out"].copy_(s["cache"][:, 0][at])


def _softmax_rows(s, seen):
    """exp(s - max) over the seen places, its sum (0 where nothing is seen) and the log-sum-exp (-inf there)."""
    s.masked_fill_(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = s.sub_(m0).exp_()
    total = p.sum(-1, keepdim=True)
    return p, total, (m0 + total.log()).squeeze(-1)


def _plain_attention(s):
    """Each request over its own tokens; who shares what makes no difference to the result."""
    q, lens, dl = s["q"].float(), s["lens"].long(), s["latent"]
    R, L, H, D = q.shape
    pages = s["table"].clamp(min=0).long()
    kv = _rows8(_parts(s["cache"], dl), pages) if s["cache"].dtype == torch.uint8 else s["cache"][pages].float()
    kv = kv.reshape(R, -1, D)
    scores = torch.matmul(q.reshape(R, L * H, D), kv.transpose(1, 2)).mul_(SCALE).view(R, L, H, -1)
    limit = lens[:, None] - torch.arange(L - 1, -1, -1, device=DEV)[None, :]
    p, total, lse = _softmax_rows(scores, torch.arange(kv.shape[1], device=DEV) < limit[:, :, None, None])
    out = torch.matmul(p.view(R, L * H, -1), kv[..., :dl]).view(R, L, H, dl)
    s["out"].copy_(out / total.clamp(min=1e-30))
    s["lse"].copy_(lse)


# -------------------------------------------------------------------- run --

def run(s):
    op = s["op"]
    if not own:
        {"write": _plain_write, "read": _plain_read, "decode": _plain_attention, "shared": _plain_attention}[op](s)
    else:
        import kimi_delta_attention_varlen_gb300 as kda
        if op in ("write", "read"):
            pt = kda.page_table_descriptor(s["table"], s["lens"], s["ref"], s["page"])
            if op == "write":
                kda.kda_latent_append8(s["x"], s["cu"], s["req"], pt, s["cache"], latent_dim=s["latent"])
            else:
                kda.kda_latent_read(s["cache"], s["cu"], s["req"], pt, s["out"], latent_dim=s["latent"], first=s["first"])
        elif op == "decode":
            kda.kda_latent_decode8(s["q"], s["cache"], s["table"], s["lens"], s["out"], s["workspace"], latent_dim=s["latent"], scale=SCALE,
                                   lse=s["lse"])
        else:
            kda.kda_latent_decode_shared(s["q"], s["cache"], s["table"], s["lens"], s["cu_groups"], s["shared"], s["out"], s["workspace"],
                                         latent_dim=s["latent"], scale=SCALE, lse=s["lse"])
    if op == "write":
        codes, rope, scales = _parts(s["cache"], s["latent"])
        return {"codes": codes, "rope": rope, "scales": scales}
    return {"out": s["out"]} if op == "read" else {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------ work, exact --

def work(case):
    op, dl, P = case["op"], case["latent"], case["page"]
    row8, row16 = dl + 132, 2 * (dl + ROPE)
    if op in ("write", "read"):
        lens = _lengths(case, case["requests"], case["lo"], case["hi"])
        if op == "write":
            n = sum(x if case["new"] == 0 else min(x, case["new"]) for x in lens)
            return {"bytes": n * (row8 + (dl + ROPE) * (2 if case["dtype"] == "bf16" else 4)), "flops": 0}
        n = sum(x - min(case["first"], x - 1) for x in lens)
        return {"bytes": n * (row16 + (row8 if case["bits"] == 8 else row16)), "flops": 0}
    L, H = case["draft"], case["heads"]
    lo, hi = max(case["lo"], L), max(case["hi"], L)
    if op == "decode":
        lens, once = _lengths(case, case["requests"], lo, hi), 0
        read = sum(lens) * row8 + sum(lens) / P * 4
    else:
        members, prefix = _groups(case)
        own_len = _lengths(case, sum(members), lo, hi)
        once = sum(m * p for m, p in zip(members, prefix))
        lens = own_len
        read = (sum(own_len) + sum(prefix)) * row16 + (sum(own_len) + once) / P * 4
    R = len(lens)
    pairs = (sum(lens) + once) * L - R * L * (L - 1) / 2
    return {"bytes": read + R * L * H * (row16 + 2 * dl + 4), "flops": 2 * H * pairs * (dl + ROPE + dl)}


def _e4m3(y):
    """64-bit values to the nearest of e4m3, ties to even: steps of 2^-9 below 2^-6, then an eighth of the power of two."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def exact(case, seed):
    """From the definitions, in 64 bits, one request at a time."""
    s = prepare(case, seed)
    op, dl, P = s["op"], s["latent"], s["page"]
    lens, table, cache = s["lens"].tolist(), s["table"].long(), s["cache"]
    if op == "write":
        parts = [t.double() for t in _parts(cache, dl)]
        cu = s["cu"].tolist()
        for i, r in enumerate(s["req"].tolist()):
            x = s["x"][cu[i]:cu[i + 1]].double()
            if not x.shape[0]:
                continue
            pos = torch.arange(lens[r] - x.shape[0], lens[r], device=DEV)
            at = (table[r, pos // P], pos % P)
            top = torch.maximum(x[:, :dl].abs().amax(1) / 448, x[:, dl:].abs().amax(1) / 2.0 ** 64).clamp(min=2.0 ** -64)
            unit = torch.exp2(torch.ceil(torch.log2(top)))
            parts[0][at] = _e4m3(x[:, :dl] / unit[:, None])
            parts[1][at] = x[:, dl:] / unit[:, None]
            parts[2][at] = unit
        return {"codes": parts[0], "rope": parts[1], "scales": parts[2]}

    def tokens(r, a, b):
        """Rows a..b-1 of request r."""
        pages = table[r, :-(-b // P)]
        if cache.dtype != torch.uint8:
            return cache[pages].reshape(-1, dl + ROPE)[a:b].double()
        codes, rope, scales = _parts(cache, dl)
        codes, rope, scales = codes.view(torch.uint8)[pages].view(torch.float8_e4m3fn), rope[pages], scales[pages]
        return (torch.cat([codes.double(), rope.double()], -1) * scales.double()[..., None]).reshape(-1, dl + ROPE)[a:b]

    if op == "read":
        first = s["first"].tolist()
        return {"out": torch.cat([tokens(r, first[i], lens[r]) for i, r in enumerate(s["req"].tolist())])}
    R, L, H, _ = s["q"].shape
    out = torch.zeros(R, L, H, dl, dtype=torch.float64, device=DEV)
    lse = torch.full((R, L, H), -math.inf, dtype=torch.float64, device=DEV)
    for r, n in enumerate(lens):
        kv = tokens(r, 0, n)
        for t in range(L):
            seen = kv[:n - (L - 1 - t)]
            if seen.shape[0]:
                z = s["q"][r, t].double() @ seen.T * SCALE
                lse[r, t] = torch.logsumexp(z, -1)
                out[r, t] = torch.softmax(z, -1) @ seen[:, :dl]
    return {"out": out, "lse": lse}
