"""Serving the attention layer of a hybrid model next to its recurrent layer.

A hybrid decoder keeps two things for a request: a recurrent state (the KDA layers) and a paged
cache of latents (the attention layers).  This example serves a batch of prompts through one layer
of each kind, forks one request into parallel samples, generates a few tokens, rolls one back,
ends another, and packs the pages, with the calls of the library only:

    kda_pages_reserve, kda_latent_append     pages and rows for the prompts' latents
    kda_latent_prefill                       the prompts' attention (expanded form)
    kda_prefill_varlen_cached                the prompts through the recurrent layer
    kda_pages_fork, kda_pages_copy           parallel samples share pages; recurrent states are copied
    kda_latent_decode_shared, kda_decode_step
                                             one token a request (absorbed form, what the samples have in
                                             common once for all of them; recurrent step)
    kda_pages_release, kda_pages_compact     requests end, pages are packed

With the latents in 8 bits, kda_latent_append8 and kda_latent_decode8 take the place of the bf16
calls, and kda_latent_read brings rows back out of the pages.

    python examples/latent_serving.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import kimi_delta_attention_varlen_gb300 as kda  # noqa: E402

H, LATENT, ROPE, DIM = 8, 512, 64, 128  # heads, latent row [LATENT | ROPE], head size
BF = torch.bfloat16


class Layer:
    """Random weights of one latent-attention layer: the two up-projections of the latent, a head's
    key [W_k c | rope] and value W_v c."""

    def __init__(self, gen, dev):
        self.wk = (torch.randn(H, LATENT, DIM, generator=gen, device=dev) / LATENT ** 0.5).to(BF)
        self.wv = (torch.randn(H, LATENT, DIM, generator=gen, device=dev) / LATENT ** 0.5).to(BF)
        self.scale = (DIM + ROPE) ** -0.5

    def expand(self, rows):
        """Keys' nope parts and values of latent rows [T, LATENT + ROPE], as slices of one projection."""
        kv = torch.einsum("td,hde->the", rows[:, :LATENT], torch.cat([self.wk, self.wv], -1))
        return kv[..., :DIM], kv[..., DIM:]

    def absorb(self, q):
        """Queries [R, H, DIM + ROPE] into the latent space: [R, 1, H, LATENT + ROPE]."""
        return torch.cat([torch.einsum("rhe,hde->rhd", q[..., :DIM], self.wk), q[..., DIM:]], -1)[:, None].contiguous()

    def values(self, out):
        """Latent outputs [R, 1, H, LATENT] to the heads' values [R, H, DIM]."""
        return torch.einsum("rhd,hde->rhe", out[:, 0], self.wv)


class Server:
    """Page tables, a latent cache (eight: in 8 bits) and recurrent states for a fixed number of requests."""

    def __init__(self, layer, requests=16, pages=64, page=16, width=16, dev="cuda", eight=False):
        i32 = dict(dtype=torch.int32, device=dev)
        self.layer, self.dev, self.eight = layer, dev, eight
        self.table, self.lens, self.ref = torch.full((requests, width), -1, **i32), torch.zeros(requests, **i32), torch.zeros(pages, **i32)
        self.pt = kda.page_table_descriptor(self.table, self.lens, self.ref, page)
        self.latents = torch.zeros(pages, 1, page, LATENT + 2 * ROPE + 4, dtype=torch.uint8, device=dev) if eight else \
            torch.zeros(pages, 1, page, LATENT + ROPE, dtype=BF, device=dev)
        self.states = torch.zeros(requests, H, DIM, DIM, device=dev)
        self.info = torch.zeros(4, **i32)
        self.page_ws = torch.empty(kda.kda_pages_workspace_size(pages, requests), dtype=torch.uint8, device=dev)
        size = kda.kda_latent_decode8_workspace_size(requests, 1, H, LATENT, ROPE) if eight else \
            kda.kda_latent_decode_shared_workspace_size(requests, requests, 1, H, LATENT, ROPE)
        self.decode_ws = torch.empty(size, dtype=torch.uint8, device=dev)

    def ints(self, x):
        return torch.tensor(x, dtype=torch.int32, device=self.dev)

    def grow(self, req, counts, rows):
        """Room for counts[i] more tokens of request req[i] and their latent rows into it."""
        req, cu = self.ints(req), self.ints([0] + counts).cumsum(0, dtype=torch.int32)
        src, dst = torch.empty_like(req), torch.empty_like(req)
        kda.kda_pages_reserve(self.pt, req, self.ints(counts), src, dst, self.info, self.page_ws)
        kda.kda_pages_copy(self.latents, src, dst)  # unfinished pages that were shared
        if self.eight:
            kda.kda_latent_append8(rows, cu, req, self.pt, self.latents, latent_dim=LATENT)
        else:
            kda.kda_latent_append(rows, cu, req, self.pt, self.latents)

    def read(self, r, first, n):
        """Latent rows first .. first + n - 1 of a request, as the cache holds them."""
        out = torch.empty(n, LATENT + ROPE, dtype=BF, device=self.dev)
        kda.kda_latent_read(self.latents, self.ints([0, n]), self.ints([r]), self.pt, out, latent_dim=LATENT, first=self.ints([first]))
        return out

    def prompts(self, req, lengths, rows, q, gates):
        """Prompts of new requests: attention outputs [T, H, DIM] and recurrent outputs of all their tokens."""
        self.grow(req, lengths, rows)
        k, v = self.layer.expand(rows)
        T, cu = rows.shape[0], self.ints([0] + lengths).cumsum(0, dtype=torch.int32)
        out = torch.empty(T, H, DIM, dtype=BF, device=self.dev)
        ws = torch.empty(kda.kda_latent_prefill_workspace_size(T, len(req), H), dtype=torch.uint8, device=self.dev)
        kda.kda_latent_prefill(q, k, rows[:, LATENT:], v, cu, cu, out, ws, scale=self.layer.scale)
        mixed = torch.empty(T, H, DIM, dtype=BF, device=self.dev)
        ws = torch.empty(kda.kda_prefill_workspace_size(T, len(req), H, DIM, DIM), dtype=torch.uint8, device=self.dev)
        kda.kda_prefill_varlen_cached(gates["q"], gates["k"], gates["v"], gates["g"], gates["beta"], cu, mixed, ws, self.states,
                                      self.ints(req), flags=torch.zeros(len(req), dtype=torch.bool, device=self.dev),
                                      idx_out=self.ints(req))
        return out, mixed

    def fork(self, src, dst):
        kda.kda_pages_fork(self.pt, self.ints(src), self.ints(dst))
        kda.kda_pages_copy(self.states, self.ints(src), self.ints(dst))

    def step(self, req, groups, rows, q, gates):
        """One token of each request: attention values and recurrent outputs [R, H, DIM].  groups: (requests, tokens that they
        have in common), in the order of req."""
        self.grow(req, [1] * len(req), rows)
        out = torch.empty(len(req), 1, H, LATENT, dtype=BF, device=self.dev)
        args = dict(latent_dim=LATENT, scale=self.layer.scale, req=self.ints(req))
        if self.eight:
            kda.kda_latent_decode8(self.layer.absorb(q), self.latents, self.table, self.lens, out, self.decode_ws, **args)
        else:
            cu = self.ints([0] + [n for n, _ in groups]).cumsum(0, dtype=torch.int32)
            kda.kda_latent_decode_shared(self.layer.absorb(q), self.latents, self.table, self.lens, cu, self.ints([t for _, t in groups]), out,
                                         self.decode_ws, **args)
        mixed = torch.empty(len(req), H, DIM, dtype=BF, device=self.dev)
        kda.kda_decode_step(gates["q"], gates["k"], gates["v"], gates["g"], gates["beta"], self.states, self.ints(req), mixed)
        return self.layer.values(out), mixed

    def release(self, req, keep=None):
        kda.kda_pages_release(self.pt, self.ints(req), None if keep is None else self.ints(keep))

    def pack(self):
        """Live pages to the lowest numbers; the number of live pages."""
        src, dst = (torch.empty(self.ref.numel() // 2, dtype=torch.int32, device=self.dev) for _ in range(2))
        kda.kda_pages_compact(self.pt, src, dst, self.info, self.page_ws)
        kda.kda_pages_copy(self.latents, src, dst)
        return int(self.info[2])


def attention(layer, rows, q):
    """The attention of the last of the tokens `rows` in 64 bits: q [H, DIM + ROPE] -> [H, DIM]."""
    k, v = (t.double() for t in layer.expand(rows))
    z = (torch.einsum("he,the->ht", q[:, :DIM].double(), k) + q[:, DIM:].double() @ rows[:, LATENT:].double().T) * layer.scale
    return torch.einsum("ht,the->he", torch.softmax(z, -1), v)


def main(seed=0, dev="cuda", eight=False):
    """Serves and checks every attention output against the 64-bit form on the request's own tokens; the largest error."""
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    layer = Layer(gen, dev)
    server = Server(layer, dev=dev, eight=eight)
    history, worst = {}, 0.0

    def draw(n):
        rows = torch.randn(n, LATENT + ROPE, generator=gen, device=dev).to(BF)
        q = torch.randn(n, H, DIM + ROPE, generator=gen, device=dev).to(BF)
        gates = {x: torch.randn(n, H, DIM, generator=gen, device=dev).to(BF) for x in "qkv"}
        gates["g"] = -torch.nn.functional.softplus(torch.randn(n, H, DIM, generator=gen, device=dev))
        gates["beta"] = torch.sigmoid(torch.randn(n, H, generator=gen, device=dev))
        return rows, q, gates

    def check(out, want):
        nonlocal worst
        worst = max(worst, float((out.double() - want).abs().max() / want.abs().max()))

    # three prompts
    lengths = [37, 100, 64]
    rows, q, gates = draw(sum(lengths))
    out, _ = server.prompts([0, 1, 2], lengths, rows, q, gates)
    at = 0
    for r, n in enumerate(lengths):
        history[r] = rows[at:at + n]
        for t in (0, n // 2, n - 1):
            check(out[at + t], attention(layer, rows[at:at + t + 1], q[at + t]))
        at += n
        if eight:  # from here on attention sees what the cache holds
            history[r] = server.read(r, 0, n)
    # request 1 samples twice in parallel
    server.fork([1, 1], [5, 6])
    history[5] = history[6] = history[1]
    live = [0, 1, 5, 6, 2]
    for token in range(6):
        rows, q, gates = draw(len(live))
        out, _ = server.step(live, [(1, 0), (3, lengths[1])] + [(1, 0)] * (len(live) - 4), rows, q, gates)
        for i, r in enumerate(live):
            row = server.read(r, history[r].shape[0], 1) if eight else rows[i:i + 1]
            history[r] = torch.cat([history[r], row])
            check(out[i], attention(layer, history[r], q[i]))
        if token == 1:  # request 5 takes its last token back
            server.release([5], [history[5].shape[0] - 1])
            history[5] = history[5][:-1]
        if token == 3:  # request 2 ends, the pages are packed
            server.release([2])
            live.remove(2)
            packed = server.pack()
            assert int((server.ref[:packed] > 0).sum()) == packed and int(server.ref[packed:].sum()) == 0
    assert int(server.info[0]) == 0
    return worst


if __name__ == "__main__":
    print(f"largest error against the 64-bit form, over the outputs' size: {main():.2e}, with latents in 8 bits {main(eight=True):.2e}")
