"""Plain 64-bit forms of latent attention and of the page tables, and the tolerances of the
kernels, for the tests.

Tolerance of an output (bf16), 1.25 * 2^-8 * sum_j p_j |x_j|: the result's rounding to bf16 takes
2^-8 of it at most (bf16's unit roundoff).  The quarter that is left covers the scores' error
below, the approximate exponential and the rounding of the probabilities to bf16, which has to be
small by the kernels' doing: normalised by the sum of the rounded weights its common part drops
out and the rest averages over the tokens, and with few tokens a second product carries it.
Tolerance of a score, and so of the log-sum-exp: the tensor cores add up to 36 partial sums of
16 products in fp32, each addition within 2^-23 of the magnitudes added, so |d| <= 2^-17 *
max_j scale * sum_c |q_c| |x_jc|; 1e-5 covers the logarithm and the sum of exponentials."""
from __future__ import annotations

import math

import torch

OUT_REL = 1.25 * 2.0 ** -8
Z_REL = 2.0 ** -17
LSE_ABS = 1e-5


def softmax_rows(z, v):
    """softmax(z) @ v, p @ |v|, lse of fp64 scores z [rows, n] (rows with nothing: 0, 0, -inf)."""
    if z.shape[1] == 0:
        return v.new_zeros(z.shape[0], v.shape[1]), v.new_zeros(z.shape[0], v.shape[1]), z.new_full((z.shape[0],), -math.inf)
    lse = torch.logsumexp(z, -1)
    p = torch.exp(z - lse.clamp(min=-1e300)[:, None])
    return p @ v, p @ v.abs(), lse


def decode_reference(q, rows_of, lens, scale, dl):
    """q [R, L, H, D]; rows_of(r, n): the first n cache rows of batch entry r, [n, D]."""
    R, L, H, _ = q.shape
    out = torch.zeros(R, L, H, dl, dtype=torch.float64)
    mag, lse, bound = torch.zeros_like(out), torch.full((R, L, H), -math.inf, dtype=torch.float64), torch.zeros(R, L, H, dtype=torch.float64)
    for r in range(R):
        n = int(lens[r])
        x = rows_of(r, n).double().cpu()
        for t in range(L):
            seen = max(0, n - (L - 1 - t))
            qq = q[r, t].double().cpu()
            out[r, t], mag[r, t], lse[r, t] = softmax_rows(qq @ x[:seen].T * scale, x[:seen, :dl])
            if seen:
                bound[r, t] = (qq.abs() @ x[:seen].abs().T * scale).amax(-1)
    return out, mag, lse, bound


def prefill_reference(q, k_nope, k_rope, v, cu_q, cu_k, scale):
    Tq, H, _ = q.shape
    dn, dv = k_nope.shape[2], v.shape[2]
    out = torch.zeros(Tq, H, dv, dtype=torch.float64)
    mag, lse, bound = torch.zeros_like(out), torch.full((Tq, H), -math.inf, dtype=torch.float64), torch.zeros(Tq, H, dtype=torch.float64)
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        qb = q[q0:q1].double().cpu()
        kb = torch.cat([k_nope[k0:k1].double().cpu(), k_rope[k0:k1, None].double().cpu().expand(-1, H, -1)], -1)
        vb = v[k0:k1].double().cpu()
        last = torch.arange(q1 - q0) + (k1 - k0) - (q1 - q0)
        hidden = torch.arange(k1 - k0)[None, :] > last[:, None]
        for h in range(H):
            z = (qb[:, h] @ kb[:, h].T * scale).masked_fill(hidden, -math.inf)
            out[q0:q1, h], mag[q0:q1, h], lse[q0:q1, h] = softmax_rows(z, vb[:, h])
            if k1 > k0 and q1 > q0:
                bound[q0:q1, h] = (qb[:, h].abs() @ kb[:, h].abs().T * scale).masked_fill(hidden, 0).amax(-1)
    return out, mag, lse, bound


def assert_attention(out, lse, ref, what=""):
    want, mag, want_lse, bound = ref
    got = out.double().cpu()
    assert torch.isfinite(got).all(), f"{what}: non-finite outputs"
    over = (got - want).abs() - (OUT_REL + bound.unsqueeze(-1) * Z_REL * 2) * mag
    assert over.max() <= 1e-30, f"{what}: output off by {float((got - want).abs().max()):.3e}, {float(over.max()):.3e} over its tolerance"
    if lse is not None:
        got = lse.double().cpu()
        none = want_lse == -math.inf
        assert torch.equal(got == -math.inf, none), f"{what}: rows without tokens"
        over = ((got - want_lse).abs() - (LSE_ABS + Z_REL * bound))[~none]
        assert over.numel() == 0 or over.max() <= 0, f"{what}: lse off ({float(over.max()):.3e} over its tolerance)"


# ------------------------------------------------------------------- pages --

class Pages:
    """Page tables in plain Python: rows of page numbers, lengths, refcounts."""

    def __init__(self, requests, width, n_pages, page):
        self.rows = [[-1] * width for _ in range(requests)]
        self.lens = [0] * requests
        self.ref = [0] * n_pages
        self.page, self.width = page, width

    def need(self, n):
        return -(-n // self.page)

    def fork(self, src, dst):
        for s, d in zip(src, dst):
            if not (0 <= s < len(self.rows) and 0 <= d < len(self.rows)) or s == d:
                continue
            n = self.need(self.lens[s])
            self.rows[d] = self.rows[s][:n] + [-1] * (self.width - n)
            self.lens[d] = self.lens[s]
            for p in self.rows[d][:n]:
                self.ref[p] += 1

    def release(self, req, keep=None):
        for i, r in enumerate(req):
            if not 0 <= r < len(self.rows):
                continue
            k = 0 if keep is None else min(max(keep[i], 0), self.lens[r])
            for j in range(self.need(k), self.need(self.lens[r])):
                self.ref[self.rows[r][j]] -= 1
                self.rows[r][j] = -1
            self.lens[r] = k

    def reserve(self, req, new):
        """(info, moves); nothing changes unless info[0] == 0."""
        free = [p for p, c in enumerate(self.ref) if c == 0]
        plan, demand, too_short = [], 0, False
        for r, add in zip(req, new):
            if not 0 <= r < len(self.rows) or add <= 0:
                plan.append(None)
                continue
            n = self.lens[r]
            have, need = self.need(n), self.need(n + add)
            cow = n % self.page != 0 and self.ref[self.rows[r][have - 1]] > 1
            too_short |= need > self.width
            demand += need - have + cow
            plan.append((have - cow, need, cow))
        moves = [(-1, -1)] * len(req)
        if too_short or demand > len(free):
            return [2 if too_short else 1, 0, demand, len(free)], moves
        at = 0
        for i, (r, p) in enumerate(zip(req, plan)):
            if p is None:
                continue
            first, need, cow = p
            for j in range(first, need):
                page = free[at]
                at += 1
                if cow and j == first:
                    moves[i] = (self.rows[r][j], page)
                    self.ref[self.rows[r][j]] -= 1
                self.rows[r][j] = page
                self.ref[page] = 1
            self.lens[r] += new[i]
        return [0, sum(m[0] >= 0 for m in moves), demand, len(free)], moves

    def compact(self):
        live = sum(c != 0 for c in self.ref)
        src = [p for p in range(live, len(self.ref)) if self.ref[p]]
        dst = [p for p in range(live) if not self.ref[p]]
        to = dict(zip(src, dst))
        for s, d in to.items():
            self.ref[d], self.ref[s] = self.ref[s], 0
        self.rows = [[to.get(p, p) for p in row] for row in self.rows]
        return [0, len(src), live, len(self.ref) - live], list(zip(src, dst))
