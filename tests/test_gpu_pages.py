"""Page upkeep on the GPU against plain Python tables (tests/latent_helpers.py): every table,
length, refcount, move and copied byte is equal."""
import random

import pytest
import torch

import kimi_delta_attention_varlen_gb300 as kda
from kimi_delta_attention_varlen_gb300 import workloads as wl
from tests.latent_helpers import Pages

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Device:
    """The same tables on the device, rows `extra` entries further apart, between guard words."""

    def __init__(self, p: Pages, extra=2):
        R, W, N = len(p.rows), p.width, len(p.ref)
        self.back = torch.full((R, W + extra), 0x5A5A5A, dtype=torch.int32, device=DEV)
        self.table = self.back[:, :W]
        self.lens = torch.zeros(R, dtype=torch.int32, device=DEV)
        self.ref_back = torch.full((N + 5,), 0x5A5A5A, dtype=torch.int32, device=DEV)
        self.ref = self.ref_back[1:N + 1]  # not 16-byte aligned
        self.put(p)
        self.desc = kda.page_table_descriptor(self.table, self.lens, self.ref, p.page)
        self.n_pages = N

    def put(self, p):
        self.table.copy_(torch.tensor(p.rows, dtype=torch.int32))
        self.lens.copy_(torch.tensor(p.lens, dtype=torch.int32))
        self.ref.copy_(torch.tensor(p.ref, dtype=torch.int32))

    def check(self, p, what):
        torch.cuda.synchronize()
        assert self.table.tolist() == p.rows, what
        assert self.lens.tolist() == p.lens, what
        assert self.ref.tolist() == p.ref, what
        W = p.width
        assert (self.back[:, W:] == 0x5A5A5A).all() and self.ref_back[0] == 0x5A5A5A and (self.ref_back[self.n_pages + 1:] == 0x5A5A5A).all()

    def reserve(self, req, new, itype=torch.int32):
        n = len(req)
        ms, md = (torch.full((n,), 7, dtype=torch.int32, device=DEV) for _ in range(2))
        info = torch.full((4,), -9, dtype=torch.int32, device=DEV)
        ws = torch.full((kda.kda_pages_workspace_size(self.n_pages, n),), 0xA5, dtype=torch.uint8, device=DEV)
        kda.kda_pages_reserve(self.desc, torch.tensor(req, dtype=itype, device=DEV), torch.tensor(new, dtype=torch.int32, device=DEV),
                              ms, md, info, ws)
        torch.cuda.synchronize()
        return info.tolist(), list(zip(ms.tolist(), md.tolist()))

    def compact(self, capacity=None):
        cap = self.n_pages // 2 if capacity is None else capacity
        ms, md = (torch.full((cap,), 7, dtype=torch.int32, device=DEV) for _ in range(2))
        info = torch.full((4,), -9, dtype=torch.int32, device=DEV)
        ws = torch.full((kda.kda_pages_workspace_size(self.n_pages, 0),), 0xA5, dtype=torch.uint8, device=DEV)
        kda.kda_pages_compact(self.desc, ms, md, info, ws)
        torch.cuda.synchronize()
        return info.tolist(), list(zip(ms.tolist(), md.tolist()))


def ints(x, dt=torch.int32):
    return torch.tensor(x, dtype=dt, device=DEV)


@pytest.mark.parametrize("requests,width,n_pages,page,seed", [(4, 3, 12, 4, 0), (20, 9, 100, 16, 1), (37, 40, 700, 8, 2),
                                                              (60, 64, 4096, 64, 3), (50, 300, 9001, 16, 4), (300, 33, 20000, 1, 5)])
def test_random_lifecycle(requests, width, n_pages, page, seed):
    rng = random.Random(seed)
    p = Pages(requests, width, n_pages, page)
    d = Device(p)
    seen = set()
    for step in range(40):
        itype = rng.choice([torch.int32, torch.int64])
        free_rows = [r for r in range(requests) if p.lens[r] == 0]
        held = [r for r in range(requests) if p.lens[r]]
        what = rng.choice(["reserve", "reserve", "reserve", "fork", "release", "compact"])
        if what == "reserve":
            req = rng.sample(range(requests), rng.randint(1, requests))
            most = rng.choice([1, 3, page, 3 * page])
            new = [rng.choice([0, -3, rng.randint(1, most), rng.randint(1, most)]) for _ in req]
            if rng.random() < 0.3:
                req += [-1, requests + 5]
                new += [10, 10]
            got, want = d.reserve(req, new, itype), p.reserve(req, new)
            assert got[0] == want[0] and got[1] == want[1]
            seen.add(("reserve", want[0][0], want[0][1] > 0))
            if want[0][0]:  # no room: give some back
                rel = rng.sample(held, len(held) // 2)
                p.release(rel)
                kda.kda_pages_release(d.desc, ints(rel, itype)) if rel else None
        elif what == "fork" and held and free_rows:
            n = rng.randint(1, len(free_rows))
            dst, src = rng.sample(free_rows, n), [rng.choice(held) for _ in range(n)]
            if rng.random() < 0.3:
                src += [-7, requests, src[0]]
                dst += [dst[0], dst[0], src[0]]
            p.fork(src, dst)
            kda.kda_pages_fork(d.desc, ints(src, itype), ints(dst, itype))
            seen.add("fork")
        elif what == "release" and held:
            rel = rng.sample(range(requests), rng.randint(1, requests))
            keep = None if rng.random() < 0.4 else [rng.choice([-2, 0, 1, page, 3 * page + 1, 10 ** 6]) for _ in rel]
            p.release(rel, keep)
            kda.kda_pages_release(d.desc, ints(rel, itype), None if keep is None else ints(keep))
            seen.add("release")
        elif what == "compact":
            got, (info, moves) = d.compact(), p.compact()
            assert got[0] == info and got[1] == moves + [(-1, -1)] * (n_pages // 2 - len(moves))
            seen.add(("compact", len(moves) > 0))
        d.check(p, f"step {step}: {what}")
    assert {"fork", "release"} <= seen
    if page > 1 and requests > 4:  # a page of one token is never unfinished; four requests are too few for every step
        assert {("compact", True), ("reserve", 0, True)} <= seen


def test_reserve_is_all_or_nothing():
    p = Pages(3, 4, 6, 8)
    d = Device(p)
    for req, new in (([0, 1], [16, 20]), ([2], [17])):  # 5 pages, then 3 of the 1 that is left
        assert d.reserve(req, new) == p.reserve(req, new)
        d.check(p, "room")
    assert d.reserve([2], [9]) == ([1, 0, 2, 1], [(-1, -1)])
    assert d.reserve([0, 2], [17, 1]) == ([2, 0, 4, 1], [(-1, -1)] * 2)  # row 0 would need 5 entries of 4
    assert d.reserve([0], [2 ** 31 - 1])[0][0] == 2
    assert d.reserve([0, 1, 2], [2 ** 31 - 1] * 3)[0][0] == 2
    d.check(p, "unchanged")


def test_every_writer_of_a_shared_page_gets_its_own():
    p = Pages(5, 4, 20, 4)
    d = Device(p)
    for s in (p, ):
        s.reserve([0], [6])
    d.reserve([0], [6])
    p.fork([0, 0, 0], [1, 2, 3])
    kda.kda_pages_fork(d.desc, ints([0, 0, 0]), ints([1, 2, 3]))
    got, want = d.reserve([3, 0, 2], [1, 1, 2]), p.reserve([3, 0, 2], [1, 1, 2])
    assert got[0] == want[0] == [0, 3, 3, 18] and got[1] == want[1] == [(1, 2), (1, 3), (1, 4)]
    d.check(p, "shared")
    assert d.reserve([1], [1]) == p.reserve([1], [1])  # the last holder writes in place
    d.check(p, "last holder")


@pytest.mark.parametrize("n_pages", [1, 2, 4095, 4096, 4097, 12288])
@pytest.mark.parametrize("fill", ["none", "all", "low", "high", "random"])
def test_compact_edges(n_pages, fill):
    p = Pages(3, n_pages, n_pages, 2)
    rng = random.Random(n_pages)
    k = {"none": 0, "all": n_pages}.get(fill, n_pages // 3)
    pages = {"low": list(range(k)), "high": list(range(n_pages - k, n_pages))}.get(fill) or rng.sample(range(n_pages), k)
    p.rows[1][:k], p.lens[1] = pages, 2 * k
    p.rows[2][:k // 2], p.lens[2] = pages[:k // 2], 2 * (k // 2)
    for row in (1, 2):
        for q in p.rows[row]:
            if q >= 0:
                p.ref[q] += 1
    d = Device(p)
    cap = n_pages // 2 + 3
    got, (info, moves) = d.compact(cap), p.compact()
    assert got == (info, moves + [(-1, -1)] * (cap - len(moves)))
    d.check(p, fill)


@pytest.mark.parametrize("dtype,shape,gap", [(torch.bfloat16, (1, 16, 576), 0), (torch.bfloat16, (1, 64, 576), 64), (torch.float32, (4, 32, 32), 16),
                                             (torch.bfloat16, (1, 3, 5), 1), (torch.float32, (1, 1, 7), 0), (torch.float32, (32, 128, 128), 0)])
@pytest.mark.parametrize("itype", [torch.int32, torch.int64])
def test_copy_moves_payloads_only(dtype, shape, gap, itype):
    N = 23
    pc = wl.paged_cache(N, *shape, dtype, shape[0] * shape[1] * shape[2] + gap, seed=1, device=DEV)
    src = [3, 5, -1, 22, 7, N, 9, 0]
    dst = [4, -1, 6, 10, N, 8, 1, 21]
    want = pc.backing.clone()
    wv = want.as_strided(pc.view.shape, pc.view.stride(), pc.front)
    for s, t in zip(src, dst):
        if 0 <= s < N and 0 <= t < N:
            wv[t] = pc.view[s]
    kda.kda_pages_copy(pc.view, ints(src, itype), ints(dst, itype))
    torch.cuda.synchronize()
    assert torch.equal(pc.backing.view(torch.uint8), want.view(torch.uint8))


def test_copy_between_rows_far_apart():
    stride, N = 1 << 31, 4  # elements; the last row starts beyond 2^32
    back = torch.empty((N - 1) * stride + 16 * 576, dtype=torch.bfloat16, device=DEV)
    cache = back.as_strided((N, 1, 16, 576), (stride, 16 * 576, 576, 1))
    cache[0], cache[3] = 1.5, -2.25
    kda.kda_pages_copy(cache, ints([3]), ints([2]))
    torch.cuda.synchronize()
    assert (cache[2] == -2.25).all() and (cache[0] == 1.5).all()


def test_copy_many_moves():
    # more moves than the grid's second dimension
    n = 70000
    cache = torch.arange(2 * n, dtype=torch.float32, device=DEV).view(2 * n, 1, 1, 1).expand(-1, 1, 1, 4).contiguous()
    kda.kda_pages_copy(cache, torch.arange(n, dtype=torch.int32, device=DEV), torch.arange(n, 2 * n, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert torch.equal(cache[n:], cache[:n])


@pytest.mark.parametrize("dtype,D,page,pad", [(torch.bfloat16, 576, 16, 0), (torch.bfloat16, 320, 64, 8), (torch.float32, 40, 3, 0), (torch.bfloat16, 9, 5, 1)])
def test_append(dtype, D, page, pad):
    p = Pages(6, 8, 40, page)
    d = Device(p)
    for req, new in (([0, 1, 2, 4], [page, 2 * page + 1, 3, 1]), ([1, 4, 0, 3], [page + 2, 1, 1, 2 * page])):
        p.reserve(req, new)
        d.reserve(req, new)
    pc = wl.paged_cache(40, 1, page, D, dtype, page * D + 8, seed=2, device=DEV)
    req, counts = [1, -3, 4, 0, 5, 3], [page + 2, 4, 1, 0, 2, 2 * page]
    cu = [3]
    for c in counts:
        cu.append(cu[-1] + c)
    x = torch.randn(cu[-1] + 4, D + pad, generator=wl.generator(4, DEV), device=DEV).to(dtype)[:, :D]
    want = pc.backing.clone()
    wv = want.as_strided(pc.view.shape, pc.view.stride(), pc.front)
    for i, r in enumerate(req):
        for e in range(counts[i]):
            pos = p.lens[r] - counts[i] + e if 0 <= r < 6 else -1
            if pos >= 0:
                wv[p.rows[r][pos // page], 0, pos % page] = x[cu[i] + e]
    for itype in (torch.int32, torch.int64):
        kda.kda_latent_append(x, ints(cu), ints(req, itype), d.desc, pc.view)
        torch.cuda.synchronize()
        assert torch.equal(pc.backing.view(torch.uint8), want.view(torch.uint8))


def test_a_step_in_a_graph():
    p = Pages(8, 16, 100, 4)
    p.reserve([0, 1, 2], [5, 9, 4])
    d = Device(p)
    ms, md, info = (torch.empty(n, dtype=torch.int32, device=DEV) for n in (4, 4, 4))
    ws = torch.empty(kda.kda_pages_workspace_size(100, 4), dtype=torch.uint8, device=DEV)
    src, dst, req, new = ints([1]), ints([3]), ints([3, 0, 1, 2]), ints([2, 2, 2, 2])
    cache = torch.randn(100, 1, 4, 16, generator=wl.generator(1, DEV), device=DEV)

    def step():
        kda.kda_pages_fork(d.desc, src, dst)
        kda.kda_pages_reserve(d.desc, req, new, ms, md, info, ws)
        kda.kda_pages_copy(cache, ms, md)
        kda.kda_pages_release(d.desc, dst)

    step()
    torch.cuda.synchronize()
    d.put(p)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        before = cache.clone()
        graph.replay()
        p.fork([1], [3])
        want_info, moves = p.reserve([3, 0, 1, 2], [2, 2, 2, 2])
        p.release([3])
        torch.cuda.synchronize()
        assert info.tolist() == want_info and list(zip(ms.tolist(), md.tolist())) == moves
        for s, t in moves:
            if s >= 0:
                assert torch.equal(cache[t], before[s])
        d.check(p, "graph")


def test_append_with_offsets_that_fall_stays_in_the_requests_pages():
    """Offsets that break the contract: rows of the named requests may be written, nothing else."""
    p = Pages(40, 8, 200, 4)
    req = list(range(36))
    p.reserve(req, [9] * 36)
    d = Device(p)
    pc = wl.paged_cache(200, 1, 4, 24, torch.float32, 4 * 24 + 8, seed=2, device=DEV)
    before = pc.backing.clone()
    cu = [0, 9, 30, 2, 5] + [50, 4] * 16
    x = torch.ones(60, 24, device=DEV)
    kda.kda_latent_append(x, ints(cu), ints(req), d.desc, pc.view)
    torch.cuda.synchronize()
    d.check(p, "tables")
    changed = before != pc.backing
    after = torch.zeros_like(before, dtype=torch.bool)
    view = after.as_strided(pc.view.shape, pc.view.stride(), pc.front)
    for r in req:
        for j, page in enumerate(p.rows[r]):
            if page >= 0:
                view[page, 0, :min(4, 9 - 4 * j)] = True
    assert not (changed & ~after).any()


@pytest.mark.parametrize("n_pages,requests", [(32769, 5), (70001, 2100)])
def test_pools_of_many_blocks(n_pages, requests):
    """Requests that take pages from many stretches of the pool, more of them than one pass of threads, and holes."""
    rng = random.Random(n_pages)
    width = 2 * n_pages // requests + 2
    p = Pages(requests, width, n_pages, 3)
    d = Device(p)
    for step in range(3):
        req = rng.sample(range(requests), requests)
        new = [rng.randrange(0, width) for _ in req]
        got, want = d.reserve(req, new), p.reserve(req, new)
        assert got == want
        d.check(p, step)
        gone = rng.sample(range(requests), requests // 3 + 1)
        kda.kda_pages_release(d.desc, ints(gone))
        p.release(gone)
    info, moves = p.compact()
    assert d.compact() == (info, moves + [(-1, -1)] * (n_pages // 2 - len(moves)))
    d.check(p, "compact")
