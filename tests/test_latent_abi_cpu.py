"""Latent attention and page upkeep on a machine without a GPU: every refusal is a host check on
metadata (the pointers below are never dereferenced), and empty calls launch nothing."""
import ctypes

import pytest
import torch

import kimi_delta_attention_varlen_gb300 as kda
from kimi_delta_attention_varlen_gb300 import _abi, build

OK, NULL, DTYPE, LAYOUT, SHAPE, RANGE, WORKSPACE, CUDA, UNSUPPORTED, ALIGN = 0, -1, -2, -3, -4, -5, -6, -7, -8, -9
A = 0x10000  # a 256-byte aligned fake device address (never dereferenced)


@pytest.fixture(scope="module")
def L():
    build.build()
    return _abi.lib()


def cache(n=8, h=1, v=64, k=576, dtype=1, data=A, stride=None, reserved=0):
    return _abi.KdaCache(data, dtype, reserved, n, h, v, k, h * v * k if stride is None else stride)


def table(requests=4, width=8, stride=None, n_pages=8, page=64, reserved=0, bt=A, lens=A, ref=A):
    return _abi.KdaPageTable(bt, lens, ref, requests, width, width if stride is None else stride, n_pages, page, reserved)


def decode(L, **kw):
    a = dict(q=A, io=1, batch=2, drafts=1, h=32, dl=512, dr=64, scale=0.1, cache=cache(), bt=A, requests=4, width=8, stride=8, lens=A,
             req=None, it=0, out=A, lse=A, ws=A, ws_bytes=1 << 40)
    a.update(kw)
    c = ctypes.byref(a["cache"]) if a["cache"] is not None else None
    return L.kda_latent_decode(a["q"], a["io"], a["batch"], a["drafts"], a["h"], a["dl"], a["dr"], a["scale"], c, a["bt"], a["requests"],
                               a["width"], a["stride"], a["lens"], a["req"], a["it"], a["out"], a["lse"], a["ws"], a["ws_bytes"], None)


def test_decode_refusals(L):
    assert decode(L, cache=None) == NULL
    assert decode(L, cache=cache(data=0)) == NULL
    assert decode(L, io=0) == DTYPE and decode(L, cache=cache(dtype=0)) == DTYPE and decode(L, req=A, it=4) == DTYPE
    assert decode(L, cache=cache(n=0)) == LAYOUT and decode(L, cache=cache(stride=64 * 576 - 1)) == LAYOUT
    for bad in (dict(batch=-1), dict(drafts=0), dict(h=0), dict(dl=0), dict(dr=0), dict(requests=0), dict(width=0), dict(stride=7),
                dict(cache=cache(h=2)), dict(cache=cache(k=575)), dict(requests=1)):
        assert decode(L, **bad) == SHAPE, bad
    assert decode(L, dl=384, cache=cache(k=448)) == UNSUPPORTED
    assert decode(L, dl=512, dr=32, cache=cache(k=544)) == UNSUPPORTED
    assert decode(L, cache=cache(v=60)) == UNSUPPORTED  # a page of 60 tokens
    assert decode(L, drafts=1 << 14, h=128) == RANGE
    assert decode(L, batch=1 << 27, requests=1 << 27, h=32) == RANGE
    assert decode(L, width=1 << 25, stride=1 << 25) == RANGE  # positions beyond 31 bits
    assert decode(L, cache=cache(n=1 << 31)) == RANGE
    for name in ("q", "bt", "lens", "out", "ws"):
        assert decode(L, **{name: None}) == NULL, name
    for bad in (dict(q=A + 8), dict(out=A + 8), dict(cache=cache(data=A + 8)), dict(cache=cache(stride=64 * 576 + 4)), dict(bt=A + 2),
                dict(lens=A + 1), dict(lse=A + 2), dict(req=A + 4, it=1)):
        assert decode(L, **bad) == ALIGN, bad
    need = L.kda_latent_decode_workspace_size(2, 1, 32, 512, 64)
    assert need > 0 and decode(L, ws_bytes=need - 1) == WORKSPACE and decode(L, ws=A + 128) == WORKSPACE
    assert decode(L, batch=0, q=None, out=None, ws=None) == OK


def test_decode_workspace_size(L):
    f = L.kda_latent_decode_workspace_size
    assert f(1, 1, 32, 384, 64) == 0 and f(1, 1, 32, 512, 32) == 0 and f(-1, 1, 32, 512, 64) == 0 and f(1, 0, 32, 512, 64) == 0
    assert f(1 << 27, 1, 32, 512, 64) == 0 and f(0, 1, 32, 512, 64) > 0
    assert f(4096, 1, 128, 512, 64) < 1 << 30  # bounded by the GPU, not by the batch's length


def prefill(L, **kw):
    a = dict(q=A, io=1, kn=A, kn_t=2048, kn_h=256, kr=A, kr_t=576, v=A, v_t=2048, v_h=256, cu_q=A, cu_k=A, B=2, Tq=100, Tk=200, h=8, dn=128,
             dr=64, dv=128, scale=0.1, out=A, lse=A, ws=A, ws_bytes=1 << 40)
    a.update(kw)
    return L.kda_latent_prefill(a["q"], a["io"], a["kn"], a["kn_t"], a["kn_h"], a["kr"], a["kr_t"], a["v"], a["v_t"], a["v_h"], a["cu_q"],
                                a["cu_k"], a["B"], a["Tq"], a["Tk"], a["h"], a["dn"], a["dr"], a["dv"], a["scale"], a["out"], a["lse"],
                                a["ws"], a["ws_bytes"], None)


def test_prefill_refusals(L):
    assert prefill(L, io=0) == DTYPE
    for bad in (dict(B=0), dict(Tq=-1), dict(Tk=-1), dict(h=0), dict(dn=0), dict(dr=0), dict(dv=0), dict(kn_t=-8), dict(v_h=-8)):
        assert prefill(L, **bad) == SHAPE, bad
    assert prefill(L, dn=64) == UNSUPPORTED and prefill(L, dv=64) == UNSUPPORTED and prefill(L, dr=32) == UNSUPPORTED
    for bad in (dict(Tq=(1 << 31) - 256), dict(Tk=1 << 31), dict(B=1 << 24), dict(h=1025), dict(kr_t=1 << 38)):
        assert prefill(L, **bad) == RANGE, bad
    for name in ("q", "kn", "kr", "v", "cu_q", "cu_k", "out", "ws"):
        assert prefill(L, **{name: None}) == NULL, name
    for bad in (dict(q=A + 2), dict(kn=A + 8), dict(kr=A + 8), dict(v=A + 8), dict(out=A + 4), dict(kn_t=2052), dict(kr_t=580), dict(v_h=4),
                dict(cu_q=A + 1), dict(lse=A + 1)):
        assert prefill(L, **bad) == ALIGN, bad
    need = L.kda_latent_prefill_workspace_size(100, 2, 8)
    assert need > 0 and prefill(L, ws_bytes=need - 1) == WORKSPACE and prefill(L, ws=A + 16) == WORKSPACE
    assert prefill(L, Tq=0, q=None, out=None, ws=None) == OK
    assert L.kda_latent_prefill_workspace_size(100, 0, 8) == 0 and L.kda_latent_prefill_workspace_size(-1, 1, 8) == 0


def call(L, name, t, *args):
    return getattr(L, name)(ctypes.byref(t) if t is not None else None, *args)


def lists(L, t=None, it=0, count=3, req=A, ws=A, ws_bytes=1 << 40, x=A):
    """Each call that takes a list of requests, with the same arguments."""
    return [call(L, "kda_pages_fork", t, req, x, it, count, None),
            call(L, "kda_pages_release", t, req, it, None, count, None),
            call(L, "kda_pages_reserve", t, req, it, x, count, A, A, A, ws, ws_bytes, None),
            L.kda_latent_append(A, 576, 5, x, req, it, count, ctypes.byref(t) if t is not None else None, ctypes.byref(cache()), None)]


def test_page_table_refusals(L):
    def every(want, t, **kw):
        assert set(lists(L, t, **kw)) == {want}

    every(NULL, None)
    for bad in (dict(bt=0), dict(lens=0), dict(ref=0)):
        every(NULL, table(**bad))
        assert call(L, "kda_pages_compact", table(**bad), A, A, 4, A, A, 1 << 40, None) == NULL
    for bad in (dict(requests=0), dict(width=0), dict(stride=7), dict(n_pages=0), dict(page=0), dict(reserved=1)):
        every(LAYOUT, table(**bad))
    for bad in (dict(n_pages=1 << 31), dict(width=1 << 26), dict(requests=1 << 31), dict(stride=1 << 41)):
        every(RANGE, table(**bad))
    for bad in (dict(bt=A + 2), dict(lens=A + 1), dict(ref=A + 3)):
        every(ALIGN, table(**bad))
    every(DTYPE, table(), it=2)
    every(SHAPE, table(), count=-1)
    every(RANGE, table(), count=1 << 30)
    every(NULL, table(), req=None)
    every(ALIGN, table(), req=A + 4, it=1)
    every(OK, table(), count=0, req=None, ws=None)
    assert call(L, "kda_pages_fork", table(), A, None, 0, 3, None) == NULL
    assert call(L, "kda_pages_release", table(), A, 0, A + 1, 3, None) == ALIGN


def test_reserve_and_compact_refusals(L):
    need = L.kda_pages_workspace_size(8, 3)
    assert L.kda_pages_workspace_size(0, 3) == 0 and L.kda_pages_workspace_size(8, -1) == 0 and need > 0
    args = [A, 0, A, 3, A, A, A, A, need, None]
    for i, want in ((2, NULL), (4, NULL), (5, NULL), (6, NULL), (7, NULL)):
        assert call(L, "kda_pages_reserve", table(), *[None if j == i else x for j, x in enumerate(args)]) == want
    for i in (2, 4, 5, 6):
        assert call(L, "kda_pages_reserve", table(), *[A + 2 if j == i else x for j, x in enumerate(args)]) == ALIGN
    assert call(L, "kda_pages_reserve", table(), *args[:8], need - 1, None) == WORKSPACE
    assert call(L, "kda_pages_reserve", table(), *args[:7], A + 4, need, None) == WORKSPACE
    need = L.kda_pages_workspace_size(8, 0)
    assert call(L, "kda_pages_compact", table(), A, A, 3, A, A, need, None) == SHAPE  # capacity below n_pages / 2
    assert call(L, "kda_pages_compact", table(), A, A, 1 << 31, A, A, need, None) == RANGE
    assert call(L, "kda_pages_compact", table(), None, A, 4, A, A, need, None) == NULL
    assert call(L, "kda_pages_compact", table(), A, A, 4, None, A, need, None) == NULL
    assert call(L, "kda_pages_compact", table(), A, A + 2, 4, A, A, need, None) == ALIGN
    assert call(L, "kda_pages_compact", table(), A, A, 4, A, A, need - 1, None) == WORKSPACE


def test_copy_and_append_refusals(L):
    def copy(c=None, src=A, dst=A, it=0, count=4):
        return L.kda_pages_copy(ctypes.byref(cache() if c is None else c), src, dst, it, count, None)
    assert copy(cache(n=0)) == LAYOUT and copy(it=7) == DTYPE and copy(count=-1) == SHAPE
    assert copy(src=None) == NULL and copy(dst=None) == NULL and copy(src=A + 2) == ALIGN and copy(dst=A + 4, it=1) == ALIGN
    assert copy(count=0, src=None, dst=None) == OK

    def append(x=A, stride=576, total=5, cu=A, count=3, t=None, c=None):
        return L.kda_latent_append(x, stride, total, cu, A, 0, count, ctypes.byref(t or table()), ctypes.byref(c or cache()), None)
    assert append(c=cache(h=2, v=32)) == SHAPE and append(t=table(page=32)) == SHAPE and append(c=cache(n=7)) == SHAPE
    assert append(stride=575) == SHAPE and append(total=-1) == SHAPE and append(total=1 << 31) == RANGE
    assert append(x=None) == NULL and append(cu=None) == NULL and append(x=A + 1) == ALIGN and append(cu=A + 2) == ALIGN
    assert append(total=0, x=None) == OK


def test_binding_refusals():
    bf = torch.bfloat16
    q, out = torch.zeros(2, 1, 4, 576, dtype=bf), torch.zeros(2, 1, 4, 512, dtype=bf)
    c, bt, sl = torch.zeros(3, 1, 16, 576, dtype=bf), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    ws = torch.zeros(256, dtype=torch.uint8)

    def decode(**kw):
        a = dict(q=q, cache=c, block_table=bt, seq_lens=sl, out=out, workspace=ws, latent_dim=512, scale=1.0, stream=0)
        a.update(kw)
        kda.kda_latent_decode(**a)
    for bad in (dict(q=q[0]), dict(q=q.transpose(1, 2)), dict(out=out[..., :256]), dict(out=out.float()), dict(block_table=bt.long()),
                dict(block_table=torch.zeros(2, 4, dtype=torch.int32)[:, ::2]), dict(seq_lens=sl[:1]), dict(seq_lens=sl.long()),
                dict(req=torch.zeros(3, dtype=torch.int32)), dict(lse=torch.zeros(2, 4)), dict(workspace=ws.view(torch.int32)),
                dict(cache=c.transpose(2, 3))):
        with pytest.raises(ValueError):
            decode(**bad)
    with pytest.raises(TypeError):
        decode(q=q.half(), out=out.half())
    with pytest.raises(kda.KdaError):
        decode(q=q.float(), out=out.float())

    qp, kn, kr = torch.zeros(5, 4, 192, dtype=bf), torch.zeros(7, 4, 128, dtype=bf), torch.zeros(7, 64, dtype=bf)
    cu = torch.zeros(2, dtype=torch.int32)

    def prefill(**kw):
        a = dict(q=qp, k_nope=kn, k_rope=kr, v=kn, cu_q=cu, cu_k=cu, out=torch.zeros(5, 4, 128, dtype=bf), workspace=ws, stream=0)
        a.update(kw)
        kda.kda_latent_prefill(**a)
    for bad in (dict(k_nope=kn[:, :3]), dict(k_rope=kr[:6]), dict(v=kn[:6]), dict(q=qp[..., :190]), dict(k_rope=kr.float()), dict(cu_k=cu.long()),
                dict(cu_q=cu[:1]), dict(out=torch.zeros(5, 4, 64, dtype=bf)), dict(lse=torch.zeros(4, 5)),
                dict(v=torch.zeros(7, 4, 256, dtype=bf)[..., ::2])):
        with pytest.raises(ValueError):
            prefill(**bad)

    with pytest.raises(ValueError):
        kda.page_table_descriptor(bt.long(), sl, sl, 16)
    with pytest.raises(ValueError):
        kda.page_table_descriptor(bt, sl[:1], sl, 16)
    t = kda.page_table_descriptor(bt, sl, torch.zeros(3, dtype=torch.int32), 16)
    i3 = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        kda.kda_pages_fork(t, i3, i3.long(), stream=0)
    with pytest.raises(ValueError):
        kda.kda_pages_reserve(t, i3, i3.long(), i3, i3, torch.zeros(4, dtype=torch.int32), ws, stream=0)
    with pytest.raises(ValueError):
        kda.kda_pages_compact(t, i3, i3, i3, ws, stream=0)
    with pytest.raises(ValueError):
        kda.kda_latent_append(torch.zeros(3, 576), i3, i3[:2], t, c, stream=0)
    with pytest.raises(TypeError):
        kda.kda_pages_copy(c, i3.float(), i3.float(), stream=0)


@pytest.mark.parametrize("scale,want", [(0.0, RANGE), (-1.0, RANGE), (float("nan"), RANGE), (float("inf"), RANGE), (3.0e38, RANGE), (2.4e38, RANGE),
                                        (2.35e38, WORKSPACE), (1e-45, WORKSPACE)])
def test_scales(L, scale, want):
    """The kernels multiply the scale by log2(e) in fp32: what overflows there is refused (a scale that passes goes on to
    the workspace, which is too small here)."""
    assert decode(L, scale=scale, ws_bytes=0) == want
    assert prefill(L, scale=scale, ws_bytes=0) == want
