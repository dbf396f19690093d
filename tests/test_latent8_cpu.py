"""8-bit latent pages and shared-prefix decode on a machine without a GPU: the layout and the quantiser of the plain form, every
refusal as a host check on metadata (the pointers below are never dereferenced), empty calls that launch nothing."""
import ctypes
import math

import pytest
import torch

import kimi_delta_attention_varlen_gb300 as kda
from kimi_delta_attention_varlen_gb300 import _abi, build
from tests import latent8_helpers as h8

OK, NULL, DTYPE, LAYOUT, SHAPE, RANGE, WORKSPACE, CUDA, UNSUPPORTED, ALIGN = 0, -1, -2, -3, -4, -5, -6, -7, -8, -9
A = 0x10000  # a 256-byte aligned fake device address (never dereferenced)


@pytest.fixture(scope="module")
def L():
    build.build()
    return _abi.lib()


def cache(n=8, h=1, v=64, k=576, dtype=1, data=A, stride=None, reserved=0):
    return _abi.KdaCache(data, dtype, reserved, n, h, v, k, h * v * k if stride is None else stride)


def cache8(k=644, **kw):
    return cache(k=k, dtype=2, **kw)


def table(requests=4, width=8, stride=None, n_pages=8, page=64, reserved=0, bt=A, lens=A, ref=A):
    return _abi.KdaPageTable(bt, lens, ref, requests, width, width if stride is None else stride, n_pages, page, reserved)


def decode8(L, name="kda_latent_decode8", **kw):
    a = dict(q=A, io=1, batch=2, drafts=1, h=32, dl=512, dr=64, scale=0.1, cache=cache8() if name.endswith("8") else cache(), bt=A,
             requests=4, width=8, stride=8, lens=A, req=None, it=0, out=A, lse=A, ws=A, ws_bytes=1 << 40, cu=A, shared=A, groups=2)
    a.update(kw)
    c = ctypes.byref(a["cache"]) if a["cache"] is not None else None
    more = () if name.endswith("8") else (a["cu"], a["shared"], a["groups"])
    return getattr(L, name)(a["q"], a["io"], a["batch"], a["drafts"], a["h"], a["dl"], a["dr"], a["scale"], c, a["bt"], a["requests"],
                            a["width"], a["stride"], a["lens"], a["req"], a["it"], *more, a["out"], a["lse"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("name", ["kda_latent_decode8", "kda_latent_decode_shared"])
def test_decode_refusals(L, name):
    def call(**kw):
        return decode8(L, name, **kw)
    eight = name.endswith("8")
    mk, k = (cache8, 644) if eight else (cache, 576)
    assert call(cache=None) == NULL and call(cache=mk(data=0)) == NULL
    assert call(io=0) == DTYPE and call(cache=cache(dtype=0)) == DTYPE and call(req=A, it=4) == DTYPE
    assert call(cache=cache() if eight else cache8()) == DTYPE
    assert call(cache=mk(n=0)) == LAYOUT and call(cache=mk(stride=64 * k - 1)) == LAYOUT
    for bad in (dict(batch=-1), dict(drafts=0), dict(h=0), dict(dl=0), dict(dr=0), dict(requests=0), dict(width=0), dict(stride=7),
                dict(cache=mk(h=2)), dict(cache=mk(k=k - 1)), dict(cache=mk(k=k + 4)), dict(requests=1)):
        assert call(**bad) == SHAPE, bad
    assert call(dl=384, cache=mk(k=k - 128 if eight else 448)) == UNSUPPORTED
    assert call(cache=mk(v=60)) == UNSUPPORTED
    assert call(drafts=1 << 14, h=128) == RANGE and call(batch=1 << 27, requests=1 << 27) == RANGE
    assert call(width=1 << 25, stride=1 << 25) == RANGE and call(cache=mk(n=1 << 31)) == RANGE
    for scale in (0.0, -1.0, math.nan, math.inf, 2.4e38):
        assert call(scale=scale) == RANGE
    for n in ("q", "bt", "lens", "out", "ws") + (() if eight else ("cu", "shared")):
        assert call(**{n: None}) == NULL, n
    for bad in (dict(q=A + 8), dict(out=A + 8), dict(cache=mk(data=A + 8)), dict(cache=mk(stride=64 * k + 4)), dict(bt=A + 2),
                dict(lens=A + 1), dict(lse=A + 2), dict(req=A + 4, it=1)) + (() if eight else (dict(cu=A + 2), dict(shared=A + 1))):
        assert call(**bad) == ALIGN, bad
    need = L.kda_latent_decode8_workspace_size(2, 1, 32, 512, 64) if eight else L.kda_latent_decode_shared_workspace_size(2, 2, 1, 32, 512, 64)
    assert need > 0 and call(ws_bytes=need - 1) == WORKSPACE and call(ws=A + 128) == WORKSPACE
    assert call(batch=0, q=None, out=None, ws=None, cu=None, shared=None) == OK
    if not eight:
        assert call(groups=0) == SHAPE and call(groups=-1) == SHAPE and call(groups=1 << 24) == RANGE and call(requests=1 << 31) == RANGE


def test_workspace_sizes(L):
    f, g = L.kda_latent_decode8_workspace_size, L.kda_latent_decode_shared_workspace_size
    for bad in ((1, 1, 32, 384, 64), (1, 1, 32, 512, 32), (-1, 1, 32, 512, 64), (1, 0, 32, 512, 64), (1 << 27, 1, 32, 512, 64)):
        assert f(*bad) == 0 and g(bad[0], 1, *bad[1:]) == 0
    assert g(4, 0, 1, 32, 512, 64) == 0 and g(4, 1 << 24, 1, 32, 512, 64) == 0 and g(0, 1, 1, 32, 512, 64) > 0 and f(0, 1, 32, 512, 64) > 0
    assert f(4096, 1, 128, 512, 64) < 1 << 30  # bounded by the GPU, not by the batch


def append8(L, x=A, dt=1, stride=576, total=5, dl=512, dr=64, cu=A, req=A, it=0, count=3, t=None, c=None):
    return L.kda_latent_append8(x, dt, stride, total, dl, dr, cu, req, it, count, ctypes.byref(t or table()), ctypes.byref(c or cache8()), None)


def read(L, x=A, stride=576, total=5, dl=512, dr=64, cu=A, req=A, it=0, count=3, t=None, c=None, first=None):
    return L.kda_latent_read(ctypes.byref(c or cache8()), dl, dr, cu, req, it, count, first, ctypes.byref(t or table()), x, stride, total, None)


@pytest.mark.parametrize("f", [append8, read])
def test_row_refusals(L, f):
    for bad in (dict(bt=0), dict(lens=0), dict(ref=0)):
        assert f(L, t=table(**bad)) == NULL
    assert f(L, t=table(reserved=1)) == LAYOUT and f(L, c=cache8(n=0)) == LAYOUT and f(L, c=cache8(reserved=1)) == LAYOUT
    assert f(L, it=3) == DTYPE and f(L, c=cache(dtype=0)) == DTYPE and f(L, c=cache(dtype=3)) == DTYPE
    for bad in (dict(total=-1), dict(count=-1), dict(stride=575), dict(dl=0), dict(dr=0), dict(c=cache8(k=640)), dict(c=cache8(h=2, v=32)),
                dict(t=table(page=32)), dict(c=cache8(n=7))):
        assert f(L, **bad) == SHAPE, bad
    assert f(L, dl=384, c=cache8(k=516)) == UNSUPPORTED and f(L, dl=512, dr=32, c=cache8(k=580)) == UNSUPPORTED
    assert f(L, t=table(page=60), c=cache8(v=60)) == UNSUPPORTED
    assert f(L, total=1 << 31) == RANGE and f(L, stride=1 << 50, total=1 << 20) == RANGE and f(L, count=1 << 30) == RANGE
    for n in ("x", "cu", "req"):
        assert f(L, **{n: None}) == NULL, n
    for bad in (dict(x=A + 8), dict(stride=580), dict(cu=A + 2), dict(req=A + 4, it=1), dict(c=cache8(data=A + 8)),
                dict(c=cache8(stride=64 * 644 + 8))):
        assert f(L, **bad) == ALIGN, bad
    assert f(L, total=0, x=None) == OK and f(L, count=0, req=None, cu=None, x=None) == OK


def test_row_refusals_of_one_call(L):
    assert append8(L, dt=2) == DTYPE and append8(L, c=cache()) == DTYPE  # bf16 pages are kda_latent_append's
    assert append8(L, dt=0, stride=578) == ALIGN
    assert read(L, first=A + 2) == ALIGN and read(L, c=cache(k=644)) == SHAPE  # bf16 pages have dl + dr elements


def test_other_calls_take_no_byte_caches(L):
    c = ctypes.byref(cache8())
    assert L.kda_state_gather(c, A, 0, 1, None, A, None) == DTYPE
    assert L.kda_latent_append(A, 644, 5, A, A, 0, 3, ctypes.byref(table()), c, None) == DTYPE
    assert L.kda_pages_copy(c, A, A, 0, 0, None) == OK


def test_binding_refusals():
    bf, i32 = torch.bfloat16, torch.int32
    q, out = torch.zeros(2, 1, 4, 576, dtype=bf), torch.zeros(2, 1, 4, 512, dtype=bf)
    c8, c16 = torch.zeros(3, 1, 16, 644, dtype=torch.uint8), torch.zeros(3, 1, 16, 576, dtype=bf)
    bt, sl, ws = torch.zeros(2, 2, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(256, dtype=torch.uint8)
    cu2, sh = torch.zeros(2, dtype=i32), torch.zeros(1, dtype=i32)
    base = dict(q=q, block_table=bt, seq_lens=sl, out=out, workspace=ws, latent_dim=512, scale=1.0, stream=0)
    bads = (dict(q=q[0]), dict(out=out[..., :256]), dict(block_table=bt.long()), dict(seq_lens=sl[:1]), dict(lse=torch.zeros(2, 4)),
            dict(workspace=ws.view(i32)), dict(req=torch.zeros(3, dtype=i32)))
    for bad in bads + (dict(cache=c8.transpose(2, 3)),):
        with pytest.raises(ValueError):
            kda.kda_latent_decode8(**{**base, "cache": c8, **bad})
    with pytest.raises(kda.KdaError):
        kda.kda_latent_decode8(**{**base, "cache": c16})
    for bad in bads + (dict(cu_groups=cu2[:1]), dict(cu_groups=cu2.long()), dict(shared=torch.zeros(2, dtype=i32)), dict(shared=sh.long())):
        with pytest.raises(ValueError):
            kda.kda_latent_decode_shared(**{**base, "cache": c16, "cu_groups": cu2, "shared": sh, **bad})
    for f, kw in ((kda.kda_latent_decode_shared, dict(cu_groups=cu2, shared=sh)), (kda.kda_latent_decode, {})):
        with pytest.raises(TypeError):  # bytes are the 8-bit calls'
            f(**{**base, "cache": c8, **kw})
    t = kda.page_table_descriptor(bt, sl, torch.zeros(3, dtype=i32), 16)
    x, req, cu = torch.zeros(5, 576, dtype=bf), torch.zeros(2, dtype=i32), torch.zeros(3, dtype=i32)
    for bad in (dict(x=x[0]), dict(x=x[:, ::2]), dict(cu=cu[:2]), dict(cu=cu.long()), dict(req=req[:1])):
        with pytest.raises(ValueError):
            kda.kda_latent_append8(**{**dict(x=x, cu=cu, req=req, table=t, cache=c8, latent_dim=512, stream=0), **bad})
    with pytest.raises(TypeError):
        kda.kda_latent_append8(x.half(), cu, req, t, c8, latent_dim=512, stream=0)
    for bad in (dict(out=x.float()), dict(out=x[:, ::2]), dict(cu=cu[:2]), dict(first=cu), dict(first=req.long())):
        with pytest.raises(ValueError):
            kda.kda_latent_read(**{**dict(cache=c8, cu=cu, req=req, table=t, out=x, latent_dim=512, stream=0), **bad})


def test_quantiser_of_the_plain_form():
    """By hand: 448 and 1.75 * 2^k fit their unit, the next value up takes the next; ties to even; torch's own conversion."""
    x = torch.zeros(6, 320)
    x[0, 0], x[1, 0], x[2, 0], x[3, 0] = 448.0, 448.5, 1.75, -0.0
    x[4, 300], x[5, 5] = 2.0 ** 70, math.inf  # a rope key beyond 2^64; an infinity
    codes, rope, scale = h8.quantise(x, 256)
    assert scale.tolist() == [1.0, 2.0, 2.0 ** -8, 2.0 ** -64, 2.0 ** 6, 2.0 ** -64]
    assert codes[0, 0] == 448 and codes[1, 0] == 224 and codes[2, 0] == 448 and rope[4, 44] == 2.0 ** 64 and math.isnan(codes[5, 5])
    y = torch.cat([torch.linspace(-448, 448, 9001), torch.exp2(torch.linspace(-12, 8, 4001)), torch.arange(0, 64) * 2.0 ** -10])
    assert torch.equal(h8.e4m3(y.double()).float(), y.to(torch.float8_e4m3fn).float())


def test_layout_of_the_plain_form():
    cache = h8.poisoned_pages(4, 8, 256, gap=16, device="cpu")
    assert torch.isnan(h8.values(cache, 256)).all()
    x = torch.randn(3, 320)
    rows = h8.put(cache, 256, 2, slice(5, 8), x)
    raw = cache.as_strided((4, 8 * 388), (cache.stride(0), 1))[2]
    assert raw[5 * 256] == (rows[0, 0] / h8.quantise(x, 256)[2][0]).float().to(torch.float8_e4m3fn).view(torch.uint8)
    assert raw[8 * 256 + 6 * 128:][:128].view(torch.bfloat16)[3] == (rows[1, 259] / h8.quantise(x, 256)[2][1]).to(torch.bfloat16)
    assert raw[8 * 384 + 7 * 4:][:4].view(torch.float32)[0] == h8.quantise(x, 256)[2][2]
    assert torch.equal(h8.values(cache, 256)[2, 5:], rows)
    assert ((rows[:, :256] - x[:, :256].double()).abs() <= 2.0 ** -4 * x[:, :256].abs() + 2.0 ** -10 * h8.quantise(x, 256)[2][:, None]).all()
