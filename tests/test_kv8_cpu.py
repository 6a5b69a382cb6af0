"""Rotary positions and the 8-bit cache without a GPU: the rotation's set-up, and every refusal before a launch."""
import ctypes
import math

import pytest
import torch

import bit_quantized_routed_router_gb300 as ds
import kv8_ref
from bit_quantized_routed_router_gb300 import build as dsbuild
from test_serving_cpu import BAD_CACHES, BAD_SHAPES, cache, on_device, shape

OK, ARG, UNSUP = ds.DS_OK, ds.DS_ERR_INVALID_ARG, ds.DS_ERR_UNSUPPORTED
P = 4096  # an address that no accepted call gets to


@pytest.fixture(scope="module")
def L():
    dsbuild.build()
    return ds.lib()


@pytest.mark.parametrize("kw", [dict(dim=128), dict(dim=64, base=500000.0), dict(dim=2), dict(dim=128, base=1.0),
                                dict(dim=96, scaling="linear", factor=8.0), dict(dim=64, scaling="ntk", factor=4.0),
                                dict(dim=128, scaling="yarn", factor=32.0, original=4096),
                                dict(dim=64, base=150000.0, scaling="yarn", factor=40.0, original=4096, fast=16.0, slow=2.0)])
def test_frequencies(L, kw):
    kind = {"none": ds.ROPE_NONE, "linear": ds.ROPE_LINEAR, "ntk": ds.ROPE_NTK, "yarn": ds.ROPE_YARN}[kw.get("scaling", "none")]
    rope = ds.Rope(kw["dim"], base=kw.get("base", 10000.0), scaling=kind, factor=kw.get("factor", 1.0), original=kw.get("original", 0),
                   beta_fast=kw.get("fast", 32.0), beta_slow=kw.get("slow", 1.0))
    f, amplitude = kv8_ref.frequencies(**kw)
    assert rope.c.amplitude == pytest.approx(amplitude, rel=1e-7)
    for i in range(64):
        want = float(f[i]) / (2 * math.pi) if i < kw["dim"] // 2 else 0.0
        # 64 bits' relative precision, through pow and two products
        assert abs(rope.c.turns[i] / 2.0 ** 64 - want) <= 2.0 ** -49 * want + 2.0 ** -64, i
    assert ds.Rope(kw["dim"], amplitude=0.5).c.amplitude == 0.5


def test_rope_init_refuses(L):
    good = dict(dim=64, first=0, inter=0, base=10000.0, kind=0, factor=1.0, original=0, fast=0.0, slow=0.0, amp=0.0)

    def call(**kw):
        a = good | kw
        r = ds.RopeC()
        return L.ds_moe_rope_init(ctypes.byref(r), a["dim"], a["first"], a["inter"], a["base"], a["kind"], a["factor"], a["original"],
                                  a["fast"], a["slow"], a["amp"], None, 0)
    nan, inf = math.nan, math.inf
    for kw in (dict(dim=0), dict(dim=63), dict(dim=130), dict(dim=-2), dict(first=-1), dict(first=65), dict(inter=2), dict(base=0.5),
               dict(base=nan), dict(base=inf), dict(kind=-1), dict(kind=4), dict(kind=1, factor=0.5), dict(kind=1, factor=nan),
               dict(kind=2, dim=2, factor=2.0), dict(kind=2, base=1e300, factor=1e300), dict(kind=3, factor=4.0),
               dict(kind=3, factor=4.0, original=4096, fast=1.0, slow=2.0), dict(kind=3, factor=4.0, original=4096, fast=nan, slow=1.0),
               dict(kind=3, factor=4.0, original=4096, base=1.0), dict(amp=-1.0), dict(amp=nan), dict(amp=inf), dict(amp=1e39)):
        assert call(**kw) == ARG, kw
    assert call(kind=0, factor=nan) == OK  # not used
    assert call(kind=3, factor=4.0, original=4096) == OK
    assert L.ds_moe_rope_init(None, 64, 0, 0, 10000.0, 0, 1.0, 0, 0.0, 0.0, 0.0, None, 0) == ARG


def rope(**kw):
    r = ds.RopeC(64, 0, 0, 1.0)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def rows(**kw):
    a = dict(x=P, token_stride=4096, head_stride=128, out=2 * P, out_token_stride=4096, out_head_stride=128) | kw
    return ds.RopeRowsC(*[a[f] for f, _ in ds.RopeRowsC._fields_])


BAD_ROPES = [dict(dim=0), dict(dim=3), dict(dim=130), dict(dim=-4), dict(first=-1), dict(first=65), dict(interleaved=2),
             dict(amplitude=math.nan), dict(amplitude=math.inf)]
BAD_ROWS = [dict(x=None), dict(out=None), dict(x=P + 1), dict(out=P + 1), dict(token_stride=-1), dict(head_stride=-1),
            dict(out_token_stride=127), dict(out_head_stride=127), dict(out=P, head_stride=256), dict(out=P, token_stride=8192),
            dict(out_token_stride=-4096), dict(out_head_stride=-1), dict(out_token_stride=128), dict(out_token_stride=4095)]


def test_rotary_refuses(L):
    def call(r=None, rw=None, **kw):
        a = dict(dt=ds.DS_BF16, heads=32, D=128, pos=P, T=3) | kw
        return L.ds_moe_rotary(ctypes.byref(r or rope()), a["dt"], a["heads"], a["D"], ctypes.byref(rw or rows()), a["pos"], a["T"],
                               None, None, 0)
    for kw in BAD_ROPES:
        assert call(r=rope(**kw)) == ARG, kw
    for kw in BAD_ROWS:
        assert call(rw=rows(**kw)) == ARG, kw
    for kw in (dict(dt=ds.DS_F32), dict(heads=0), dict(heads=1025), dict(D=62), dict(pos=None), dict(pos=P + 2), dict(T=-1), dict(T=1 << 25)):
        assert call(**kw) == ARG, kw
    assert call(D=0) == UNSUP and call(D=129) == UNSUP
    assert call(T=0, pos=None) == OK
    # rows [heads][tokens] are apart as well
    assert call(rw=rows(out_token_stride=128, out_head_stride=3 * 128), pos=None) == ARG  # (positions: what is refused is not the rows)
    err = ctypes.create_string_buffer(200)
    L.ds_moe_rotary(ctypes.byref(rope()), ds.DS_BF16, 32, 128, ctypes.byref(rows(out_token_stride=128, out_head_stride=3 * 128)), P + 2, 3,
                    None, err, 200)
    assert b"positions" in err.value
    assert L.ds_moe_rotary(None, 1, 1, 128, ctypes.byref(rows()), P, 1, None, None, 0) == ARG
    assert L.ds_moe_rotary(ctypes.byref(rope()), 1, 1, 128, None, P, 1, None, None, 0) == ARG


def test_append_rotary_refuses(L):
    def call(sh=None, kv=None, r=None, q=None, **kw):
        a = dict(k=P, v=P, ts=1024, hs=128, slots=P, pos=P, T=2) | kw
        return L.ds_moe_kv_append_rotary(ctypes.byref(sh or shape()), ctypes.byref(kv or cache()), ctypes.byref(r or rope()), a["k"], a["v"],
                                         a["ts"], a["hs"], ctypes.byref(q) if q else None, a["slots"], a["pos"], a["T"], None, None, 0)
    for kw, code in BAD_SHAPES:
        assert call(shape(**kw)) == code
    for kw in BAD_CACHES:
        assert call(kv=cache(**kw)) == ARG
    for kw in BAD_ROPES:
        assert call(r=rope(**kw)) == ARG
    for kw in BAD_ROWS:
        assert call(q=rows(**kw)) == ARG
    for kw in (dict(k=None), dict(v=None), dict(slots=None), dict(pos=None), dict(k=P + 1), dict(slots=P + 4), dict(pos=P + 1), dict(T=-1),
               dict(T=1 << 25), dict(ts=-1), dict(hs=-1)):
        assert call(**kw) == ARG, kw
    assert call(T=0, k=None) == OK
    assert L.ds_moe_kv_append_rotary(ctypes.byref(shape()), ctypes.byref(cache()), None, P, P, 1024, 128, None, P, P, 2, None, None, 0) == ARG


def cache8(**kw):
    a = dict(k=P, v=P, k_scale=P, v_scale=P, n_pages=10, page_stride=16 * 8 * 128, row_stride=8 * 128, head_stride=128, scale_page_stride=16,
             scale_block_stride=8, scale_head_stride=1, block_rows=8) | kw
    return ds.KVCache8C(*[a[f] for f, _ in ds.KVCache8C._fields_])


BAD_CACHES8 = [dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None), dict(k_scale=P + 2), dict(v_scale=P + 1),
               dict(n_pages=-1), dict(n_pages=1 << 31), dict(page_stride=-1), dict(row_stride=64), dict(head_stride=127), dict(page_stride=0),
               dict(scale_head_stride=-1), dict(scale_page_stride=-16), dict(block_rows=0), dict(block_rows=5), dict(block_rows=32),
               dict(block_rows=-8)]
# strides that an append refuses, and attention does not mind
SHARED8 = [dict(scale_page_stride=0), dict(scale_block_stride=0), dict(scale_head_stride=0), dict(scale_block_stride=7),
           dict(scale_page_stride=15), dict(page_stride=16 * 8 * 128 - 1), dict(row_stride=128)]


def test_append8_refuses(L):
    def call(sh=None, kv=None, r=None, q=None, **kw):
        a = dict(k=P, v=P, ts=1024, hs=128, table=P, width=4, tstride=4, cu=P, seq=P, R=2, T=3, mx=2) | kw
        return L.ds_moe_kv8_append(ctypes.byref(sh or shape()), ctypes.byref(kv or cache8()), ctypes.byref(r) if r else None, a["k"], a["v"],
                                   a["ts"], a["hs"], ctypes.byref(q) if q else None, a["table"], a["width"], a["tstride"], a["cu"], a["seq"],
                                   a["R"], a["T"], a["mx"], None, None, 0)
    for kw, code in BAD_SHAPES:
        assert call(shape(**kw)) == code
    for kw in BAD_CACHES8 + SHARED8:
        assert call(kv=cache8(**kw)) == ARG, kw
    for kw in BAD_ROPES:
        assert call(r=rope(**kw)) == ARG
    for kw in BAD_ROWS:
        assert call(r=rope(), q=rows(**kw)) == ARG
    assert call(q=rows()) == ARG  # without rope
    for kw in (dict(k=None), dict(v=None), dict(table=None), dict(cu=None), dict(seq=None), dict(k=P + 1), dict(table=P + 2), dict(cu=P + 1),
               dict(seq=P + 2), dict(T=-1), dict(T=1 << 25), dict(ts=-1), dict(hs=-1), dict(R=-1), dict(mx=-1), dict(width=-1), dict(tstride=3)):
        assert call(**kw) == ARG, kw
    for kw in (dict(T=0, k=None), dict(R=0, cu=None), dict(mx=0)):
        assert call(**kw) == OK, kw


def attention8(L, sh, kv, **kw):
    a = dict(table=P, width=4, tstride=4, q=P, qs=32 * 128, T=3, cu=P, seq=P, R=2, max_new=2, out=P, os=32 * 128, lse=None, ws=P,
             wsb=1 << 40) | kw
    return L.ds_moe_paged_attention8(ctypes.byref(sh) if sh else None, ctypes.byref(kv) if kv else None, a["table"], a["width"],
                                     a["tstride"], a["q"], a["qs"], a["T"], a["cu"], a["seq"], a["R"], a["max_new"], a["out"],
                                     a["os"], a["lse"], a["ws"], a["wsb"], None, None, 0)


def test_attention8_refuses(L):
    n = ctypes.c_size_t()
    for kw, code in BAD_SHAPES:
        assert attention8(L, shape(**kw), cache8()) == code, kw
        assert L.ds_moe_attention8_workspace_bytes(ctypes.byref(shape(**kw)), 1, 1, 1, ctypes.byref(n), None, 0) == code
        assert L.ds_moe_attention8_path(ctypes.byref(shape(**kw)), ctypes.byref(cache8()), P, 4096, 1) < 0
    for kw in BAD_CACHES8:
        assert attention8(L, shape(), cache8(**kw)) == ARG, kw
    for kw in SHARED8:
        assert attention8(L, shape(), cache8(**kw), T=0) == OK, kw
    assert attention8(L, None, cache8()) == ARG and attention8(L, shape(), None) == ARG
    for kw in (dict(width=-1), dict(tstride=3), dict(table=None), dict(q=None), dict(cu=None), dict(seq=None), dict(out=None),
               dict(ws=None), dict(T=-1), dict(T=1 << 25), dict(R=-1), dict(max_new=-1), dict(q=P + 1), dict(out=P + 1), dict(lse=P + 2),
               dict(cu=P + 2), dict(seq=P + 1), dict(table=P + 2), dict(qs=-8), dict(os=32 * 128 - 1), dict(ws=P + 16), dict(wsb=0)):
        assert attention8(L, shape(), cache8(), **kw) == ARG, kw
    for kw in (dict(T=0, q=None, out=None), dict(R=0, cu=None), dict(max_new=0)):
        assert attention8(L, shape(), cache8(), **kw) == OK, kw


def test_binding_refuses(L, monkeypatch):
    called = []
    sh, b16, u8, f32 = ds.AttentionShape(4, 2, 64, 16), torch.bfloat16, torch.uint8, torch.float32
    good = [on_device(4, 16, 2, 64, dtype=u8)] * 2 + [on_device(4, 2, 2, dtype=f32)] * 2
    kv, r = ds.KVCache8(*good), ds.Rope(64)
    assert kv.block_rows == 8
    for i, bad in ((0, torch.zeros(4, 16, 2, 64, dtype=u8)), (0, on_device(4, 16, 2, 32, dtype=u8)), (0, on_device(4, 16, 2, 64, dtype=b16)),
                   (2, on_device(4, 3, 2, dtype=f32)), (2, on_device(3, 2, 2, dtype=f32)), (2, on_device(4, 2, 2, dtype=b16)),
                   (3, on_device(4, 2, 1, dtype=f32)), (3, on_device(4, 1, 2, dtype=f32))):
        with pytest.raises(ValueError):
            ds.KVCache8(*[bad if j == i else t for j, t in enumerate(good)])
    with pytest.raises(ds.DsMoeError):
        ds.Rope(63)
    monkeypatch.setattr(ds, "_call", lambda fn, *args: called.append(fn.__name__))
    x, pos = on_device(3, 4, 64, dtype=b16), on_device(3)
    ds.rotary(r, x, pos, x, stream=0)
    ds.rotary(r, x.transpose(0, 1).contiguous().transpose(0, 1), pos, x, stream=0)
    kn = on_device(3, 2, 64, dtype=b16)
    table, cu, seq = on_device(2, 3), on_device(3), on_device(2)
    ds.kv8_append(sh, kv, kn, kn, table, cu, seq, 2, stream=0)
    ds.kv8_append(sh, kv, kn, kn, table, cu, seq, 2, rope=r, q=x, q_out=x, stream=0)
    kv16 = ds.KVCache(on_device(4, 16, 2, 64, dtype=b16), on_device(4, 16, 2, 64, dtype=b16))
    ds.kv_append_rotary(sh, kv16, r, kn, kn, on_device(3, dtype=torch.int64), pos, q=x, q_out=x, stream=0)
    ws = on_device(1 << 10, dtype=u8)
    ds.paged_attention8(sh, kv, table, x, cu, seq, 2, x, ws, stream=0)
    assert called == ["ds_moe_rotary"] * 2 + ["ds_moe_kv8_append"] * 2 + ["ds_moe_kv_append_rotary", "ds_moe_paged_attention8"]
    half = on_device(3, 4, 64, dtype=torch.float16)
    for bad in (lambda: ds.rotary(r, torch.zeros(3, 4, 64, dtype=b16), pos, x, stream=0), lambda: ds.rotary(r, x, pos.long(), x, stream=0),
                lambda: ds.rotary(r, x, on_device(2), x, stream=0), lambda: ds.rotary(r, x, pos, half, stream=0),
                lambda: ds.rotary(r, on_device(3, 4, 64, dtype=f32), pos, on_device(3, 4, 64, dtype=f32), stream=0),
                lambda: ds.rotary(r, x, pos, on_device(3, 4, 32, dtype=b16), stream=0),
                lambda: ds.kv8_append(sh, kv, kn, kn, table, cu, seq, 2, rope=r, q=x, stream=0),
                lambda: ds.kv8_append(sh, kv, kn, kn, table, cu, seq, 2, rope=r, q=half, q_out=half, stream=0),
                lambda: ds.kv8_append(sh, kv, kn, kn, table, cu, seq, 2, rope=r, q=on_device(2, 4, 64, dtype=b16), q_out=on_device(2, 4, 64, dtype=b16), stream=0),
                lambda: ds.kv8_append(sh, kv, kn, kn, table, cu, on_device(3), 2, stream=0),
                lambda: ds.kv8_append(sh, kv, half[:, :2], half[:, :2], table, cu, seq, 2, stream=0),
                lambda: ds.kv8_append(ds.AttentionShape(4, 2, 64, 32), kv, kn, kn, table, cu, seq, 2, stream=0),
                lambda: ds.kv_append_rotary(sh, kv16, r, kn, kn, on_device(3), pos, stream=0),
                lambda: ds.kv_append_rotary(sh, kv16, r, kn, kn, on_device(3, dtype=torch.int64), on_device(2), stream=0),
                lambda: ds.paged_attention8(sh, kv, table, half, cu, seq, 2, half, ws, stream=0),
                lambda: ds.paged_attention8(sh, kv, table, x, cu, seq, 2, on_device(2, 4, 64, dtype=b16), ws, stream=0)):
        with pytest.raises(ValueError):
            bad()
    assert len(called) == 6


@pytest.mark.parametrize("kw", [dict(row_stride=128), dict(page_stride=16 * 8 * 128 - 1), dict(head_stride=8 * 128, row_stride=8 * 128),
                                dict(page_stride=128, row_stride=8 * 128, n_pages=9), dict(row_stride=8 * 128 - 1)])
def test_16_bit_appends_refuse_rows_that_overlap(L, kw):
    """Where a row of one head is a row of another, or of another page, what an append leaves would depend on its order;
    attention may read such a cache."""
    sh, kv = shape(), cache(**kw)
    err = ctypes.create_string_buffer(200)
    assert L.ds_moe_kv_append(ctypes.byref(sh), ctypes.byref(kv), P, P, 1024, 128, P, 2, None, err, 200) == ARG and b"overlap" in err.value
    err = ctypes.create_string_buffer(200)
    assert L.ds_moe_kv_append_rotary(ctypes.byref(sh), ctypes.byref(kv), ctypes.byref(rope()), P, P, 1024, 128, None, P, P, 2, None, err,
                                     200) == ARG and b"overlap" in err.value
    a = [P, 4, 4, P, 32 * 128, 0, P, P, 2, 2, P, 32 * 128, None, P, 1 << 40]
    assert L.ds_moe_paged_attention(ctypes.byref(sh), ctypes.byref(kv), *a, None, None, 0) == OK


@pytest.mark.parametrize("kw", [dict(), dict(row_stride=128, head_stride=16 * 128), dict(page_stride=2 * 16 * 8 * 128),
                                dict(row_stride=10 * 8 * 128, page_stride=8 * 128), dict(row_stride=8 * 136, head_stride=136, page_stride=16 * 8 * 136),
                                dict(n_pages=1, page_stride=0)])
def test_16_bit_appends_take_any_order_of_the_axes(L, kw):
    """(Refused for its rows' address, which is looked at behind the cache: nothing runs.)"""
    err = ctypes.create_string_buffer(200)
    assert L.ds_moe_kv_append(ctypes.byref(shape()), ctypes.byref(cache(**kw)), P + 1, P, 1024, 128, P, 2, None, err, 200) == ARG
    assert b"aligned" in err.value
