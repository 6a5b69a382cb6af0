"""Refusals of the serving entry points, which need no GPU: every bad argument is turned down before a launch."""
import ctypes

import pytest
import torch

import bit_quantized_routed_router_gb300 as ds
from bit_quantized_routed_router_gb300 import build as dsbuild

OK, ARG, UNSUP = ds.DS_OK, ds.DS_ERR_INVALID_ARG, ds.DS_ERR_UNSUPPORTED
P = 4096  # an address that no accepted call gets to


@pytest.fixture(scope="module")
def L():
    dsbuild.build()
    return ds.lib()


def shape(**kw):
    a = dict(n_head=32, n_head_kv=8, head_dim=128, page_size=16, dtype=ds.DS_BF16, scale=0.0, window=0) | kw
    return ds.AttnShapeC(*[a[f] for f, _ in ds.AttnShapeC._fields_])


def cache(**kw):
    a = dict(k=P, v=P, n_pages=10, page_stride=16 * 8 * 128, row_stride=8 * 128, head_stride=128) | kw
    return ds.KVCacheC(*[a[f] for f, _ in ds.KVCacheC._fields_])


BAD_SHAPES = [(dict(n_head=0), ARG), (dict(n_head=33), ARG), (dict(n_head_kv=0), ARG), (dict(n_head=2048), ARG),
              (dict(head_dim=0), UNSUP), (dict(head_dim=129), UNSUP), (dict(page_size=0), ARG), (dict(page_size=65537), ARG),
              (dict(dtype=ds.DS_F32), ARG), (dict(dtype=7), ARG), (dict(scale=float("nan")), ARG), (dict(scale=-1.0), ARG),
              (dict(window=-1), ARG)]
BAD_CACHES = [dict(k=None), dict(v=None), dict(k=P + 1), dict(n_pages=-1), dict(n_pages=1 << 31), dict(page_stride=-1),
              dict(row_stride=64), dict(head_stride=127), dict(page_stride=0)]


def attention(L, sh, kv, **kw):
    a = dict(table=P, width=4, tstride=4, q=P, qs=32 * 128, T=3, cu=P, seq=P, R=2, max_new=2, out=P, os=32 * 128, lse=None, ws=P,
             wsb=1 << 40) | kw
    err = ctypes.create_string_buffer(256)
    return L.ds_moe_paged_attention(ctypes.byref(sh) if sh else None, ctypes.byref(kv) if kv else None, a["table"], a["width"],
                                    a["tstride"], a["q"], a["qs"], a["T"], a["cu"], a["seq"], a["R"], a["max_new"], a["out"],
                                    a["os"], a["lse"], a["ws"], a["wsb"], None, err, 256), err.value


def test_attention_refuses_bad_shapes_and_caches(L):
    n = ctypes.c_size_t()
    for kw, code in BAD_SHAPES:
        assert attention(L, shape(**kw), cache())[0] == code, kw
        assert L.ds_moe_attention_workspace_bytes(ctypes.byref(shape(**kw)), 1, 1, 1, ctypes.byref(n), None, 0) == code
        assert L.ds_moe_attention_path(ctypes.byref(shape(**kw)), ctypes.byref(cache()), P, 4096, 1) < 0
    for kw in BAD_CACHES:
        assert attention(L, shape(), cache(**kw))[0] == ARG, kw
    assert attention(L, None, cache())[0] == ARG and attention(L, shape(), None)[0] == ARG


def test_attention_refuses_bad_arguments(L):
    for kw in (dict(width=-1), dict(tstride=3), dict(table=None), dict(q=None), dict(cu=None), dict(seq=None), dict(out=None),
               dict(ws=None), dict(T=-1), dict(T=1 << 25), dict(R=-1), dict(max_new=-1), dict(q=P + 1), dict(out=P + 1), dict(lse=P + 2),
               dict(cu=P + 2), dict(seq=P + 1), dict(table=P + 2), dict(qs=-8), dict(os=32 * 128 - 1), dict(ws=P + 16), dict(wsb=0)):
        rc, msg = attention(L, shape(), cache(), **kw)
        assert rc == ARG and msg, kw
    for kw in (dict(T=0, q=None, out=None), dict(R=0, cu=None), dict(max_new=0)):  # nothing to do
        assert attention(L, shape(), cache(), **kw)[0] == OK, kw


def test_workspace_bytes(L):
    sh = ds.AttentionShape(32, 8, 128, 16)
    assert ds.attention_workspace_bytes(sh, 0, 0, 0) > 0
    assert ds.attention_workspace_bytes(sh, 1, 1, 1) % 256 == 0
    for bad in ((-1, 1, 1), (1, -1, 1), (1, 1, -1), (1, 1 << 25, 1)):
        with pytest.raises(ds.DsMoeError):
            ds.attention_workspace_bytes(sh, *bad)
    assert L.ds_moe_attention_workspace_bytes(ctypes.byref(shape()), 1, 1, 1, None, None, 0) == ARG


def test_append_refuses(L):
    def call(sh=None, kv=None, **kw):
        a = dict(k=P, v=P, ts=1024, hs=128, slots=P, T=2) | kw
        return L.ds_moe_kv_append(ctypes.byref(sh or shape()), ctypes.byref(kv or cache()), a["k"], a["v"], a["ts"], a["hs"],
                                  a["slots"], a["T"], None, None, 0)
    for kw, code in BAD_SHAPES:
        assert call(shape(**kw)) == code
    for kw in BAD_CACHES:
        assert call(kv=cache(**kw)) == ARG
    for kw in (dict(k=None), dict(v=None), dict(slots=None), dict(k=P + 1), dict(slots=P + 4), dict(T=-1), dict(T=1 << 25),
               dict(ts=-1), dict(hs=-1)):
        assert call(**kw) == ARG, kw
    assert call(T=0, k=None) == OK


def test_page_map_refuses(L):
    def call(**kw):
        a = dict(ctx=P, new=P, R=2, page=16, free=P, n_free=3, table=P, width=4, ts=4, slots=P, pos=P, cap=8, cu=P, seq=P, taken=P) | kw
        return L.ds_moe_page_map(a["ctx"], a["new"], a["R"], a["page"], a["free"], a["n_free"], a["table"], a["width"], a["ts"],
                                 a["slots"], a["pos"], a["cap"], a["cu"], a["seq"], a["taken"], None, None, 0)
    for kw in (dict(R=-1), dict(R=16385), dict(page=0), dict(page=65537), dict(n_free=-1), dict(width=-1), dict(cap=-1),
               dict(cap=(1 << 24) + 1), dict(ts=3), dict(ctx=None), dict(new=None), dict(free=None), dict(table=None), dict(slots=None),
               dict(pos=None), dict(cu=None), dict(seq=None), dict(taken=None), dict(ctx=P + 1), dict(slots=P + 4), dict(cu=P + 2)):
        assert call(**kw) == ARG, kw


def test_verify_refuses(L):
    def call(**kw):
        a = dict(p=P, ps=100, q=P, qs=100, dt=ds.DS_F32, T=6, V=100, tok=P, cu=P, R=2, mx=3, ua=P, us=P, out=P, n=P) | kw
        return L.ds_moe_verify_drafts(a["p"], a["ps"], a["q"], a["qs"], a["dt"], a["T"], a["V"], a["tok"], a["cu"], a["R"], a["mx"],
                                      a["ua"], a["us"], a["out"], a["n"], None, None, 0)
    for kw in (dict(dt=ds.DS_F16), dict(dt=-1), dict(V=0), dict(V=(1 << 22) + 1), dict(T=-1), dict(T=1 << 25), dict(R=-1), dict(mx=-1),
               dict(mx=0), dict(p=None), dict(tok=None), dict(ua=None), dict(us=None), dict(cu=None), dict(out=None), dict(n=None),
               dict(ps=99), dict(qs=99), dict(p=P + 2), dict(q=P + 1), dict(tok=P + 2), dict(n=P + 1)):
        assert call(**kw) == ARG, kw
    assert call(R=0, p=None) == OK


def test_binding_refuses_host_tensors_and_wrong_types(L):
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        ds.page_map(i, i, i, i.view(2, 2), 16, i.long(), i, i, i, i)
    with pytest.raises(ValueError):
        ds.KVCache(torch.zeros(2, 16, 8, 128, dtype=torch.bfloat16), torch.zeros(2, 16, 8, 128, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        ds.verify_drafts(torch.zeros(2, 9), None, i, i, i, i, i.view(2, 2), i)


class OnDevice(torch.Tensor):
    """A host tensor that says it is on the device: arguments that the binding turns down before it calls."""
    is_cuda = True


def on_device(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)


@pytest.fixture
def calls(L, monkeypatch):
    """What the binding would hand to the library, which is not called."""
    seen = []
    monkeypatch.setattr(ds, "_call", lambda fn, *args: seen.append(fn.__name__))
    return seen


def attend(**kw):
    bf16 = torch.bfloat16
    a = dict(table=on_device(2, 3), q=on_device(3, 4, 64, dtype=bf16), cu=on_device(3), seq=on_device(2),
             out=on_device(3, 4, 64, dtype=bf16), workspace=on_device(1 << 20, dtype=torch.uint8), lse=None) | kw
    cache = ds.KVCache(on_device(4, 16, 2, 64, dtype=bf16), on_device(4, 16, 2, 64, dtype=bf16))
    ds.paged_attention(ds.AttentionShape(4, 2, 64, 16), cache, a["table"], a["q"], a["cu"], a["seq"], 2, a["out"], a["workspace"],
                       lse=a["lse"], stream=0)


def test_binding_refuses_a_workspace_on_the_host(calls):
    for bad in (torch.zeros(1 << 20, dtype=torch.uint8), torch.zeros(1 << 17, dtype=torch.float64),
                on_device(1 << 20, 2, dtype=torch.uint8)[:, 0]):
        with pytest.raises(ValueError, match="workspace"):
            attend(workspace=bad)
    assert not calls
    attend()
    attend(workspace=on_device(1 << 17, dtype=torch.float64))
    assert calls == ["ds_moe_paged_attention"] * 2


# the binding's calls, with arguments that it lets through
F32, I64, BF16 = torch.float32, torch.int64, torch.bfloat16
CALLS = {
    "page_map": (lambda a: ds.page_map(*a.values(), stream=0),
                 dict(context_lens=on_device(2), new_lens=on_device(2), free_pages=on_device(9), block_table=on_device(2, 3), page_size=16,
                      slots=on_device(8, dtype=I64), positions=on_device(8), cu_new=on_device(3), seq_lens=on_device(2), n_taken=on_device(1))),
    "kv_append": (lambda a: ds.kv_append(ds.AttentionShape(4, 2, 64, 16), ds.KVCache(a["k"], a["v"]), a["k_new"], a["v_new"], a["slots"], stream=0),
                  dict(k=on_device(4, 16, 2, 64, dtype=BF16), v=on_device(4, 16, 2, 64, dtype=BF16), k_new=on_device(3, 2, 64, dtype=BF16),
                       v_new=on_device(3, 2, 64, dtype=BF16), slots=on_device(3, dtype=I64))),
    "paged_attention": (lambda a: attend(**a),
                        dict(table=on_device(2, 3), q=on_device(3, 4, 64, dtype=BF16), cu=on_device(3), seq=on_device(2),
                             out=on_device(3, 4, 64, dtype=BF16), lse=on_device(3, 4, dtype=F32))),
    "verify_drafts": (lambda a: ds.verify_drafts(*a.values(), stream=0),
                      dict(target=on_device(5, 9, dtype=F32), draft=on_device(5, 9, dtype=F32), tokens=on_device(5), cu_new=on_device(3),
                           u_accept=on_device(5, dtype=F32), u_sample=on_device(2, dtype=F32), out_tokens=on_device(2, 3),
                           n_accepted=on_device(2))),
}


@pytest.mark.parametrize("name", CALLS)
def test_binding_refuses_other_types_and_host_tensors_in_every_place(calls, name):
    call, args = CALLS[name]
    call(args)
    assert calls == ["ds_moe_" + name]
    for key, t in args.items():
        if not torch.is_tensor(t):
            continue
        plain = t.as_subclass(torch.Tensor)
        # floats for whole numbers of the same width and the other way round, another width, and the host
        others = {torch.int32: (F32, I64), I64: (torch.float64, torch.int32), F32: (torch.int32, torch.float64), BF16: (torch.float16, F32)}
        for bad in [plain] + [plain.to(d).as_subclass(OnDevice) for d in others[t.dtype]]:
            with pytest.raises(ValueError):
                call(args | {key: bad})
    assert len(calls) == 1
