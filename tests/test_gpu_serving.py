"""The serving operators on the GPU against their plain 64-bit forms, at the sizes and masks where they can go wrong."""
import math
import random

import numpy as np
import pytest
import torch

import bit_quantized_routed_router_gb300 as ds
import serving_ref as ref

pytestmark = pytest.mark.gpu


def shape_of(c):
    return ds.AttentionShape(c.H, c.G, c.D, c.page, ds.DS_F16 if c.dtype == "f16" else ds.DS_BF16, window=c.window)


def attend(c, max_new=None, workspace=None, lse=True, out=None, stream=None):
    sh, cache = shape_of(c), ds.KVCache(c.k, c.v)
    max_new = max([1] + c.new) if max_new is None else max_new
    if workspace is None:
        workspace = torch.full((ds.attention_workspace_bytes(sh, c.R, c.T, max_new),), 0xFF, dtype=torch.uint8, device="cuda")
    if out is None:
        out = torch.full((c.T, c.H, c.D), 7.0, dtype=c.dt, device="cuda")
    z = torch.full((c.T, c.H), 7.0, device="cuda") if lse else None
    ds.paged_attention(sh, cache, c.table, c.q, c.cu, c.seq_lens, max_new, out, workspace, lse=z, stream=stream)
    c.path = ds.attention_path(sh, cache, c.q, max_new)
    return out, z


def check(c, out, lse, rows=None):
    want, wlse, mag = c.reference()
    rows = torch.ones(c.T, dtype=torch.bool) if rows is None else rows
    tol, ltol = c.tolerances(want, mag, c.path != ds.ATTN_GENERIC)
    off = (out.cpu().double() - want).abs()
    assert bool((off <= tol)[rows].all()), f"out off by {float((off / tol.clamp(min=1e-30))[rows].max()):.3g} of the tolerance"
    if lse is not None:
        got = lse.cpu().double()
        none = torch.isinf(wlse)
        assert torch.equal(torch.isneginf(got)[rows], none[rows])
        assert bool(((got - wlse).abs()[rows] <= ltol + 2.0 ** -24 * wlse.abs()[rows])[~none[rows]].all())


R = random.Random(5)
CASES = {
    # ctx, new, heads, key heads, dim, page, options
    "one_key": ([0], [1], 1, 1, 64, 16, {}),
    "one_token": ([136], [1], 32, 8, 128, 16, {}),
    "tile_edges": ([126, 127, 128, 255, 256], [1, 1, 1, 1, 1], 8, 2, 128, 32, {}),
    "some_without_tokens": ([5, 0, 300, 9], [0, 1, 0, 2], 8, 2, 64, 8, {}),
    "none_cached": ([0, 0, 0], [1, 7, 130], 4, 2, 128, 16, {}),
    "drafts": (ref.lengths(R, 9, 0, 700), ref.lengths(R, 9, 1, 6), 28, 4, 64, 24, {}),
    "drafts_f16": (ref.lengths(R, 9, 0, 700), ref.lengths(R, 9, 1, 6), 28, 4, 128, 48, dict(dtype="f16")),
    "long": ([9000], [1], 8, 1, 128, 16, {}),
    "long_few_heads": ([20011, 3], [2, 1], 2, 1, 64, 64, {}),
    "rows_16": ([500], [2], 16, 2, 128, 16, {}),
    "rows_17": ([500], [17], 1, 1, 128, 16, {}),
    "rows_64": ([333], [8], 8, 1, 128, 16, {}),
    "rows_65": ([333], [13], 5, 1, 128, 16, {}),
    "rows_128": ([200], [16], 8, 1, 64, 16, {}),
    "rows_129": ([200], [129], 1, 1, 64, 16, {}),
    "rows_300": ([77], [75], 4, 1, 128, 32, {}),
    "group_7": ([100, 31], [50, 64], 14, 2, 128, 16, {}),
    "group_128": ([40], [3], 128, 1, 64, 16, {}),
    "group_200": ([40], [2], 200, 1, 64, 16, {}),
    "own_heads": ([64, 200], [90, 33], 6, 6, 64, 48, dict(dtype="f16")),
    "mixed": ([700, 0, 1, 300, 128], [1, 200, 3, 129, 1], 8, 2, 128, 64, {}),
    "chunk": ([515], [400], 4, 2, 128, 128, dict(dtype="f16")),
    "window_1": ([50, 0], [3, 40], 4, 2, 128, 16, dict(window=1)),
    "window_100": ([500, 40, 0], [3, 300, 140], 4, 2, 128, 16, dict(window=100)),
    "window_decode": ([1000, 129, 5], [1, 1, 2], 8, 2, 64, 32, dict(window=128)),
    "window_wide": ([100], [60], 4, 2, 64, 16, dict(window=5000)),
    "dim_40": ([60, 200], [1, 2], 8, 2, 40, 16, {}),
    "dim_80": ([60, 200], [70, 2], 8, 2, 80, 8, {}),
    "dim_96": ([300], [4], 8, 2, 96, 256, {}),
    "dim_72_f16": ([130], [100], 4, 2, 72, 64, dict(dtype="f16")),
    "dim_1": ([70], [3], 2, 1, 1, 16, {}),
    "dim_37": ([70], [3], 2, 1, 37, 16, {}),
    "page_1": ([70], [3], 4, 2, 64, 1, {}),
    "page_20": ([170], [3], 4, 2, 64, 20, {}),
    "page_8": ([170, 1000], [3, 1], 4, 2, 128, 8, {}),
    "page_40": ([170, 1000], [3, 200], 4, 2, 128, 40, {}),
    "page_1024": ([170, 1500], [3, 200], 4, 2, 128, 1024, {}),
    "heads_first": ([170, 1000], [3, 150], 4, 2, 128, 16, dict(layout="heads")),
    "both_in_one": ([170, 1000], [3, 1], 4, 2, 128, 16, dict(layout="both")),
    "padded_rows": ([170, 1000], [3, 150], 4, 2, 64, 16, dict(layout="padded")),
    "odd_strides": ([170, 300], [3, 1], 4, 2, 64, 16, dict(layout="odd")),
    "fused_q": ([170, 300], [3, 100], 4, 2, 64, 16, dict(qkv=True)),
    "shorter_than_chunk": ([0, 0], [5, 200], 4, 2, 128, 16, dict(seq=[3, 40])),
    "empty_sequence": ([0, 30], [5, 1], 4, 2, 128, 16, dict(seq=[0, 31])),
    "many_requests": (ref.lengths(R, 70, 0, 300), ref.lengths(R, 70, 0, 3), 8, 2, 64, 16, {}),
    "many_chunks": (ref.lengths(R, 40, 0, 900), [9] * 40, 16, 2, 128, 64, {}),
    "many_chunks_64": (ref.lengths(R, 60, 0, 300), ref.lengths(R, 60, 1, 40), 14, 2, 64, 16, dict(dtype="f16")),
    "chunks_and_windows": (ref.lengths(R, 24, 0, 700), ref.lengths(R, 24, 1, 300), 2, 2, 64, 48, dict(window=200)),
    "sharp": ([700], [40], 4, 2, 128, 16, dict(qscale=12.0)),
    "sharp_decode": ([2000], [2], 4, 2, 128, 16, dict(qscale=12.0, dtype="f16")),
}


@pytest.mark.parametrize("name", CASES)
def test_attention(name):
    ctx, new, H, G, D, page, kw = CASES[name]
    c = ref.Case(ctx, new, H, G, D, page, **kw).put()
    out, lse = attend(c)
    ds.sync_status()
    check(c, out, lse)
    # without lse, and again: the same bits
    again, _ = attend(c, lse=False)
    assert torch.equal(out, again)


def growing(c, order):
    """Keys whose scores grow (or fall) along the sequence, so that the running maximum keeps moving (or never does)."""
    for r, s in enumerate(c.seq):
        k = torch.zeros(s, c.G, c.D)
        ramp = torch.arange(s, dtype=torch.float32) / 16
        k[..., 0] = (ramp if order > 0 else ramp.flip(0))[:, None]
        c.keys[r] = (k + 0.01 * c.keys[r].float()).to(c.dt)
    c.q_cpu = (0.1 * c.q_cpu.float()).to(c.dt)
    c.q_cpu[..., 0] = 8.0
    return c


@pytest.mark.parametrize("order", [1, -1])
@pytest.mark.parametrize("new", [1, 4, 150])
def test_attention_moving_maximum(order, new):
    c = growing(ref.Case([900, 20], [new, 1], 8, 2, 128, 16), order).put()
    out, lse = attend(c)
    ds.sync_status()
    check(c, out, lse)


@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("new", [2, 4, 150, 300])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_later_tokens_have_no_influence(what, new, D):
    """The last new token's key or value is not a number: rows before it do not see it."""
    for side in ("values", "keys"):
        c = ref.Case([120, 40], [new, 3], 8, 2, D, 16)
        getattr(c, side)[0][-1, :, 3:9] = what
        c.put()
        out, lse = attend(c)
        ds.sync_status()
        rows = torch.ones(c.T, dtype=torch.bool)
        rows[new - 1] = False
        check(c, out, lse, rows)
        if side == "values":
            o = out[new - 1, :, 3:9].cpu().double()
            assert bool((torch.isnan(o) if math.isnan(what) else o == what).all())
            assert bool(torch.isfinite(out[new - 1, :, 9:]).all()) and bool(torch.isfinite(out[new - 1, :, :3]).all())


@pytest.mark.parametrize("new", [8, 20, 100, 150, 300])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_attention_many_infinities_in_a_tile(new, D, dtype):
    """Several values that are not finite in one tile, each seen by some rows only, where the maxima rise from tile to
    tile: rows that do not see them keep their sums, the others get what the formula gives."""
    ctx = 120
    c = growing(ref.Case([ctx, 40], [new, 3], 8, 2, D, 16, dtype=dtype), 1)
    for i, (at, what) in enumerate(((1, math.inf), (2, math.inf), (3, -math.inf), (new // 2, math.nan), (new - 4, math.inf),
                                    (new - 3, -math.inf), (new - 1, math.nan))):
        c.values[0][ctx + at, :, 5 * i: 5 * i + 7] = what  # (neighbours share elements)
    c.put()
    out, lse = attend(c)
    ds.sync_status()
    want, wlse, mag = c.reference()
    tol, ltol = c.tolerances(want, mag, True)
    got, fin = out.cpu().double(), torch.isfinite(want)
    assert not bool(fin.all()) and torch.equal(torch.isfinite(got), fin)
    assert torch.equal(got[~fin].nan_to_num(7.0), want[~fin].nan_to_num(7.0))
    assert bool(((got - want).abs() <= tol)[fin].all())
    assert bool(((lse.cpu().double() - wlse).abs() <= ltol + 2.0 ** -24 * wlse.abs()).all())


@pytest.mark.parametrize("new", [1, 3, 150])
def test_attention_keys_before_the_window_have_no_influence(new):
    c = ref.Case([400], [new], 4, 2, 128, 16, window=90)
    first = 400 + 1 - 90
    c.values[0][:first], c.keys[0][:first] = math.nan, math.inf
    c.put()
    out, lse = attend(c)
    ds.sync_status()
    check(c, out, lse)


@pytest.mark.parametrize("new", [1, 100])
def test_attention_bad_page_is_zeros_and_reported(new):
    for bad in (-1, -(1 << 30), 1 << 30, None):
        c = ref.Case([200, 50], [new, 1], 4, 2, 128, 16)
        c.table_cpu_bad = c.n_pages if bad is None else bad
        c.put()
        c.table[0, 3] = c.table_cpu_bad
        c.keys[0][48:64] = 0
        c.values[0][48:64] = 0
        out, lse = attend(c)
        with pytest.raises(ds.DsMoeError) as e:
            ds.sync_status()
        assert e.value.code == ds.DS_ERR_DEVICE_CHECK
        check(c, out, lse)
    ds.sync_status()


@pytest.mark.parametrize("new", [1, 40])
def test_attention_bad_lengths_are_reported_and_bounded(new):
    c = ref.Case([100, 90, 80], [new, new, new], 4, 2, 64, 16).put()
    out0, lse0 = attend(c)
    ds.sync_status()
    for name, at, v in (("seq_lens", 1, 1 << 30), ("seq_lens", 1, -5), ("cu", 3, 1 << 20), ("cu", 0, -3)):
        t = getattr(c, name)
        keep = int(t[at])
        t[at] = v
        out, lse = attend(c)
        with pytest.raises(ds.DsMoeError) as e:
            ds.sync_status()
        assert e.value.code == ds.DS_ERR_DEVICE_CHECK
        other = slice(0, new) if name == "seq_lens" else slice(new, 2 * new)  # a request that the bad entry is not of
        assert torch.equal(out[other], out0[other]) and torch.equal(lse[other], lse0[other])
        t[at] = keep
    # more new tokens than max_new: dropped, their rows kept as they were
    if new > 1:
        out, _ = attend(c, max_new=new - 1)
        with pytest.raises(ds.DsMoeError):
            ds.sync_status()
        assert bool((out[new - 1] == 7.0).all())
        sh = shape_of(c)
        if ds.attention_path(sh, ds.KVCache(c.k, c.v), c.q, new - 1) == ds.attention_path(sh, ds.KVCache(c.k, c.v), c.q, new):
            tol = 2 * torch.finfo(c.dt).eps
            assert bool(((out[: new - 1] - out0[: new - 1]).abs() <= tol * (1 + out0[: new - 1].abs())).all())
    ds.sync_status()


def test_attention_rows_beyond_the_last_are_kept():
    c = ref.Case([100, 90], [3, 2], 4, 2, 64, 16).put()
    c.T += 4
    c.q = torch.cat([c.q, torch.full((4, 4, 64), math.nan, dtype=c.dt, device="cuda")])
    out, lse = attend(c)
    ds.sync_status()
    assert bool((out[5:] == 7.0).all()) and bool((lse[5:] == 7.0).all())
    c.T -= 4
    check(c, out[:5], lse[:5])


def test_attention_out_strided_and_in_a_stream_and_a_graph():
    for new in (2, 150):
        c = ref.Case([300, 41], [new, 1], 8, 2, 128, 16).put()
        out0, lse0 = attend(c)
        sh, cache = shape_of(c), ds.KVCache(c.k, c.v)
        ws = torch.empty(ds.attention_workspace_bytes(sh, c.R, c.T, new), dtype=torch.uint8, device="cuda")
        wide = torch.full((c.T, c.H + 3, c.D), 7.0, dtype=c.dt, device="cuda")
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            attend(c, workspace=ws, out=wide[:, : c.H])
        s.synchronize()
        assert torch.equal(wide[:, : c.H], out0) and bool((wide[:, c.H:] == 7.0).all())
        out, lse = torch.empty_like(out0), torch.empty_like(lse0)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ds.paged_attention(sh, cache, c.table, c.q, c.cu, c.seq_lens, new, out, ws, lse=lse)
        for _ in range(3):
            out.zero_(), lse.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, out0) and torch.equal(lse, lse0)
    ds.sync_status()


def test_attention_offsets_beyond_32_bits():
    """Pages whose elements lie beyond 2^31 of the cache's first (and bytes beyond 2^32)."""
    n_pages, page, G, D = 36000, 64, 8, 128
    for new in (1, 40):
        c = ref.Case([500], [new], 16, G, D, page)
        k, v = (torch.empty(n_pages, page, G, D, dtype=c.dt, device="cuda") for _ in range(2))
        c.put()
        used = ref.cdiv(500 + new, page)
        for j in range(used):
            k[n_pages - 1 - j], v[n_pages - 1 - j] = c.k[c.table[0, j].long()], c.v[c.table[0, j].long()]
            c.table[0, j] = n_pages - 1 - j
        c.k, c.v = k, v
        out, lse = attend(c)
        ds.sync_status()
        check(c, out, lse)


@pytest.mark.parametrize("page,D,new,window", [(16, 128, 1, 0), (64, 64, 2, 0), (24, 128, 33, 700)])
def test_attention_long_sequences(page, D, new, window):
    """Tens of thousands of keys against a 64-bit form on the device, all heads at once."""
    H, G, L = 8, 2, 70001
    g = torch.Generator(device="cuda").manual_seed(3)
    n = ref.cdiv(L, page)
    table = torch.randperm(n, generator=g, device="cuda").to(torch.int32).view(1, n)
    k, v = (torch.randn(n, page, G, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(new, H, D, generator=g, device="cuda").bfloat16()
    cu = torch.tensor([0, new], dtype=torch.int32, device="cuda")
    seq = torch.tensor([L], dtype=torch.int32, device="cuda")
    sh = ds.AttentionShape(H, G, D, page, window=window)
    ws = torch.empty(ds.attention_workspace_bytes(sh, 1, new, new), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(new, H, device="cuda")
    ds.paged_attention(sh, ds.KVCache(k, v), table, q, cu, seq, new, out, ws, lse=lse)
    ds.sync_status()
    kk, vv = (t[table[0].long()].reshape(-1, G, D)[:L].double() for t in (k, v))
    s = torch.einsum("ighd,jgd->ighj", q.double().view(new, G, H // G, D), kk) / math.sqrt(D)
    far = torch.arange(L - new, L, device="cuda")[:, None] - torch.arange(L, device="cuda")
    hidden = (far < 0) | ((far >= window) if window else (far < 0))
    s = s.masked_fill(hidden[:, None, None], -math.inf)
    z = torch.logsumexp(s, -1)
    p = torch.exp(s - z[..., None])
    want = torch.einsum("ighj,jgd->ighd", p, vv).reshape(new, H, D)
    mag = torch.einsum("ighj,jgd->ighd", p, vv.abs()).reshape(new, H, D)
    # a score's fp32 sum: D products of magnitude at most |q||k|; sums of n terms in order are off by at most
    # (n / 128 + 256) 2^-24 of their magnitude when taken in tiles of 128
    score = (D + 4) * 2.0 ** -24 * float(q.double().norm(dim=-1).max() * kk.norm(dim=-1).max()) / math.sqrt(D)
    sums = (L / 128 + 256) * 2.0 ** -24
    u = 2.0 ** -8
    tol = u * want.abs() + (u + 2 * score + 2 * sums) * mag
    assert bool(((out.double() - want).abs() <= tol).all())
    assert bool(((lse.double() - z.reshape(new, H)).abs() <= score + sums + 2.0 ** -20).all())


def test_attention_path():
    """Which kernel serves which geometry: the fast ones want 8-element alignment, pages of whole 8-row groups and heads
    of a multiple of 8; up to 32 query rows a key head the decode kernel, above it the chunk kernel."""
    def path(new, H=8, G=2, D=128, page=16, **kw):
        c = ref.Case([20], [new], H, G, D, page, **kw).put()
        return ds.attention_path(shape_of(c), ds.KVCache(c.k, c.v), c.q, new)
    assert path(1) == path(8) == path(1, H=32, G=1) == path(2, D=64, page=8, layout="heads") == ds.ATTN_DECODE
    assert path(9) == path(1, H=33, G=1) == path(1, H=128, G=1) == path(300, D=72, layout="both") == ds.ATTN_CHUNK
    assert path(1, page=20) == path(1, D=36) == path(9, layout="odd", D=64) == path(1, H=129, G=1) == ds.ATTN_GENERIC


def test_example_runs():
    import importlib.util
    import os
    at = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serving_step.py")
    spec = importlib.util.spec_from_file_location("serving_step", at)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    kept = example.run(steps=5)
    assert all(len(k) > 40 for k in kept)


# -------------------------------------------------------------------- page map


def run_page_map(ctx, new, page, free, table, cap):
    i32 = dict(dtype=torch.int32, device="cuda")
    R_ = len(ctx)
    dev = table.cuda()
    out = dict(slots=torch.full((cap,), 99, dtype=torch.int64, device="cuda"), positions=torch.full((cap,), 99, **i32),
               cu_new=torch.full((R_ + 1,), 99, **i32), seq_lens=torch.full((R_,), 99, **i32), n_taken=torch.full((1,), 99, **i32))
    args = (torch.tensor(ctx, **i32), torch.tensor(new, **i32), torch.tensor(free, **i32), dev, page)
    for _ in range(2):  # the same call again gives the same
        ds.page_map(*args, **out)
    try:
        ds.sync_status()
        bad = False
    except ds.DsMoeError as e:
        assert e.code == ds.DS_ERR_DEVICE_CHECK
        bad = True
    return dev.cpu(), {k: v.cpu().tolist() for k, v in out.items()}, bad


def held_table(rng, ctx, page, width, n_extra):
    ids = list(range(sum(ref.cdiv(max(0, c), page) for c in ctx) + n_extra))
    rng.shuffle(ids)
    table = torch.full((len(ctx), width), -7, dtype=torch.int32)
    for r, c in enumerate(ctx):
        for j in range(min(width, ref.cdiv(max(0, c), page))):
            table[r, j] = ids.pop()
    return table, ids


@pytest.mark.parametrize("n,ctx_hi,new_hi,page", [(1, 0, 1, 16), (1, 40, 1, 1), (7, 100, 5, 16), (64, 3000, 9, 64), (33, 70, 200, 24),
                                                  (600, 50, 3, 8), (513, 50, 40, 7), (5, 2, 3000, 100), (3, 5, 0, 16)])
def test_page_map(n, ctx_hi, new_hi, page):
    rng = random.Random(n)
    ctx, new = ref.lengths(rng, n, 0, ctx_hi), ref.lengths(rng, n, 0, new_hi)
    width = max(1, max(ref.cdiv(a + b, page) for a, b in zip(ctx, new)))
    table, free = held_table(rng, ctx, page, width, 5 + sum(new))
    cap = sum(new) + rng.randint(0, 9)
    got_table, got, bad = run_page_map(ctx, new, page, free, table, cap)
    slots, positions, cu, seq, taken, want_bad = ref.page_map(ctx, new, page, free, table, cap)
    assert not bad and not want_bad
    assert torch.equal(got_table, table)
    assert got == dict(slots=slots, positions=positions, cu_new=cu, seq_lens=seq, n_taken=[taken])


@pytest.mark.parametrize("what", ["few_pages", "no_pages", "narrow", "no_columns", "room", "no_room", "negative", "huge", "hole"])
def test_page_map_reports(what):
    rng = random.Random(8)
    ctx, new = ref.lengths(rng, 9, 0, 50), ref.lengths(rng, 9, 1, 40)
    width = max(ref.cdiv(a + b, 16) for a, b in zip(ctx, new))
    cap = sum(new) + 3
    if what == "narrow":
        width = 2
    if what == "negative":
        ctx[2], new[4], new[5] = -1, -3, -(1 << 31)
    if what == "huge":
        ctx[2], new[4] = 1 << 30, (1 << 31) - 1
    if what == "no_columns":
        width = 0
    table, free = held_table(rng, [c if c < 1 << 20 else 0 for c in ctx], 16, width, sum(max(0, v) for v in new if v < 1 << 20))
    if what == "few_pages":
        free = free[:4]
    if what == "no_pages":
        free = []
    if what == "room":
        cap = sum(new) // 2
    if what == "no_room":
        cap = 0
    if what == "hole":
        ctx[3] = 20
        table[3, 1] = -1
    got_table, got, bad = run_page_map(ctx, new, 16, free, table, cap)
    slots, positions, cu, seq, taken, want_bad = ref.page_map(ctx, new, 16, free, table, cap)
    assert bad and want_bad
    assert torch.equal(got_table, table)
    assert got == dict(slots=slots, positions=positions, cu_new=cu, seq_lens=seq, n_taken=[taken])
    ds.sync_status()


def test_page_map_no_requests_and_many():
    _, got, bad = run_page_map([], [], 16, [3], torch.zeros(0, 1, dtype=torch.int32), 4)
    assert not bad and got == dict(slots=[-1] * 4, positions=[-1] * 4, cu_new=[0], seq_lens=[], n_taken=[0])
    n = 16384
    rng = random.Random(1)
    ctx, new = ref.lengths(rng, n, 0, 20), ref.lengths(rng, n, 0, 2)
    table, free = held_table(rng, ctx, 16, 2, 2 * n)
    cap = sum(new)
    got_table, got, bad = run_page_map(ctx, new, 16, free, table, cap)
    slots, positions, cu, seq, taken, _ = ref.page_map(ctx, new, 16, free, table, cap)
    assert not bad and torch.equal(got_table, table)
    assert got == dict(slots=slots, positions=positions, cu_new=cu, seq_lens=seq, n_taken=[taken])


# ------------------------------------------------------------------- kv append


@pytest.mark.parametrize("T,G,D,page,layout", [(1, 1, 64, 16, "pages"), (37, 8, 128, 16, "pages"), (300, 3, 80, 24, "heads"),
                                               (65, 2, 37, 5, "pages"), (20, 4, 64, 16, "both"), (20, 4, 64, 16, "odd"),
                                               (20, 4, 64, 16, "padded"), (3000, 2, 128, 64, "pages")])
@pytest.mark.parametrize("fused", [False, True])
def test_kv_append(T, G, D, page, layout, fused):
    c = ref.Case([T], [1], G, G, D, page, layout=layout).put()
    g = torch.Generator().manual_seed(T)
    places = torch.randperm(c.n_pages * page, generator=g)[:T]
    slots = torch.where(torch.rand(T, generator=g) < 0.2, -1 - places, places) if T > 1 else places
    if fused:  # slices of one projection
        kv = torch.randn(T, 2 * G + 1, D, generator=g).to(c.dt).cuda()
        kn, vn = kv[:, 1: G + 1], kv[:, G + 1:]
    else:
        kn, vn = (torch.randn(T, G, D, generator=g).to(c.dt).cuda() for _ in range(2))
    bits = lambda t: t.cpu().contiguous().view(torch.int16)  # noqa: E731  (NaN are compared too)
    want = [bits(t).reshape(-1, G, D).clone() for t in (c.k, c.v)]
    for w, n in zip(want, (kn, vn)):
        w[slots[slots >= 0]] = bits(n)[slots >= 0]
    ds.kv_append(shape_of(c), ds.KVCache(c.k, c.v), kn, vn, slots.cuda())
    ds.sync_status()
    for t, w in zip((c.k, c.v), want):
        assert torch.equal(bits(t).reshape(-1, G, D), w)
    # a slot beyond the cache is skipped and reported
    slots[0] = c.n_pages * page
    ds.kv_append(shape_of(c), ds.KVCache(c.k, c.v), kn, vn, slots.cuda())
    with pytest.raises(ds.DsMoeError) as e:
        ds.sync_status()
    assert e.value.code == ds.DS_ERR_DEVICE_CHECK
    for t, w in zip((c.k, c.v), want):
        assert torch.equal(bits(t).reshape(-1, G, D), w)


# ---------------------------------------------------------------------- verify


def run_verify(p, q, tokens, cu, ua, us, max_new, bad=False, pad=0):
    dev = lambda t: None if t is None else torch.nn.functional.pad(t, (0, pad)).cuda()[:, : t.shape[1]]  # noqa: E731
    R_ = len(cu) - 1
    out = torch.full((R_, max_new), 99, dtype=torch.int32, device="cuda")
    n = torch.full((R_,), 99, dtype=torch.int32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    ds.verify_drafts(dev(p), dev(q), torch.tensor(tokens, **i32), torch.tensor(cu, **i32), torch.tensor(ua, dtype=torch.float32, device="cuda"),
                     torch.tensor(us, dtype=torch.float32, device="cuda"), out, n)
    if bad:
        with pytest.raises(ds.DsMoeError) as e:
            ds.sync_status()
        assert e.value.code == ds.DS_ERR_DEVICE_CHECK
    else:
        ds.sync_status()
    return out.cpu().numpy(), n.cpu().numpy()


def draws(seed, n_requests, new_lo, new_hi, V, sharp=3.0, dtype=torch.float32, drafted=True):
    rng = random.Random(seed)
    g = torch.Generator().manual_seed(seed)
    new = ref.lengths(rng, n_requests, new_lo, new_hi)
    cu = [0] + np.cumsum(new).tolist()
    T = cu[-1]
    logits = sharp * torch.randn(T, V, generator=g)
    p = torch.softmax(logits, -1).to(dtype)
    qf = torch.softmax(logits + torch.randn(T, V, generator=g), -1)
    tokens = np.roll(torch.multinomial(qf, 1, generator=g)[:, 0].numpy(), 1).astype(np.int32) if T else np.zeros(0, np.int32)
    ua, us = torch.rand(T, generator=g).numpy(), torch.rand(n_requests, generator=g).numpy()
    return p, qf.to(dtype) if drafted else None, tokens, cu, ua, us


@pytest.mark.parametrize("n,new_lo,new_hi,V", [(1, 1, 1, 1), (1, 4, 4, 5), (7, 0, 4, 33), (20, 1, 6, 1000), (9, 2, 3, 1024), (9, 2, 3, 1025),
                                               (5, 1, 4, 32768), (40, 1, 8, 100003), (3, 1, 2, 300001), (300, 1, 2, 2049)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("drafted", [True, False])
def test_verify(n, new_lo, new_hi, V, dtype, drafted):
    p, q, tokens, cu, ua, us = draws(n + V, n, new_lo, new_hi, V, dtype=dtype, drafted=drafted)
    mx = new_hi + 1
    got = run_verify(p, q, tokens, cu, ua, us, mx, pad=3 if V % 2 else 0)
    want = ref.verify(p.float().numpy(), None if q is None else q.float().numpy(), tokens, cu, ua, us, mx)
    assert np.array_equal(got[1], want[1]) and np.array_equal(got[0], want[0])


def test_verify_edges():
    V = 6
    p = torch.tensor([[.1, .2, .3, .4, 0, 0], [.25, .25, .25, .25, 0, 0], [0, 0, 0, 0, 0, 1.0]])
    tok = [0, 3, 1]
    # u q < p holds strictly: u = 0.5 and p = q / 2 is a refusal; just below is not
    q = torch.tensor([[.1, .05, .05, .8, 0, 0], [.25, .25, .25, .25, 0, 0], [0, 0, 0, 0, 0, 1.0]])
    for u, kept in ((.5, 0), (float(np.nextafter(np.float32(.5), np.float32(0))), 2)):
        out, n = run_verify(p, q, tok, [0, 3], [u, .999, 0], [.5], 3)
        assert n[0] == kept
    # draws at both ends of the line, and entries of no weight in between
    for u, x in ((0.0, 1), (float(np.nextafter(np.float32(1), np.float32(0))), 2)):
        out, n = run_verify(p, q, tok, [0, 3], [.99, 0, 0], [u], 4)
        assert n[0] == 0 and out[0].tolist() == [x, -1, -1, -1]
    # the draft's distribution is the target's: nothing is left at a refusal, so the target itself is drawn from
    out, n = run_verify(p, p.clone(), [0, 4, 1], [0, 3], [0, 0, 0], [.95], 3)
    assert n[0] == 0 and out[0].tolist() == [3, -1, -1]
    # a zero probability of the draft: kept where the target has some
    out, n = run_verify(p, torch.zeros(3, V), tok, [0, 3], [.9, .9, 0], [.2], 3)
    assert n[0] == 2 and out[0].tolist() == [3, 1, 5]
    # a sure drafter: refused, the draft cannot be drawn
    out, n = run_verify(p, None, [0, 3, 1], [0, 3], [.4, .9, 0], [.9999], 3)
    assert n[0] == 0 and out[0].tolist() == [2, -1, -1]


def test_verify_reports():
    p, q, tokens, cu, ua, us = draws(4, 6, 3, 3, 700)
    good = run_verify(p, q, tokens, cu, ua, us, 3)
    t = tokens.copy()
    t[cu[2] + 1] = 700                     # a draft that is no token
    t[cu[4] + 1] = -1
    out, n = run_verify(p, q, t, cu, ua, us, 3, bad=True)
    want = ref.verify(p.numpy(), q.numpy(), t, cu, ua, us, 3)
    assert np.array_equal(out, want[0]) and np.array_equal(n, want[1]) and n[2] == 0 and n[4] == 0
    for v in (math.nan, -0.25, 2.0):       # a row that is sampled from
        pp = p.clone()
        row = cu[3] + int(good[1][3])
        pp[row, 5] = v
        out, n = run_verify(pp, q, tokens, cu, ua, us, 3, bad=True)
        want = ref.verify(pp.numpy(), q.numpy(), tokens, cu, ua, us, 3)
        assert np.array_equal(out, want[0]) and np.array_equal(n, want[1])
    pp = p.clone()
    pp[cu[1] + int(good[1][1])] = 0.0      # nothing to draw from
    out, n = run_verify(pp, q, tokens, cu, ua, us, 3, bad=True)
    assert out[1, n[1]] == -1
    for bad_cu in ([-2, 3, 6, 9, 12, 15, 18], [0, 3, 6, 9, 12, 15, 1 << 20]):
        run_verify(p, q, tokens, bad_cu, ua, us, 3, bad=True)
    run_verify(p, q, tokens, cu, ua, us, 2, bad=True)    # more new tokens than out has room for
    assert np.array_equal(run_verify(p, q, tokens, cu, ua, us, 3)[0], good[0])


def test_verify_keeps_the_targets_distribution():
    """Of many requests with one draft each, the first token kept is distributed as the target (within five standard
    deviations of a multinomial count)."""
    n, V = 40000, 7
    g = torch.Generator().manual_seed(2)
    p, q = torch.softmax(torch.randn(V, generator=g), -1), torch.softmax(torch.randn(V, generator=g), -1)
    tokens = torch.zeros(2 * n, dtype=torch.int32)
    tokens[1::2] = torch.multinomial(q, n, True, generator=g).int()
    ua, us = torch.rand(2 * n, generator=g).numpy(), torch.rand(n, generator=g).numpy()
    out, _ = run_verify(p.repeat(2 * n, 1), q.repeat(2 * n, 1), tokens.numpy(), list(range(0, 2 * n + 1, 2)), ua, us, 2)
    count = np.bincount(out[:, 0], minlength=V)
    pe = p.double().numpy()
    assert np.all(np.abs(count - n * pe) <= 5 * np.sqrt(n * pe * (1 - pe)))


def test_verify_beside_other_work():
    """Blocks of a cluster that begin when another stream's kernels leave them room exchange their totals all the same."""
    n, V, mx = 70, 20011, 4
    p, q, tokens, cu, ua, us = draws(11, n, 0, 4, V)
    want = ref.verify(p.numpy(), q.numpy(), tokens, cu, ua, us, mx)
    dev = lambda a, t: torch.as_tensor(a).to(t).cuda()  # noqa: E731
    args = (p.cuda(), q.cuda(), dev(tokens, torch.int32), dev(cu, torch.int32), dev(ua, torch.float32), dev(us, torch.float32))
    turns = 24
    out = torch.full((turns, n, mx), 99, dtype=torch.int32, device="cuda")
    kept = torch.full((turns, n), 99, dtype=torch.int32, device="cuda")
    m = torch.randn(2048, 2048, device="cuda").bfloat16()
    busy, own = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(turns):
        with torch.cuda.stream(busy):
            for _ in range(3):
                m @ m
        with torch.cuda.stream(own):
            ds.verify_drafts(*args, out[i], kept[i])
    torch.cuda.synchronize()
    ds.sync_status()
    for i in range(turns):
        assert np.array_equal(out[i].cpu().numpy(), want[0]) and np.array_equal(kept[i].cpu().numpy(), want[1])


def drawn(w, u):
    """The least entry whose cumulative weight exceeds u times the total: whole numbers throughout."""
    total, m = sum(w), int(float(np.float32(u)) * 2 ** 48)  # (u here is a multiple of 2^-48)
    run = 0
    for x, v in enumerate(w):
        run += v
        if run << 48 > m * total:
            return x
    return -1


@pytest.mark.parametrize("V", [262145, 524287, 524288, 600000, 1048577, 1200000, 1 << 22])
@pytest.mark.parametrize("drafted", [True, False])
def test_verify_large_rows_that_are_not_normalised(V, drafted):
    """Entries of 1 throughout add up to the vocabulary's size; u times that is exact here, and so is the entry drawn."""
    us = [0.0, 0.25, 0.3, 0.625, float(np.nextafter(np.float32(1), np.float32(0)))]
    p = torch.ones(1, V).cuda()
    for u in us:
        want = int(float(np.float32(u)) * V)
        out, n = run_verify(p, None, [0], [0, 1], [0.0], [u], 1)
        assert n[0] == 0 and out[0].tolist() == [want]
    # a refused draft, entry 3, of which the target has nothing: the others weigh the same
    p = p.repeat(2, 1)
    p[:, 3] = 0
    q = torch.full((2, V), 0.25).cuda() if drafted else None
    for u in us:
        out, n = run_verify(p, q, [0, 3], [0, 2], [0.0, 0.0], [u], 2)
        at = int(float(np.float32(u)) * (V - 1))
        assert n[0] == 0 and out[0].tolist() == [at + (at >= 3), -1]


def test_verify_small_entries():
    """Entries that are whole multiples of 2^-44 count as they are, whatever their sum; less than half of it is none."""
    rng = np.random.default_rng(3)
    w = rng.integers(0, 9, 3000)
    for u in (0.0, 0.125, 0.7, float(np.nextafter(np.float32(1), np.float32(0)))):
        p = torch.tensor(w * 2.0 ** -44, dtype=torch.float32)[None]
        out, n = run_verify(p, None, [0], [0, 1], [0.0], [u], 1)
        assert n[0] == 0 and out[0, 0] == drawn(w.tolist(), u)
    p = torch.full((1, 500), 2.0 ** -46)
    p[0, 77] = 0.75 * 2.0 ** -44
    assert run_verify(p, None, [0], [0, 1], [0.0], [0.9], 1)[0][0, 0] == 77
    p[0, 77] = 0
    out, n = run_verify(p, None, [0], [0, 1], [0.0], [0.9], 1, bad=True)
    assert n[0] == 0 and out[0, 0] == -1
    # nothing that counts is left above the draft: the target itself is drawn from
    p = torch.tensor([[2.0 ** -30, 0.5, 0.0, 0.5]] * 2)
    q = p.clone()
    q[:, 0] -= 2.0 ** -50
    out, n = run_verify(p, q, [0, 2], [0, 2], [0.0, 0.0], [0.75], 2)
    assert n[0] == 0 and out[0].tolist() == [3, -1]


@pytest.mark.parametrize("seed", range(4))
def test_verify_draws_by_exact_products(seed):
    """u times the total lies just below a whole number, which a cumulative sum reaches: that entry is drawn, not the next."""
    rng, found = random.Random(seed), 0
    while found < 5:
        total, m = rng.randrange(1 << 43, 1 << 44) | 1, rng.randrange(1 << 23, 1 << 24) | 1
        below = -(m * total) % (1 << 24)  # u = m 2^-24: what is missing to the whole number above, in 2^-24
        if not 0 < below < 1 << 12:
            continue
        found += 1
        reach = (m * total >> 24) + 1
        parts = lambda n: [n >> 20 << 20, n & (1 << 20) - 1]  # noqa: E731  (24 bits each)
        w = parts(reach) + parts(total - reach)
        assert sum(w) == total and all(v > 0 for v in w)
        p = torch.tensor([v * 2.0 ** -44 for v in w])[None]
        assert [int(v * 2.0 ** 44) for v in p[0].tolist()] == w
        out, n = run_verify(p, None, [0], [0, 1], [0.0], [m * 2.0 ** -24], 1)
        assert n[0] == 0 and out[0, 0] == drawn(w, m * 2.0 ** -24) == 1


@pytest.mark.parametrize("new", [1, 8, 30, 70])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attention_flat_tail_below_a_sharp_key(new, D, dtype):
    """Two keys that take nearly all of the probability and have no values; what the others, 2^-25.5 of them each, add up
    to is the output.  In fp16 a probability is off by 2^-11 of itself, or of 2^-21 of the row's largest where it is
    below that (fp16's steps end at 2^-24, and the largest is taken as 2^7 or more): half of 2^-31."""
    c = ref.Case([1500 - new] * 76, [new] * 76, 8, 2, D, 16, dtype=dtype, seed=new)
    c.q_cpu = torch.zeros_like(c.q_cpu)
    c.q_cpu[..., 0] = 16.0
    for k, v in zip(c.keys, c.values):
        k *= 0.01
        k[[5, 133]] = 0
        k[[5, 133], :, 0] = 25.5 * math.log(2) * math.sqrt(D) / 16
        v += 1
        v[[5, 133]] = 0
    c.put()
    out, lse = attend(c)
    ds.sync_status()
    assert c.path != ds.ATTN_GENERIC
    want, wlse, mag = c.reference()
    tol, ltol = c.tolerances(want, mag, True)
    if dtype == "f16":
        sums = torch.stack([v.double().abs().sum(0) for v in c.values])  # [requests][key heads][D]
        tol = tol + 2.0 ** -32 * sums.repeat_interleave(4, 1).repeat_interleave(new, 0)
    assert bool(((out.cpu().double() - want).abs() <= tol).all())
    assert bool(((lse.cpu().double() - wlse).abs() <= ltol + 2.0 ** -24 * wlse.abs()).all())


def test_attention_path_of_a_single_token():
    """A lone token's stride is not used, so it does not keep the call from the tensor cores; q given the same way to both."""
    c = ref.Case([20], [1], 8, 2, 64, 16).put()
    room = torch.empty(2, 8 * 64 + 3, dtype=c.dt, device="cuda")
    q, q2 = (room.as_strided((n, 8, 64), (8 * 64 + 3, 64, 1)) for n in (1, 2))
    assert q.stride(0) % 8
    sh, cache = shape_of(c), ds.KVCache(c.k, c.v)
    assert ds.attention_path(sh, cache, q, 1) == ds.ATTN_DECODE
    assert ds.attention_path(sh, cache, q2, 1) == ds.ATTN_GENERIC
    q.copy_(c.q)
    out, _ = attend(c)
    c.q = q
    assert torch.equal(attend(c)[0], out)


def test_example_takes_the_decode_kernel_behind_the_prompts(monkeypatch):
    import importlib.util
    import os
    at = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serving_step.py")
    spec = importlib.util.spec_from_file_location("serving_step", at)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    paths, attention = [], ds.paged_attention

    def watched(shape, cache, table, q, cu, seq, max_new, *args, **kw):
        paths.append(ds.attention_path(shape, cache, q, max_new))
        return attention(shape, cache, table, q, cu, seq, max_new, *args, **kw)

    monkeypatch.setattr(ds, "paged_attention", watched)
    example.run(steps=3)
    assert paths == [ds.ATTN_CHUNK, ds.ATTN_DECODE, ds.ATTN_DECODE]


@pytest.mark.parametrize("max_new,path", [(8, ds.ATTN_DECODE), (40, ds.ATTN_CHUNK)])
def test_a_captured_step_serves_other_lengths(max_new, path):
    """page_map, kv_append, paged_attention and verify_drafts in one graph, with the lengths and the list of free pages
    moved on by it on the device: replayed with other lengths, each step is the eager one's."""
    R_, H, G, D, page, cap, V, width = 3, 8, 2, 64, 16, 3 * max_new, 501, 12
    rng, g = random.Random(max_new), torch.Generator().manual_seed(max_new)
    i32 = dict(dtype=torch.int32, device="cuda")
    n_pages = R_ * width + 5
    ids = list(range(n_pages))
    rng.shuffle(ids)
    free, table = torch.tensor(ids, **i32), torch.full((R_, width), -1, **i32)
    context, new = torch.zeros(R_, **i32), torch.zeros(R_, **i32)
    slots, positions = torch.empty(cap, dtype=torch.int64, device="cuda"), torch.empty(cap, **i32)
    cu, seq, taken = torch.empty(R_ + 1, **i32), torch.empty(R_, **i32), torch.empty(1, **i32)
    sh = ds.AttentionShape(H, G, D, page)
    cache = ds.KVCache(*(torch.full((n_pages, page, G, D), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    q = torch.zeros(cap, H, D, dtype=torch.bfloat16, device="cuda")
    kn, vn = (torch.zeros(cap, G, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    out, ws = torch.zeros_like(q), torch.empty(ds.attention_workspace_bytes(sh, R_, cap, max_new), dtype=torch.uint8, device="cuda")
    p, d, ua, us = (torch.zeros(*s, device="cuda") for s in ((cap, V), (cap, V), (cap,), (R_,)))
    tokens, drawn_, kept = torch.zeros(cap, **i32), torch.empty(R_, max_new, **i32), torch.empty(R_, **i32)
    turn = torch.arange(n_pages, device="cuda")
    assert ds.attention_path(sh, cache, q, max_new) == path

    def step():
        ds.page_map(context, new, free, table, page, slots, positions, cu, seq, taken)
        ds.kv_append(sh, cache, kn, vn, slots)
        ds.paged_attention(sh, cache, table, q, cu, seq, max_new, out, ws)
        ds.verify_drafts(p, d, tokens, cu, ua, us, drawn_, kept)
        context.copy_(seq)
        free.copy_(free[(turn + taken) % n_pages])  # the pages taken go behind the others

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()  # (no new tokens: a step that changes nothing)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    ctx, host_table, host_free = [0] * R_, torch.full((R_, width), -1, dtype=torch.int32), list(ids)
    keys, values = [torch.zeros(0, G, D) for _ in range(R_)], [torch.zeros(0, G, D) for _ in range(R_)]
    most = [max_new, 1, max_new // 2]
    for lens in ([max_new, 1, 5], [1, 1, 1], [0, 7, 2], [0, 0, 0], most, [3, 0, max_new]):
        T = sum(lens)
        a = [torch.randn(cap, n, D, generator=g).bfloat16() for n in (H, G, G)]
        pp, qq, tok, _, aa, uu = draws(T + 1, 1, cap, cap, V)
        uu = torch.rand(R_, generator=g).numpy()
        for t, v in ((q, a[0]), (kn, a[1]), (vn, a[2]), (p, pp), (d, qq), (tokens, torch.as_tensor(tok)), (ua, torch.as_tensor(aa)),
                     (us, torch.as_tensor(uu)), (new, torch.tensor(lens))):
            t.copy_(v)
        out.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        ds.sync_status()
        w_slots, w_pos, w_cu, w_seq, w_taken, bad = ref.page_map(ctx, lens, page, host_free, host_table, cap)
        assert not bad and torch.equal(table.cpu(), host_table)
        assert (slots.tolist(), positions.tolist(), cu.tolist(), seq.tolist(), int(taken)) == (w_slots, w_pos, w_cu, w_seq, w_taken)
        host_free = host_free[w_taken:] + host_free[:w_taken]
        for r in range(R_):
            at = slice(w_cu[r], w_cu[r + 1])
            keys[r], values[r] = torch.cat([keys[r], a[1][at].float()]), torch.cat([values[r], a[2][at].float()])
        c = ref.Case(ctx, lens, H, G, D, page, seq=w_seq)
        c.keys, c.values, c.q_cpu, c.path = keys, values, a[0][:T], path
        if T:
            check(c, out[:T], None)
        assert bool((out[T:] == 7.0).all())
        want = ref.verify(pp.numpy(), qq.numpy(), tok, w_cu, aa, uu, max_new)
        assert np.array_equal(drawn_.cpu().numpy(), want[0]) and np.array_equal(kept.cpu().numpy(), want[1])
        ctx = w_seq


@pytest.mark.parametrize("new", [3, 8, 20, 150])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_attention_infinities_that_leave_the_window(new, D, dtype):
    """Values that are not finite, before the first new token and among them: rows whose window has passed them, or that
    come before them, keep their sums."""
    ctx, window = 400, 90
    c = ref.Case([ctx, 40], [new, 3], 8, 2, D, 16, dtype=dtype, window=window, qscale=0.5)
    first = ctx + 1 - window
    for i, (at, what) in enumerate(((first - 1, math.nan), (first, math.inf), (first + 1, -math.inf), (first + new // 2, math.nan),
                                    (ctx, math.inf), (ctx + new // 2, -math.inf), (ctx + new - 1, math.nan))):
        c.values[0][at, :, 5 * i: 5 * i + 7] = what
    c.put()
    out, lse = attend(c)
    ds.sync_status()
    want, wlse, mag = c.reference()
    tol, ltol = c.tolerances(want, mag, True)
    got, fin = out.cpu().double(), torch.isfinite(want)
    assert not bool(fin.all()) and torch.equal(torch.isfinite(got), fin)
    assert torch.equal(got[~fin].nan_to_num(7.0), want[~fin].nan_to_num(7.0))
    assert bool(((got - want).abs() <= tol)[fin].all())
    assert bool(((lse.cpu().double() - wlse).abs() <= ltol + 2.0 ** -24 * wlse.abs()).all())


@pytest.mark.parametrize("new_hi,D", [(1, 128), (4, 64), (12, 64), (12, 128)])
def test_attention_more_requests_than_threads(new_hi, D):
    """Every thread of a block then takes several requests, some without new tokens, and most items are of one tile."""
    rng = random.Random(new_hi)
    n = 1100
    c = ref.Case(ref.lengths(rng, n, 0, 150), ref.lengths(rng, n, 0, new_hi), 8, 2, D, 8).put()
    out, lse = attend(c)
    ds.sync_status()
    check(c, out, lse)
