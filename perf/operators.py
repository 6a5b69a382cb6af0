"""One serving step around a routed layer, operator by operator.

A server that runs the layer keeps the keys and values of earlier tokens in
pages.  Each step it maps the step's new tokens to pages (``page_map``),
writes their keys and values there (``kv_append``), attends from the new
tokens over the pages (``attention``) and, when the new tokens were drafted,
checks them against the model's probabilities (``verify``).

Each case is timed through ``run``: in the operators' plain form (elementary
torch operations) or, with ``own`` set, through the package's entry points.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one user's chat: one new token on a short history; latency counts
        _attention("attention_one_short", 1, 137, 137, 1, 1, 32, 8, 128, 16, 0, "bf16"),
        # an ordinary decode batch of unlike histories, one token each
        _attention("attention_decode_batch", 64, 200, 8200, 1, 1, 32, 8, 128, 64, 0, "bf16"),
        # few users with long documents: the work has to be split along the history
        _attention("attention_decode_long", 3, 60000, 131000, 1, 1, 64, 8, 128, 16, 0, "f16"),
        # drafted tokens checked at once: one to six tokens a request, seven heads share a key
        _attention("attention_drafted", 29, 17, 5000, 1, 6, 28, 4, 64, 24, 0, "bf16"),
        # a long prompt's next chunk
        _attention("attention_chunk_long", 1, 30011, 30011, 2048, 2048, 32, 8, 128, 32, 0, "bf16"),
        # chunks and single tokens in one batch, own keys for each head, a sliding window
        _attention("attention_mixed_window", 17, 0, 4000, 1, 700, 16, 16, 64, 48, 1024, "f16"),
        # a handful of requests, one step of drafted tokens
        _page_map("page_map_few", 7, 0, 3000, 1, 5, 16),
        # many requests, prompts among them
        _page_map("page_map_many", 2048, 0, 8000, 1, 150, 64),
        # one decode step's keys and values
        _append("kv_append_step", 24, 1, 5, 8, 128, 16, "bf16"),
        # prompts' keys and values
        _append("kv_append_prompts", 13, 100, 2500, 8, 128, 64, "bf16"),
        # one user, three drafts, a small vocabulary; latency counts
        _verify("verify_one", 1, 4, 4, 32768, True, "f32"),
        # a batch with an odd vocabulary
        _verify("verify_batch", 96, 1, 6, 100003, True, "f32"),
    ]


def _attention(name, requests, ctx_lo, ctx_hi, new_lo, new_hi, heads, kv_heads, dim, page, window, dtype, lens=1):
    return {"name": name, "op": "attention", "requests": requests, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "new_lo": new_lo,
            "new_hi": new_hi, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "window": window,
            "dtype": dtype, "lens": lens}


def _page_map(name, requests, ctx_lo, ctx_hi, new_lo, new_hi, page, lens=1):
    return {"name": name, "op": "page_map", "requests": requests, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "new_lo": new_lo,
            "new_hi": new_hi, "page": page, "lens": lens}


def _append(name, requests, new_lo, new_hi, kv_heads, dim, page, dtype, lens=1):
    return {"name": name, "op": "kv_append", "requests": requests, "ctx_lo": 0, "ctx_hi": 2000, "new_lo": new_lo,
            "new_hi": new_hi, "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype, "lens": lens}


def _verify(name, requests, new_lo, new_hi, vocab, drafted, dtype, lens=1):
    return {"name": name, "op": "verify", "requests": requests, "ctx_lo": 0, "ctx_hi": 0, "new_lo": new_lo,
            "new_hi": new_hi, "vocab": vocab, "drafted": drafted, "dtype": dtype, "lens": lens}


def _log(rng, lo, hi):
    """A whole number from lo to hi, spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    lens = rng.randrange(2, 1 << 20)
    op = rng.choice(["attention", "attention", "attention", "page_map", "kv_append", "verify"])
    if op == "page_map":
        hi = _log(rng, 1, 150)
        c = _page_map("", _log(rng, 1, 2048), 0, _log(rng, 1, 8000), rng.randint(0, min(1, hi)), hi,
                      rng.choice([1, 8, 16, 24, 32, 64, 100, 128]), lens)
    elif op == "kv_append":
        hi = _log(rng, 1, 1500)
        c = _append("", _log(rng, 1, max(1, min(64, 16000 // hi))), 1, hi, rng.choice([1, 2, 4, 8]),
                    rng.choice([64, 80, 96, 128]), rng.choice([8, 16, 24, 32, 64, 128]), rng.choice(["bf16", "f16"]), lens)
    elif op == "verify":
        hi = rng.randint(1, 6)
        c = _verify("", _log(rng, 1, 96), 1, hi, _log(rng, 1000, 100003), rng.random() < 0.75, rng.choice(["f32", "f32", "bf16"]), lens)
    else:
        while True:
            heads, kv = rng.choice([(32, 8), (64, 8), (28, 4), (16, 16), (40, 8), (24, 2), (8, 1), (12, 12)])
            hi = rng.randint(1, 8) if rng.random() < 0.5 else _log(rng, 9, 2500)
            ctx = _log(rng, 1, 131000)
            c = _attention("", _log(rng, 1, 64), rng.randint(0, ctx), ctx, rng.randint(1, hi), hi, heads, kv,
                           rng.choice([64, 80, 96, 128, 128]), rng.choice([8, 16, 24, 32, 48, 64, 128, 256]),
                           rng.choice([0, 0, 0, _log(rng, 1, 4096)]), rng.choice(["bf16", "bf16", "f16"]), lens)
            # no dearer than the listed ones: padded scores, and cached keys
            if c["requests"] * (ctx + hi) * hi * heads <= 1 << 31 and c["requests"] * (ctx + hi) * kv * c["dim"] <= 1 << 29:
                break
    del c["name"]
    return c


def _lengths(case):
    """(cached tokens, new tokens) of each request: the case alone decides them."""
    rng = random.Random(case["lens"])
    return ([rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["requests"])],
            [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["requests"])])


def _pages(lengths, page, width, g, spare):
    """A block table whose requests hold the pages of their lengths, in no order; and the pages left over."""
    held = torch.tensor([-(-n // page) for n in lengths], device="cuda")
    total = int(held.sum())
    order = torch.randperm(total + spare, generator=g, device="cuda").to(torch.int32)
    j = torch.arange(width, device="cuda")[None]
    at = (held.cumsum(0) - held)[:, None] + j
    table = torch.where(j < held[:, None], order[at.clamp(max=total + spare - 1)], -1).to(torch.int32).contiguous()
    return table, order[total:].contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ctx, new = _lengths(case)
    R, T = case["requests"], sum(new)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    cu = ints([sum(new[:r]) for r in range(R + 1)])
    st = {"case": case, "T": T, "max_new": max(1, max(new)), "cu_new": cu}
    if case["op"] == "verify":
        V, dt = case["vocab"], DTYPES[case["dtype"]]
        logits = 4 * torch.randn(T, V, generator=g, device="cuda")
        st["target"] = torch.softmax(logits, -1).to(dt)
        logits += torch.randn(T, V, generator=g, device="cuda")
        draft = torch.softmax(logits, -1)
        tokens = torch.multinomial(draft, 1, generator=g)[:, 0].to(torch.int32)
        st["draft"] = draft.to(dt) if case["drafted"] else None
        st["tokens"] = torch.roll(tokens, 1).contiguous()  # row i's draft is the token that row i + 1 was fed
        st["u_accept"] = torch.rand(T, generator=g, device="cuda")
        st["u_sample"] = torch.rand(R, generator=g, device="cuda")
        st["out_tokens"] = torch.empty(R, st["max_new"], dtype=torch.int32, device="cuda")
        st["n_accepted"] = torch.empty(R, dtype=torch.int32, device="cuda")
        return st
    page = case["page"]
    total = [a + b for a, b in zip(ctx, new)]
    width = max(1, max(-(-n // page) for n in total))
    if case["op"] == "page_map":
        st["table"], st["free"] = _pages(ctx, page, width, g, sum(-(-a // page) - -(-b // page) for a, b in zip(total, ctx)) + 5)
        st["context"], st["new"] = ints(ctx), ints(new)
        cap = T + 7  # a captured step has room to spare
        st["slots"] = torch.empty(cap, dtype=torch.int64, device="cuda")
        st["positions"] = torch.empty(cap, dtype=torch.int32, device="cuda")
        st["seq"] = torch.empty(R, dtype=torch.int32, device="cuda")
        st["cu_out"] = torch.empty(R + 1, dtype=torch.int32, device="cuda")
        st["taken"] = torch.empty(1, dtype=torch.int32, device="cuda")
        return st
    dt, kv, D = DTYPES[case["dtype"]], case["kv_heads"], case["dim"]
    st["table"], _ = _pages(total, page, width, g, 3)
    n_pages = sum(-(-n // page) for n in total) + 3
    for name in ("k", "v"):
        st[name] = torch.randn(n_pages, page, kv, D, generator=g, device="cuda", dtype=dt)
    if case["op"] == "kv_append":
        st["k_new"] = torch.randn(T, kv, D, generator=g, device="cuda", dtype=dt)
        st["v_new"] = torch.randn(T, kv, D, generator=g, device="cuda", dtype=dt)
        r = torch.repeat_interleave(torch.arange(R, device="cuda"), torch.tensor(new, device="cuda"))
        pos = ints(ctx)[r] + torch.arange(T, device="cuda") - cu[r]
        slots = st["table"][r, pos // page].long() * page + pos % page
        st["slots"] = torch.cat([slots, slots.new_full((3,), -1)])  # a captured step's spare places
        for name in ("k_new", "v_new"):
            st[name] = torch.cat([st[name], st[name].new_zeros(3, kv, D)])
        return st
    st["q"] = (1.5 * torch.randn(T, case["heads"], D, generator=g, device="cuda")).to(dt)
    st["seq"] = ints(total)
    st["max_seq"] = max(total)
    st["out"] = torch.empty(T, case["heads"], D, dtype=dt, device="cuda")
    st["lse"] = torch.empty(T, case["heads"], dtype=torch.float32, device="cuda")
    return st


def run(st):
    op = st["case"]["op"]
    if own:
        return {"attention": _own_attention, "page_map": _own_page_map, "kv_append": _own_append, "verify": _own_verify}[op](st)
    return {"attention": _plain_attention, "page_map": _plain_page_map, "kv_append": _plain_append, "verify": _plain_verify}[op](st)


# ------------------------------------------------------- the package's calls


def _shape(st):
    import bit_quantized_routed_router_gb300 as ds
    c = st["case"]
    if "shape" not in st:
        st["shape"] = ds.AttentionShape(c.get("heads", c["kv_heads"]), c["kv_heads"], c["dim"], c["page"],
                                        ds.DS_F16 if c["dtype"] == "f16" else ds.DS_BF16, window=c.get("window", 0))
        st["cache"] = ds.KVCache(st["k"], st["v"])
    return ds, st["shape"], st["cache"]


def _own_attention(st):
    ds, shape, cache = _shape(st)
    if "workspace" not in st:
        n = ds.attention_workspace_bytes(shape, st["case"]["requests"], st["T"], st["max_new"])
        st["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    ds.paged_attention(shape, cache, st["table"], st["q"], st["cu_new"], st["seq"], st["max_new"], st["out"], st["workspace"],
                       lse=st["lse"])
    return {"out": st["out"], "lse": st["lse"]}


def _own_page_map(st):
    import bit_quantized_routed_router_gb300 as ds
    ds.page_map(st["context"], st["new"], st["free"], st["table"], st["case"]["page"], st["slots"], st["positions"], st["cu_out"],
                st["seq"], st["taken"])
    return [st[n] for n in ("table", "slots", "positions", "cu_out", "seq", "taken")]


def _own_append(st):
    ds, shape, cache = _shape(st)
    ds.kv_append(shape, cache, st["k_new"], st["v_new"], st["slots"])
    return {"k": st["k"], "v": st["v"]}


def _own_verify(st):
    import bit_quantized_routed_router_gb300 as ds
    ds.verify_drafts(st["target"], st["draft"], st["tokens"], st["cu_new"], st["u_accept"], st["u_sample"], st["out_tokens"],
                     st["n_accepted"])
    return {"tokens": st["out_tokens"], "accepted": st["n_accepted"]}


# ----------------------------------------------------------- the plain forms


def _plain_attention(st):
    """softmax(scale q k^T) v over the keys that each new token sees: those up to itself, and within the window."""
    c = st["case"]
    R, H, G, D, page = c["requests"], c["heads"], c["kv_heads"], c["dim"], c["page"]
    N, L, g = st["max_new"], st["max_seq"], H // G
    cu, seq = st["cu_new"].long(), st["seq"].long()
    i, j = torch.arange(N, device="cuda"), torch.arange(L, device="cuda")
    new = cu[1:] - cu[:-1]
    row = (cu[:-1, None] + i).clamp(max=st["T"] - 1)                              # [R][N] rows of q
    pos = seq[:, None] - new[:, None] + i
    slot = st["table"][:, j // page].clamp(min=0).long() * page + j % page           # [R][L]
    k = st["k"].view(-1, G, D)[slot].float().permute(0, 2, 3, 1)                     # [R][G][D][L]
    v = st["v"].view(-1, G, D)[slot].float().permute(0, 2, 1, 3)                     # [R][G][L][D]
    q = st["q"].float()[row].view(R, N, G, g, D).permute(0, 2, 1, 3, 4).reshape(R, G, N * g, D)
    s = torch.matmul(q * D ** -0.5, k).view(R, G, N, g, L)
    sees = j <= pos[..., None]
    if c["window"]:
        sees = sees & (j > pos[..., None] - c["window"])
    s = torch.where(sees[:, None, :, None], s, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(R, G, N * g, L), v).view(R, G, N, g, D) / torch.where(total == 0, 1.0, total)
    lse = (m + torch.log(total))[..., 0]
    # back to rows: row t of q is token t - cu[r] of request r
    t = torch.arange(st["T"], device="cuda")
    r = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    at = t - cu[r]
    out = o.permute(0, 2, 1, 3, 4).reshape(R, N, H, D)[r, at].to(st["q"].dtype)
    return {"out": out, "lse": lse.permute(0, 2, 1, 3).reshape(R, N, H)[r, at]}


def _plain_page_map(st):
    """Pages for the new tokens, in request order from the list of free ones, and each new token's place."""
    page, table, free = st["case"]["page"], st["table"], st["free"]
    ctx, new = st["context"].long(), st["new"].long()
    seq = ctx + new
    held, need = (ctx + page - 1) // page, (seq + page - 1) // page
    take = need - held
    first = take.cumsum(0) - take
    j = torch.arange(table.shape[1], device="cuda")
    fresh = (j >= held[:, None]) & (j < need[:, None])
    table = torch.where(fresh, free[(first[:, None] + j - held[:, None]).clamp(0, free.shape[0] - 1)], table)
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
    t = torch.arange(st["slots"].shape[0], device="cuda")
    r = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=ctx.shape[0] - 1)
    valid = t < cu[-1]
    pos = torch.where(valid, ctx[r] + t - cu[r], 0)
    slots = torch.where(valid, table[r, pos // page].long() * page + pos % page, -1)
    return [table, slots, torch.where(valid, pos, -1).int(), cu.int(), seq.int(), take.sum().view(1).int()]


def _plain_append(st):
    """Rows of the new keys and values to their places; a place below zero is none."""
    slots = st["slots"]
    valid = slots >= 0
    at = torch.where(valid, slots, slots[0])
    for_kv = valid[:, None, None]
    k, v = (st[n].view(-1, *st[n].shape[2:]) for n in ("k", "v"))
    k[at] = torch.where(for_kv, st["k_new"], st["k_new"][:1])
    v[at] = torch.where(for_kv, st["v_new"], st["v_new"][:1])
    return {"k": st["k"], "v": st["v"]}


def _plain_verify(st):
    """Drafts are taken while u q(x) < p(x); then one token of max(p - q, 0), or of p when all were taken."""
    cu, target, draft = st["cu_new"].long(), st["target"], st["draft"]
    T, V = target.shape
    K = st["max_new"] - 1
    new = cu[1:] - cu[:-1]
    i = torch.arange(K, device="cuda")
    row = (cu[:-1, None] + i).clamp(max=T - 1)                                      # the row that each draft is checked against
    x = st["tokens"].long()[(row + 1).clamp(max=T - 1)]
    p = target[row, x].double()
    q = draft[row, x].double() if draft is not None else torch.ones_like(p)
    taken = (st["u_accept"].double()[row] * q < p) & (i < new[:, None] - 1)
    n = taken.long().cumprod(1).sum(1)
    row = cu[:-1] + n
    refused = (n < new - 1)[:, None]
    p = target[row].double()
    y = st["tokens"].long()[(row + 1).clamp(max=T - 1)]
    q = draft[row].double() if draft is not None else (torch.arange(V, device="cuda") == y[:, None]).double()
    rest = torch.where(refused, (p - q).clamp(min=0), p)
    rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, p)
    c = rest.cumsum(-1)
    z = (c <= st["u_sample"].double()[:, None] * c[:, -1:]).sum(-1)
    i = torch.arange(K + 1, device="cuda")
    fed = st["tokens"].long()[(cu[:-1, None] + 1 + i).clamp(max=T - 1)]
    out = torch.where(i < n[:, None], fed, torch.where(i == n[:, None], z[:, None], -1))
    return {"tokens": out.int(), "accepted": n.int()}


# --------------------------------------------------------------- what is due


def work(case):
    ctx, new = _lengths(case)
    R, T = case["requests"], sum(new)
    if case["op"] == "page_map":
        page = case["page"]
        took = sum(-(-(a + b) // page) - -(-a // page) for a, b in zip(ctx, new))
        touched = sum(-(-(a + b) // page) - a // page for a, b in zip(ctx, new) if b)
        return {"bytes": 8 * R + 8 * took + 4 * touched + 12 * T + 8 * R, "flops": 0}
    if case["op"] == "kv_append":
        return {"bytes": 8 * T + 8 * T * case["kv_heads"] * case["dim"], "flops": 0}
    if case["op"] == "verify":
        e = 2 if case["dtype"] == "bf16" else 4
        rows = sum(1 + (case["drafted"] and n > 1) for n in new)
        return {"bytes": e * case["vocab"] * rows + 20 * T + 8 * R, "flops": 2 * case["vocab"] * R}
    H, G, D, w = case["heads"], case["kv_heads"], case["dim"], case["window"]
    keys = sum(a + b - (max(0, a + 1 - w) if w else 0) for a, b in zip(ctx, new))
    pairs = sum(sum(min(a + i + 1, w or a + i + 1) for i in range(b)) for a, b in zip(ctx, new))
    return {"bytes": 4 * keys * G * D + 4 * T * H * D + 4 * T * H + 4 * (keys // case["page"] + 3 * R), "flops": 4 * pairs * H * D}


def exact(case, seed):
    """Attention in 64 bits, one request and one shared head at a time.  The other operators give whole numbers or copies."""
    if case["op"] != "attention" or work(case)["flops"] > 4e12:
        return None
    st = prepare(case, seed)
    ctx, new = _lengths(case)
    page, g, w = case["page"], case["heads"] // case["kv_heads"], case["window"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    t0 = 0
    for r in range(case["requests"]):
        n, pages = new[r], st["table"][r, : -(-(ctx[r] + new[r]) // page)].long()
        far = torch.arange(ctx[r], ctx[r] + n, device="cuda")[:, None] - torch.arange(ctx[r] + n, device="cuda")[None]
        hidden = (far < 0) | (far >= w) if w else far < 0
        for h in range(case["kv_heads"]):
            k = st["k"][pages, :, h].reshape(-1, case["dim"])[: ctx[r] + n].double()
            v = st["v"][pages, :, h].reshape(-1, case["dim"])[: ctx[r] + n].double()
            for a in range(h * g, h * g + g):
                s = (st["q"][t0:t0 + n, a].double() @ k.T / math.sqrt(case["dim"])).masked_fill_(hidden, -math.inf)
                z = torch.logsumexp(s, -1)
                lse[t0:t0 + n, a] = z
                out[t0:t0 + n, a] = torch.exp(s - z[:, None]) @ v
        t0 += n
    return {"out": out, "lse": lse}
