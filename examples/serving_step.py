"""A few speculative decoding steps of a one-layer model, with every operator of a serving step around the routed layer:

    page_map         pages and places for the step's new tokens
    kv_append        their keys and values into the pages
    paged_attention  attention from the new tokens over the pages
    layer            the routed layer on the attention's output
    verify_drafts    which drafted tokens stand, and one token more

The weights are random and the drafter is the model itself on stale states, so the text means nothing; each step's attention
is checked against a plain one in 64 bits, and the keys a request ends with against the tokens it kept.

    python examples/serving_step.py
"""
import math
import os
import sys
from dataclasses import replace

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
for _p in (ROOT, os.path.join(ROOT, "gen")):
    if _p not in sys.path:
        sys.path.insert(0, _p)

import torch  # noqa: E402

import bit_quantized_routed_router_gb300 as ds  # noqa: E402


class Model:
    """Embeddings, projections and one routed layer of width 1024 (16 experts, 4 a token); bf16."""

    def __init__(self, vocab=5003, heads=8, kv_heads=2, dim=64, page=16, seed=0):
        import dsgen
        from bit_quantized_routed_router_gb300 import synthetic
        cfg = replace(dsgen.TINY, name="serving step", T=8, D=1024, F=1024, E=16, k=4, Fs=1024, shared_sigma=0.02, x_dtype="bf16",
                      router_dtype="bf16", router_sigma=0.02, seed=5)
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, sigma):
            return (sigma * torch.randn(*shape, generator=g, device="cuda")).bfloat16()

        self.vocab, self.heads, self.kv, self.dim, self.D = vocab, heads, kv_heads, dim, cfg.D
        self.embed = normal(vocab, cfg.D, sigma=1.0)
        self.place = normal(4096, cfg.D, sigma=0.3)
        self.qkv = normal(cfg.D, (heads + 2 * kv_heads) * dim, sigma=cfg.D ** -0.5)
        self.back = normal(heads * dim, cfg.D, sigma=(heads * dim) ** -0.5)
        self.head = normal(cfg.D, vocab, sigma=0.7 * cfg.D ** -0.5)
        self.moe, self.weights = synthetic.shape_of(cfg), synthetic.build_layer(cfg)
        self.shape = ds.AttentionShape(heads, kv_heads, dim, page)


def plain_attention(keys, values, q):
    """The last len(q) tokens of a sequence over its keys and values, in 64 bits."""
    n, L, g = q.shape[0], keys.shape[0], q.shape[1] // keys.shape[1]
    k, v = (t.double().repeat_interleave(g, 1) for t in (keys, values))
    s = torch.einsum("ihd,jhd->hij", q.double(), k) / math.sqrt(q.shape[2])
    far = torch.arange(L - n, L, device=q.device)[:, None] - torch.arange(L, device=q.device)
    return torch.einsum("hij,jhd->ihd", torch.softmax(s.masked_fill(far < 0, -math.inf), -1), v)


def run(steps=4, requests=3, drafts=3, prompt=40, check=True):
    m, dev, page = Model(), "cuda", 16
    i32 = dict(dtype=torch.int32, device=dev)
    max_new, width, n_pages = max(prompt, drafts + 1), 16, requests * 16
    room = requests * max_new
    cache = ds.KVCache(*(torch.zeros(n_pages, page, m.kv, m.dim, dtype=torch.bfloat16, device=dev) for _ in range(2)))
    table, free = torch.full((requests, width), -1, **i32), torch.arange(n_pages, **i32)
    slots, positions = torch.empty(room, dtype=torch.int64, device=dev), torch.empty(room, **i32)
    cu, seq, taken = torch.empty(requests + 1, **i32), torch.empty(requests, **i32), torch.empty(1, **i32)
    workspace = torch.empty(ds.attention_workspace_bytes(m.shape, requests, room, max_new), dtype=torch.uint8, device=dev)
    scratch = torch.empty(ds.workspace_bytes(m.moe, room), dtype=torch.uint8, device=dev)
    g = torch.Generator(device=dev).manual_seed(1)

    context = torch.zeros(requests, **i32)
    fed = [torch.randint(m.vocab, (prompt - r,), generator=g, **i32) for r in range(requests)]  # prompts, of unlike lengths
    kept = [f.tolist() for f in fed]
    guess = None
    for step in range(steps):
        new = torch.tensor([len(f) for f in fed], **i32)
        tokens = torch.cat(fed)
        T = tokens.numel()
        ds.page_map(context, new, free, table, page, slots, positions, cu, seq, taken)
        x = m.embed[tokens.long()] + m.place[positions[:T].long()]
        qkv = (x @ m.qkv).unflatten(1, (m.heads + 2 * m.kv, m.dim))
        q, k, v = qkv[:, : m.heads], qkv[:, m.heads: m.heads + m.kv], qkv[:, m.heads + m.kv:]
        ds.kv_append(m.shape, cache, k, v, slots)
        out = torch.empty(T, m.heads, m.dim, dtype=torch.bfloat16, device=dev)
        # (the step's own largest number of new tokens, not the prompts': drafts then take the kernel for few rows)
        ds.paged_attention(m.shape, cache, table, q, cu, seq, max(len(f) for f in fed), out, workspace)
        x = (x + out.flatten(1) @ m.back).contiguous()
        y = torch.empty(T, m.D, dtype=torch.float32, device=dev)
        normed = torch.nn.functional.rms_norm(x.float(), (m.D,)).bfloat16()
        ds.layer(m.moe, m.weights, normed, y, scratch)
        target = torch.softmax((torch.nn.functional.rms_norm(x.float() + y, (m.D,)).bfloat16() @ m.head).float(), -1)

        # the drafts' own distributions: rows of the step before, for each request's drafts
        if guess is None:  # prompts have none: each request's last row is the one to draw from
            rows = torch.tensor([int(c) - 1 for c in cu[1:]], device=dev)
            one = torch.arange(requests + 1, **i32)
            p, d, tok, lay = target[rows].contiguous(), None, tokens[rows].contiguous(), one
        else:
            p, d, tok, lay = target, guess, tokens, cu
        n_accepted, drawn = torch.empty(requests, **i32), torch.empty(requests, drafts + 1, **i32)
        ds.verify_drafts(p, d, tok, lay, torch.rand(tok.numel(), generator=g, device=dev),
                         torch.rand(requests, generator=g, device=dev), drawn, n_accepted)
        ds.sync_status()

        if check:
            pages, ends = table.cpu(), seq.tolist()
            for r in range(requests):
                at = torch.arange(ends[r])
                place = (pages[r, at // page].long().to(dev), (at % page).to(dev))
                a, b = int(cu[r]), int(cu[r + 1])
                want = plain_attention(cache.k[place], cache.v[place], q[a:b])
                # rounded once, the weights once: bf16 steps of the values' magnitude
                far = float((out[a:b].double() - want).abs().max())
                assert far <= 2 * 2.0 ** -8 * float(cache.v[place].abs().max()), f"request {r}: attention off by {far:.3g}"

        # what stands: the accepted drafts and the token drawn; pages behind them go back to the free list
        accepted = n_accepted.tolist()
        context = context + (new if guess is None else n_accepted + 1)
        used = int(taken)
        held = (context + page - 1) // page
        j = torch.arange(width, **i32)
        back = table[(j >= held[:, None]) & (j < ((seq + page - 1) // page)[:, None])]
        free = torch.cat([free[used:], back])
        fresh = [drawn[r, : accepted[r] + 1].tolist() for r in range(requests)]
        for r in range(requests):
            kept[r] += fresh[r]
        # the next drafts come from the distribution behind the last token, which the model then judges afresh
        last = torch.tensor([(int(cu[r + 1]) - 1 if guess is None else int(cu[r]) + accepted[r]) for r in range(requests)], device=dev)
        q_rows = target[last]
        drafted = torch.multinomial(q_rows, drafts, True, generator=g).int()
        fed = [torch.cat([torch.tensor(fresh[r][-1:], **i32), drafted[r]]) for r in range(requests)]
        guess = q_rows.repeat_interleave(drafts + 1, 0)
        print(f"step {step}: new tokens {new.tolist()}, drafts accepted {accepted}, pages free {free.numel()}")
    for r in range(requests):
        assert int(context[r]) == len(kept[r]) - 1  # all but the token drawn last have their keys in the pages
    return kept


if __name__ == "__main__":
    run()
