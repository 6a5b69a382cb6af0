"""Plain 64-bit forms of the serving operators, and cases to run them on (test infrastructure)."""
import math
import random

import numpy as np
import torch

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def cdiv(a, b):
    return -(-a // b)


class Case:
    """Requests with ctx cached and new new tokens over paged keys and values.  What no request may see is NaN:
    pages of no request, rows behind a sequence's end, table columns beyond its pages (ids out of the cache)."""

    def __init__(self, ctx, new, H, G, D, page, dtype="bf16", window=0, layout="pages", seed=0, seq=None, device="cuda", qscale=1.5,
                 qkv=False):
        self.ctx, self.new, self.H, self.G, self.D, self.page, self.window = ctx, new, H, G, D, page, window
        self.dtype, self.dt, self.device = dtype, DT[dtype], device
        self.R, self.T = len(new), sum(new)
        g = torch.Generator().manual_seed(seed)
        # the sequence's length; shorter than its chunk where seq says so
        self.seq = [a + b for a, b in zip(ctx, new)] if seq is None else seq
        n_pages = sum(cdiv(s, page) for s in self.seq) + 3
        order = torch.randperm(n_pages, generator=g).tolist()
        self.width = max([1] + [cdiv(s, page) for s in self.seq]) + 2
        table = torch.full((self.R, self.width), n_pages + 7, dtype=torch.int32)
        table[:, -1] = -1
        kv = torch.full((2, n_pages, page, G, D), math.nan, dtype=self.dt)
        self.keys, self.values = [], []
        for r, s in enumerate(self.seq):
            for j in range(cdiv(s, page)):
                table[r, j] = order.pop()
            k, v = torch.randn(2, s, G, D, generator=g).to(self.dt)
            self.keys.append(k)
            self.values.append(v)
        self.table_cpu = table
        self.n_pages, self.kv_cpu, self.layout = n_pages, kv, layout
        q = (qscale * torch.randn(self.T, H, D, generator=g)).to(self.dt)
        self.q_cpu = q
        self.qkv = qkv

    def put(self):
        """Everything onto the device (after a test changed self.keys or self.values)."""
        kv, dev = self.kv_cpu, self.device
        for r, s in enumerate(self.seq):
            j = torch.arange(s)
            pg = self.table_cpu[r, j // self.page].long()
            kv[0][pg, j % self.page] = self.keys[r]
            kv[1][pg, j % self.page] = self.values[r]
        if self.layout == "pages":      # [pages][rows][heads][D]
            self.k, self.v = kv[0].to(dev), kv[1].to(dev)
        elif self.layout == "heads":    # [pages][heads][rows][D]
            self.k, self.v = (t.transpose(1, 2).contiguous().to(dev).transpose(1, 2) for t in kv)
        elif self.layout == "both":     # [pages][2][rows][heads][D]
            b = kv.transpose(0, 1).contiguous().to(dev)
            self.k, self.v = b[:, 0], b[:, 1]
        elif self.layout == "padded":   # rows 8 elements longer than they need be
            b = torch.nn.functional.pad(kv, (0, 8), value=math.nan).to(dev)
            self.k, self.v = b[0][..., : self.D], b[1][..., : self.D]
        elif self.layout == "odd":      # strides that no vector load can take
            b = torch.nn.functional.pad(kv, (1, 2), value=math.nan).to(dev)
            self.k, self.v = b[0][..., 1: 1 + self.D], b[1][..., 1: 1 + self.D]
        q = self.q_cpu
        if self.qkv:  # q as the first part of a fused projection
            q = torch.nn.functional.pad(q.reshape(self.T, -1), (0, 2 * self.G * self.D), value=math.nan).to(dev)
            self.q = q[:, : self.H * self.D].unflatten(1, (self.H, self.D))
        else:
            self.q = q.to(dev)
        self.table = self.table_cpu.to(dev)
        self.cu = torch.tensor([0] + np.cumsum(self.new).tolist(), dtype=torch.int32, device=dev)
        self.seq_lens = torch.tensor(self.seq, dtype=torch.int32, device=dev)
        return self

    def reference(self):
        """out, lse and the scale of out's error (the weights' sum of |v|) in 64 bits, one token at a time."""
        g = self.H // self.G
        out = torch.zeros(self.T, self.H, self.D, dtype=torch.float64)
        mag = torch.zeros_like(out)
        lse = torch.full((self.T, self.H), -math.inf, dtype=torch.float64)
        t, worst = 0, 0.0
        for r in range(self.R):
            k, v = self.keys[r].double().permute(1, 0, 2), self.values[r].double().permute(1, 0, 2)
            for i in range(self.new[r]):
                hi = self.seq[r] - self.new[r] + i + 1
                lo = max(0, hi - self.window) if self.window else 0
                if hi > 0:
                    q = self.q_cpu[t].double().view(self.G, g, self.D)
                    s = torch.einsum("gid,gjd->gij", q, k[:, lo:hi]) / math.sqrt(self.D)
                    worst = max(worst, float((torch.einsum("gid,gjd->gij", q.abs(), k[:, lo:hi].abs()) / math.sqrt(self.D)).nan_to_num(0, 0, 0).max()))
                    z = torch.logsumexp(s, -1, keepdim=True)
                    p = torch.exp(s - z)
                    out[t] = torch.einsum("gij,gjd->gid", p, v[:, lo:hi]).reshape(self.H, self.D)
                    mag[t] = torch.einsum("gij,gjd->gid", p, v[:, lo:hi].abs()).reshape(self.H, self.D)
                    lse[t] = z.reshape(self.H)
                t += 1
        self.worst = worst
        return out, lse, mag

    def tolerances(self, out, mag, rounded_p):
        """How far out and lse may be off.  With u half a step of the type: out is rounded once (u |out|), the
        probabilities once where the second product runs on tensor cores (u mag); a score's fp32 sum of D products
        is off by (D + 4) 2^-24 of the sum of their magnitudes, which moves weights by twice as much; sums of up to
        n terms, the running rescales and the exponential by (n + 64) 2^-24."""
        u = torch.finfo(self.dt).eps / 2
        n = max([1] + self.seq)
        score = (self.D + 4) * 2.0 ** -24 * self.worst
        sums = (n + 64) * 2.0 ** -24
        tiny = 2.0 ** -24 if self.dtype == "f16" else 0.0  # fp16's smallest step
        return u * out.abs() + (u * rounded_p + 2 * score + 2 * sums) * mag + tiny, score + sums + 2.0 ** -22


def page_map(ctx, new, page, free, table, cap):
    """ds_moe_page_map, request by request; table is changed in place.  Returns slots, positions, cu, seq, taken, bad."""
    width, bad = table.shape[1], False
    slots, positions = [-1] * cap, [-1] * cap
    cu, seq, p = [0], [], 0
    taken = 0
    for r in range(len(ctx)):
        c, n = ctx[r], new[r]
        if not 0 <= c < 1 << 30:
            c, bad = 0, True
        if not 0 <= n < 1 << 30:
            n, bad = 0, True
        if cu[-1] + n > cap:
            n, bad = cap - cu[-1], True
        held, need = min(cdiv(c, page), width), cdiv(c + n, page)
        bad |= need > width
        for j in range(held, min(need, width)):
            ok = p < len(free)
            table[r, j] = free[p] if ok else -1
            taken += ok
            bad |= not ok
            p += 1
        for i in range(n):
            pos, t = c + i, cu[-1] + i
            col = pos // page
            pg = int(table[r, col]) if col < width else -1
            bad |= pg < 0
            slots[t] = pg * page + pos % page if pg >= 0 else -1
            positions[t] = pos
        cu.append(cu[-1] + n)
        seq.append(c + n)
    return slots, positions, cu, seq, taken, bad


def verify(p, q, tokens, cu, u_accept, u_sample, max_new):
    """ds_moe_verify_drafts on numpy fp32 rows, in 64 bits."""
    p = p.astype(np.float64)
    q = None if q is None else q.astype(np.float64)
    out, kept = [], []
    V = p.shape[1]
    for r in range(len(cu) - 1):
        t0, n = cu[r], cu[r + 1] - cu[r]
        row, k, x = [-1] * max_new, 0, None
        while k < n - 1:
            x = int(tokens[t0 + k + 1])
            if not 0 <= x < V or not float(u_accept[t0 + k]) * (1.0 if q is None else q[t0 + k, x]) < p[t0 + k, x]:
                break
            row[k] = x
            k += 1
        if n > 0:
            w = np.clip(np.nan_to_num(p[t0 + k], nan=0.0), 0, 1)
            if k < n - 1:
                d = np.clip(np.nan_to_num(q[t0 + k], nan=0.0), 0, 1) if q is not None else (np.arange(V) == x).astype(np.float64)
                rest = np.maximum(w - d, 0)
                w = rest if rest.sum() > 0 else w
            c = np.cumsum(w)
            row[k] = int(np.searchsorted(c, float(u_sample[r]) * c[-1], side="right")) if c[-1] > 0 else -1
        out.append(row)
        kept.append(k)
    return np.array(out, np.int32).reshape(len(cu) - 1, max_new), np.array(kept, np.int32)


def lengths(rng: random.Random, n, lo, hi):
    return [rng.randint(lo, hi) for _ in range(n)]
