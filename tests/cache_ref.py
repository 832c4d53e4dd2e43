"""The session-cache operators in 64 bits, from their definitions, and random
caches to run them on.  Plain loops over sessions, heads and rows."""
import math

import numpy as np
import torch

import prefix_aware_decode_b200 as pad

P = 16


class Cache:
    """A paged cache of sessions with given lengths and new rows, everything that
    no session holds poisoned with NaN.  holes: (session, logical page) entries set
    to ids outside the pool."""

    def __init__(self, kv, rows, Hq, Hkv, D, seed=0, holes=(), extra_rows=0, extra_pages=1, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.kv, self.rows, self.Hq, self.Hkv, self.D = list(kv), list(rows), Hq, Hkv, D
        S = len(kv)
        pages = [-(-n // P) for n in kv]
        self.width = max(pages + [1]) + extra_pages
        self.num_pages = sum(pages) + 3
        perm = torch.randperm(self.num_pages, generator=g).int()
        self.table = torch.full((S, self.width), -1, dtype=torch.int32)
        self.k = torch.full((self.num_pages, Hkv, P, D), math.nan).bfloat16()
        self.v = self.k.clone()
        at = 0
        for s in range(S):
            for j in range(pages[s]):
                p = int(perm[at])
                at += 1
                self.table[s, j] = p
                n = min(P, kv[s] - j * P)
                self.k[p, :, :n] = torch.randn(Hkv, n, D, generator=g).bfloat16()
                self.v[p, :, :n] = torch.randn(Hkv, n, D, generator=g).bfloat16()
        for i, (s, j) in enumerate(holes):
            self.table[s, j] = (-1, self.num_pages, 2 ** 31 - 1, -2 ** 31)[i % 4]
        self.cu = torch.tensor([0] + list(np.cumsum(rows)), dtype=torch.int32)
        self.n = int(self.cu[-1])
        self.q = torch.randn(self.n + extra_rows, Hq, D, generator=g).bfloat16()
        self.gen, self.device = g, device

    def dev(self, *names):
        return [getattr(self, n).to(self.device) for n in names]

    @property
    def lens(self):
        return torch.tensor(self.kv, dtype=torch.int32)

    def tokens(self, pool, s, h):
        """(indices, rows in fp64) of the session's cached tokens that are not in holes."""
        t = [i for i in range(self.kv[s]) if 0 <= int(self.table[s, i // P]) < self.num_pages]
        t = torch.tensor(t, dtype=torch.long)
        p = self.table[s, t // P].long()
        return t, pool[p, h, t % P].double()


def sees(p, t, window, sinks):
    m = t[None, :] <= p[:, None]
    if window:
        m &= (t[None, :] > p[:, None] - window) | (t[None, :] < sinks)
    return m


def logits(c, s, h, window, sinks, scale):
    """(indices, masked logits, bound of a logit's fp32 error) of a session's rows at query head h."""
    r0, n = int(c.cu[s]), c.rows[s]
    t, k = c.tokens(c.k, s, h // (c.Hq // c.Hkv))
    q = c.q[r0:r0 + n, h].double()
    x = q @ k.t() * scale
    # a sum of D products, each step off by at most 2^-23 (a tensor core may truncate)
    err = c.D * 2.0 ** -23 * abs(scale) * float(q.norm(dim=1).max() * k.norm(dim=1).max()) if k.numel() and n else 0.0
    p = torch.arange(c.kv[s] - n, c.kv[s])
    return t, x.masked_fill(~sees(p, t, window, sinks), -math.inf), err


def attend(c, window=0, sinks=0, scale=None):
    """out, lse, and the bounds that the kernels' roundings allow."""
    scale = scale or 1 / math.sqrt(c.D)
    out = torch.zeros(c.n, c.Hq, c.D, dtype=torch.float64)
    tol = torch.zeros_like(out)
    lse = torch.full((c.n, c.Hq), -math.inf, dtype=torch.float64)
    ltol = torch.zeros_like(lse)
    for s in range(len(c.kv)):
        r = slice(int(c.cu[s]), int(c.cu[s + 1]))
        for h in range(c.Hq):
            t, x, err = logits(c, s, h, window, sinks, scale)
            if not len(t) or not c.rows[s]:
                continue
            v = c.tokens(c.v, s, h // (c.Hq // c.Hkv))[1]
            l = torch.logsumexp(x, 1)
            p = torch.where(l[:, None] > -math.inf, (x - l[:, None]).exp(), 0.0)
            o, a = p @ v, p @ v.abs()
            out[r, h], lse[r, h] = o, l
            # one bf16 rounding of the weights and one of the result, each half a step
            # (2^-8); the logits' error moves a weight by twice itself; 2^-15 for fp32 sums
            tol[r, h] = 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2 * err + 2.0 ** -15) * a * (1 + 2.0 ** -7)
            ltol[r, h] = err + 2.0 ** -20 + 2.0 ** -22 * torch.where(l > -math.inf, l.abs(), 0.0)
    return out, lse, tol, ltol


def weigh(c, lse, window=0, sinks=0, scale=None):
    """The weights added to [S][Hkv][max kv] and the bound of their error."""
    scale = scale or 1 / math.sqrt(c.D)
    w = torch.zeros(len(c.kv), c.Hkv, max(c.kv + [1]), dtype=torch.float64)
    tol = torch.zeros_like(w)
    for s in range(len(c.kv)):
        r = slice(int(c.cu[s]), int(c.cu[s + 1]))
        for h in range(c.Hq):
            t, x, err = logits(c, s, h, window, sinks, scale)
            if not len(t) or not c.rows[s]:
                continue
            l = lse[r, h].double()[:, None]
            y = torch.where(l > -math.inf, (x - l).exp(), 0.0).sum(0)
            w[s, h // (c.Hq // c.Hkv), t] += y
            # a weight's exponent is off by the logit's error and by roundings of the
            # scaled logit and lse (2^-22 of their size); fp32 sums over the rows
            big = float(torch.where(x > -math.inf, x.abs(), 0.0).max()) + float(torch.where(l > -math.inf, l.abs(), 0.0).max())
            tol[s, h // (c.Hq // c.Hkv), t] += y * (2 * err + 2.0 ** -20 + 2.0 ** -21 * big + c.rows[s] * 2.0 ** -24)
    return w, tol


def evict(scores, kv, budget, sinks, recent):
    """kept[s][h]: the kept tokens' indices, ascending."""
    kept = []
    for s, n in enumerate(kv):
        n = min(n, scores.shape[2])
        kept.append([])
        for h in range(scores.shape[1]):
            if n <= budget:
                kept[s].append(list(range(n)))
                continue
            x = scores[s, h, :n].tolist()
            key = [math.inf if f != f else f for f in x]
            nan = [f != f for f in x]
            rest = sorted(range(sinks, n - recent), key=lambda t: (not nan[t], -key[t], t))[:budget - sinks - recent]
            kept[s].append(sorted(list(range(sinks)) + rest + list(range(n - recent, n))))
    return kept


def rotate(x, positions, inv_freq, axes, interleaved):
    """x fp64 [rows][heads][D] rotated, and the bound of the result's error."""
    y, tol = x.clone(), torch.zeros_like(x)
    R = 2 * len(inv_freq)
    for i, f in enumerate(inv_freq.tolist()):
        a = positions[axes[i]].double() * f
        co, si = a.cos()[:, None], a.sin()[:, None]
        m, n = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        y[..., m], y[..., n] = x[..., m] * co - x[..., n] * si, x[..., m] * si + x[..., n] * co
        # fp32 products and a sine, each 2^-22; then one bf16 rounding
        size = x[..., m].abs() + x[..., n].abs()
        for d in (m, n):
            tol[..., d] = 2.0 ** -8 * y[..., d].abs() + 2.0 ** -20 * size
    return y, tol


def check(got, want, tol, what):
    got = got.double().cpu()
    same = (got == want) | ((got - want).abs() <= tol)
    assert bool(same.all()), (what, int((~same).sum()), float(torch.where(same, 0.0, (got - want).abs()).max()),
                              torch.nonzero(~same)[:4].tolist())


def run_attend(c, window=0, sinks=0, scale=0.0, **kw):
    q, k, v, table, lens, cu = c.dev("q", "k", "v", "table", "lens", "cu")
    return pad.window_attend(q, k, v, table, lens, cu, window=window, sinks=sinks, softmax_scale=scale, **kw)
