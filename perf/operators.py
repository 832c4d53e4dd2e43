"""Cases of the session-cache operators: rope_append, window_attend, weigh_tokens and evict_tokens.

The life of a session's paged cache: new tokens are rotated and written into
their pages, attend over the cache (causal, with a sliding window and sinks),
their attention weights are accumulated per cached token, and the tokens with
the least weight are evicted.  `run` makes one call of one operator: in its
plain form (elementary torch operations in fp32, angles in fp64) or, with
`own`, through the package's public entry points.
"""
import math
import random

import torch

own = False

P = 16  # tokens of a page


def listed():
    return [
        # one decode step of 4 short sessions with few heads: the smallest call, launch latency
        _attend("attend decode tiny", 4, 8, 2, 64, 272, 320, 1, 1, 0, 0, 1),
        # decode of long streaming sessions that keep a window and a few first tokens
        _attend("attend decode window", 64, 32, 8, 128, 8192, 65536, 1, 1, 4096, 16, 2),
        # decode of two very long sessions over their whole context: few rows, a long axis
        _attend("attend decode long", 2, 32, 8, 128, 100001, 131072, 1, 1, 0, 0, 3),
        # several proposed tokens of every request checked at once, wide head groups
        _attend("attend verify", 16, 32, 4, 128, 500, 9000, 2, 7, 0, 0, 4),
        # ragged chunks of streamed data under a window, one kv head per query head
        _attend("attend chunk window", 8, 16, 16, 64, 700, 5000, 1, 700, 512, 4, 5),
        # a long chunk of a prompt over the session's context
        _attend("attend prefill", 1, 32, 8, 128, 32768, 32768, 4096, 4096, 0, 0, 6),
        # the weights of a decode step of 64 sessions
        _weigh("weigh decode", 64, 32, 8, 128, 2000, 20000, 1, 1, 0, 0, 7),
        # the weights of a prompt's chunk
        _weigh("weigh prefill", 2, 32, 8, 128, 9000, 16384, 1500, 2048, 0, 0, 8),
        # short sessions back to their budget
        _evict("evict small", 4, 2, 64, 300, 320, 256, 4, 32, 9),
        # long sessions pruned to an eighth
        _evict("evict large", 16, 8, 128, 20000, 32768, 4096, 16, 512, 10),
        # the new token of each of 64 sessions
        _rope("rope decode", 64, 32, 8, 128, 128, 1, 0, 2048, 8192, 1, 1, 11),
        # chunks of text, images and video: three axes
        _rope("rope chunk", 4, 32, 8, 128, 128, 3, 0, 4096, 16384, 1000, 4096, 12),
    ]


def _attend(name, S, Hq, Hkv, D, ctx_lo, ctx_hi, rows_lo, rows_hi, window, sinks, shape, op="attend"):
    """ctx: cached tokens of a session, its new rows among them; shape: seeds the sessions' lengths."""
    return {"name": name, "op": op, "S": S, "Hq": Hq, "Hkv": Hkv, "D": D, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi,
            "rows_lo": rows_lo, "rows_hi": rows_hi, "window": window, "sinks": sinks, "shape": shape}


def _weigh(*a):
    return _attend(*a, op="weigh")


def _evict(name, S, Hkv, D, ctx_lo, ctx_hi, budget, sinks, recent, shape):
    return {"name": name, "op": "evict", "S": S, "Hkv": Hkv, "D": D, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi,
            "budget": budget, "sinks": sinks, "recent": recent, "shape": shape}


def _rope(name, S, Hq, Hkv, D, R, n_axes, interleaved, ctx_lo, ctx_hi, rows_lo, rows_hi, shape):
    return {"name": name, "op": "rope", "S": S, "Hq": Hq, "Hkv": Hkv, "D": D, "R": R, "n_axes": n_axes,
            "interleaved": interleaved, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "rows_lo": rows_lo, "rows_hi": rows_hi,
            "shape": shape}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "weigh", "evict", "rope"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 8])
    shape = rng.randrange(1 << 20)
    if op in ("attend", "weigh"):
        hi = _log(rng, 20, 65536)
        rows = _log(rng, 1, min(hi, 2048)) if rng.random() < 0.5 else rng.randint(1, min(hi, 6))
        # pairs of rows and keys, and cached tokens, stay below the largest listed cases'
        S = max(1, min(_log(rng, 1, 64), (1 << 25) // (rows * hi), (1 << 18) // hi))
        window = rng.choice([0, 0, _log(rng, 16, 8192)])
        sinks = rng.choice([0, 1, 4, 37]) if window else 0
        f = _attend if op == "attend" else _weigh
        c = f("", S, Hq, Hkv, D, max(rows, rng.randint(hi // 4, hi)), hi, rng.randint(1, rows), rows, window, sinks, shape)
    elif op == "evict":
        hi = _log(rng, 64, 65536)
        S = max(1, min(_log(rng, 1, 32), (1 << 17) // hi))
        budget = rng.randint(20, hi)
        sinks = rng.randint(0, 16)
        c = _evict("", S, Hkv, D, rng.randint(hi // 2, hi), hi, budget, sinks, rng.randint(0, budget - sinks), shape)
    else:
        rows = _log(rng, 1, 2048)
        hi = rows + _log(rng, 1, 16384)
        S = max(1, min(_log(rng, 1, 64), 8192 // rows))
        R = rng.choice([D, D, D // 2])
        c = _rope("", S, Hq, Hkv, D, R, rng.choice([1, 3, 3, 4]), rng.choice([0, 1]), rows, hi, rng.randint(1, rows), rows,
                  shape)
    del c["name"]
    return c


def _lens(c):
    """The sessions' cached tokens and new rows: a property of the case, so that its work is known."""
    r = random.Random(c["shape"])
    kv = [r.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["S"])]
    kv[-1] = c["ctx_hi"]
    rows = [min(k, r.randint(c.get("rows_lo", 1), c.get("rows_hi", 1))) for k in kv]
    return kv, rows


def _axes(c):
    """The axis of every rotated pair: contiguous sections, the first axis (time) the shortest."""
    n, a = c["R"] // 2, c["n_axes"]
    first = n // a if a == 1 else n // (a + 1)
    return [0 if i < first or a == 1 else 1 + (i - first) * (a - 1) // (n - first) for i in range(n)]


def prepare(case, seed):
    c, dev = case, "cuda"
    kv, rows = _lens(c)
    S, Hkv, D = c["S"], c["Hkv"], c["D"]
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    pages = [-(-k // P) for k in kv]
    width = max(pages)
    n_dst = -(-c["budget"] // P) if c["op"] == "evict" else 0
    total = sum(pages) + S * n_dst
    num_pages = total + max(1, total // 20)  # some spare pages, as a pool has
    perm = torch.randperm(num_pages, generator=g, device=dev, dtype=torch.int32)
    table = torch.full((S, width), -1, dtype=torch.int32, device=dev)
    at = 0
    for s, n in enumerate(pages):
        table[s, :n] = perm[at:at + n]
        at += n
    st = {"case": c, "kv_lens": torch.tensor(kv, dtype=torch.int32, device=dev), "table": table,
          "n_max": max(rows), "t_max": max(kv)}
    st["cu_rows"] = torch.tensor([0] + [sum(rows[:i + 1]) for i in range(S)], dtype=torch.int32, device=dev)
    n = sum(rows)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.bfloat16)

    if c["op"] == "rope":
        st["k_pool"] = torch.zeros(num_pages, Hkv, P, D, dtype=torch.bfloat16, device=dev)
        st["v_pool"] = torch.zeros_like(st["k_pool"])
        # q, k and v come out of one projection: rows of one matrix
        fused = normal(n, (c["Hq"] + 2 * Hkv) * D)
        hq, hk = c["Hq"] * D, Hkv * D
        st["q"] = fused[:, :hq].view(n, c["Hq"], D)
        st["k"] = fused[:, hq:hq + hk].view(n, Hkv, D)
        st["v"] = fused[:, hq + hk:].view(n, Hkv, D)
        start = torch.cat([torch.arange(k - r, k, dtype=torch.int32) for k, r in zip(kv, rows)]).to(dev)
        pos = start.repeat(c["n_axes"], 1)
        for a in range(1, c["n_axes"]):  # height, width, ...: coordinates inside a frame
            pos[a] = (start // 7 ** (a - 1)) % 61 + start // 1000
        st["positions"] = pos.contiguous()
        i = torch.arange(c["R"] // 2, dtype=torch.float64, device=dev)
        st["inv_freq"] = 10000.0 ** (-2.0 * i / c["R"])
        st["axes"] = _axes(c)
        return st
    st["k_pool"], st["v_pool"] = normal(num_pages, Hkv, P, D), normal(num_pages, Hkv, P, D)
    if c["op"] == "evict":
        st["dst_table"] = perm[at:at + S * n_dst].view(S, n_dst).contiguous()
        # weights of a long tail, many tokens with none at all
        x = torch.rand(S, Hkv, width * P, generator=g, device=dev)
        x = x.pow(6.0) * 40.0
        st["scores"] = torch.where(x < 1e-4, torch.zeros_like(x), x)
        return st
    # queries and the first cached tokens share a direction, so that the first tokens draw weight as they do in earnest
    u = normal(Hkv, 1, D)
    q = normal(n, c["Hq"], D).view(n, Hkv, c["Hq"] // Hkv, D) + 0.5 * u
    st["q"] = q.view(n, c["Hq"], D).contiguous()
    first = table[:, 0].long()
    st["k_pool"][first, :, :2] += 0.8 * u * math.sqrt(64.0 / D)
    if c["op"] == "weigh":
        st["scores"] = torch.rand(S, Hkv, width * P, generator=g, device=dev)
        st["lse"] = _softmax(st, want_out=False)
    return st


# ------------------------------------------------------------------------------------------------ plain forms


def _rows_of(st):
    """Row of the batch and cached position of each (session, row): [S, n_max], and which of them exist."""
    cu = st["cu_rows"].long()
    n = cu[1:] - cu[:-1]
    i = torch.arange(st["n_max"], device=cu.device)
    valid = i < n[:, None]
    return (cu[:-1, None] + i).clamp(max=st["q"].shape[0] - 1), st["kv_lens"].long()[:, None] - n[:, None] + i, valid


def _keys_of(st):
    """Cached tokens that some row of the session may see: [S, W] token indices, and which of them exist."""
    c, kv = st["case"], st["kv_lens"].long()
    n = (st["cu_rows"][1:] - st["cu_rows"][:-1]).long()
    w, dev = c["window"], kv.device
    if w == 0 or c["sinks"] + w + st["n_max"] >= st["t_max"]:
        t = torch.arange(st["t_max"], device=dev).expand(c["S"], -1)
        return t, t < kv[:, None]
    lo = (kv - n - w + 1).clamp(min=c["sinks"])
    t = torch.cat([torch.arange(c["sinks"], device=dev).expand(c["S"], -1),
                   lo[:, None] + torch.arange(w + st["n_max"] - 1, device=dev)], 1)
    ok = t < kv[:, None]
    return t.clamp(max=st["t_max"] - 1), ok


def _logits(st):
    c = st["case"]
    S, Hkv, D, G, n = c["S"], c["Hkv"], c["D"], c["Hq"] // c["Hkv"], st["n_max"]
    row, pos, valid = _rows_of(st)
    t, ok = _keys_of(st)
    page = st["table"].long().gather(1, t // P).clamp(min=0)
    k = st["k_pool"][page, :, t % P].float()  # [S, W, Hkv, D]
    q = st["q"][row].float().view(S, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(S, Hkv, n * G, D)
    x = torch.matmul(q * (1.0 / math.sqrt(D)), k.permute(0, 2, 3, 1))
    sees = ok[:, None, :] & (t[:, None, :] <= pos[:, :, None]) & valid[:, :, None]
    if c["window"]:
        sees &= (t[:, None, :] > pos[:, :, None] - c["window"]) | (t[:, None, :] < c["sinks"])
    x.view(S, Hkv, n, G, -1).masked_fill_(~sees[:, None, :, None, :], -math.inf)
    return x, t, page, valid


def _softmax(st, want_out=True):
    c = st["case"]
    S, Hkv, D, G, n = c["S"], c["Hkv"], c["D"], c["Hq"] // c["Hkv"], st["n_max"]
    x, t, page, valid = _logits(st)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    lse = (m + l.log()).view(S, Hkv, n, G).permute(0, 2, 1, 3).reshape(S, n, c["Hq"])[valid].contiguous()
    if not want_out:
        return lse
    v = st["v_pool"][page, :, t % P].float()
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(l > 0, l, torch.ones_like(l))
    o = o.view(S, Hkv, n, G, D).permute(0, 2, 1, 3, 4).reshape(S, n, c["Hq"], D)[valid]
    return {"out": o.to(torch.bfloat16), "lse": lse}


def _weigh_plain(st):
    c = st["case"]
    S, Hkv, G, n = c["S"], c["Hkv"], c["Hq"] // c["Hkv"], st["n_max"]
    x, t, _, valid = _logits(st)
    row = _rows_of(st)[0]
    lse = st["lse"][row].view(S, n, Hkv, G).permute(0, 2, 1, 3).reshape(S, Hkv, n * G, 1)
    w = x.sub_(lse).exp_().sum(2)
    st["scores"].scatter_add_(2, t[:, None, :].expand(-1, Hkv, -1), w)
    return {"scores": st["scores"]}


def _evict_plain(st):
    c = st["case"]
    S, Hkv, B = c["S"], c["Hkv"], c["budget"]
    kv, dev = st["kv_lens"].long(), st["scores"].device
    T = st["scores"].shape[2]
    t = torch.arange(T, device=dev)
    hold = (t < c["sinks"]) | (t >= kv[:, None] - c["recent"])
    key = torch.where(hold[:, None, :], math.inf, st["scores"]).masked_fill(t >= kv[:, None, None], -math.inf)
    if T < B:
        key = torch.nn.functional.pad(key, (0, B - T), value=-math.inf)
    order = key.sort(dim=-1, descending=True, stable=True).indices[..., :B]
    new = kv.clamp(max=B)
    j = torch.arange(B, device=dev)
    there = (j < new[:, None])[:, None, :].expand(-1, Hkv, -1)
    kept = torch.where(there, order, 1 << 40).sort(dim=-1).values
    kept = torch.where(there, kept, 0)
    out = torch.zeros_like(st["scores"])
    out[..., :min(B, T)] = torch.where(there, st["scores"].gather(2, kept), 0.0)[..., :T]
    s, h, d = there.nonzero(as_tuple=True)
    src = kept[s, h, d]
    sp, dp = st["table"][s, src // P].long(), st["dst_table"][s, d // P].long()
    st["k_pool"][dp, h, d % P] = st["k_pool"][sp, h, src % P]
    st["v_pool"][dp, h, d % P] = st["v_pool"][sp, h, src % P]
    return {"new_lens": new.int(), "kept": torch.where(there, kept, -1).int(), "scores": out,
            "k_pool": st["k_pool"], "v_pool": st["v_pool"]}


def _rotate(x, cos, sin, R, interleaved):
    x = x.float()
    r = x[..., :R]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :R // 2], r[..., R // 2:])
    u, w = a * cos - b * sin, a * sin + b * cos
    r = torch.stack([u, w], -1).flatten(-2) if interleaved else torch.cat([u, w], -1)
    return torch.cat([r, x[..., R:]], -1).to(torch.bfloat16)


def _rope_plain(st):
    c = st["case"]
    axes = torch.tensor(st["axes"], device=st["q"].device)
    angle = st["positions"][axes].double().t() * st["inv_freq"]  # [rows, R / 2]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    row, pos, valid = _rows_of(st)
    pos = pos.clamp(min=0, max=st["t_max"] - 1)
    page = st["table"].long().gather(1, pos // P)[valid]
    slot = (pos % P)[valid]
    st["k_pool"][page, :, slot] = _rotate(st["k"], cos, sin, c["R"], c["interleaved"])
    st["v_pool"][page, :, slot] = st["v"]
    return {"q": _rotate(st["q"], cos, sin, c["R"], c["interleaved"]), "k_pool": st["k_pool"], "v_pool": st["v_pool"]}


def run(st):
    c = st["case"]
    if own:
        import prefix_aware_decode_b200 as pad
        if c["op"] == "attend":
            out, lse = pad.window_attend(st["q"], st["k_pool"], st["v_pool"], st["table"], st["kv_lens"], st["cu_rows"],
                                         window=c["window"], sinks=c["sinks"])
            return {"out": out, "lse": lse}
        if c["op"] == "weigh":
            pad.weigh_tokens(st["q"], st["k_pool"], st["lse"], st["table"], st["kv_lens"], st["cu_rows"], st["scores"],
                             window=c["window"], sinks=c["sinks"])
            return {"scores": st["scores"]}
        if c["op"] == "evict":
            new_lens, kept, scores = pad.evict_tokens(st["scores"], st["k_pool"], st["v_pool"], st["table"],
                                                      st["kv_lens"], st["dst_table"], c["budget"], sinks=c["sinks"],
                                                      recent=c["recent"])
            return {"new_lens": new_lens, "kept": kept, "scores": scores, "k_pool": st["k_pool"], "v_pool": st["v_pool"]}
        q = pad.rope_append(st["q"], st["k"], st["v"], st["positions"], st["inv_freq"], st["k_pool"], st["v_pool"],
                            st["table"], st["kv_lens"], st["cu_rows"], axes=st["axes"],
                            interleaved=bool(c["interleaved"]))
        return {"q": q, "k_pool": st["k_pool"], "v_pool": st["v_pool"]}
    return {"attend": _softmax, "weigh": _weigh_plain, "evict": _evict_plain, "rope": _rope_plain}[c["op"]](st)


# ------------------------------------------------------------------------------------------------ the definitions in 64 bits


def exact(case, seed):
    """Session by session and head by head, in float64, from the definitions."""
    c = case
    st = prepare(c, seed)
    kv, rows = _lens(c)
    table = st["table"].cpu()

    def cached(pool, s, h):  # the session's tokens of one kv head, in order
        p = table[s, :-(-kv[s] // P)].long().to(pool.device)
        return pool[p, h].reshape(-1, c["D"])[:kv[s]].double()

    if c["op"] == "rope":
        inv = [10000.0 ** (-2.0 * i / c["R"]) for i in range(c["R"] // 2)]
        q, kp, vp = st["q"].double(), st["k_pool"].double(), st["v_pool"].double()
        k, at = st["k"].double(), 0

        def turn(x):
            y = x.clone()
            for i, f in enumerate(inv):
                a = st["positions"][st["axes"][i]].double() * f
                co, si = torch.cos(a)[:, None], torch.sin(a)[:, None]
                m, n = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + c["R"] // 2)
                y[..., m], y[..., n] = x[..., m] * co - x[..., n] * si, x[..., m] * si + x[..., n] * co
            return y

        q, k = turn(q), turn(k)
        for s in range(c["S"]):
            t = torch.arange(kv[s] - rows[s], kv[s])
            p, o = table[s, t // P].long().to(q.device), (t % P).to(q.device)
            kp[p, :, o] = k[at:at + rows[s]]
            vp[p, :, o] = st["v"][at:at + rows[s]].double()
            at += rows[s]
        return {"q": q, "k_pool": kp, "v_pool": vp}
    if c["op"] == "evict":
        T = st["scores"].shape[2]
        out = torch.zeros(c["S"], c["Hkv"], T, dtype=torch.float64)
        x = st["scores"].cpu()
        for s in range(c["S"]):
            n = min(kv[s], c["budget"])
            held = set(range(min(c["sinks"], kv[s]))) | set(range(max(0, kv[s] - c["recent"]), kv[s]))
            for h in range(c["Hkv"]):
                v = x[s, h, :kv[s]].double().tolist()
                rest = sorted((t for t in range(kv[s]) if t not in held), key=lambda t: (-v[t], t))
                ids = list(range(kv[s])) if kv[s] <= c["budget"] else sorted(list(held) + rest[:n - len(held)])
                out[s, h, :n] = torch.tensor([v[t] for t in ids], dtype=torch.float64)
        return {"new_lens": None, "kept": None, "scores": out.to(st["q"].device if "q" in st else "cuda"),
                "k_pool": None, "v_pool": None}
    G, scale = c["Hq"] // c["Hkv"], 1.0 / math.sqrt(c["D"])
    n = sum(rows)
    out = torch.zeros(n, c["Hq"], c["D"], dtype=torch.float64, device="cuda")
    lse = torch.zeros(n, c["Hq"], dtype=torch.float64, device="cuda")
    scores = st["scores"].double() if c["op"] == "weigh" else None
    at = 0
    for s in range(c["S"]):
        r = rows[s]
        p = torch.arange(kv[s] - r, kv[s], device="cuda")[:, None]
        lo = max(0, kv[s] - r - c["window"] + 1) if c["window"] else 0
        t = torch.arange(kv[s], device="cuda")
        t = t[(t < c["sinks"]) | (t >= lo)]
        see = t <= p
        if c["window"]:
            see &= (t > p - c["window"]) | (t < c["sinks"])
        for h in range(c["Hq"]):
            k = cached(st["k_pool"], s, h // G)[t]
            x = (st["q"][at:at + r, h].double() @ k.t() * scale).masked_fill_(~see, -math.inf)
            if c["op"] == "weigh":
                scores[s, h // G].index_add_(0, t, torch.exp(x - st["lse"][at:at + r, h].double()[:, None]).sum(0))
                continue
            lse[at:at + r, h] = torch.logsumexp(x, 1)
            out[at:at + r, h] = torch.softmax(x, 1) @ cached(st["v_pool"], s, h // G)[t]
        at += r
    return {"scores": scores} if c["op"] == "weigh" else {"out": out, "lse": lse}


# ------------------------------------------------------------------------------------------------ what a pass cannot do without


def _seen(c):
    """Visible (row, key) pairs of a query head, and cached tokens that some row sees, over all sessions."""
    pairs = tokens = 0
    w, k = c["window"], c["sinks"]
    for kv, r in zip(*_lens(c)):
        for p in range(kv - r, kv):
            first = max(0, p - w + 1) if w else 0
            pairs += p + 1 - first + min(k, first)
        first = max(0, kv - r - w + 1) if w else 0
        tokens += kv - first + min(k, first)
    return pairs, tokens


def work(case):
    c = case
    kv, rows = _lens(c)
    S, Hkv, D, n = c["S"], c["Hkv"], c["D"], sum(rows)
    table = 4 * sum(-(-k // P) for k in kv) + 8 * S
    if c["op"] == "rope":
        return {"bytes": 2 * n * (c["Hq"] + 2 * Hkv) * D * 2 + 4 * n * c["n_axes"] + 8 * S + 4 * n,
                "flops": 3 * n * (c["Hq"] + Hkv) * c["R"]}
    if c["op"] == "evict":
        kept = sum(min(k, c["budget"]) for k in kv)
        T = -(-max(kv) // P) * P
        return {"bytes": Hkv * (4 * sum(kv) + kept * (2 * 2 * 2 * D) + 4 * S * c["budget"] + 4 * S * T) + table + 4 * S,
                "flops": 0}
    pairs, tokens = _seen(c)
    if c["op"] == "weigh":
        return {"bytes": tokens * Hkv * (2 * D + 8) + n * c["Hq"] * (2 * D + 4) + table,
                "flops": 2 * D * c["Hq"] * pairs}
    return {"bytes": tokens * Hkv * 4 * D + n * c["Hq"] * (4 * D + 4) + table, "flops": 4 * D * c["Hq"] * pairs}
