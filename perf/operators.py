"""The operators around the W12 GEMMs of a verify step's attention layer, as cases to be measured.

  norm   residual addition + root-mean-square norm, output in BF16 (a W12 GEMM's input) or in 8 bits
         (e4m3) with one FP32 scale per 128 columns
  rope   rotary positions with one or several axes on q and k, optional per-head norms, and the write of
         the new keys and values into a paged cache
  attn   attention of the nodes of draft trees over a paged cache (one node per request: plain decode)

With `own` the framework's entry points are called; without it the same mathematics runs as elementary
torch operations in 32 bits.  Head layout and widths are those of the 27B-class layer shapes: 5120 columns,
QKV 7168 = (40 + 2*8) heads of 128.
"""
import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------
def _norm(name, M, K, residual=True, out8=False):
    return {"name": name, "op": "norm", "M": M, "K": K, "residual": residual, "out8": out8}


def _rope(name, n, Hq, Hkv, D, rot, axes=1, append=True, interleaved=False, qk_norm=False, page=64, top=131072):
    return {"name": name, "op": "rope", "n": n, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot, "axes": axes,
            "append": append, "interleaved": interleaved, "qk_norm": qk_norm, "page": page, "top": top}


def _attn(name, R, nodes, ctx, Hq=40, Hkv=8, D=128, page=64, tree="draft", shared=False, window=0, softcap=0.0):
    """nodes: per request (shared: on average); ctx: the longest request's cached tokens."""
    return {"name": name, "op": "attn", "R": R, "nodes": nodes, "ctx": ctx, "Hq": Hq, "Hkv": Hkv, "D": D,
            "page": page, "tree": tree, "shared": shared, "window": window, "softcap": softcap}


def listed():
    return [
        # one token of one request: between two GEMMs of a decode step, latency is all there is
        _norm("norm, 1 token", 1, 5120),
        # the 256 nodes of a verify pass, the next GEMM reads 8 bits
        _norm("norm, 256 nodes, 8 bit", 256, 5120, out8=True),
        # a long prompt's prefill, odd number of tokens
        _norm("norm, 16383 tokens", 16383, 5120),
        # a tree's nodes: keys stay with the step until acceptance, nothing is written into the cache
        _rope("rope, 256 nodes", 256, 40, 8, 128, 128, append=False),
        # a prompt with images: time / height / width positions, normed heads, written into pages
        _rope("rope, 12345 tokens, 3 axes", 12345, 40, 8, 128, 128, axes=3, qk_norm=True),
        # plain decode of one short request
        _attn("attn, 1 token, 1000 cached", 1, 1, 1000),
        # plain decode of a ragged batch: the cache is what is read
        _attn("attn, 64 x 1 token, 16k", 64, 1, 16384),
        # the usual verify pass: 256 nodes shared by 8 requests
        _attn("attn, 8 requests, 256 nodes", 8, 32, 4096, shared=True),
        # one request with a very long context and a small tree
        _attn("attn, 64 nodes, 128k", 1, 64, 131072),
        # the largest trees: tensor work
        _attn("attn, 8 x 256 nodes, 8k", 8, 256, 8192, page=128),
        # a sliding-window layer with capped scores, small heads, small pages
        _attn("attn, window, capped", 4, 63, 32768, Hq=16, Hkv=4, D=64, page=16, window=4096, softcap=50.0),
        # chains (prompt chunks, one axis of speculation), heads not shared
        _attn("attn, 3 x 200 chained", 3, 200, 3001, Hq=12, Hkv=12, D=128, page=32, tree="chain"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "rope", "attn", "attn"])
    if op == "norm":
        K = rng.choice([5120, 8 * _log(rng, 8, 2176), 8 * _log(rng, 8, 2176), _log(rng, 64, 17408)])
        M = min(_log(rng, 2, 16383), 16383 * 5120 // K)
        c = _norm("", M, K, residual=rng.random() < 0.75, out8=rng.random() < 0.5)
    elif op == "rope":
        D = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        c = _rope("", _log(rng, 1, 12345), Hkv * rng.choice([1, 2, 4, 5]), Hkv, D, rng.choice([D, D, D // 2, D // 4]),
                  axes=rng.choice([1, 2, 3]), append=rng.random() < 0.5, interleaved=rng.random() < 0.3,
                  qk_norm=rng.random() < 0.5, page=rng.choice([16, 32, 64, 128]), top=_log(rng, 100, 131072))
    else:
        D = rng.choice([64, 128, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 4, 5, 7])
        R = _log(rng, 1, 64)
        ctx = min(_log(rng, 1, 131072), (64 * 16384 * 8 * 128) // (R * Hkv * D), 131072)
        most = max(1, min(256, (8 * 256 * 8192 * 40 * 128) // (R * ctx * Hq * D)))
        c = _attn("", R, _log(rng, 1, most), ctx, Hq, Hkv, D, page=rng.choice([16, 32, 64, 128]), shared=rng.random() < 0.3,
                  tree=rng.choice(["draft", "draft", "chain"]), window=rng.choice([0, 0, 0, _log(rng, 1, 8192)]),
                  softcap=rng.choice([0.0, 0.0, 30.0]))
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------
def _ctx_lens(c):
    """Cached tokens of every request, from ctx / 2 to ctx."""
    R, ctx = c["R"], c["ctx"]
    return [ctx - (r * 7919) % (ctx // 2 + 1) for r in range(R)]


def _counts(c):
    """Nodes of every request: all the same, or uneven with the same sum and at most 256."""
    R, m = c["R"], c["nodes"]
    got = [m] * R
    if c["shared"]:
        for r in range(R // 2):
            d = min((m * (r + 1) * 2) // (R + 1), m - 1, 256 - m)
            got[2 * r] -= d
            got[2 * r + 1] += d
    return got


def _tree(c, g):
    """req and parent (index in the whole list, -1: the root) of every node, a parent before its children."""
    counts = _counts(c)
    req = torch.repeat_interleave(torch.arange(c["R"]), torch.tensor(counts))
    if c["shared"]:  # a shared budget's nodes come best first over all requests
        req = req[torch.randperm(len(req), generator=g)]
    pick = torch.rand(len(req), generator=g).tolist()
    seen, depth, parent = {}, [], []
    for i, r in enumerate(req.tolist()):
        mine = seen.setdefault(r, [])
        if not mine:
            p = -1
        elif c["tree"] == "chain":
            p = mine[-1]
        else:  # best-first lists mostly deepen what was just added
            k = int(pick[i] ** 2 * (min(len(mine), 24) + 1))
            p = mine[-1 - k] if k < len(mine) else -1
            if p >= 0 and depth[p] >= 16:
                p = -1
        depth.append(1 if p < 0 else depth[p] + 1)
        parent.append(p)
        mine.append(i)
    return req.to(torch.int32), torch.tensor(parent, dtype=torch.int32)


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    h = torch.Generator()
    h.manual_seed(int(seed))

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * scale).to(torch.bfloat16)

    if c["op"] == "norm":
        s = {"x": normal(c["M"], c["K"]), "weight": (1 + 0.2 * torch.randn(c["K"], generator=g, device=dev)).to(torch.bfloat16)}
        s["residual"] = normal(c["M"], c["K"], scale=3.0) if c["residual"] else None
    elif c["op"] == "rope":
        n, Hq, Hkv, D, half = c["n"], c["Hq"], c["Hkv"], c["D"], c["rot"] // 2
        qkv = normal(n, (Hq + 2 * Hkv) * D)  # the QKV GEMM's output: q, k and v are views of its rows
        s = {"q": qkv[:, :Hq * D].view(n, Hq, D), "k": qkv[:, Hq * D:(Hq + Hkv) * D].view(n, Hkv, D),
             "v": qkv[:, (Hq + Hkv) * D:].view(n, Hkv, D)}
        s["pos"] = torch.randint(0, c["top"], (c["axes"], n), generator=g, device=dev, dtype=torch.int32)
        s["inv_freq"] = 10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float32) / half)
        part = -(-half // c["axes"])
        s["axis"] = [j // part for j in range(half)] if c["axes"] > 1 else None
        s["axis_dev"] = torch.tensor(s["axis"] or [0] * half, device=dev)
        s["q_norm"], s["k_norm"] = (normal(D, scale=0.2) + 1, normal(D, scale=0.2) + 1) if c["qk_norm"] else (None, None)
        if c["append"]:
            pages = -(-n // c["page"]) + 2
            s["kc"] = torch.zeros(pages, c["page"], Hkv, D, dtype=torch.bfloat16, device=dev)
            s["vc"] = torch.zeros_like(s["kc"])
            s["slots"] = torch.randperm(pages * c["page"], generator=g, device=dev)[:n]
        else:
            s["kc"] = s["vc"] = s["slots"] = None
    else:
        R, Hq, Hkv, D, page = c["R"], c["Hq"], c["Hkv"], c["D"], c["page"]
        lens = _ctx_lens(c)
        wide = -(-c["ctx"] // page)
        pages = sum(-(-x // page) for x in lens) + 1
        s = {"kc": normal(pages, page, Hkv, D), "vc": normal(pages, page, Hkv, D)}
        perm = torch.randperm(pages, generator=h).tolist()
        table = torch.zeros(R, wide, dtype=torch.int32)
        at = 0
        for r, x in enumerate(lens):
            m = -(-x // page)
            table[r, :m] = torch.tensor(perm[at:at + m], dtype=torch.int32)
            at += m
        req, parent = _tree(c, h)
        n = len(req)
        s.update(table=table.to(dev), ctx_len=torch.tensor(lens, dtype=torch.int32, device=dev), req=req.to(dev),
                 parent=parent.to(dev), most=max(_counts(c)))
        qkv = normal(n, (Hq + 2 * Hkv) * D)
        s.update(q=qkv[:, :Hq * D].view(n, Hq, D), k=qkv[:, Hq * D:(Hq + Hkv) * D].view(n, Hkv, D),
                 v=qkv[:, (Hq + Hkv) * D:].view(n, Hkv, D))
    s["case"] = c
    return s


# ---------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------
def _plain_norm(s):
    c = s["case"]
    x = s["x"].float()
    if s["residual"] is not None:
        x = x + s["residual"].float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    out = {}
    if s["residual"] is not None:
        out["h"] = x.to(torch.bfloat16)
    if not c["out8"]:
        out["y"] = y.to(torch.bfloat16)
        return out
    M, K = y.shape
    G = -(-K // 128)
    t = torch.nn.functional.pad(y, (0, G * 128 - K)).view(M, G, 128)
    top = t.abs().amax(-1)
    scale = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
    q8 = (t / scale[..., None]).to(torch.float8_e4m3fn).view(M, G * 128)[:, :K]
    out["scale"] = scale
    out["q8"] = q8
    return out


def _rotate(x, cos, sin, rot, interleaved):
    a, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        lo, hi = a[..., 0::2], a[..., 1::2]
        y = torch.stack((lo * cos - hi * sin, hi * cos + lo * sin), -1).flatten(-2)
    else:
        lo, hi = a[..., :rot // 2], a[..., rot // 2:]
        y = torch.cat((lo * cos - hi * sin, hi * cos + lo * sin), -1)
    return torch.cat((y, rest), -1)


def _rope_values(s, kind):
    c = s["case"]
    pos = s["pos"].to(kind)[s["axis_dev"]].t()  # [n, rot / 2]
    angle = (pos * s["inv_freq"].to(kind)).unsqueeze(1)
    cos, sin = angle.cos(), angle.sin()
    q, k = s["q"].to(kind), s["k"].to(kind)
    if c["qk_norm"]:
        q = q * torch.rsqrt((q * q).mean(-1, keepdim=True) + EPS) * s["q_norm"].to(kind)
        k = k * torch.rsqrt((k * k).mean(-1, keepdim=True) + EPS) * s["k_norm"].to(kind)
    return _rotate(q, cos, sin, c["rot"], c["interleaved"]), _rotate(k, cos, sin, c["rot"], c["interleaved"])


def _plain_rope(s):
    c = s["case"]
    q, k = _rope_values(s, torch.float32)
    q, k = q.to(torch.bfloat16), k.to(torch.bfloat16)
    if not c["append"]:
        return {"q": q, "k": k}
    s["kc"].view(-1, c["Hkv"], c["D"])[s["slots"]] = k
    s["vc"].view(-1, c["Hkv"], c["D"])[s["slots"]] = s["v"]
    return {"q": q, "kc": s["kc"], "vc": s["vc"]}


def _plain_attn(s):
    c = s["case"]
    R, N, Hq, Hkv, D, page = c["R"], s["most"], c["Hq"], c["Hkv"], c["D"], c["page"]
    G, T, n, dev = Hq // Hkv, c["ctx"], s["q"].shape[0], s["q"].device
    # nodes by request, padded to N
    req = s["req"].long()
    order = torch.argsort(req, stable=True)
    count = torch.zeros(R, dtype=torch.long, device=dev).scatter_add_(0, req, torch.ones_like(req))
    start = count.cumsum(0) - count
    rank = torch.empty_like(order).scatter_(0, order, torch.arange(n, device=dev) - start[req[order]])
    idx = order[(start[:, None] + torch.arange(N, device=dev)).clamp(max=n - 1)]  # [R, N]
    live = torch.arange(N, device=dev) < count[:, None]
    # who descends from whom: a node's line of ancestors doubles in length with each product
    up = s["parent"].long()[idx]
    line = torch.nn.functional.one_hot(torch.where(live & (up >= 0), rank[up.clamp(min=0)], N), N + 1)[..., :N].float()
    line = line + torch.eye(N, device=dev)
    for _ in range((N - 1).bit_length()):
        line = (line @ line).clamp(max=1.0)
    above = line > 0.5
    depth = above.sum(-1)
    # cached keys and values, padded to T
    t = torch.arange(T, device=dev)
    at = s["table"].long()[:, t // page]
    kc, vc = s["kc"][at, t % page].float(), s["vc"][at, t % page].float()  # [R, T, Hkv, D]
    K = torch.cat((kc, s["k"][idx].float()), 1)
    V = torch.cat((vc, s["v"][idx].float()), 1)
    seen = (t < s["ctx_len"][:, None])[:, None, :].expand(R, N, T)
    tree = above
    if c["window"]:
        here = s["ctx_len"][:, None] + depth - 1
        seen = seen & (here[..., None] - t < c["window"])
        tree = tree & (depth[:, :, None] - depth[:, None, :] < c["window"])
    mask = torch.cat((seen, tree), 2)  # [R, N, T + N]
    q = s["q"][idx].float().view(R, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(R, Hkv, N * G, D)
    x = (q @ K.permute(0, 2, 3, 1)) * (D ** -0.5)
    if c["softcap"]:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    x = x.view(R, Hkv, N, G, T + N).masked_fill(~mask[:, None, :, None, :], float("-inf"))
    p = torch.exp(x - x.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    o = p.view(R, Hkv, N * G, T + N) @ V.permute(0, 2, 1, 3)
    o = o.view(R, Hkv, N, G, D).permute(0, 2, 1, 3, 4).reshape(R * N, Hq, D)
    return o[req * N + rank].to(torch.bfloat16)


# ---------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------
def run(state):
    s = state
    c = s["case"]
    if not own:
        return {"norm": _plain_norm, "rope": _plain_rope, "attn": _plain_attn}[c["op"]](s)
    import lossless_bit_weight_02_gb300 as w12

    if c["op"] == "norm":
        r = w12.w12_rmsnorm(s["x"], s["weight"], eps=EPS, residual=s["residual"], out8=c["out8"])
        out = {"h": r["h"]} if c["residual"] else {}
        if c["out8"]:
            out["scale"] = r["scale"]
            out["q8"] = r["q8"]
        else:
            out["y"] = r["y"]
        return out
    if c["op"] == "rope":
        cache = w12.KvCache(s["kc"], s["vc"]) if c["append"] else None
        q, k = w12.w12_rope_append(s["q"], s["k"], s["pos"], s["inv_freq"], axis=s["axis"],
                                   interleaved=c["interleaved"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS,
                                   v=s["v"] if c["append"] else None, cache=cache, slots=s["slots"])
        return {"q": q, "kc": s["kc"], "vc": s["vc"]} if c["append"] else {"q": q, "k": k}
    return w12.w12_tree_attn(s["q"], s["k"], s["v"], w12.KvCache(s["kc"], s["vc"]), s["table"], s["ctx_len"],
                             s["parent"], s["req"], window=c["window"], softcap=c["softcap"])


def work(case):
    c = case
    if c["op"] == "norm":
        M, K = c["M"], c["K"]
        out = K + 4 * -(-K // 128) if c["out8"] else 2 * K
        return {"bytes": M * (2 * K + (4 * K if c["residual"] else 0) + out) + 2 * K, "flops": 5 * M * K}
    if c["op"] == "rope":
        heads = 2 * (c["Hq"] + c["Hkv"]) + (2 * c["Hkv"] if c["append"] else 0)
        return {"bytes": c["n"] * (heads * c["D"] * 2 + 4 * c["axes"] + (8 if c["append"] else 0)),
                "flops": c["n"] * (c["Hq"] + c["Hkv"]) * (3 * c["rot"] + (4 * c["D"] if c["qk_norm"] else 0))}
    n = keys = pairs = 0
    for x, m in zip(_ctx_lens(c), _counts(c)):
        seen = min(x, c["window"]) if c["window"] else x
        n += m
        keys += seen + m
        above = (m + 1) / 2 if c["tree"] == "chain" else min(m, 8)
        pairs += m * (seen + (min(above, c["window"]) if c["window"] else above))
    return {"bytes": 4 * n * c["Hq"] * c["D"] + 4 * keys * c["Hkv"] * c["D"] + 4 * -(-keys // c["page"]) + 8 * n,
            "flops": int(4 * pairs * c["Hq"] * c["D"])}


# ---------------------------------------------------------------------------------------------------
# 64 bits
# ---------------------------------------------------------------------------------------------------
def _exact_attn(s):
    """Request by request and head by head, the ancestors of a node walked up one by one."""
    c = s["case"]
    D, G, page = c["D"], c["Hq"] // c["Hkv"], c["page"]
    req, parent = s["req"].tolist(), s["parent"].tolist()
    out = torch.zeros(len(req), c["Hq"], D, dtype=torch.float64, device=s["q"].device)
    for r in range(c["R"]):
        mine = [i for i, x in enumerate(req) if x == r]
        if not mine:
            continue
        place = {i: j for j, i in enumerate(mine)}
        L, m = int(s["ctx_len"][r]), len(mine)
        lines = []
        for i in mine:
            line, at = [], i
            while at >= 0:
                line.append(place[at])
                at = parent[at]
            lines.append(line)
        see = torch.zeros(m, L + m, dtype=torch.bool)
        for j, line in enumerate(lines):
            pos = L + len(line) - 1
            first = max(0, pos - c["window"] + 1) if c["window"] else 0
            see[j, first:L] = True
            for up in (line[:c["window"]] if c["window"] else line):
                see[j, L + up] = True
        see = see.to(out.device)
        tok = torch.arange(L, device=out.device)
        at = s["table"][r].long()[tok // page]
        rows = torch.tensor(mine, device=out.device)
        for h in range(c["Hkv"]):
            K = torch.cat((s["kc"][at, tok % page, h], s["k"][rows, h])).double()
            V = torch.cat((s["vc"][at, tok % page, h], s["v"][rows, h])).double()
            for g in range(G):
                x = s["q"][rows, h * G + g].double() @ K.t() / math.sqrt(D)
                if c["softcap"]:
                    x = c["softcap"] * torch.tanh(x / c["softcap"])
                x = torch.where(see, x, torch.full_like(x, -math.inf))
                out[rows, h * G + g] = torch.softmax(x, -1) @ V
    return out


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "norm":
        x = s["x"].double()
        if s["residual"] is not None:
            x = x + s["residual"].double()
        y = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / c["K"] + EPS) * s["weight"].double()
        out = {"h": x} if c["residual"] else {}
        if not c["out8"]:
            out["y"] = y
            return out
        scale = torch.stack([y[:, k:k + 128].abs().max(1).values for k in range(0, c["K"], 128)], 1) / E4M3_MAX
        out["scale"] = torch.where(scale > 0, scale, torch.ones_like(scale))
        out["q8"] = y / out["scale"].repeat_interleave(128, 1)[:, :c["K"]]
        return out
    if c["op"] == "attn":
        return _exact_attn(s)
    half = c["rot"] // 2
    z = {}
    for name, w in (("q", s["q_norm"]), ("k", s["k_norm"])):
        x = s[name].double()
        if w is not None:
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / c["D"] + EPS) * w.double()
        x = x.clone()
        for j in range(half):
            a, b = (2 * j, 2 * j + 1) if c["interleaved"] else (j, j + half)
            turn = s["pos"][s["axis"][j] if s["axis"] else 0].double() * s["inv_freq"][j].double()
            turned = torch.complex(x[..., a], x[..., b]) * torch.exp(1j * turn)[:, None]
            x[..., a], x[..., b] = turned.real, turned.imag
        z[name] = x
    if not c["append"]:
        return z
    for name, old, new in (("kc", s["kc"], z["k"]), ("vc", s["vc"], s["v"])):
        full = old.double().view(-1, c["Hkv"], c["D"])
        full[s["slots"]] = new.double()
        z[name] = full.view_as(old)
    return {"q": z["q"], "kc": z["kc"], "vc": z["vc"]}
