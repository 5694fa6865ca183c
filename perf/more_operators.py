"""The operators that end a verify step of a hybrid model and carry its recurrent layers on, as cases to be measured.

  accept  verification of drafted tokens against the target's probabilities, from given random numbers: how far down
          its draft tree each request goes, and the token that follows
  scan    the gated delta rule over sequences of any length with the state read and written: prompts in chunks, one
          token a request, or the accepted nodes of a tree

With `own` the framework's entry points are called; without it the same mathematics runs as elementary torch
operations.  Heads are those of the recurrent layers that the tree operator serves: 32 of 128, or of 64.
"""
import math

import torch

own = False

CHUNK = 64  # tokens of a chunk of the plain form


# ---------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------
def _scan(name, R, tokens, H=32, Hk=16, D=128, out32=False, nodes=0, fresh=False):
    """tokens: the longest request's (nodes > 0: of the accepted nodes among so many); fresh: states of zero."""
    return {"name": name, "op": "scan", "R": R, "tokens": tokens, "H": H, "Hk": Hk, "D": D, "out32": out32,
            "nodes": nodes, "fresh": fresh}


def _accept(name, R, nodes, V, draft="none", logits32=False, temp="one", wide=4):
    """nodes: of a request; draft: none (the tree's tokens are given), drawn (each drawn from its row of
    probabilities); temp: one, mixed (some requests greedy), zero; wide: most children of a node (1: chains)."""
    return {"name": name, "op": "accept", "R": R, "nodes": nodes, "V": V, "draft": draft, "logits32": logits32,
            "temp": temp, "wide": wide}


def listed():
    return [
        # decode of one request: a state is read and written, latency counts
        _scan("scan, 1 token", 1, 1),
        # decode of a batch: the states are what is moved
        _scan("scan, 64 x 1 token", 64, 1),
        # after a verify pass: the states go on along the accepted nodes of 8 requests' trees, no outputs
        _scan("scan, accepted nodes", 8, 12, Hk=32, nodes=256),
        # prefill of one long prompt, odd length, from nothing
        _scan("scan, 8191 tokens", 1, 8191, fresh=True),
        # a ragged batch of prompts that go on from a state
        _scan("scan, 16 x 1999 tokens", 16, 1999),
        # heads of 64, outputs in 32 bits, heads not shared
        _scan("scan, 3 x 1000, heads of 64", 3, 1000, H=16, Hk=16, D=64, out32=True),
        # a large prefill: four long prompts
        _scan("scan, 4 x 8192 tokens", 4, 8192),
        # one request, a short chain, greedy: latency
        _accept("accept, chain of 4, greedy", 1, 4, 32000, temp="zero", wide=1),
        # the usual verify pass: 256 nodes of 8 requests, best-first trees
        _accept("accept, 8 x 32 nodes", 8, 32, 131072),
        # chains drawn from the drafter's probabilities
        _accept("accept, 64 chains of 7, drawn", 64, 7, 131072, draft="drawn", wide=1),
        # trees whose siblings are drawn from one row of probabilities, odd vocabulary
        _accept("accept, 4 x 40 nodes, drawn", 4, 40, 50001, draft="drawn", wide=3),
        # a large batch, logits in 32 bits, greedy and sampled requests
        _accept("accept, 32 x 64 nodes, mixed", 32, 64, 100003, logits32=True, temp="mixed", wide=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.6:
        D = rng.choice([64, 128, 128])
        Hk = rng.choice([1, 2, 4, 8, 16])
        H = Hk * rng.choice([1, 1, 2, 3])
        R = _log(rng, 1, 64)
        kind = rng.choice(["few", "long", "long", "nodes"])
        if kind == "nodes":
            return _strip(_scan("", min(R, 32), rng.randint(1, 16), H, Hk, D, nodes=32 * min(R, 32)))
        most = max(1, (4 * 8192 * 32 * 128) // (R * H * D))
        tokens = min(rng.randint(1, 16) if kind == "few" else _log(rng, 17, 8192), most)
        return _strip(_scan("", R, tokens, H, Hk, D, out32=rng.random() < 0.3, fresh=rng.random() < 0.3))
    R = _log(rng, 1, 64)
    V = min(_log(rng, 1000, 131072), (64 * 131072) // R)
    draft = rng.choice(["none", "none", "drawn"])
    nodes = _log(rng, 1, 256 if draft == "none" else 48)
    while (nodes + 1) * R * V > 32 * 65 * 100003:
        nodes = max(1, nodes // 2)
    return _strip(_accept("", R, nodes, V, draft=draft, logits32=rng.random() < 0.4,
                          temp=rng.choice(["one", "one", "mixed", "zero"]) if draft == "none" else rng.choice(["one", "mixed"]),
                          wide=rng.choice([1, 2, 4, 8] if draft == "none" else [1, 1, 2, 3])))


def _strip(c):
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------
def _lens(c):
    """Tokens of every request, from half of the longest to the longest (the largest prefill: all the same)."""
    R, L = c["R"], c["tokens"]
    if c["op"] == "scan" and L % 64 == 0 and R > 1:
        return [L] * R
    return [L - (r * 7919) % (L // 2 + 1) for r in range(R)]


def _unit(x):
    return x / (x * x).sum(-1, keepdim=True).sqrt()


def _prepare_scan(c, g, h, dev):
    R, H, Hk, D = c["R"], c["H"], c["Hk"], c["D"]
    lens = _lens(c)
    n = c["nodes"] or sum(lens)
    bf = torch.bfloat16

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    # queries and keys of unit length (they were normalised and scaled before), neighbours alike
    drift = _unit(normal(Hk, D))
    q = (_unit(normal(n, Hk, D)) * D ** -0.5).to(bf)
    k = _unit(normal(n, Hk, D) * D ** -0.5 + 0.5 * drift).to(bf)
    s = {"q": q, "k": k, "v": normal(n, H, D).to(bf), "lens": lens}
    # decays from a rate of each head and a step of each token, most close to 1; write strengths in (0, 1)
    rate = torch.exp(normal(H) * 1.2 - 2.5)
    s["alpha"] = torch.exp(-rate * torch.nn.functional.softplus(normal(n, H)))
    s["beta"] = torch.sigmoid(normal(n, H))
    s["S"] = torch.zeros(R, H, D, D, device=dev) if c["fresh"] else normal(R, H, D, D) * 0.3
    s["S_new"] = torch.empty_like(s["S"])
    if c["nodes"]:
        rows = torch.full((R, 16), -1, dtype=torch.int32)
        perm = torch.randperm(n, generator=h)
        for r, m in enumerate(lens):  # accepted nodes: somewhere in the list of all trees, a parent before its child
            rows[r, :m] = perm[r * (n // R):r * (n // R) + m].sort().values.int()
        s["rows"], s["count"] = rows.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev)
        s["most"] = 16
    else:
        s["start"] = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).to(torch.int32).to(dev)
        s["out"] = torch.empty(n, H, D, dtype=torch.float32 if c["out32"] else bf, device=dev)
        s["most"] = max(lens)
    return s


def _trees(c, h):
    """Parents (index in the whole list, -1: the root) and requests of every node, a request's nodes in best-first
    order and the requests' lists mixed; a node has at most `wide` children and stands at most 16 deep."""
    R, m, wide = c["R"], c["nodes"], c["wide"]
    req = torch.arange(R).repeat_interleave(m)
    if wide > 1:
        req = req[torch.randperm(R * m, generator=h)]
    pick = torch.rand(R * m, generator=h).tolist()
    seen = [[-1] for _ in range(R)]  # who may still have a child
    kids, depth, parent = {}, {}, []
    for i, r in enumerate(req.tolist()):
        mine = seen[r]
        p = mine[-1 - int(pick[i] ** 2 * min(len(mine), 12))]
        parent.append(p)
        kids[r, p] = kids.get((r, p), 0) + 1
        if kids[r, p] >= wide:
            mine.remove(p)
        depth[i] = 1 + depth.get(p, 0) if p >= 0 else 1
        if depth[i] < 16:
            mine.append(i)
        if not mine:  # a chain that is as deep as it may be: another from the root
            mine.append(-1)
            kids[r, -1] = 0
    return req.to(torch.int32), torch.tensor(parent, dtype=torch.int32)


def _prepare_accept(c, g, h, dev):
    R, m, V = c["R"], c["nodes"], c["V"]
    n = R * m
    req, parent = _trees(c, h)
    up = torch.where(parent >= 0, parent, n + req).long().to(dev)  # the row that a node's token was drafted for
    kind = torch.float32 if c["logits32"] else torch.bfloat16
    logits = torch.randn(n + R, V, generator=g, device=dev).mul_(2.5)
    s = {"req": req.to(dev), "parent": parent.to(dev)}
    if c["draft"] == "drawn":
        # a row of the drafter's probabilities for every row that has children: near the target's
        rows, at = torch.unique(up, return_inverse=True)
        q = torch.empty(len(rows), V, device=dev)
        token = torch.empty(n, dtype=torch.int64, device=dev)
        for i in range(0, len(rows), 64):
            x = logits[rows[i:i + 64]] + 0.7 * torch.randn(len(rows[i:i + 64]), V, generator=g, device=dev)
            x = torch.exp(x - x.amax(-1, keepdim=True))
            q[i:i + 64] = x / x.sum(-1, keepdim=True)
        for i in range(0, n, 64):
            token[i:i + 64] = torch.multinomial(q[at[i:i + 64]], 1, generator=g)[:, 0]
        s["draft"], s["draft_row"] = q, at.to(torch.int32)
    else:
        # the drafter's best candidates: tokens that have a good part of the target's probability
        token = torch.randint(0, V, (n,), generator=g, device=dev)
        like = math.log(V) + 3.1 - 2.5 + 3.0 * torch.rand(n, generator=g, device=dev)
        logits[up, token] = like
        s["draft"] = s["draft_row"] = None
    s["logits"], s["token"] = logits.to(kind), token.to(torch.int32)
    s["uniform"] = torch.rand(n, generator=g, device=dev)
    s["noise"] = torch.empty(R, V, device=dev).exponential_(generator=g).clamp_(min=1e-30)
    t = torch.full((R,), 0.8, device=dev)
    if c["temp"] == "mixed":
        t = torch.where(torch.arange(R, device=dev) % 3 == 0, torch.zeros_like(t), 0.6 + 0.1 * (torch.arange(R, device=dev) % 5))
    elif c["temp"] == "zero":
        t = torch.zeros_like(t)
    s["temperature"] = t
    return s


def prepare(case, seed):
    dev = torch.device("cuda" if torch.cuda.is_available() else "cpu")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    h = torch.Generator()
    h.manual_seed(int(seed))
    s = (_prepare_scan if case["op"] == "scan" else _prepare_accept)(case, g, h, dev)
    s["case"] = case
    return s


# ---------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------
def _inverse(A):
    """(I + A)^-1 of strictly lower triangular A [..., C, C], C a power of two: blocks of twice the size each time."""
    C = A.shape[-1]
    T = torch.eye(C, device=A.device, dtype=A.dtype).expand_as(A).clone()
    half = 1
    while half < C:
        blocks = A.unflatten(-2, (-1, 2, half)).unflatten(-1, (-1, 2, half))  # [..., nb, 2, half, nb, 2, half]
        low = blocks.diagonal(0, -6, -3)[..., 1, :, 0, :, :].movedim(-1, -3)  # [..., nb, half, half]
        Tb = T.unflatten(-2, (-1, 2, half)).unflatten(-1, (-1, 2, half)).diagonal(0, -6, -3)
        hi, lo = Tb[..., 1, :, 1, :, :].movedim(-1, -3), Tb[..., 0, :, 0, :, :].movedim(-1, -3)
        Tb[..., 1, :, 0, :, :] = -(hi @ low @ lo).movedim(-3, -1)
        half *= 2
    return T


def _plain_scan(s):
    c = s["case"]
    R, H, Hk, D, most = c["R"], c["H"], c["Hk"], c["D"], s["most"]
    dev = s["q"].device
    C = min(CHUNK, 1 << (most - 1).bit_length())
    L = -(-most // C) * C
    t = torch.arange(L, device=dev)
    if c["nodes"]:
        live = t < s["count"][:, None]
        at = torch.nn.functional.pad(s["rows"].long(), (0, L - s["rows"].shape[1])).clamp(min=0)
    else:
        live = t < (s["start"][1:] - s["start"][:-1])[:, None]
        at = (s["start"][:-1].long()[:, None] + t).clamp(max=s["q"].shape[0] - 1)
    cut = lambda x: x[at].float() * live[..., None, None]  # noqa: E731  [R, L, heads, D]
    chunks = lambda x: x.unflatten(1, (-1, C)).movedim(3, 1)  # noqa: E731  [R, H, chunks, C, ...]
    k = chunks(cut(s["k"]).repeat_interleave(H // Hk, 2))
    v = chunks(cut(s["v"]))
    beta = chunks(s["beta"][at] * live[..., None])
    log_a = torch.where(live[..., None], s["alpha"][at].double().log().clamp(min=-200.0), 0.0)
    cum = chunks(log_a).cumsum(-1)  # products of decays as sums, in 64 bits
    gamma = cum.exp().float()
    low = torch.ones(C, C, device=dev, dtype=torch.bool).tril()
    G = torch.where(low, (cum[..., :, None] - cum[..., None, :]).clamp(max=80.0), -torch.inf).exp().float()
    to_end = (cum[..., -1:] - cum).exp().float()
    A = (beta[..., None] * G * (k @ k.transpose(-1, -2))).tril(-1)
    T = _inverse(A) * beta[..., None, :]
    want = not c["nodes"]
    if want:
        q = chunks(cut(s["q"]).repeat_interleave(H // Hk, 2))
        M = G * (q @ k.transpose(-1, -2))
    S = s["S"].clone()
    out = []
    for i in range(L // C):
        St = S.transpose(-1, -2)
        f = T[:, :, i] @ (v[:, :, i] - gamma[:, :, i, :, None] * (k[:, :, i] @ St))
        if want:
            out.append(gamma[:, :, i, :, None] * (q[:, :, i] @ St) + M[:, :, i] @ f)
        S = gamma[:, :, i, -1, None, None] * S + (f * to_end[:, :, i, :, None]).transpose(-1, -2) @ k[:, :, i]
    if not want:
        return {"S": S}
    o = torch.stack(out, 2).movedim(1, 3).flatten(0, 2)  # [R * L, H, D]
    row = torch.arange(s["out"].shape[0], device=dev)
    of = torch.searchsorted(s["start"][1:], row, right=True)
    return {"o": o[of * L + row - s["start"].long()[of]].to(s["out"].dtype), "S": S}


def _plain_accept(s):
    """All requests one step at a time: the row of where each stands, then its children in their order.  Comparisons
    and the sums below them in 64 bits: a token is accepted or not on the last bit."""
    c = s["case"]
    R, n, V, dev = c["R"], c["R"] * c["nodes"], c["V"], s["logits"].device
    req, parent, token = s["req"].long(), s["parent"].long(), s["token"].long()
    deep = min(16, c["nodes"])
    # children of every place (node, or n + request: its root) in the order of the list
    place = torch.where(parent >= 0, parent, n + req)
    order = torch.argsort(place, stable=True)
    first = torch.searchsorted(place[order], torch.arange(n + R + 1, device=dev))
    wide = c["wide"] if c["wide"] > 1 else -(-c["nodes"] // 16)
    here = n + torch.arange(R, device=dev)
    going = torch.ones(R, dtype=torch.bool, device=dev)
    count = torch.zeros(R, dtype=torch.int32, device=dev)
    nodes = torch.full((R, 16), -1, dtype=torch.int32, device=dev)
    greedy = s["temperature"] == 0
    temp = torch.where(greedy, 1.0, s["temperature"]).double()[:, None]
    every = torch.arange(R, device=dev)
    left = torch.zeros(R, V, dtype=torch.float64, device=dev)
    best = torch.zeros(R, dtype=torch.int64, device=dev)
    for d in range(deep + 1):
        row = s["logits"][here].float()
        top = row.argmax(-1)  # the first of equal ones
        x = row.double() / temp
        p = torch.exp(x - x.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
        taken = torch.full((R,), -1, dtype=torch.int64, device=dev)
        for j in range(wide if d < deep else 0):
            i = first[here] + j
            child = order[i.clamp(max=n - 1)]
            there = (i < first[here + 1]) & (taken < 0)
            y = token[child]
            if s["draft"] is None:
                q, qy = None, 1.0
            else:
                q = s["draft"][s["draft_row"][child].long()].double()
                qy = q[every, y]
            ok = torch.where(greedy, y == top, s["uniform"][child].double() * qy < p[every, y])
            taken = torch.where(there & ok, child, taken)
            # what is left of p after a refusal
            if q is None:
                rest = p.clone()
                rest[every, y] = 0.0
            else:
                rest = (p - q).clamp(min=0.0)
            total = rest.sum(-1, keepdim=True)
            rest = torch.where(total > 0, rest / total, p)
            p = torch.where((there & ~ok)[:, None], rest, p)
        goes = going & (taken >= 0)
        stops = going & (taken < 0)
        left = torch.where(stops[:, None], p, left)
        best = torch.where(stops, top, best)
        nodes[:, min(d, 15)] = torch.where(goes, taken.to(torch.int32), nodes[:, min(d, 15)])
        count = count + goes.to(torch.int32)
        here = torch.where(goes, taken, here)
        going = goes
    drawn = (left / s["noise"].double()).argmax(-1)
    return {"count": count, "nodes": nodes, "next": torch.where(greedy, best, drawn).to(torch.int32)}


# ---------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------
def run(state):
    s = state
    c = s["case"]
    if not own:
        return (_plain_scan if c["op"] == "scan" else _plain_accept)(s)
    import lossless_bit_weight_02_gb300 as w12

    if c["op"] == "accept":
        return w12.w12_tree_accept(s["logits"], s["token"], s["parent"], s["req"], temperature=s["temperature"],
                                   uniform=s["uniform"], noise=s["noise"], draft=s["draft"], draft_row=s["draft_row"])
    if c["nodes"]:
        _, S = w12.w12_gdn_scan(s["S"], None, s["k"], s["v"], s["alpha"], s["beta"], rows=s["rows"], count=s["count"],
                                S_out=s["S_new"])
        return {"S": S}
    o, S = w12.w12_gdn_scan(s["S"], s["q"], s["k"], s["v"], s["alpha"], s["beta"], start=s["start"], S_out=s["S_new"],
                            out=s["out"])
    return {"o": o, "S": S}


def work(case):
    c = case
    if c["op"] == "accept":
        # a request reads the row of where it begins, of where it ends and, here, of one between; noise where it is drawn
        R, V = c["R"], c["V"]
        rows = R * min(3, c["nodes"] + 1)
        drawn = {"one": R, "mixed": R - -(-R // 3), "zero": 0}[c["temp"]]
        read = rows * V * (4 if c["logits32"] else 2) + drawn * V * 4
        read += R * V * 4 if c["draft"] == "drawn" else 0
        return {"bytes": read + 16 * R * c["nodes"], "flops": 4 * rows * V}
    lens = _lens(c)
    n, H, D = sum(lens), c["H"], c["D"]
    states = 2 * c["R"] * H * D * D * 4
    rows = n * (2 * c["Hk"] * D + 2 * H * D + 8 * H)  # keys, values, decays and strengths
    if not c["nodes"]:
        rows += n * (2 * c["Hk"] * D + (4 if c["out32"] else 2) * H * D)
    return {"bytes": states + rows, "flops": n * H * D * D * (4 if c["nodes"] else 6)}


# ---------------------------------------------------------------------------------------------------
# 64 bits
# ---------------------------------------------------------------------------------------------------
def exact(case, seed):
    c = case
    if c["op"] == "accept":
        return None  # tokens and nodes are chosen, not computed
    s = prepare(case, seed)
    lens, S = s["lens"], s["S"].double()
    dev, reps = S.device, c["H"] // c["Hk"]
    begin = [0]
    for m in lens:
        begin.append(begin[-1] + m)
    o = None if c["nodes"] else torch.zeros(s["q"].shape[0], c["H"], c["D"], dtype=torch.float64, device=dev)
    heads = torch.arange(c["H"], device=dev) // reps
    lens_dev, begin_dev = torch.tensor(lens, device=dev), torch.tensor(begin[:-1], device=dev)
    sure = min(lens)  # tokens that every request has
    for t in range(max(lens)):  # token by token, as the rule is written
        who = None if t < sure else torch.nonzero(lens_dev > t)[:, 0]
        if who is None:
            at = s["rows"][:, t].long() if c["nodes"] else begin_dev + t
            now = S
        else:
            at = s["rows"][who, t].long() if c["nodes"] else begin_dev[who] + t
            now = S[who]
        key, val = s["k"][at][:, heads].double(), s["v"][at].double()
        a, b = s["alpha"][at].double()[..., None, None], s["beta"][at].double()[..., None]
        now = now * a
        wrong = val - (now * key[:, :, None, :]).sum(-1)
        now = now + (b * wrong)[..., None] * key[:, :, None, :]
        if who is None:
            S = now
        else:
            S[who] = now
        if o is not None:
            o[at] = (now * s["q"][at][:, heads].double()[:, :, None, :]).sum(-1)
    return {"S": S} if c["nodes"] else {"o": o, "S": S}
