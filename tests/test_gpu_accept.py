"""w12_tree_accept against the rule in 64 bits, request by request."""
import math

import pytest
import torch

import lossless_bit_weight_02_gb300 as w12
import step_ref as ref

pytestmark = pytest.mark.gpu


def make(R, nodes, V, seed, dtype=torch.bfloat16, drawn=False, wide=3, temps=(0.8,), shared_q=True, deep=16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.Generator().manual_seed(seed)
    n = R * nodes
    req = torch.arange(R).repeat_interleave(nodes)[torch.randperm(n, generator=h)].tolist()
    pick = torch.rand(n, generator=h).tolist()
    parent, depth, kids, seen = [], {}, {}, [[-1] for _ in range(R)]
    for i, r in enumerate(req):
        p = seen[r][-1 - int(pick[i] * min(4, len(seen[r])))]
        parent.append(p)
        kids[r, p] = kids.get((r, p), 0) + 1
        if kids[r, p] >= wide:
            seen[r].remove(p)
        depth[i] = 1 if p < 0 else depth[p] + 1
        if depth[i] < deep:
            seen[r].append(i)
        if not seen[r]:
            seen[r].append(-1)
    logits = torch.randn(n + R, V, generator=g, device="cuda") * 2.5
    up = torch.tensor([p if p >= 0 else n + r for p, r in zip(parent, req)], device="cuda")
    draft = draft_row = None
    if drawn:
        rows, at = torch.unique(up, return_inverse=True) if shared_q else (up, torch.arange(n, device="cuda"))
        draft = torch.softmax(logits[rows] + 0.7 * torch.randn(len(rows), V, generator=g, device="cuda"), -1)
        token = torch.multinomial(draft[at], 1, generator=g)[:, 0]
        draft_row = at.int()
    else:
        token = torch.randint(0, V, (n,), generator=g, device="cuda")
        logits[up, token] = math.log(V) + 1.5 + 3 * torch.rand(n, generator=g, device="cuda")
    t = torch.tensor([temps[r % len(temps)] for r in range(R)], device="cuda")
    return dict(logits=logits.to(dtype), token=token.int(), parent=torch.tensor(parent, dtype=torch.int32, device="cuda"),
                req=torch.tensor(req, dtype=torch.int32, device="cuda"), temperature=t,
                uniform=torch.rand(n, generator=g, device="cuda"),
                noise=torch.empty(R, V, device="cuda").exponential_(generator=g).clamp_(min=1e-30), draft=draft,
                draft_row=draft_row)


def expected(s, R, **kw):
    lst = lambda t: t.tolist() if t is not None else None  # noqa: E731
    return ref.accept(s["logits"].cpu().float(), lst(s["token"]), lst(s["parent"]), lst(s["req"]), R,
                      s["temperature"].tolist() if isinstance(s["temperature"], torch.Tensor) else [s["temperature"]] * R,
                      lst(s["uniform"]), s["noise"].cpu() if s["noise"] is not None else None,
                      s["draft"].cpu() if s["draft"] is not None else None, lst(s["draft_row"]), **kw)


def check(got, want, most_close=0.1):
    close = 0
    for r, (path, nxt, margin) in enumerate(want):
        mine = got["nodes"][r].tolist()
        same = (int(got["count"][r]), mine[:len(path)], int(got["next"][r])) == (len(path), path, nxt)
        assert mine[int(got["count"][r]):] == [-1] * (len(mine) - int(got["count"][r]))
        if margin < ref.MARGIN:
            close += 1
            continue
        assert same, (r, mine, int(got["next"][r]), path, nxt, margin)
    assert close <= max(1, most_close * len(want)), close


@pytest.mark.parametrize("R,nodes,V", [(1, 1, 1000), (1, 4, 32000), (3, 20, 517), (8, 32, 50001), (40, 7, 4097), (2, 256, 9000), (5, 3, 131072),
                                       (2, 5, 200003)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("temps", [(0.0,), (0.7,), (0.0, 1.0, 0.6)])
def test_given_tokens(w12lib, R, nodes, V, dtype, temps):
    s = make(R, nodes, V, 11 * R + nodes, dtype, temps=temps)
    check(w12.w12_tree_accept(**s), expected(s, R))


@pytest.mark.parametrize("R,nodes,V,wide,shared", [(1, 1, 1000, 1, True), (64, 5, 1003, 1, True), (6, 20, 50001, 3, True),
                                                   (6, 20, 5000, 4, False), (3, 12, 70000, 2, True), (9, 16, 300, 16, True)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_drawn_tokens(w12lib, R, nodes, V, wide, shared, dtype):
    s = make(R, nodes, V, 7 * R + nodes, dtype, drawn=True, wide=wide, temps=(1.0, 0.9, 0.0), shared_q=shared)
    check(w12.w12_tree_accept(**s), expected(s, R))


@pytest.mark.parametrize("V,pad,off", [(1000, 24, 8), (1001, 6, 3), (777, 0, 1), (5, 3, 2), (1, 1, 0), (8192, 8, 0), (4099, 2, 5)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_anywhere(w12lib, V, pad, off, dtype):
    """Rows that begin on any element, in another order than the nodes, between rows of NaN."""
    R, nodes = 4, 6
    s = make(R, nodes, V, V, dtype, temps=(0.0, 0.8))
    m = s["logits"].shape[0]
    for name in ("logits", "noise"):
        t = s[name]
        wide = torch.full((t.shape[0], V + pad + off), float("nan"), dtype=t.dtype, device="cuda")
        wide[:, off:off + V] = t
        s[name] = wide[:, off:off + V]
    order = torch.randperm(m, generator=torch.Generator().manual_seed(V))
    logits = torch.full((m + 3, V + pad + off), float("nan"), dtype=dtype, device="cuda")[:, off:off + V]
    logits[order.cuda()] = s["logits"]
    row, root = order[:R * nodes].int().cuda(), order[R * nodes:].int().cuda()
    want = expected(s, R)
    check(w12.w12_tree_accept(**{**s, "logits": logits}, row=row, root_row=root), want, 0.5)


@pytest.mark.parametrize("deep", [1, 3, 64, 256])
def test_depths(w12lib, deep):
    """A long chain of tokens that are nearly certain; the walk ends at max_depth."""
    n, V = 200, 600
    s = make(1, n, V, 5, wide=1, deep=1000)
    s["parent"] = torch.arange(-1, n - 1, dtype=torch.int32, device="cuda")
    s["logits"] = torch.zeros(n + 1, V, device="cuda").bfloat16()
    s["logits"][n, s["token"][0].long()] = 30.0
    s["logits"][torch.arange(n - 1), s["token"][1:].long()] = 30.0
    got = w12.w12_tree_accept(**s, max_depth=deep)
    m = min(deep, n)
    assert got["count"].tolist() == [m] and got["nodes"][0, :m].tolist() == list(range(m))
    check(got, expected(s, 1, max_depth=deep))


def test_infinities(w12lib):
    """-inf is never drawn, +inf always; a row of nothing but -inf is uniform."""
    V = 3000
    s = make(4, 3, V, 9, torch.float32, temps=(0.8, 0.0, 1.0, 1.2))
    n = 12
    s["logits"][n:, ::2] = -math.inf
    s["logits"][:n, 1::2] = -math.inf
    s["logits"][n + 2, 77] = math.inf
    s["logits"][n + 3] = -math.inf
    check(w12.w12_tree_accept(**s), expected(s, 4), 0.5)


def test_certain_and_impossible(w12lib):
    """u = 0 accepts what has any probability; a token of none is refused; two children of all the mass: one is taken."""
    V = 1000
    lg = torch.full((4 + 1, V), -math.inf, device="cuda")
    lg[4, 5], lg[4, 6] = 0.0, 0.0
    lg[0:4, 9] = 1.0
    tok = torch.tensor([5, 6, 5, 6], dtype=torch.int32, device="cuda")
    par = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    noise = torch.ones(1, V, device="cuda")
    almost = 1 - 2.0 ** -24
    for u in ([0.0] * 4, [almost] * 4, [almost, 0.0, 0.0, 0.0]):
        got = w12.w12_tree_accept(lg, tok, par, temperature=1.0, uniform=torch.tensor(u, device="cuda"), noise=noise)
        assert got["count"].tolist() == [1] and got["next"].tolist() == [9]
        assert got["nodes"][0, 0].item() == (0 if u[0] == 0 else 1)
    tok2 = torch.tensor([7, 8, 9, 7], dtype=torch.int32, device="cuda")
    got = w12.w12_tree_accept(lg, tok2, par, temperature=1.0, uniform=torch.zeros(4, device="cuda"), noise=noise)
    assert got["count"].tolist() == [0] and got["next"].tolist() == [5]


def test_no_nodes(w12lib):
    V = 5000
    lg = torch.randn(3, V, device="cuda")
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    got = w12.w12_tree_accept(lg, e, e, temperature=0)
    assert got["count"].tolist() == [0, 0, 0] and got["next"].tolist() == lg.argmax(-1).tolist()
    noise = torch.empty(3, V, device="cuda").exponential_()
    got = w12.w12_tree_accept(lg, e, e, temperature=1.0, noise=noise)
    assert got["next"].tolist() == (lg.double().softmax(-1) / noise.double()).argmax(-1).tolist()


def test_argmax_takes_the_lowest(w12lib):
    lg = torch.zeros(2, 70001, device="cuda").bfloat16()
    lg[0, [69999, 33000, 40000]] = 2.0
    tok = torch.tensor([0], dtype=torch.int32, device="cuda")
    par = torch.tensor([-1], dtype=torch.int32, device="cuda")
    got = w12.w12_tree_accept(lg, tok, par, temperature=0)
    assert got["count"].tolist() == [1] and got["next"].tolist() == [33000]


def test_rules(w12lib):
    """A request that breaks a rule gets -1; the others what they get alone."""
    R, nodes, V = 9, 5, 2000
    s = make(R, nodes, V, 21, temps=(0.8, 0.0))
    want = expected(s, R)
    who = lambda r: (s["req"] == r).nonzero()[:, 0].tolist()  # noqa: E731
    s["row"] = torch.arange(R * nodes, dtype=torch.int32, device="cuda")
    s["root_row"] = torch.arange(R * nodes, R * nodes + R, dtype=torch.int32, device="cuda")
    s["parent"][who(1)[3]] = who(2)[0] if who(2)[0] < who(1)[3] else -7
    s["token"][who(3)[1]] = V
    s["row"][who(4)[4]] = R * nodes + R
    s["root_row"][5] = -1
    s["parent"][who(6)[0]] = who(6)[0]
    s["token"][who(7)[2]] = -1
    stray = who(8)[4]
    s["req"][stray] = R + 3  # belongs to nobody
    s8 = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    got = w12.w12_tree_accept(**s)
    for r in (1, 3, 4, 5, 6, 7):
        assert got["count"][r] == -1 and got["next"][r] == -1 and (got["nodes"][r] == -1).all()
    keep = [0, 2]
    check({k: v[keep] for k, v in got.items()}, [want[r] for r in keep], 0.5)
    if not (s8["parent"] == stray).any():
        del s8["row"], s8["root_row"]
        s8["token"] = s8["token"].clamp(0, V - 1)
        want8 = expected(s8, R)[8]
        check({k: v[8:9] for k, v in got.items()}, [want8], 1.0)


def test_too_many_nodes(w12lib):
    V, n = 300, 257
    lg = torch.zeros(n + 2, V, device="cuda")
    tok = torch.zeros(n, dtype=torch.int32, device="cuda")
    par = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    req = torch.zeros(n, dtype=torch.int32, device="cuda")
    got = w12.w12_tree_accept(lg, tok, par, req, temperature=0)
    assert got["count"].tolist() == [-1, 0]
    req[100] = 1
    got = w12.w12_tree_accept(lg, tok, par, req, temperature=0)
    assert got["count"].tolist() == [1, 1]


def test_law(w12lib):
    """Over many random numbers the first token has the target's distribution, whatever was drafted."""
    V, R = 12, 20000
    g = torch.Generator(device="cuda").manual_seed(3)
    row = torch.randn(V, generator=g, device="cuda") * 1.5
    p = torch.softmax(row.double(), -1)
    q = torch.softmax(torch.randn(V, generator=g, device="cuda"), -1)
    for drawn in (False, True):
        n = 2 * R
        tok = torch.multinomial(q, n, replacement=True, generator=g).int() if drawn else torch.tensor([2, 7], device="cuda").int().repeat(R)
        got = w12.w12_tree_accept(
            row.expand(2, V).contiguous(), tok, torch.full((n,), -1, dtype=torch.int32, device="cuda"),
            torch.arange(R, device="cuda").repeat_interleave(2).int(), uniform=torch.rand(n, generator=g, device="cuda"),
            noise=torch.empty(R, V, device="cuda").exponential_(generator=g), draft=q[None].contiguous() if drawn else None,
            draft_row=torch.zeros(n, dtype=torch.int32, device="cuda") if drawn else None,
            row=torch.zeros(n, dtype=torch.int32, device="cuda"), root_row=torch.ones(R, dtype=torch.int32, device="cuda"), max_depth=1)
        first = torch.where(got["count"] > 0, tok[got["nodes"][:, 0].clamp(min=0).long()], got["next"])
        seen = torch.bincount(first.long(), minlength=V).double() / R
        # five standard deviations of a count of R draws
        assert ((seen - p).abs() <= 5 * (p * (1 - p) / R).sqrt() + 1e-9).all(), (drawn, seen, p)


def test_streams_graphs_and_repeats(w12lib):
    s = make(8, 32, 20000, 2, temps=(0.8, 0.0))
    a = w12.w12_tree_accept(**s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = w12.w12_tree_accept(**s, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = w12.w12_tree_accept(**s)
    graph.replay()
    torch.cuda.synchronize()
    for k in a:
        assert torch.equal(a[k], b[k]) and torch.equal(a[k], c[k])
    s2 = make(8, 32, 20000, 3, temps=(0.8, 0.0))
    for k in ("logits", "token", "uniform", "noise", "parent", "req"):
        s[k].copy_(s2[k])
    graph.replay()
    d = w12.w12_tree_accept(**s)
    for k in a:
        assert torch.equal(c[k], d[k])
