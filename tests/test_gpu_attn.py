"""w12_tree_attn against softmax attention in 64 bits, one row at a time.

Requests with more than 16 rows (nodes times heads of a group) per key/value
head on average take the tcgen05 kernel, the others the kernel for few rows;
every shape here says which by its sizes.
"""
import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def make_tree(counts, kind, mixed, g):
    """(req, parent) of every node: "chain", "flat" or "tree"; mixed: the requests' nodes interleaved."""
    req = [r for r, c in enumerate(counts) for _ in range(c)]
    if mixed:
        req = [req[i] for i in torch.randperm(len(req), generator=g).tolist()]
    seen, parent = {}, []
    for i, r in enumerate(req):
        mine = seen.setdefault(r, [])
        pick = int(torch.randint(0, min(len(mine), 9) + 1, (1,), generator=g))
        parent.append(-1 if not mine or kind == "flat" else mine[-1] if kind == "chain" else
                      mine[-1 - pick] if pick < len(mine) else -1)
        mine.append(i)
    return torch.tensor(req, dtype=torch.int32), torch.tensor(parent, dtype=torch.int32)


def case(counts, ctx, Hq, Hkv, D, page, kind="tree", mixed=False, head_major=False, seed=1, gain=1.0, junk=NAN):
    """Inputs of a call; every cached slot and table entry that no request owns holds junk."""
    gc = torch.Generator().manual_seed(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    req, parent = make_tree(counts, kind, mixed, gc)
    n, R = len(req), len(ctx)
    need = [(c + page - 1) // page for c in ctx]
    width, pages = max(need) + 2, sum(need) + 3
    table = torch.full((R, width), -12345, dtype=torch.int32)
    perm = torch.randperm(pages, generator=gc).int()
    shape = (pages, Hkv, page, D) if head_major else (pages, page, Hkv, D)
    kc, vc = (torch.full(shape, junk, device="cuda").bfloat16() for _ in range(2))
    if head_major:
        kc, vc = kc.permute(0, 2, 1, 3), vc.permute(0, 2, 1, 3)
    at = 0
    for r, c in enumerate(ctx):
        mine = perm[at:at + need[r]]
        at += need[r]
        table[r, :need[r]] = mine
        for j, p in enumerate(mine.tolist()):
            m = min(page, c - j * page)
            kc[p, :m] = torch.randn(m, Hkv, D, generator=g, device="cuda").bfloat16()
            vc[p, :m] = torch.randn(m, Hkv, D, generator=g, device="cuda").bfloat16()
    qkv = torch.randn(n, (Hq + 2 * Hkv) * D, generator=g, device="cuda").bfloat16()
    q = (qkv[:, :Hq * D] * gain).contiguous() if gain != 1.0 else qkv[:, :Hq * D]  # rows of the wider buffer
    return dict(q=q.view(n, Hq, D), k=qkv[:, Hq * D:(Hq + Hkv) * D].view(n, Hkv, D),
                v=qkv[:, (Hq + Hkv) * D:].view(n, Hkv, D), kc=kc, vc=vc, table=table.cuda(),
                ctx=torch.tensor(ctx, dtype=torch.int32, device="cuda"), parent=parent.cuda(), req=req.cuda())


def run(w, c, **kw):
    return w.w12_tree_attn(c["q"], c["k"], c["v"], w.KvCache(c["kc"], c["vc"]), c["table"], c["ctx"], c["parent"],
                           c["req"], **kw)


def want(c, **kw):
    return ref.tree_attn(c["q"], c["k"], c["v"], c["kc"], c["vc"], c["table"], c["ctx"], c["parent"], c["req"], **kw)


def check(w, c, **kw):
    o = run(w, c, **kw)
    assert w.default_attn_workspace(torch.device("cuda", 0)).status() == w.W12_OK
    x, mag = want(c, **kw)
    assert not o.isnan().any()
    assert ref.attn_failures(o, x, mag) == 0
    return o


FEW = [  # at most 16 rows per key/value head on average
    # counts, ctx, Hq, Hkv, D, page, kind
    ([1], [0], 1, 1, 64, 16, "flat"),
    ([1], [1], 8, 1, 128, 1, "flat"),
    ([1], [1000], 40, 8, 128, 64, "flat"),
    ([1] * 7, [63, 64, 65, 0, 1, 127, 3001], 10, 2, 128, 16, "flat"),
    ([1] * 5, [15, 16, 17, 500, 4097], 16, 1, 64, 24, "flat"),
    ([3, 0, 2, 0, 1], [100, 7, 0, 900, 33], 4, 2, 64, 8, "tree"),
    ([16], [77], 2, 2, 128, 5, "chain"),
    ([2, 3, 1], [700, 20, 129], 5, 1, 128, 128, "tree"),
]
MANY = [  # the tcgen05 kernel
    ([17], [0], 1, 1, 64, 16, "tree"),
    ([64], [1], 5, 1, 128, 64, "tree"),
    ([33], [127], 8, 2, 64, 16, "chain"),
    ([200], [128], 2, 2, 128, 32, "chain"),
    ([256], [129], 7, 1, 128, 128, "tree"),
    ([256, 1, 0, 100], [300, 5000, 640, 0], 10, 2, 128, 256, "tree"),
    ([40, 41], [1000, 77], 12, 4, 64, 1, "tree"),
    ([26, 30], [517, 383], 6, 2, 128, 24, "flat"),
    ([129], [256], 1, 1, 128, 96, "chain"),     # one row beyond a tile: the second stream nearly empty
    ([20], [2000], 72, 1, 64, 48, "tree"),      # a group wider than a copy of queries
    ([3], [700], 256, 2, 128, 16, "chain"),
]


@pytest.mark.parametrize("extra", [{}, {"window": 1}, {"window": 40}, {"window": 100000}, {"softcap": 5.0},
                                   {"window": 130, "softcap": 30.0, "scale": 0.25}],
                         ids=["plain", "w1", "w40", "wide", "cap", "all"])
@pytest.mark.parametrize("shape", FEW + MANY, ids=[f"few{i}" for i in range(len(FEW))] +
                         [f"many{i}" for i in range(len(MANY))])
def test_attention(shape, extra, w12lib):
    counts, ctx, Hq, Hkv, D, page, kind = shape
    check(w12lib, case(counts, ctx, Hq, Hkv, D, page, kind), **extra)


@pytest.mark.parametrize("counts,Hq,Hkv", [([30, 50, 9], 10, 2), ([4, 3, 2], 3, 3), ([256, 255, 250], 4, 4)])
@pytest.mark.parametrize("head_major", [False, True])
@pytest.mark.parametrize("mixed", [False, True])
def test_orders_and_layouts(counts, Hq, Hkv, head_major, mixed, w12lib):
    """Nodes in any order over the requests, both orders of a page."""
    check(w12lib, case(counts, [300, 0, 65], Hq, Hkv, 128, 16, "tree", mixed, head_major, junk=INF))


@pytest.mark.parametrize("counts,ctx,Hq,Hkv,D", [
    ([100, 37, 129, 1, 60, 90], [3000, 2500, 2049, 2700, 1000, 3100], 16, 8, 64),    # enough work for an item's end
    ([140, 30, 256], [3000, 2900, 2049], 16, 8, 128),                                # to count in the cut of the work
    ([1] * 600, [(7 * r) % 90 for r in range(600)], 4, 2, 64),                       # more requests than a CTA has
    ([2, 0, 3] * 180, [(11 * r) % 150 for r in range(540)], 16, 1, 64),              # threads, and than it keeps at hand
])
def test_much_work_and_many_requests(counts, ctx, Hq, Hkv, D, w12lib):
    c = case(counts, ctx, Hq, Hkv, D, 32, mixed=len(counts) > 100)
    o = check(w12lib, c)
    assert torch.equal(run(w12lib, c, max_ctas=37), o)


@pytest.mark.parametrize("page", [100, 512])
def test_wide_groups_and_long_pages(page, w12lib):
    """A group wider than an item's rows; pages longer than a block, of a size that is no power of two."""
    check(w12lib, case([2, 3], [700, 1100], 300, 1, 64, page))


def test_plain_decode(w12lib):
    """parent None: every node a child of the root; req None: request 0."""
    c = case([1] * 9, [9 * i * i for i in range(9)], 10, 2, 128, 16)
    c["parent"] = None
    check(w12lib, c)
    c = case([1], [333], 10, 2, 64, 16)
    c["parent"] = c["req"] = None
    check(w12lib, c)
    c = case([40], [333], 10, 2, 64, 16, "flat")
    c["parent"] = c["req"] = None
    check(w12lib, c)


@pytest.mark.parametrize("shape", [FEW[3], MANY[5]])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_large_scores(shape, softcap, w12lib):
    """Softmax weights that span all of FP32 (scores up to some hundreds): the running maximum has to follow.
    A score's FP32 error grows with it: 2^-17 of up to 700 and then that of the exponential."""
    counts, ctx, Hq, Hkv, D, page, kind = shape
    c = case(counts, ctx, Hq, Hkv, D, page, kind, gain=40.0)
    o = run(w12lib, c, softcap=softcap)
    x, mag = want(c, softcap=softcap)
    assert ((o.double() - x).abs() <= (2 * ref.BF + 700 * 2.0 ** -17) * mag + 2 * ref.BF * x.abs()).all()


@pytest.mark.parametrize("D,nodes", [(64, 60), (128, 60), (128, 2)])
def test_values_that_are_not_finite(D, nodes, w12lib):
    """NaN and Inf in a node's or a slot's K and V reach the rows that see them and no others."""
    c = case([nodes, nodes], [100, 70], 5, 1, D, 16, "tree")
    base = run(w12lib, c, window=50)
    bad = nodes // 2  # a node of request 0
    for name, value, cols in (("k", NAN, slice(3, 4)), ("v", NAN, slice(3, 4)), ("v", INF, slice(0, 7))):
        d = {n: t.clone() for n, t in c.items()}
        d[name][bad, :, cols] = value
        o = run(w12lib, d, window=50)
        par, sees = c["parent"].tolist(), set()
        for i in range(2 * nodes):
            j, steps = i, 0
            while j >= 0 and j != bad:
                j, steps = par[j], steps + 1
            if j == bad and steps < 50:
                sees.add(i)
        rest = [i for i in range(2 * nodes) if i not in sees]
        assert torch.equal(o[rest], base[rest])
        x, mag = want(d, window=50)
        finite = x.isfinite()
        assert torch.equal(o.isfinite(), finite) and finite[rest].all() and not finite[sorted(sees)].all()
        assert ref.attn_failures(o[finite], x[finite], mag[finite]) == 0
    # a cached slot that the window hides from the deeper nodes
    d = {n: t.clone() for n, t in c.items()}
    t = 100 - 49  # position 51: seen by nodes of depth 1 only (first key ctx + d - 50)
    d["vc"][int(c["table"][0, t // 16]), t % 16, :, :] = INF
    o = run(w12lib, d, window=50)
    deep = [i for i in range(nodes) if c["parent"][i] >= 0] + list(range(nodes, 2 * nodes))
    top = [i for i in range(nodes) if c["parent"][i] < 0]
    assert torch.equal(o[deep], base[deep]) and not o[top].isfinite().any()


@pytest.mark.parametrize("nodes", [3, 70])
def test_errors_found_on_the_device(nodes, w12lib):
    """A bad tree, length or page: NaN for what it touches, the right answers for the rest, and a status."""
    dev = torch.device("cuda", 0)
    ws = w12lib.default_attn_workspace(dev)
    c = case([nodes, nodes, nodes], [200, 100, 90], 5, 1, 128, 16, "chain")
    good, mag = want(c)  # (a request in error also moves the cut of the work, so not the same bits)
    first = run(w12lib, c)
    one = slice(nodes, 2 * nodes)  # request 1
    keep = [i for i in range(3 * nodes) if not nodes <= i < 2 * nodes]

    def right(o, i):
        return ref.attn_failures(o, good[i], mag[i]) == 0

    def broken(**change):
        d = {n: t.clone() for n, t in c.items()}
        for name, (at, value) in change.items():
            d[name][at] = value
        o = run(w12lib, d)
        assert ws.status() == w12lib.W12_ERR_INVALID
        assert right(o[keep], keep)
        return o[one]

    assert broken(ctx=(1, -1)).isnan().all()
    assert broken(ctx=(1, c["table"].shape[1] * 16 + 1)).isnan().all()
    assert broken(table=((1, 2), -1)).isnan().all()
    assert broken(table=((1, 0), c["kc"].shape[0])).isnan().all()
    for value in (nodes + 1, 2 * nodes, 0, -2, 3 * nodes + 5, 2 ** 31 - 1, -2 ** 31):  # of node 1 of request 1
        o = broken(parent=(nodes + 1, value))
        assert o[1:].isnan().all() and right(o[0], nodes)
    o = broken(req=(nodes + 1, 3))  # no such request; its children lose their parent
    assert o[1:].isnan().all() and right(o[0], nodes)
    assert broken(req=(nodes + 1, -1))[1:].isnan().all()
    # the next call is clean again, and the status with it
    assert torch.equal(run(w12lib, c), first) and ws.status() == w12lib.W12_OK


def test_more_nodes_than_a_request_may_have(w12lib):
    c = case([257, 3], [50, 60], 2, 1, 64, 16, "flat")
    o = run(w12lib, c)
    assert w12lib.default_attn_workspace(torch.device("cuda", 0)).status() == w12lib.W12_ERR_INVALID
    assert o[:257].isnan().all()
    x, mag = want({**c, "q": c["q"][257:], "k": c["k"][257:], "v": c["v"][257:], "parent": c["parent"][257:],
                   "req": c["req"][257:]})
    assert ref.attn_failures(o[257:], x, mag) == 0


@pytest.mark.parametrize("shape", [FEW[3], FEW[5], MANY[5], MANY[6]])
def test_same_bits(shape, w12lib):
    """Twice, on smaller grids, with the plan of the last call, into a wider buffer: the same bits."""
    counts, ctx, Hq, Hkv, D, page, kind = shape
    c = case(counts, ctx, Hq, Hkv, D, page, kind)
    ws = w12lib.AttnWorkspace("cuda")
    first = run(w12lib, c, workspace=ws)
    assert torch.equal(run(w12lib, c, workspace=ws), first)
    for ctas in (1, 3, 100):
        assert torch.equal(run(w12lib, c, workspace=ws, max_ctas=ctas), first)
    # another layer: the plan stays, queries, nodes and cache change
    d = {n: t.clone() if t.dim() > 2 else t for n, t in c.items()}
    d["q"] = c["q"].flip(0).contiguous()
    d["q"] = torch.cat((d["q"].flatten(1), c["k"].flatten(1), c["v"].flatten(1)), 1)[:, :Hq * D].view(-1, Hq, D)
    d["k"], d["v"] = c["k"], c["v"]
    plain = run(w12lib, d)
    assert torch.equal(run(w12lib, d, workspace=ws, reuse_plan=True), plain)
    wide = torch.full((len(c["req"]), Hq * D + 8), 7.0, device="cuda").bfloat16()
    out = run(w12lib, c, workspace=ws, out=wide[:, :Hq * D].view(-1, Hq, D))
    assert torch.equal(out, first) and (wide[:, Hq * D:] == 7).all()


def test_a_row_does_not_depend_on_its_siblings(w12lib):
    """The first 40 nodes' rows are within the bounds with and without 60 more of them."""
    c = case([100], [500], 4, 1, 128, 16, "tree")
    x, mag = want(c)
    part = {n: (t[:40] if n in ("q", "k", "v", "parent", "req") else t) for n, t in c.items()}
    assert ref.attn_failures(run(w12lib, c), x, mag) == 0
    assert ref.attn_failures(run(w12lib, part), x[:40], mag[:40]) == 0


@pytest.mark.parametrize("counts", [[1, 1], [60, 50]])
def test_other_stream_and_graph(counts, w12lib):
    c = case(counts, [500, 300], 10, 2, 128, 16)
    first = run(w12lib, c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = run(w12lib, c, stream=s)
    s.synchronize()
    assert torch.equal(got, first)
    ws = w12lib.AttnWorkspace("cuda")
    out = torch.empty_like(first)
    with torch.cuda.stream(s):
        run(w12lib, c, out=out, workspace=ws)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        run(w12lib, c, out=out, workspace=ws)
    c["q"].mul_(0.5)
    c["ctx"].sub_(40)  # lengths and trees are read on the device: a captured call follows them
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, run(w12lib, c))


@pytest.mark.parametrize("nodes", [1, 30])
def test_offsets_beyond_32_bits(nodes, w12lib):
    """Pages 2^30 + 2^12 elements apart: the last ones begin beyond 2^32 bytes and 2^31 elements."""
    c = case([nodes], [100], 5, 1, 128, 32)
    pages, page, H, D = c["kc"].shape
    stride = (1 << 30) + 4096
    buf = torch.empty((pages - 1) * stride + 2 * page * D, dtype=torch.bfloat16, device="cuda")
    far = []
    for at, t in ((0, c["kc"]), (page * D, c["vc"])):
        f = torch.as_strided(buf, (pages, page, H, D), (stride, D, D, 1), at)
        f.copy_(t)
        far.append(f)
    first = run(w12lib, c)
    c["kc"], c["vc"] = far
    assert torch.equal(run(w12lib, c), first)
    # and the append to the last page
    slots = torch.arange(nodes, device="cuda") % page + (pages - 1) * page
    w12lib.w12_kv_append(c["k"], c["v"], w12lib.KvCache(*far), slots)
    m = min(nodes, page)
    assert torch.equal(far[0][pages - 1, :m], c["k"][:m]) and torch.equal(far[1][pages - 1, :m], c["v"][:m])


@pytest.mark.parametrize("counts,D", [([40, 30], 128), ([200], 64)])
def test_stalled_wait_reports_timeout_and_the_next_call_is_right(counts, D, w12lib, monkeypatch):
    """With W12_ATTN_TEST_STALL the queries never come: the bounded waits give up (about a second), the call
    ends, the status says so once, and the next call on the workspace is right."""
    c = case(counts, [700, 90][:len(counts)], 10, 2, D, 16)
    ws = w12lib.AttnWorkspace("cuda")
    first = run(w12lib, c, workspace=ws)
    with monkeypatch.context() as m:
        m.setattr(w12lib, "W12_ATTN_REUSE_PLAN", w12lib.W12_ATTN_TEST_STALL)  # the flag that reuse_plan passes
        run(w12lib, c, workspace=ws, reuse_plan=True)
    assert ws.status() == w12lib.W12_ERR_TIMEOUT
    assert ws.status() == w12lib.W12_OK
    assert torch.equal(run(w12lib, c, workspace=ws), first) and ws.status() == w12lib.W12_OK


def test_no_nodes(w12lib):
    c = case([1], [10], 4, 2, 64, 16)
    none = {n: (t[:0] if n in ("q", "k", "v", "parent", "req") else t) for n, t in c.items()}
    assert run(w12lib, none).shape == (0, 4, 64)


def test_refusals(w12lib):
    c = case([2, 2], [10, 20], 4, 2, 64, 16)

    def call(**change):
        return run(w12lib, {**c, **{n: t for n, t in change.items() if n in c}},
                   **{n: t for n, t in change.items() if n not in c})

    for change in ({"q": c["q"].float()}, {"q": c["q"].flatten(1)}, {"q": c["q"][:, :3].contiguous()},
                   {"k": c["k"][:3]}, {"v": c["v"].half()}, {"table": c["table"].long()}, {"ctx": c["ctx"][:1]},
                   {"parent": c["parent"].long()}, {"req": c["req"][:3]}, {"out": torch.empty_like(c["k"])},
                   {"workspace": w12lib.AttnWorkspace("cuda"), "reuse_plan": True}):
        with pytest.raises(ValueError):
            call(**change)
    for change in ({"scale": -1.0}, {"softcap": -1.0}, {"softcap": 2000.0}, {"window": -1}, {"max_ctas": -1},
                   {"scale": NAN}, {"softcap": NAN}):
        with pytest.raises(w12lib.W12Error) as e:
            call(**change)
        assert e.value.status == w12lib.W12_ERR_INVALID
    odd = torch.zeros(4, 4 * 64 + 4, device="cuda").bfloat16()[:, 4:].view(4, 4, 64)
    with pytest.raises(w12lib.W12Error) as e:
        call(q=odd)
    assert e.value.status == w12lib.W12_ERR_ALIGN
    wide = torch.zeros(2, 16, 2, 96, device="cuda").bfloat16()
    with pytest.raises(w12lib.W12Error):
        call(q=torch.zeros(4, 4, 96, device="cuda").bfloat16(), k=torch.zeros(4, 2, 96, device="cuda").bfloat16(),
             v=torch.zeros(4, 2, 96, device="cuda").bfloat16(), kc=wide, vc=wide.clone())
