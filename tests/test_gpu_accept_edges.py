"""w12_tree_accept at its edges: nothing drafted, rows with NaN, draws that rounding leaves nothing of, waits that give up."""
import pytest
import torch

import lossless_bit_weight_02_gb300 as w12
import step_ref as ref
from test_gpu_accept import expected, make

pytestmark = pytest.mark.gpu


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("R", [1, 3, 200])
def test_no_nodes_behind_large_trees(w12lib, R):
    """Without nodes a call is a plain draw, whatever the call before left in shared memory: trees of 200 nodes, all of
    them children of the root, on every multiprocessor."""
    V, nodes, big = 5000, 200, 608
    g = torch.Generator(device="cuda").manual_seed(R)
    n = big * nodes
    row = torch.zeros(n, dtype=torch.int32, device="cuda")
    lg = torch.randn(2, V, generator=g, device="cuda")
    before = dict(token=torch.randint(0, V, (n,), generator=g, device="cuda").int(), parent=row - 1,
                  req=torch.arange(big, device="cuda").repeat_interleave(nodes).int(), row=row,
                  root_row=torch.ones(big, dtype=torch.int32, device="cuda"))
    noise = torch.empty(R, V, device="cuda").exponential_(generator=g).clamp_(min=1e-30)
    x = torch.randn(R, V, generator=g, device="cuda")
    e = ints()
    # an exact draw: the two highest scores of every row lie further apart than FP32 moves them
    score = x.double().softmax(-1) / noise.double()
    top = score.topk(2, -1).values
    sure = (top[:, 0] - top[:, 1]) > 2.0 ** -14 * top[:, 0]
    assert sure.any()
    for _ in range(20):
        w12.w12_tree_accept(lg, temperature=0, **before)
        got = w12.w12_tree_accept(x, e, e, temperature=0)
        assert (got["count"] == 0).all() and (got["nodes"] == -1).all() and torch.equal(got["next"].long(), x.argmax(-1))
        w12.w12_tree_accept(lg, temperature=0, **before)
        got = w12.w12_tree_accept(x, e, e, temperature=1.0, noise=noise)
        assert (got["count"] == 0).all() and (got["nodes"] == -1).all()
        assert torch.equal(got["next"].long()[sure], score.argmax(-1)[sure])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [0.0, 1.0])
@pytest.mark.parametrize("beside", ["finite", "masked", "inf"])
@pytest.mark.parametrize("at", [0, 1500, 3000])
@pytest.mark.parametrize("drawn", [False, True])
@pytest.mark.parametrize("R", [1, 20])
def test_nan_accepts_nothing(w12lib, dtype, T, beside, at, drawn, R):
    """A row with a NaN accepts none of its children, whatever else is in it; places above it are not affected."""
    V, n = 3001, 2 * R
    row = torch.zeros(V, device="cuda")
    if beside == "masked":
        row[:] = -float("inf")
    row[[7, 1501]] = 1.0
    row[7] = float("inf") if beside == "inf" else 5.0
    good, bad = row.clone(), row.clone()
    bad[at] = float("nan")
    tok, par = ints(*[7] * n), ints(*[x for r in range(R) for x in (-1, 2 * r)])
    kw = dict(req=torch.arange(R, device="cuda").repeat_interleave(2).int(), temperature=T,
              uniform=torch.zeros(n, device="cuda"), noise=torch.ones(R, V, device="cuda"))
    if drawn:
        q = torch.zeros(1, V, device="cuda")
        q[0, 7] = 1.0
        kw.update(draft=q, draft_row=ints(*[0] * n))
    for lg, count in (([bad, bad], 0), ([good, bad], 1), ([good, good], 2)):
        got = w12.w12_tree_accept(torch.stack(lg[1:] + lg[:1]).to(dtype), tok, par, **kw, max_depth=3,
                                  row=ints(*[0] * n), root_row=ints(*[1] * R))
        want = [[2 * r, 2 * r + 1][:count] + [-1] * (3 - count) for r in range(R)]
        assert got["count"].tolist() == [count] * R and got["nodes"].tolist() == want
        assert ((got["next"] >= 0) & (got["next"] < V)).all()
        if count == 2:
            assert (got["next"] == 7).all()


@pytest.mark.parametrize("T", [0.0, 1.0])
def test_nothing_drafted_with_a_draft(w12lib, T):
    """A step in which no request drafted a node takes the drafter's tensors all the same, rows or none in them."""
    V, R = 1000, 3
    g = torch.Generator(device="cuda").manual_seed(1)
    x, noise = torch.randn(R, V, generator=g, device="cuda"), torch.empty(R, V, device="cuda").exponential_(generator=g)
    e, u = ints(), torch.zeros(0, device="cuda")
    want = w12.w12_tree_accept(x, e, e, temperature=T, uniform=u, noise=noise)
    for rows in (0, 4):
        got = w12.w12_tree_accept(x, e, e, e, T, u, noise, draft=torch.full((rows, V), 1.0 / V, device="cuda"), draft_row=e, row=e)
        assert all(torch.equal(got[k], want[k]) for k in want)


@pytest.mark.parametrize("V", [5, 7, 12, 60])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_nothing_left_by_rounding(w12lib, V, dtype):
    """Every token is a child and is refused, which only rounding can bring about: V equal probabilities, taken off one
    after the other, leave more than the last one.  The draw is from p as it was, the lowest of equal scores."""
    step = next(s for s in (3, 5, 7) if V % s)
    for order in (range(V - 1, -1, -1), range(V), [(step * i + 1) % V for i in range(V)]):
        order = list(order)
        assert sorted(order) == list(range(V))
        kw = dict(uniform=torch.full((V,), 1 - 2.0 ** -24, device="cuda"))
        lg = torch.zeros(V + 1, V, device="cuda", dtype=dtype)
        noise = torch.ones(1, V, device="cuda")
        got = w12.w12_tree_accept(lg, ints(*order), ints(*[-1] * V), noise=noise, **kw)
        assert got["count"].tolist() == [0] and got["next"].tolist() == [0]
        noise[0, [1, V - 1]] = 0.5
        got = w12.w12_tree_accept(lg, ints(*order), ints(*[-1] * V), noise=noise, **kw)
        assert got["count"].tolist() == [0] and got["next"].tolist() == [1]


@pytest.mark.parametrize("how", ["greedy", "proposed", "drawn"])
@pytest.mark.parametrize("R", [1, 3, 20])
def test_a_wait_runs_out(w12lib, how, R):
    """The numbers of one warp of a cluster never come, at the second place of the walk: its waits give up after about a
    second, the request gets -1 everywhere, the node accepted before among them, and the next call is right."""
    V, n = 20000, 3 * R
    tok = ints(*[9] * n)
    par = ints(*[x for r in range(R) for x in (-1, 3 * r, 3 * r + 1)])
    lg = torch.zeros(n + R, V, device="cuda")
    lg[:, 9] = 30.0
    kw = dict(req=torch.arange(R, device="cuda").repeat_interleave(3).int(), temperature=0.0 if how == "greedy" else 1.0,
              uniform=torch.zeros(n, device="cuda"), noise=torch.ones(R, V, device="cuda"))
    if how == "drawn":
        kw.update(draft=torch.full((1, V), 1.0 / V, device="cuda"), draft_row=ints(*[0] * n))
    for stall in (0, w12.W12_ACCEPT_TEST_STALL, 0):
        old = torch.full((R, 5), 77, dtype=torch.int32, device="cuda")  # what the outputs' memory may hold
        del old
        got = w12.w12_tree_accept(lg, tok, par, **kw, max_depth=5 | stall)
        nodes = [[-1] * 5 if stall else [3 * r, 3 * r + 1, 3 * r + 2, -1, -1] for r in range(R)]
        assert got["nodes"].tolist() == nodes
        assert got["count"].tolist() == [-1 if stall else 3] * R and got["next"].tolist() == [-1 if stall else 9] * R


@pytest.mark.parametrize("nodes,V,drawn", [(1, 1000, False), (4, 32000, False), (1, 1000, True), (5, 1003, True), (20, 517, False), (12, 70000, True)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_one_request(w12lib, nodes, V, drawn, dtype):
    """A request alone, over ten seeds: nearly all of them are decided by more than the arithmetic's error, and those
    are compared."""
    compared = 0
    for seed in range(10):
        s = make(1, nodes, V, 100 + seed, dtype, drawn=drawn, wide=2, temps=(0.9,))
        path, nxt, margin = expected(s, 1)[0]
        got = w12.w12_tree_accept(**s)
        if margin >= ref.MARGIN:
            compared += 1
            assert got["nodes"][0].tolist() == path + [-1] * (16 - len(path))
            assert (int(got["count"]), int(got["next"])) == (len(path), nxt)
    assert compared >= 8, compared
