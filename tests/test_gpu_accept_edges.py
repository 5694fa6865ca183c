"""w12_tree_accept at its edges: nothing drafted, rows with NaN, draws that rounding leaves nothing of, waits that give up."""
import pytest
import torch

import lossless_bit_weight_02_gb300 as w12

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
