"""Values that are not finite, seen with a weight that underflows: one rule in
both kernels and in whole and masked blocks."""
import pytest
import torch

from test_gpu_attn import case, run, want
import layer_ref as ref

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("value", [INF, -INF, NAN])
@pytest.mark.parametrize("at", ["whole", "masked", "node"])
@pytest.mark.parametrize("nodes,D", [(1, 64), (3, 128), (3, 64), (40, 128), (40, 64)])
def test_seen_with_a_weight_that_underflows(nodes, D, at, value, w12lib):
    """The last node's score is 700 and more above every other, whose weights are 0 in FP32.  A seen value that is not
    finite makes its column of the row not finite all the same, and nothing else."""
    if at == "node" and nodes == 1:
        pytest.skip("one node sees no other")
    c = case([nodes], [300], 5, 1, D, 16, "chain")
    c = {n: t.clone() for n, t in c.items()}
    c["q"].fill_(8.0)
    c["kc"].copy_(torch.where(c["kc"].isnan(), c["kc"], 0.0))
    c["k"].zero_()
    c["k"][-1] = 90.0 / D ** 0.5  # score 8 * 90 = 720
    clean = run(w12lib, c)
    x, mag = want(c)
    assert clean.isfinite().all() and ref.attn_failures(clean, x, mag) == 0
    d = {n: t.clone() for n, t in c.items()}
    # few rows walk blocks of 16 keys, many rows of 128: 5 and 299 lie in a whole block and in the masked one of either
    if at == "node":
        d["v"][0, :, 3:5] = value
    else:
        t = 5 if at == "whole" else 299
        d["vc"][int(c["table"][0, t // 16]), t % 16, :, 3:5] = value
    o = run(w12lib, d)
    last = nodes - 1
    hit = torch.zeros(D, dtype=torch.bool, device="cuda")
    hit[3:5] = True
    assert not o[last][:, hit].isfinite().any()
    assert torch.equal(o[last][:, ~hit], clean[last][:, ~hit])
    assert not o[:, :, hit].isfinite().any() and o[:, :, ~hit].isfinite().all()  # every row of the chain sees it
