"""The attention tests that count failures against the 64-bit formula, once
more with a count in which NaN is a failure (a comparison with NaN is false, so
layer_ref.attn_failures passes over it)."""
import os
import sys

import pytest
import torch

import layer_ref as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
count = ref.attn_failures


def failures(o, want, mag):
    """Entries of o beyond the bound, and NaN where the formula has a number."""
    return count(o, want, mag) + (o.isnan() & ~want.isnan()).sum().item()


def test_nan_is_a_failure():
    want, mag = torch.randn(3, 2, 64, dtype=torch.float64), torch.ones(3, 2, 64, dtype=torch.float64)
    assert failures(want.bfloat16(), want, mag) == 0
    assert failures(torch.full_like(want, float("nan")), want, mag) == want.numel()
    o = want.bfloat16()
    o[1, 0, 5] = float("nan")
    o[2, 1, 7] = float("inf")
    assert failures(o, want, mag) == 2


@pytest.fixture(autouse=True)
def nan_counts(monkeypatch):
    monkeypatch.setattr(ref, "attn_failures", failures)


@pytest.mark.gpu
class TestAttention:
    @pytest.mark.parametrize("nodes", [3, 70])
    def test_errors_found_on_the_device(self, nodes, w12lib):
        import test_gpu_attn as t
        t.test_errors_found_on_the_device(nodes, w12lib)

    def test_more_nodes_than_a_request_may_have(self, w12lib):
        import test_gpu_attn as t
        t.test_more_nodes_than_a_request_may_have(w12lib)

    def test_a_row_does_not_depend_on_its_siblings(self, w12lib):
        import test_gpu_attn as t
        t.test_a_row_does_not_depend_on_its_siblings(w12lib)

    def test_verify_step(self, w12lib, monkeypatch):
        import test_gpu_verify_layer as t
        t.test_verify_step(w12lib, monkeypatch)


@pytest.mark.gpu
@pytest.mark.parametrize("counts", [[2, 1, 3], [70, 60, 50]])
def test_a_request_in_error_leaves_the_others_alone(counts, w12lib):
    """Lengths, pages, parents and requests in error: NaN in that request's rows, none in the others, for nodes that lie
    mixed in the call."""
    import test_gpu_attn as t
    c = t.case(counts, [200, 100, 90], 5, 1, 128, 16, "chain", mixed=True)
    x, mag = t.want(c)
    mine = c["req"] == 1
    node = int(mine.nonzero()[0])
    for name, at, value in (("ctx", 1, -1), ("ctx", 1, 2 ** 30), ("table", (1, 0), -1), ("table", (1, 0), 2 ** 30),
                            ("parent", node, len(c["req"])), ("req", node, 3), ("req", node, -1)):
        d = {n: v.clone() for n, v in c.items()}
        d[name][at] = value
        o = t.run(w12lib, d)
        assert w12lib.default_attn_workspace(torch.device("cuda", 0)).status() == w12lib.W12_ERR_INVALID
        assert o[mine].isnan().all()
        assert failures(o[~mine], x[~mine], mag[~mine]) == 0
