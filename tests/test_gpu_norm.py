"""w12_rmsnorm against the 64-bit formula."""
import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu
EPS = 1e-6


def make(M, K, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(M, K, generator=g, device="cuda") * scale).bfloat16()


def weights(K, seed=5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (1 + 0.3 * torch.randn(K, generator=g, device="cuda")).bfloat16()


def check(out, x, w, residual, eps=EPS):
    h, t = ref.rmsnorm(x, w, eps, residual)
    if residual is not None:
        assert ((out["h"].double() - h).abs() <= (ref.BF + ref.FP) * h.abs()).all()
    if "y" in out:
        assert ((out["y"].double() - t).abs() <= (ref.BF + ref.FP) * t.abs() + 1e-38).all()
    if "q8" in out:
        s = ref.group_scales(t)
        assert ((out["scale"].double() - s).abs() <= ref.FP * s).all()
        z = t / out["scale"].double().repeat_interleave(128, 1)[:, :t.shape[1]]
        q = out["q8"].float().double()
        assert ((q - z).abs() <= (2.0 ** -4 + ref.FP) * z.abs() + 2.0 ** -10 * (1 + ref.FP)).all()


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("out8", [False, True])
@pytest.mark.parametrize("M,K", [(1, 5120), (3, 1), (5, 7), (2, 130), (4, 1000), (257, 64), (3, 8200), (2, 17408),
                                 (1, 16385), (2, 40000), (1, 65536), (300, 128)])
def test_norm(M, K, out8, residual, w12lib):
    x, w = make(M, K, 1), weights(K)
    r = make(M, K, 2, 3.0) if residual else None
    check(w12lib.w12_rmsnorm(x, w, eps=EPS, residual=r, out8=out8), x, w, r)


@pytest.mark.parametrize("K,pad", [(256, 8), (256, 3), (250, 6)])
def test_strided_rows(K, pad, w12lib):
    """Rows inside wider buffers, aligned or not; nothing outside the rows is written."""
    M = 9
    wide = [make(M, K + pad, s) for s in (1, 2)]
    x, r = wide[0][:, :K], wide[1][:, pad:]
    w = weights(K)
    h = torch.full((M, K + pad), 7.0, device="cuda").bfloat16()
    y = torch.full((M, K + pad), 7.0, device="cuda").bfloat16()
    out = w12lib.w12_rmsnorm(x, w, eps=EPS, residual=r, h_out=h[:, :K], y_out=y[:, pad:])
    check(out, x, w, r)
    assert (h[:, K:] == 7).all() and (y[:, :pad] == 7).all()


def test_in_place(w12lib):
    x, r, w = make(33, 5120, 1), make(33, 5120, 2), weights(5120)
    want = w12lib.w12_rmsnorm(x, w, residual=r)
    x2, r2 = x.clone(), r.clone()
    out = w12lib.w12_rmsnorm(x2, w, residual=r2, h_out=r2, y_out=x2)
    assert torch.equal(out["h"], want["h"]) and torch.equal(out["y"], want["y"])
    assert out["h"].data_ptr() == r2.data_ptr() and out["y"].data_ptr() == x2.data_ptr()


def test_row_does_not_depend_on_the_others(w12lib):
    x, r, w = make(301, 5120, 1), make(301, 5120, 2), weights(5120)
    many = w12lib.w12_rmsnorm(x, w, residual=r, out8=True)
    one = w12lib.w12_rmsnorm(x[7:8], w, residual=r[7:8], out8=True)
    for k in many:
        assert torch.equal(many[k][7:8].view(torch.uint8), one[k].view(torch.uint8)), k


def test_zero_rows_and_groups(w12lib):
    x, w = make(4, 512, 1), weights(512)
    x[1] = 0
    x[2, 128:256] = 0
    out = w12lib.w12_rmsnorm(x, w, eps=EPS, out8=True)
    assert (out["q8"][1].float() == 0).all() and (out["scale"][1] == 1).all()
    assert (out["q8"][2, 128:256].float() == 0).all() and out["scale"][2, 1] == 1
    zero = w12lib.w12_rmsnorm(x, w, eps=0.0)["y"]  # 0 / 0 in the row of zeros only
    assert zero[1].isnan().all() and not zero[[0, 2, 3]].isnan().any()


def test_not_finite(w12lib):
    x, w = make(3, 384, 1), torch.ones(384, device="cuda").bfloat16()
    x[0, 5] = float("nan")
    out = w12lib.w12_rmsnorm(x, w, eps=EPS)["y"]
    assert out[0].isnan().all() and not out[1:].isnan().any()
    big = torch.ones(384, device="cuda").bfloat16()
    big[200] = float("inf")  # an infinite weight: one column, so one group
    q = w12lib.w12_rmsnorm(x[1:], big, eps=EPS, out8=True)
    assert q["scale"][:, 1].isinf().all() and not q["scale"][:, [0, 2]].isinf().any()
    vals = q["q8"].float()
    assert vals[:, 200].isnan().all()
    rest = torch.cat((vals[:, 128:200], vals[:, 201:256]), 1)
    assert (rest == 0).all()
    nan = torch.ones(384, device="cuda").bfloat16()
    nan[200] = float("nan")
    q = w12lib.w12_rmsnorm(x[1:], nan, eps=EPS, out8=True)
    assert q["scale"][:, 1].isnan().all() and q["q8"].float()[:, 128:256].isnan().all()
    assert not q["q8"].float()[:, :128].isnan().any()


def test_no_rows_and_other_stream(w12lib):
    w = weights(256)
    out = w12lib.w12_rmsnorm(torch.empty(0, 256, device="cuda").bfloat16(), w)
    assert out["y"].shape == (0, 256)
    x = make(64, 256, 3)
    want = w12lib.w12_rmsnorm(x, w)["y"]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = w12lib.w12_rmsnorm(x, w, stream=s)["y"]
    s.synchronize()
    assert torch.equal(got, want)


def test_refusals(w12lib):
    x, w = make(4, 256, 1), weights(256)
    for bad in (lambda: w12lib.w12_rmsnorm(x.float(), w), lambda: w12lib.w12_rmsnorm(x, w[:255]),
                lambda: w12lib.w12_rmsnorm(x, w, residual=x[:3]), lambda: w12lib.w12_rmsnorm(x.t(), w[:4]),
                lambda: w12lib.w12_rmsnorm(x.cpu(), w), lambda: w12lib.w12_rmsnorm(x, w, out8=True, y_out=x)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(w12lib.W12Error) as e:
        w12lib.w12_rmsnorm(x, w, eps=-1.0)
    assert e.value.status == w12lib.W12_ERR_INVALID
    wide = torch.empty(1, 65537, device="cuda").bfloat16()
    with pytest.raises(w12lib.W12Error):
        w12lib.w12_rmsnorm(wide, torch.empty(65537, device="cuda").bfloat16())
