"""The Python binding's checks of the norm, rotary and attention operators'
tensors: what a kernel would read or write beyond a tensor is refused before
any launch."""
import pytest
import torch

import lossless_bit_weight_02_gb300 as w12

CPU = torch.device("cpu")
BF = torch.bfloat16


def rows(t):
    return w12._rows(t, "t", t.shape, t.dtype, t.device)


@pytest.mark.parametrize("t,stride", [
    (torch.zeros(4, 6), 6), (torch.zeros(4, 9)[:, :6], 9), (torch.zeros(4, 6)[::2], 12), (torch.zeros(1, 6).expand(1, 6), 6),
    (torch.zeros(6).as_strided((1, 6), (0, 1)), 6), (torch.zeros(0, 6), 6), (torch.zeros(4, 0), 0),
    (torch.zeros(3, 4, 6), 24), (torch.zeros(3, 40)[:, :24].view(3, 4, 6), 40), (torch.zeros(3, 1, 6)[:, :, :], 6),
])
def test_row_strides(t, stride):
    got = rows(t)
    assert got == stride or (t.numel() == 0 and got >= stride)


@pytest.mark.parametrize("t", [
    torch.zeros(1, 6).expand(4, 6), torch.zeros(10).as_strided((4, 6), (1, 1)), torch.zeros(40).as_strided((4, 6), (5, 1)),
    torch.zeros(1, 4, 6).expand(3, 4, 6), torch.zeros(80).as_strided((3, 4, 6), (23, 6, 1)),
    torch.zeros(1, 16, dtype=torch.int32).expand(8, 16),
])
def test_rows_that_overlap_are_refused(t):
    with pytest.raises(ValueError, match="overlap"):
        rows(t)


@pytest.mark.gpu
def test_norm_refuses_rows_that_overlap(w12lib):
    g = torch.Generator(device="cuda").manual_seed(1)
    x, w = torch.randn(4, 256, generator=g, device="cuda").to(BF), torch.ones(256, device="cuda").to(BF)
    over = torch.zeros(4 * 256, device="cuda").to(BF).as_strided((4, 256), (255, 1))
    for call in (lambda: w12lib.w12_rmsnorm(x[:1].expand(4, 256), w), lambda: w12lib.w12_rmsnorm(x, w, residual=x[:1].expand(4, 256)),
                 lambda: w12lib.w12_rmsnorm(x, w, y_out=over), lambda: w12lib.w12_rmsnorm(x, w, residual=x, h_out=over)):
        with pytest.raises(ValueError, match="overlap"):
            call()
    bias = x[:1].expand(4, 256)
    y = w12lib.w12_rmsnorm(x, w, residual=bias.contiguous())
    assert torch.equal(y["h"], (x.float() + bias.float()).to(BF))


@pytest.mark.gpu
def test_rotary_refuses_rows_that_overlap(w12lib):
    q, k, f = torch.zeros(8, 4, 64, device="cuda").to(BF), torch.zeros(8, 2, 64, device="cuda").to(BF), torch.ones(32, device="cuda")
    pos = torch.zeros(8, dtype=torch.int32, device="cuda")
    kc = torch.zeros(2, 16, 2, 64, device="cuda").to(BF)
    cache, slots = w12lib.KvCache(kc, kc.clone()), torch.arange(8, device="cuda")
    q1, k1 = q[:1].expand(8, 4, 64), k[:1].expand(8, 2, 64)
    for call in (lambda: w12lib.w12_rope_append(q1, k, pos, f), lambda: w12lib.w12_rope_append(q, k1, pos, f),
                 lambda: w12lib.w12_rope_append(q, k, pos, f, q_out=q1), lambda: w12lib.w12_rope_append(q, k, pos, f, k_out=k1),
                 lambda: w12lib.w12_rope_append(q, k, pos, f, v=k1, cache=cache, slots=slots),
                 lambda: w12lib.w12_kv_append(k1, k, cache, slots)):
        with pytest.raises(ValueError, match="overlap"):
            call()


@pytest.mark.gpu
def test_attention_refuses_rows_that_overlap(w12lib):
    g = torch.Generator(device="cuda").manual_seed(2)
    kc, vc = torch.randn(2, 3, 16, 2, 64, generator=g, device="cuda").to(BF)
    q, k, v = (torch.randn(4, h, 64, generator=g, device="cuda").to(BF) for h in (4, 2, 2))
    table = torch.tensor([[2, 0]], dtype=torch.int32, device="cuda")  # one prefix that all requests share
    base = dict(q=q, k=k, v=v, cache=w12lib.KvCache(kc, vc), block_table=table.repeat(4, 1),
                ctx_len=torch.full((4,), 20, dtype=torch.int32, device="cuda"),
                req=torch.arange(4, dtype=torch.int32, device="cuda"))
    for change in (dict(block_table=table.expand(4, 2)), dict(q=q[:1].expand(4, 4, 64)), dict(k=k[:1].expand(4, 2, 64)),
                   dict(v=v[:1].expand(4, 2, 64)), dict(out=q[:1].expand(4, 4, 64))):
        with pytest.raises(ValueError, match="overlap"):
            w12lib.w12_tree_attn(**{**base, **change})
    assert w12lib.w12_tree_attn(**base).isfinite().all()
