"""Refusals of the operators that end a verify step, on the host: C ABI and binding."""
import ctypes

import pytest
import torch

import lossless_bit_weight_02_gb300 as w12

P = 1 << 20  # an address that is never read: every call here is refused before a launch


def accept(lib, **kw):
    a = dict(logits=P, ldl=100, rows=12, V=100, logits32=0, token=P, parent=P, req=0, row=0, root_row=0, n=8, R=4,
             temperature=0, temperature1=1.0, uniform=P, noise=P, ld_noise=100, draft=0, ldd=0, draft_rows=0, draft_row=0,
             max_depth=16, count=P, nodes=P, next=P, ld_nodes=16)
    a.update(kw)
    return lib.w12_tree_accept(w12._accept_args.pack(*a.values()), None)


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(n=1 << 21), dict(R=0), dict(R=65537), dict(V=0), dict(V=1 << 25), dict(rows=-1), dict(max_depth=0),
    dict(max_depth=257), dict(logits32=2), dict(logits=0), dict(ldl=99), dict(count=0), dict(nodes=0), dict(next=0),
    dict(ld_nodes=15), dict(token=0), dict(parent=0), dict(temperature1=-1.0), dict(temperature1=float("nan")),
    dict(temperature1=float("inf")), dict(noise=0), dict(uniform=0), dict(ld_noise=99), dict(temperature=P, temperature1=0.0, noise=0),
    dict(draft=P), dict(draft_row=P), dict(draft=P, draft_row=P, ldd=99), dict(draft=P, draft_row=P, ldd=100, draft_rows=-1)])
def test_accept_refuses(w12lib, kw):
    assert accept(w12lib.load(), **kw) == w12.W12_ERR_INVALID


@pytest.mark.parametrize("kw", [dict(logits=P + 1), dict(logits=P + 2, logits32=1), dict(token=P + 2), dict(noise=P + 1), dict(count=P + 3)])
def test_accept_alignment(w12lib, kw):
    assert accept(w12lib.load(), **kw) == w12.W12_ERR_ALIGN


def scan(lib, ws=P, size=1 << 40, **kw):
    a = dict(S=1 << 30, S_out=1 << 31, q=P, k=P, v=P, ldq=256, ldk=256, ldv=512, alpha=P, beta=P, o=P, ldo=512, o32=0,
             start=P, rows=0, count=0, ld_rows=0, width=0, n=100, R=2, H=4, key_heads=2, D=128, mode=2, status=0)
    a.update(kw)
    return lib.w12_gdn_scan(w12._scan_args.pack(*a.values()), ws, size, None)


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(n=1 << 25), dict(R=0), dict(R=65537), dict(H=0), dict(H=1025), dict(D=96), dict(D=256), dict(mode=-1),
    dict(mode=3), dict(key_heads=0), dict(key_heads=3), dict(o32=2), dict(S=0), dict(S_out=0), dict(start=0),
    dict(rows=P), dict(count=P), dict(start=0, rows=P), dict(start=0, rows=0, count=P, width=3, ld_rows=3),
    dict(start=0, rows=P, count=P, width=-1), dict(start=0, rows=P, count=P, width=4, ld_rows=3),
    dict(start=0, rows=P, count=P, width=4, ld_rows=4, mode=1), dict(start=0, rows=P, count=P, width=65537, ld_rows=65537),
    dict(q=0), dict(o=0), dict(k=0), dict(v=0), dict(alpha=0), dict(beta=0), dict(ldk=255), dict(ldv=504), dict(ldq=248),
    dict(ldo=504), dict(S_out=(1 << 30) + 4096), dict(S_out=(1 << 30) - 4096)])
def test_scan_refuses(w12lib, kw):
    assert scan(w12lib.load(), **kw) == w12.W12_ERR_INVALID


@pytest.mark.parametrize("kw", [dict(S=(1 << 30) + 8), dict(q=P + 8), dict(k=P + 2), dict(ldv=516), dict(ldo=516), dict(start=P + 2),
                                dict(status=P + 1), dict(o=P + 8, o32=1)])
def test_scan_alignment(w12lib, kw):
    assert scan(w12lib.load(), **kw) == w12.W12_ERR_ALIGN


def test_scan_workspace(w12lib):
    lib = w12lib.load()
    assert lib.w12_gdn_scan_workspace_bytes(100, 2, 4, 128, w12.W12_GDN_PATH) == 0
    need = lib.w12_gdn_scan_workspace_bytes(100, 2, 4, 128, w12.W12_GDN_WY)
    if need:
        assert scan(lib, mode=w12.W12_GDN_WY, size=need - 1) == w12.W12_ERR_CAPACITY
        assert scan(lib, mode=w12.W12_GDN_WY, ws=0) == w12.W12_ERR_CAPACITY
        assert scan(lib, mode=w12.W12_GDN_WY, ws=P + 16) == w12.W12_ERR_ALIGN


@pytest.mark.gpu
def test_binding_refuses(w12lib):
    V, n, R = 64, 4, 2
    lg = torch.zeros(n + R, V, device="cuda")
    i32 = lambda m: torch.zeros(m, dtype=torch.int32, device="cuda")  # noqa: E731
    tok, par, u, e = i32(n), i32(n) - 1, torch.zeros(n, device="cuda"), torch.ones(R, V, device="cuda")
    good = dict(logits=lg, token=tok, parent=par, req=i32(n), uniform=u, noise=e)
    w12.w12_tree_accept(**good)
    for bad in (dict(logits=lg.half()), dict(logits=lg.cpu()), dict(logits=lg[:n]), dict(logits=lg[:1].expand(n + R, V)), dict(noise=None),
                dict(uniform=None), dict(noise=e[:1]), dict(noise=e[:1].expand(R, V)), dict(token=tok.long()), dict(req=i32(n + 1)),
                dict(max_depth=0), dict(max_depth=257), dict(draft=e), dict(draft_row=tok), dict(draft=e[:, :9], draft_row=tok),
                dict(temperature=torch.ones(R + 1, device="cuda")), dict(row=i32(n - 1)), dict(parent=par.cpu())):
        with pytest.raises((ValueError, w12.W12Error)):
            w12.w12_tree_accept(**{**good, **bad})
    for t in (-1.0, float("nan")):
        with pytest.raises(w12.W12Error):
            w12.w12_tree_accept(**good, temperature=t)

    S = torch.zeros(R, 2, 64, 64, device="cuda")
    q = torch.zeros(n, 1, 64, device="cuda").bfloat16()
    v = torch.zeros(n, 2, 64, device="cuda").bfloat16()
    ab = torch.ones(n, 2, device="cuda")
    st = i32(R + 1)
    good = dict(S=S, q=q, k=q, v=v, alpha=ab, beta=ab, start=st)
    w12.w12_gdn_scan(**good)
    for bad in (dict(S=S.double()), dict(S=S[:, :, :32]), dict(S=S.transpose(2, 3)), dict(S_out=S[:1]), dict(q=q.float()), dict(k=q[:3]),
                dict(v=v[:, :1].expand(n, 2, 64)), dict(q=q[:1].expand(n, 1, 64)), dict(alpha=ab[:, :1]), dict(beta=ab.half()),
                dict(start=None), dict(start=st.long()), dict(start=st[:2]), dict(rows=i32(4).view(2, 2)), dict(count=i32(2)),
                dict(start=None, rows=i32(4).view(2, 2)), dict(start=None, rows=i32(2).view(1, 2).expand(2, 2), count=i32(2)),
                dict(q=None, out=v), dict(out=v.half()), dict(out=v[:3]), dict(status=i32(2)), dict(mode=7),
                dict(S_out=torch.zeros(2 * S.numel(), device="cuda")[64:64 + S.numel()].view(S.shape), S=S, mode=5)):
        with pytest.raises((ValueError, w12.W12Error)):
            w12.w12_gdn_scan(**{**good, **bad})


@pytest.mark.parametrize("kw", [
    dict(q=1 << 22, k=1 << 23, v=P), dict(q=P, k=1 << 23, v=1 << 22), dict(q=1 << 22, k=P, v=1 << 23),
    dict(q=P + 99 * 512, k=1 << 22, v=1 << 23),  # the last row of o is the first of q
    dict(q=1 << 22, k=1 << 23, v=P + 1008, ldv=1024, ldo=1024), dict(q=1 << 22, k=1 << 23, v=P - 1008, ldv=1024, ldo=1024),
    dict(q=1 << 22, k=1 << 23, v=P + 1024, ldv=1024, ldo=1024, o32=1)])
def test_scan_output_over_inputs(w12lib, kw):
    assert scan(w12lib.load(), **kw) == w12.W12_ERR_INVALID


@pytest.mark.gpu
def test_scan_output_beside_inputs(w12lib):
    """q, k, v and o as columns of one buffer give what tensors of their own do; o over one of them is refused."""
    for n, mode in ((5, w12.W12_GDN_PATH), (130, w12.W12_GDN_WY)):
        g = torch.Generator("cuda").manual_seed(n)
        both = torch.randn(n, 64 * 6, device="cuda", generator=g).bfloat16()
        q, k, v, o = both[:, :64].view(n, 1, 64), both[:, 64:128].view(n, 1, 64), both[:, 128:256].view(n, 2, 64), both[:, 256:].view(n, 2, 64)
        k.copy_(torch.nn.functional.normalize(k.float(), dim=-1))
        S = torch.randn(1, 2, 64, 64, device="cuda", generator=g)
        ab = torch.rand(n, 2, device="cuda", generator=g)
        want, after = w12.w12_gdn_scan(S.clone(), q.clone(), k.clone(), v.clone(), ab, ab, mode=mode)
        got, S2 = w12.w12_gdn_scan(S.clone(), q, k, v, ab, ab, out=o, mode=mode)
        assert torch.equal(got, want) and torch.equal(S2, after) and got.data_ptr() == o.data_ptr()
        for bad in (v, both[:, 192:320].view(n, 2, 64), both[:, :128].view(n, 2, 64)):
            with pytest.raises(w12.W12Error):
                w12.w12_gdn_scan(S.clone(), q, k, v, ab, ab, out=bad, mode=mode)
