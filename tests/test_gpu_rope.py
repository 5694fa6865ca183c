"""w12_rope_append against the 64-bit formula, and its cache writes."""
import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu
EPS = 1e-5


def inputs(n, Hq, Hkv, D, axes, top=200000, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn(n, (Hq + 2 * Hkv) * D, generator=g, device="cuda").bfloat16()
    q = qkv[:, :Hq * D].view(n, Hq, D)
    k = qkv[:, Hq * D:(Hq + Hkv) * D].view(n, Hkv, D)
    v = qkv[:, (Hq + Hkv) * D:].view(n, Hkv, D)
    pos = torch.randint(0, top, (axes, n), generator=g, device="cuda", dtype=torch.int32)
    return q, k, v, pos, g


def freqs(rot):
    return 10000.0 ** (-torch.arange(rot // 2, device="cuda", dtype=torch.float32) / max(1, rot // 2))


def check(out, x, pos, f, axis, inter, norm=None):
    """Angles: the reduction, sines and products in FP32 leave less than 4e-6 of a radian; beyond 2^24 the
    fraction of a turn comes from numbers of |pos| 2^-26 turns held to 2^-24, summed a few times."""
    want, mag = ref.rope(x, pos, f, axis, inter, norm, EPS)
    top = pos.double().abs().max().item()
    tol = 4e-6 + (2 * 3.1416 * 0.16 * top * 2.0 ** -46 if top >= 1 << 24 else 0.0)
    assert ((out.double() - want).abs() <= (ref.BF + ref.FP) * want.abs() + tol * mag).all()


@pytest.mark.parametrize("n,Hq,Hkv,D,rot,axes,inter,norm", [
    (1, 40, 8, 128, 128, 1, False, False),
    (17, 5, 1, 128, 128, 3, False, True),
    (608, 4, 2, 64, 64, 1, True, False),   # the last size of the one-token kernel
    (609, 4, 2, 64, 32, 2, False, True),   # the first of the four-token kernel, an odd number of tokens
    (613, 3, 3, 128, 32, 4, True, True),
    (5, 1, 1, 256, 256, 1, False, True),
    (7, 2, 1, 256, 64, 2, True, False),
    (9, 7, 7, 64, 16, 1, False, False),
    (700, 65, 1, 64, 64, 1, False, True),  # more heads than the CTA holds at once
])
def test_rope(n, Hq, Hkv, D, rot, axes, inter, norm, w12lib):
    q, k, v, pos, g = inputs(n, Hq, Hkv, D, axes)
    f = freqs(rot)
    axis = [j % axes for j in range(rot // 2)]
    qn, kn = ((1 + 0.2 * torch.randn(2, D, generator=g, device="cuda")).bfloat16() if norm else (None, None))
    qo, ko = w12lib.w12_rope_append(q, k, pos, f, axis=axis, interleaved=inter, q_norm=qn, k_norm=kn, eps=EPS)
    check(qo, q, pos, f, axis, inter, qn)
    check(ko, k, pos, f, axis, inter, kn)
    assert torch.equal(qo[..., rot:], q[..., rot:]) or norm


@pytest.mark.parametrize("head_major", [False, True])
@pytest.mark.parametrize("page", [1, 5, 16, 64])
def test_append(page, head_major, w12lib):
    n, Hkv, D, pages = 77, 3, 128, 120 // page + 1
    q, k, v, pos, g = inputs(n, 6, Hkv, D, 1)
    shape = (pages, Hkv, page, D) if head_major else (pages, page, Hkv, D)
    kc, vc = (torch.full(shape, 9.0, device="cuda").bfloat16() for _ in range(2))
    if head_major:
        kc, vc = kc.permute(0, 2, 1, 3), vc.permute(0, 2, 1, 3)
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:n]
    slots[3], slots[11], slots[20] = -1, pages * page, -5  # skipped
    f = freqs(D)
    qo, ko = w12lib.w12_rope_append(q, k, pos[0], f, v=v, cache=w12lib.KvCache(kc, vc), slots=slots)
    assert ko is None
    _, want = w12lib.w12_rope_append(q, k, pos[0], f)
    check(qo, q, pos, f, [0] * (D // 2), False)
    keep = [i for i in range(n) if i not in (3, 11, 20)]
    flat_k, flat_v = kc.reshape(-1, Hkv, D), vc.reshape(-1, Hkv, D)
    assert torch.equal(flat_k[slots[keep]], want[keep]) and torch.equal(flat_v[slots[keep]], v[keep])
    rest = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    rest[slots[keep]] = False
    assert (flat_k[rest] == 9).all() and (flat_v[rest] == 9).all()


def test_plain_append_and_norm_without_rotation(w12lib):
    n, Hkv, D = 31, 2, 64
    q, k, v, pos, g = inputs(n, 4, Hkv, D, 1)
    kc, vc = (torch.zeros(4, 16, Hkv, D, device="cuda").bfloat16() for _ in range(2))
    slots = torch.randperm(64, generator=g, device="cuda")[:n]
    w12lib.w12_kv_append(k, v, w12lib.KvCache(kc, vc), slots)
    assert torch.equal(kc.view(-1, Hkv, D)[slots], k) and torch.equal(vc.view(-1, Hkv, D)[slots], v)
    w = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).bfloat16()
    qo, _ = w12lib.w12_rope_append(q, None, None, None, q_norm=w, eps=EPS)
    check(qo, q, pos, freqs(0), [], False, w)


def test_in_place_and_keys_only(w12lib):
    q, k, v, pos, g = inputs(50, 4, 2, 128, 2)
    f, axis = freqs(64), [1] * 32
    qo, ko = w12lib.w12_rope_append(q, k, pos, f, axis=axis)
    q2, k2 = q.clone(), k.clone()
    w12lib.w12_rope_append(q2, k2, pos, f, axis=axis, q_out=q2, k_out=k2)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)
    none, k3 = w12lib.w12_rope_append(None, k, pos, f, axis=axis)
    assert none is None and torch.equal(k3, ko)


@pytest.mark.parametrize("p", [0, 4095, 4096, (1 << 24) + 1, (1 << 30) + 12345, (1 << 31) - 1, -7, -(1 << 31)])
def test_positions(p, w12lib):
    """Every int32 position works."""
    q, k, v, pos, g = inputs(3, 2, 1, 64, 1)
    pos.fill_(p)
    f = freqs(64) * 0.9
    qo, _ = w12lib.w12_rope_append(q, k, pos[0], f)
    check(qo, q, pos, f, [0] * 32, False)


def test_empty_and_other_stream(w12lib):
    q, k, v, pos, g = inputs(40, 4, 2, 64, 1)
    f = freqs(64)
    qo, ko = w12lib.w12_rope_append(q[:0], k[:0], pos[:, :0], f)
    assert qo.shape == (0, 4, 64) and ko.shape == (0, 2, 64)
    want, _ = w12lib.w12_rope_append(q, k, pos, f)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, _ = w12lib.w12_rope_append(q, k, pos, f, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


def test_refusals(w12lib):
    q, k, v, pos, g = inputs(8, 4, 2, 64, 2)
    f = freqs(64)
    kc = torch.zeros(2, 16, 2, 64, device="cuda").bfloat16()
    cache = w12lib.KvCache(kc, kc.clone())
    slots = torch.arange(8, device="cuda")
    call = w12lib.w12_rope_append
    for bad in (lambda: call(q.float(), k, pos, f), lambda: call(q, k[:7], pos, f), lambda: call(q, k, pos.long(), f),
                lambda: call(q, k, pos, f, axis=[0] * 31), lambda: call(q, k, pos, f, slots=slots),
                lambda: call(q, k, pos, f, cache=cache, slots=slots), lambda: call(None, None, pos, f),
                lambda: call(q, k, pos, f, v=v, cache=cache, slots=slots.int()),
                lambda: call(q, k, pos, f, q_norm=f), lambda: w12lib.KvCache(kc, kc.float())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: call(q, k, pos, freqs(24)), lambda: call(q, k, pos, freqs(128)),
                lambda: call(q, k, pos, f, axis=[2] * 32),
                lambda: call(torch.zeros(8, 2, 96, device="cuda").bfloat16(), None, pos, f),
                lambda: call(q, torch.zeros(8, 3, 64, device="cuda").bfloat16(), pos, f,
                             v=torch.zeros(8, 3, 64, device="cuda").bfloat16(), cache=cache, slots=slots)):
        with pytest.raises(w12lib.W12Error) as e:
            bad()
        assert e.value.status == w12lib.W12_ERR_INVALID
    odd = torch.zeros(8, 4 * 64 + 4, device="cuda").bfloat16()[:, 4:].view(8, 4, 64)
    with pytest.raises(w12lib.W12Error) as e:
        call(odd, k, pos, f)
    assert e.value.status == w12lib.W12_ERR_ALIGN
