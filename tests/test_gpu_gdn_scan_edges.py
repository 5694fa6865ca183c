"""w12_gdn_scan at its edges: waits that give up, chunks that are ill-conditioned, the automatic mode, every head by itself."""
import pytest
import torch

import lossless_bit_weight_02_gb300 as w12
import step_ref as ref

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def make(R, n, H, Hk, D, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    nrm = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    return [nrm(R, H, D, D) * 0.3, unit(nrm(n, Hk, D)).to(BF), unit(nrm(n, Hk, D)).to(BF), nrm(n, H, D).to(BF),
            torch.rand(n, H, generator=g, device="cuda") * 0.1 + 0.9, torch.sigmoid(nrm(n, H))]


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("out32,in_place,states_only", [(False, False, False), (True, True, False), (False, False, True)])
def test_a_wait_that_gave_up_shows(w12lib, D, out32, in_place, states_only):
    """Also without a status: the states and outputs of the sequences are NaN, not what was there before.  Sequences
    without tokens and rows in no sequence are as ever, and the next call is right."""
    H = 2
    S, q, k, v, alpha, beta = make(3, 200, H, 1, D, D)
    q = None if states_only else q
    start = ints(5, 105, 105, 190)
    want_o, want = w12.w12_gdn_scan(S.clone(), q, k, v, alpha, beta, start=start, out32=out32, mode=w12.W12_GDN_WY)
    for stall in (w12.W12_GDN_TEST_STALL, 0):
        S2 = S.clone()
        out = None if states_only else torch.full((200, H, D), 3.0, dtype=torch.float32 if out32 else BF, device="cuda")
        o, after = w12.w12_gdn_scan(S2, q, k, v, alpha, beta, start=start, S_out=None if in_place else torch.zeros_like(S), out=out,
                                    mode=w12.W12_GDN_WY | stall)
        assert torch.equal(after[1], S[1])
        if not states_only:
            assert (o[:5] == 3.0).all() and (o[190:] == 3.0).all()
        if stall:
            assert after[[0, 2]].isnan().all() and (states_only or o[5:190].isnan().all())
        else:
            assert torch.equal(after, want) and (states_only or torch.equal(o[5:190], want_o[5:190]))


def alike(n, Hk, D, g, like):
    """Unit keys whose cosines are about `like`."""
    nrm = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    return unit((1 - like) ** 0.5 * unit(nrm(n, Hk, D)) + like ** 0.5 * unit(nrm(Hk, D))).to(BF)


@pytest.mark.parametrize("mode", [w12.W12_GDN_WY, w12.W12_GDN_AUTO])
@pytest.mark.parametrize("D,lens,out32", [(64, [500], True), (128, [130, 0, 700], False), (128, [64, 65, 63], True)])
@pytest.mark.parametrize("in_place", [False, True])
def test_ill_conditioned_chunks(w12lib, mode, D, lens, out32, in_place):
    """Equal keys and beta = 2: every write flips what is there and nothing decays.  A head with such a chunk anywhere is
    what it is token by token, bit for bit; the others stay within the chunks' error."""
    H, Hk, R, n = 4, 2, len(lens), sum(lens) + 7
    g = torch.Generator(device="cuda").manual_seed(D + n)
    S, q, k, v, alpha, beta = make(R, n, H, Hk, D, D + n)
    k = alike(n, Hk, D, g, 1.0)
    alpha[:, 1], beta[:, 1] = 1.0, 2.0   # all of head 1
    start = ints(*[4 + sum(lens[:i]) for i in range(R + 1)])
    first, last = 4, 4 + sum(lens)
    alpha[last - 63:last, 2], beta[last - 63:last, 2] = 1.0, 2.0  # the end of the last sequence, in head 2
    run = lambda m, S, S_out: w12.w12_gdn_scan(S, q, k, v, alpha, beta, start=start, S_out=S_out, mode=m,  # noqa: E731
                                               out=torch.full((n, H, D), 3.0, dtype=torch.float32 if out32 else BF, device="cuda"))
    o, after = run(mode, S.clone(), None) if in_place else run(mode, S, torch.empty_like(S))
    po, pafter = run(w12.W12_GDN_PATH, S, torch.empty_like(S))
    assert torch.equal(o[:, 1], po[:, 1]) and torch.equal(after[:, 1], pafter[:, 1])
    a, b = start.tolist()[-2:]
    assert torch.equal(o[a:b, 2], po[a:b, 2]) and torch.equal(after[-1, 2], pafter[-1, 2])
    assert (o[:first] == 3.0).all() and (o[last:] == 3.0).all()
    seqs = [list(range(x, y)) for x, y in zip(start.tolist(), start.tolist()[1:])]
    o64, S64, _, _ = ref.scan(S, q, k, v, alpha, beta, seqs)
    want = torch.stack([o64[i] for i in range(first, last)])
    err = lambda x, y: float(torch.linalg.norm(x.double() - y) / torch.linalg.norm(y))  # noqa: E731
    half = 0.0 if out32 else 2.0 ** -8
    for h in range(H):
        # by token 1e-5, as test_gpu_gdn_scan has it.  In chunks 3e-4: the algorithm in 64 bits with every operand rounded as
        # the kernels round it comes to 2.8e-4 at most for equal keys and beta <= 1
        bound = 1e-5 if h == 1 else 3e-4
        for r in range(R):
            assert err(after[r, h], S64[r, h]) <= bound, (r, h, err(after[r, h], S64[r, h]))
        assert err(o[first:last, h], want[:, h]) <= bound + half, (h, err(o[first:last, h], want[:, h]))


@pytest.mark.parametrize("what", ["k", "beta", "alpha"])
def test_not_a_number_in_a_key(w12lib, what):
    """A NaN or Inf in k, beta or alpha reaches the outputs of its token and those after it, as the rule has it, and no
    other head."""
    H, D, n = 2, 128, 200
    args = make(1, n, H, 2, D, 3)
    clean = [t.clone() for t in args]
    bad = {"k": 2, "beta": 5, "alpha": 4}[what]
    args[bad][70, 0] = float("nan")
    args[bad][90, 0] = float("inf")
    o, S = w12.w12_gdn_scan(*args, S_out=torch.empty_like(args[0]), mode=w12.W12_GDN_WY)
    po, pS = w12.w12_gdn_scan(*args, S_out=torch.empty_like(args[0]), mode=w12.W12_GDN_PATH)
    co, cS = w12.w12_gdn_scan(*clean, S_out=torch.empty_like(args[0]), mode=w12.W12_GDN_WY)
    assert torch.equal(o[:70, 0], po[:70, 0]) and o[70:, 0].isnan().all() and S[0, 0].isnan().all() and pS[0, 0].isnan().all()
    assert torch.equal(o[:, 1], co[:, 1]) and torch.equal(S[0, 1], cS[0, 1])


@pytest.mark.parametrize("D,lens,H,mode", [(128, [100, 3, 44], 2, "WY"), (128, [100, 3, 37], 2, "PATH"), (64, [1, 200], 4, "WY"),
                                           (128, [90] + [1] * 31, 4, "PATH"), (128, [737] + [1] * 31, 4, "WY"), (64, [20] * 3, 40, "PATH")])
def test_the_automatic_mode(w12lib, D, lens, H, mode):
    """One mode for the whole call, by n / R, bit for bit."""
    n, R = sum(lens), len(lens)
    S, q, k, v, alpha, beta = make(R, n, H, H // 2, D, n)
    start = ints(*[sum(lens[:i]) for i in range(R + 1)])
    runs = [w12.w12_gdn_scan(S, q, k, v, alpha, beta, start=start, S_out=torch.empty_like(S), out32=True, mode=m)
            for m in (w12.W12_GDN_AUTO, getattr(w12, "W12_GDN_" + mode), w12.W12_GDN_PATH if mode == "WY" else w12.W12_GDN_WY)]
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])
    assert not torch.equal(runs[0][0], runs[2][0])


@pytest.mark.parametrize("D,H,Hk,lens", [(128, 6, 2, [300, 64, 0, 1, 129]), (64, 5, 5, [700, 65])])
@pytest.mark.parametrize("like,bound", [(0.0, 2e-5), (0.9, 7e-5), (1.0, 6e-4)])
@pytest.mark.parametrize("write", ["sigmoid", "one", "most"])
@pytest.mark.parametrize("decay,zero", [(0.0, True), (0.02, False)])
def test_accuracy_of_every_head(w12lib, D, H, Hk, lens, like, bound, write, decay, zero):
    """In chunks, the state and the FP32 outputs of every head of every request by themselves.  The bounds are twice what the
    algorithm comes to in 64 bits with every operand of a product rounded as the kernels round it (two BF16 numbers, the
    product of the two low ones left out): 9.6e-6, 3.4e-5 and 2.8e-4 at most for independent keys, cosines of 0.9 and
    equal keys, beta <= 1, up to 1024 tokens of 64 columns."""
    n, R = sum(lens), len(lens)
    g = torch.Generator(device="cuda").manual_seed(n + int(10 * like))
    S, q, k, v, alpha, beta = make(R, n, H, Hk, D, n + H)
    S = torch.zeros_like(S) if zero else S
    k = alike(n, Hk, D, g, like)
    alpha = torch.exp(-decay * torch.rand(n, H, generator=g, device="cuda"))
    beta = {"sigmoid": beta, "one": torch.ones_like(beta), "most": torch.full_like(beta, 0.9)}[write]
    start = [sum(lens[:i]) for i in range(R + 1)]
    o, after = w12.w12_gdn_scan(S, q, k, v, alpha, beta, start=ints(*start), S_out=torch.empty_like(S), out32=True, mode=w12.W12_GDN_WY)
    o64, S64, _, _ = ref.scan(S, q, k, v, alpha, beta, [list(range(a, b)) for a, b in zip(start, start[1:])])
    want = torch.stack([o64[i] for i in range(n)])
    for r, (a, b) in enumerate(zip(start, start[1:])):
        if a == b:
            assert torch.equal(after[r], S[r])
            continue
        for got, true in ((after[r].flatten(1), S64[r].flatten(1)), (o[a:b].transpose(0, 1).flatten(1), want[a:b].transpose(0, 1).flatten(1))):
            err = torch.linalg.vector_norm(got.double() - true, dim=1) / torch.linalg.vector_norm(true, dim=1)
            assert (err <= bound).all(), (r, err.tolist())
