"""w12_gdn_scan at its edges: waits that give up."""
import pytest
import torch

import lossless_bit_weight_02_gb300 as w12

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
