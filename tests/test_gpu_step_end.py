"""The end of a verify step as it is used: drafted trees are selected, a recurrent layer computes their nodes, the
target's logits decide which are accepted, and the layer's states, and the attention layers' caches, go on along them,
all without a trip to the host."""
import pytest
import torch

import lossless_bit_weight_02_gb300 as w12
import step_ref as ref

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def make(R, budget, H, Hk, D, V, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    nrm = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    lp = (nrm(R, 16, 8) * 2).log_softmax(-1)
    sel = w12.w12_tree_select(lp, budget=budget, shared=True)
    n = int(sel["count"][0])
    req, depth, parent, path = (sel[k][:n].contiguous() for k in ("req", "depth", "parent", "path"))
    # candidate c of position d of request r is one token for all nodes
    vocab = torch.argsort(torch.rand(R, 16, V, generator=g, device="cuda"), -1)[..., :8]
    cand = (path >> (4 * (depth.long() - 1))) & 15
    token = vocab[req.long(), depth.long() - 1, cand.long()].int()
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(BF)  # noqa: E731
    s = dict(S=nrm(R, H, D, D) * 0.3, q=unit(nrm(n, Hk, D)), k=unit(nrm(n, Hk, D)), v=nrm(n, H, D).to(BF),
             alpha=torch.rand(n, H, generator=g, device="cuda") * 0.15 + 0.85, beta=torch.sigmoid(nrm(n, H)))
    logits = nrm(n + R, V) * 2
    up = torch.where(parent >= 0, parent.long(), n + req.long())
    logits[up, token.long()] += 7.0
    t = torch.full((R,), 0.8, device="cuda")
    t[::3] = 0.0
    a = dict(logits=logits.to(BF), token=token, parent=parent, req=req, temperature=t,
             uniform=torch.rand(n, generator=g, device="cuda"),
             noise=torch.empty(R, V, device="cuda").exponential_(generator=g).clamp_(min=1e-30))
    return n, s, a, depth


@pytest.mark.parametrize("R,budget,H,Hk,D,V", [(8, 256, 4, 4, 128, 5000), (3, 40, 6, 2, 64, 32000), (1, 16, 2, 1, 128, 1001)])
def test_step(w12lib, R, budget, H, Hk, D, V):
    n, s, a, depth = make(R, budget, H, Hk, D, V, 7 * R + H)
    if H == Hk:  # (the tree operator's heads are not shared)
        tree = w12.w12_gdn_tree(s["S"], s["q"], s["k"], s["v"], s["alpha"], s["beta"], a["parent"], a["req"])
    got = w12.w12_tree_accept(**a)
    status = torch.ones(1, dtype=torch.int32, device="cuda")
    before = s["S"].clone()
    out = torch.zeros(n, H, D, device="cuda")
    o, S = w12.w12_gdn_scan(**s, rows=got["nodes"], count=got["count"], out=out, status=status)
    assert S is s["S"] and o is out and status.item() == 0
    # what was accepted
    lst = lambda t: t.tolist()  # noqa: E731
    want = ref.accept(a["logits"].cpu().float(), lst(a["token"]), lst(a["parent"]), lst(a["req"]), R, lst(a["temperature"]),
                      lst(a["uniform"]), a["noise"].cpu())
    seqs = [got["nodes"][r, :int(got["count"][r])].tolist() for r in range(R)]
    for r, (path, nxt, margin) in enumerate(want):
        assert margin < ref.MARGIN or (seqs[r] == path and int(got["next"][r]) == nxt)
        assert depth[seqs[r]].tolist() == list(range(1, len(seqs[r]) + 1)) and (a["req"][seqs[r]] == r).all()
    assert sum(map(len, seqs)) > 0
    # the states behind them, and their outputs, which are those of the tree
    o64, S64, _, _ = ref.scan(before, s["q"], s["k"], s["v"], s["alpha"], s["beta"], seqs)
    assert torch.linalg.norm(S.double() - S64) <= 1e-5 * torch.linalg.norm(S64)
    for i, x in o64.items():
        assert torch.linalg.norm(o[i].double() - x) <= 1e-5 * torch.linalg.norm(x) + 1e-6
        if H == Hk:
            assert (o[i] - tree[i]).abs().max() <= 1e-5 * tree[i].abs().max() + 1e-6
    # an attention layer's cache takes the same nodes, from the lists as they are
    page, ctx = 16, torch.arange(R, device="cuda") * 5 + 3
    table = torch.arange(R * 4, device="cuda").view(R, 4)
    cache = w12.KvCache(*torch.zeros(2, R * 4, page, 2, 64, device="cuda").to(BF))
    k, v = torch.randn(2, n, 2, 64, device="cuda").to(BF)
    at = got["nodes"].clamp(min=0).long()
    pos = ctx[:, None] + torch.arange(at.shape[1], device="cuda")
    slots = torch.where(got["nodes"] >= 0, torch.gather(table, 1, pos // page) * page + pos % page, -1)
    w12.w12_kv_append(k[at.flatten()], v[at.flatten()], cache, slots.flatten())
    for r, nodes in enumerate(seqs):
        for d, i in enumerate(nodes):
            p = int(ctx[r]) + d
            assert torch.equal(cache.k[int(table[r, p // page]), p % page], k[i])


def test_step_in_a_graph(w12lib):
    """Captured as a whole and replayed on other inputs."""
    n, s, a, _ = make(4, 64, 2, 2, 128, 4000, 3)
    S0 = s.pop("S")
    S = S0.clone()

    def step(S):
        got = w12.w12_tree_accept(**a)
        w12.w12_gdn_scan(S, None, s["k"], s["v"], s["alpha"], s["beta"], rows=got["nodes"], count=got["count"])
        return got

    step(S)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step(S)
    for seed in (5, 6):
        g = torch.Generator(device="cuda").manual_seed(seed)
        a["uniform"].copy_(torch.rand(n, generator=g, device="cuda"))
        S.copy_(S0)
        graph.replay()
        S2 = S0.clone()
        got = step(S2)
        assert torch.equal(S, S2) and all(torch.equal(kept[k], got[k]) for k in got)


def test_prompt_then_steps(w12lib):
    """A prompt in chunks, then tokens one at a time: the states of the whole at once."""
    H, Hk, D, n, m = 4, 2, 128, 333, 5
    g = torch.Generator(device="cuda").manual_seed(4)
    nrm = lambda *x: torch.randn(*x, generator=g, device="cuda")  # noqa: E731
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(BF)  # noqa: E731
    q, k, v = unit(nrm(n, Hk, D)), unit(nrm(n, Hk, D)), nrm(n, H, D).to(BF)
    alpha, beta = torch.rand(n, H, generator=g, device="cuda") * 0.1 + 0.9, torch.sigmoid(nrm(n, H))
    S = torch.zeros(1, H, D, D, device="cuda")
    o = torch.empty(n, H, D, device="cuda")
    first = n - m
    w12.w12_gdn_scan(S, q[:first], k[:first], v[:first], alpha[:first], beta[:first], out=o[:first], mode=w12.W12_GDN_WY)
    for t in range(first, n):
        w12.w12_gdn_scan(S, q[t:t + 1], k[t:t + 1], v[t:t + 1], alpha[t:t + 1], beta[t:t + 1], out=o[t:t + 1])
    o64, S64, _, _ = ref.scan(torch.zeros_like(S), q, k, v, alpha, beta, [list(range(n))])
    assert torch.linalg.norm(S.double() - S64) <= 1e-5 * torch.linalg.norm(S64)
    whole = torch.stack([o64[i] for i in range(n)])
    assert torch.linalg.norm(o.double() - whole) <= 3e-5 * torch.linalg.norm(whole)


def test_two_threads(w12lib):
    """Calls of two threads on streams of their own do not come between one another."""
    import threading
    n, s, a, _ = make(4, 64, 2, 2, 128, 4000, 9)
    S0 = s.pop("S")
    start = torch.tensor([0, 20, 20, 50, n], dtype=torch.int32, device="cuda")
    want = w12.w12_gdn_scan(S0, s["q"], s["k"], s["v"], s["alpha"], s["beta"], start=start, S_out=torch.empty_like(S0), mode=w12.W12_GDN_WY)
    wa = w12.w12_tree_accept(**a)
    torch.cuda.synchronize()
    bad = []

    def work():
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(50):
                o, S = w12.w12_gdn_scan(S0, s["q"], s["k"], s["v"], s["alpha"], s["beta"], start=start, S_out=torch.empty_like(S0),
                                        mode=w12.W12_GDN_WY)
                got = w12.w12_tree_accept(**a)
                stream.synchronize()
                if not (torch.equal(o, want[0]) and torch.equal(S, want[1]) and all(torch.equal(got[x], wa[x]) for x in wa)):
                    bad.append(1)

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
