"""w12_gdn_scan against the recurrence in 64 bits."""
import pytest
import torch

import lossless_bit_weight_02_gb300 as w12
import step_ref as ref

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def make(R, n, H, Hk, D, seed, unit=True, decay=1.0, zero=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    nrm = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q, k, v = nrm(n, Hk, D), nrm(n, Hk, D) + 0.5 * nrm(Hk, D), nrm(n, H, D)
    if unit:
        q, k = q / q.norm(dim=-1, keepdim=True), k / k.norm(dim=-1, keepdim=True)
    alpha = torch.exp(-decay * 0.1 * torch.rand(n, H, generator=g, device="cuda") ** 2)
    beta = torch.sigmoid(nrm(n, H))
    S = torch.zeros(R, H, D, D, device="cuda") if zero else nrm(R, H, D, D) * 0.3
    return [S, q.to(BF), k.to(BF), v.to(BF), alpha, beta]


def cuts(lens, gap=0):
    c = [gap]
    for m in lens:
        c.append(c[-1] + m)
    return torch.tensor(c, dtype=torch.int32, device="cuda")


def check(args, seqs, out, S_new, mode):
    """Errors in the 2-norm of a head against the bound of the reference's docstring, and element by element."""
    S, q, k, v, alpha, beta = args
    D = S.shape[-1]
    o, S64, oa, A = ref.scan(S, q, k, v, alpha, beta, seqs)
    longest = max([len(x) for x in seqs] + [1])
    eps = (2 * D + 8) * 2.0 ** -24 * min(longest, 64) + 2.0 ** -21 + (2.0 ** -14 if mode != w12.W12_GDN_PATH else 0)
    assert ((S_new.double() - S64).abs() <= eps * A + 1e-30).all(), ((S_new.double() - S64).abs() / (A + 1e-30)).max()
    assert torch.linalg.norm(S_new.double() - S64) <= 1e-5 * torch.linalg.norm(S64) + 1e-30
    if q is None or not o:
        return
    rows = sorted(o)
    want, mag = torch.stack([o[i] for i in rows]), torch.stack([oa[i] for i in rows])
    got = out[rows].double()
    half = 2.0 ** -8 if out.dtype is BF else 0.0
    assert ((got - want).abs() <= half * want.abs() * (1 + eps) + 2 * eps * mag + 1e-30).all()
    # the magnitudes grow with every token where signs cancel: the whole's error against the states'
    assert torch.linalg.norm(got - want) <= (half + 3e-5) * torch.linalg.norm(want) + 1e-30


MODES = [w12.W12_GDN_PATH, w12.W12_GDN_WY, w12.W12_GDN_AUTO]


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("D,H,Hk", [(128, 4, 2), (64, 3, 3), (128, 3, 1), (64, 6, 2)])
@pytest.mark.parametrize("lens", [[1], [5], [64], [65], [63, 0, 1, 130], [200, 17], [1, 1, 1, 1], [0], [0, 0, 3], [127, 129, 128]])
def test_sequences(w12lib, lens, D, H, Hk, mode):
    n = sum(lens)
    args = make(len(lens), n, H, Hk, D, 3 * n + D + H)
    start = cuts(lens)
    out32 = (n + H) % 2 == 0
    S_out = torch.full_like(args[0], float("nan"))
    o, S_new = w12.w12_gdn_scan(*args, start=start, S_out=S_out, out32=out32, mode=mode)
    assert S_new is S_out and o.dtype is (torch.float32 if out32 else BF)
    c = start.tolist()
    seqs = [list(range(a, b)) for a, b in zip(c, c[1:])]
    check(args, seqs, o, S_new, mode)
    # in place, and without outputs: the same states
    S2 = args[0].clone()
    _, again = w12.w12_gdn_scan(S2, None, *args[2:], start=start, mode=mode)
    assert again is S2 and torch.equal(S2, S_new)


@pytest.mark.parametrize("mode", MODES)
def test_long(w12lib, mode):
    args = make(2, 1500, 2, 1, 128, 5)
    start = cuts([1001, 499])
    o, S = w12.w12_gdn_scan(*args, start=start, S_out=torch.empty_like(args[0]), mode=mode)
    check(args, [list(range(1001)), list(range(1001, 1500))], o, S, mode)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("width,counts", [(16, [0, 1, 16, 7]), (1, [1, 0, 1, 1]), (40, [33, 40, 0, 2])])
def test_listed_rows(w12lib, D, width, counts):
    R, n, H = 4, 300, 4
    args = make(R, n, H, 2, D, width)
    perm = torch.randperm(n, generator=torch.Generator().manual_seed(1))
    rows = torch.full((R, width + 3), -1, dtype=torch.int32)
    seqs, at = [], 0
    for r, c in enumerate(counts):
        seqs.append(perm[at:at + c].tolist())
        rows[r, :c] = perm[at:at + c].int()
        at += c
    rows = rows.cuda()[:, :width]
    count = torch.tensor(counts, dtype=torch.int32, device="cuda")
    out = torch.full((n, H, D), 7.0, dtype=BF, device="cuda")
    status = torch.full((1,), 5, dtype=torch.int32, device="cuda")
    o, S = w12.w12_gdn_scan(*args, rows=rows, count=count, S_out=torch.empty_like(args[0]), out=out, status=status)
    assert o is out and status.item() == 0
    check(args, seqs, o, S, w12.W12_GDN_PATH)
    rest = sorted(set(range(n)) - {i for s in seqs for i in s})
    assert (out[rest] == 7.0).all()


@pytest.mark.parametrize("mode", MODES)
def test_views_and_rows_behind(w12lib, mode):
    """q, k, v as views of one matrix, outputs into a wider one; rows before and behind the sequences stay."""
    H, Hk, D, lens = 4, 2, 128, [70, 3, 100]
    n = sum(lens) + 9
    S, q, k, v, alpha, beta = make(3, n, H, Hk, D, 8)
    both = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1), torch.full((n, 8), float("nan"), device="cuda").to(BF)], 1)
    q, k, v = (both[:, a:b].unflatten(1, (-1, D)) for a, b in ((0, Hk * D), (Hk * D, 2 * Hk * D), (2 * Hk * D, (2 * Hk + H) * D)))
    for t in (q, k, v):
        t[:4] = float("nan")
        t[n - 5:] = float("inf")
    alpha[:4] = float("nan")
    beta[n - 5:] = float("nan")
    wide = torch.full((n, H * D + 16), 3.0, device="cuda").to(BF)
    out = wide[:, :H * D].unflatten(1, (H, D))
    start = cuts(lens, gap=4)
    args = [S, q, k, v, alpha, beta]
    o, S_new = w12.w12_gdn_scan(*args, start=start, S_out=torch.empty_like(S), out=out, mode=mode)
    c = start.tolist()
    check(args, [list(range(a, b)) for a, b in zip(c, c[1:])], o, S_new, mode)
    assert (wide[:, H * D:] == 3.0).all() and (wide[:4] == 3.0).all() and (wide[n - 5:] == 3.0).all()


@pytest.mark.parametrize("mode", MODES)
def test_a_bad_neighbour_stays_alone(w12lib, mode):
    """NaN and Inf in one sequence reach no other."""
    lens = [70, 40, 90]
    args = make(3, 200, 2, 2, 128, 4)
    clean = [t.clone() for t in args]
    for t in args[1:4]:
        t[70:110] = float("nan")
        t[80] = float("inf")
    args[0][1] = float("inf")
    start = cuts(lens)
    o, S = w12.w12_gdn_scan(*args, start=start, S_out=torch.empty_like(args[0]), mode=mode)
    o2, S2 = w12.w12_gdn_scan(*clean, start=start, S_out=torch.empty_like(args[0]), mode=mode)
    for r, (a, b) in enumerate(((0, 70), (70, 110), (110, 200))):
        if r != 1:
            assert torch.equal(o[a:b], o2[a:b]) and torch.equal(S[r], S2[r])


@pytest.mark.parametrize("mode", MODES)
def test_requests_do_not_matter_to_each_other(w12lib, mode):
    """A request's results are bitwise those that it gets alone."""
    lens = [129, 1, 66]
    args = make(3, 196, 4, 2, 128, 6)
    start = cuts(lens)
    o, S = w12.w12_gdn_scan(*args, start=start, S_out=torch.empty_like(args[0]), mode=mode if mode != w12.W12_GDN_AUTO else w12.W12_GDN_WY)
    c = start.tolist()
    for r in range(3):
        part = [args[0][r:r + 1].contiguous()] + [t[c[r]:c[r + 1]].contiguous() for t in args[1:]]
        o1, S1 = w12.w12_gdn_scan(*part, S_out=torch.empty_like(part[0]), mode=mode if mode != w12.W12_GDN_AUTO else w12.W12_GDN_WY)
        assert torch.equal(o[c[r]:c[r + 1]], o1) and torch.equal(S[r:r + 1], S1)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("D", [64, 128])
def test_resets_and_extremes(w12lib, mode, D):
    """Decays of 0 (a document's border) and 1, writes of 0 and 1, equal keys."""
    n, H = 150, 2
    args = make(1, n, H, 1, D, 12)
    alpha, beta = args[4], args[5]
    alpha[::3] = 1.0
    alpha[[0, 40, 41, 64, 100]] = 0.0
    alpha[120:, 1] = 1e-30
    beta[::4], beta[1::4] = 0.0, 1.0
    args[2][50:90] = args[2][50]
    o, S = w12.w12_gdn_scan(*args, S_out=torch.empty_like(args[0]), mode=mode)
    check(args, [list(range(n))], o, S, mode)


def test_rules(w12lib):
    """A sequence that breaks a rule is left out and reported; its states are copied, its rows left."""
    n, H, D = 40, 2, 64
    for mode in MODES:
        args = make(4, n, H, 1, D, 1)
        start = torch.tensor([0, 10, 5, 30, 41], dtype=torch.int32, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((n, H, D), 7.0, dtype=BF, device="cuda")
        _, S = w12.w12_gdn_scan(*args, start=start, S_out=torch.empty_like(args[0]), out=out, mode=mode, status=status)
        assert status.item() == 1
        assert torch.equal(S[1], args[0][1]) and torch.equal(S[3], args[0][3]) and (out[30:] == 7.0).all()
        start = torch.tensor([0, 10, 20, 30, 40], dtype=torch.int32, device="cuda")
        w12.w12_gdn_scan(*args, start=start, S_out=torch.empty_like(args[0]), out=out, mode=mode, status=status)
        assert status.item() == 0
    rows = torch.tensor([[0, 1, 2], [3, 40, 4], [5, -1, 6], [7, 8, 9]], dtype=torch.int32, device="cuda")
    count = torch.tensor([3, 3, 3, 4], dtype=torch.int32, device="cuda")
    out.fill_(7.0)
    _, S = w12.w12_gdn_scan(*args, rows=rows, count=count, S_out=torch.empty_like(args[0]), out=out, status=status)
    assert status.item() == 1
    for r in (1, 2, 3):
        assert torch.equal(S[r], args[0][r])
    assert (out[3:] == 7.0).all()
    check([args[0][:1]] + args[1:], [[0, 1, 2]], out, S[:1], w12.W12_GDN_PATH)
    count[:] = -1
    w12.w12_gdn_scan(*args, rows=rows, count=count, S_out=S, status=status)
    assert status.item() == 1 and torch.equal(S, args[0])


def test_as_the_tree(w12lib):
    """The outputs of a tree's root path are those of the sequence of its nodes."""
    n, H, D = 12, 3, 128
    args = make(1, n, H, H, D, 14)
    parent = torch.arange(-1, n - 1, dtype=torch.int32, device="cuda")
    want = w12.w12_gdn_tree(*args, parent)
    o, _ = w12.w12_gdn_scan(*args, S_out=torch.empty_like(args[0]), out32=True)
    assert (o - want).abs().max() <= 1e-5 * want.abs().max()


@pytest.mark.parametrize("mode", MODES)
def test_streams_graphs_and_repeats(w12lib, mode):
    lens = [100, 1, 70]
    args = make(3, 171, 2, 2, 128, 15)
    start = cuts(lens)
    new = lambda: torch.empty_like(args[0])  # noqa: E731
    o, S = w12.w12_gdn_scan(*args, start=start, S_out=new(), mode=mode)
    side = torch.cuda.Stream()
    Ss = new()
    side.wait_stream(torch.cuda.current_stream())
    o2, _ = w12.w12_gdn_scan(*args, start=start, S_out=Ss, mode=mode, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    Sg, graphs = [new(), new()], []
    for k in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            og, _ = w12.w12_gdn_scan(*args, start=start, S_out=Sg[k], mode=mode)
        graphs.append((graph, og))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):  # at the same time
        for (graph, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(S, Ss)
    for k in range(2):
        assert torch.equal(o, graphs[k][1]) and torch.equal(S, Sg[k])


def test_a_wait_runs_out(w12lib):
    """The loads of the chunked kernel never come: its waits give up after about a second, the status says so, and the
    next call is right."""
    args = make(2, 200, 2, 2, 128, 16)
    start = cuts([100, 100])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, S = w12.w12_gdn_scan(*args, start=start, S_out=torch.empty_like(args[0]), mode=w12.W12_GDN_WY, status=status)
    assert status.item() == 0
    w12.w12_gdn_scan(*args, start=start, S_out=torch.empty_like(args[0]), mode=w12.W12_GDN_WY | w12.W12_GDN_TEST_STALL, status=status)
    assert status.item() == 1
    o2, S2 = w12.w12_gdn_scan(*args, start=start, S_out=torch.empty_like(args[0]), mode=w12.W12_GDN_WY, status=status)
    assert status.item() == 0 and torch.equal(o, o2) and torch.equal(S, S2)


@pytest.mark.parametrize("mode", [w12.W12_GDN_PATH, w12.W12_GDN_WY])
@pytest.mark.parametrize("n,start", [(228, [0, 64, 1000, 100, 228]), (256, [64, 256, 0, 64]), (1280, [0, 640, 1280, 5, 70]),
                                     (400, [0, 100, -7, 100, 200, 190, 200, 400]), (300, [0, 5000, 0, 10, 5, 10, 300]), (64, [64, 0, 64])])
def test_starts_in_disorder(w12lib, mode, n, start):
    """A sequence is what it is alone, or left out; where `start` ascends to n again some sequences still keep the rules."""
    R, H, Hk, D = len(start) - 1, 2, 1, 64
    args = make(R, n, H, Hk, D, n + R)
    S = args[0]
    st = torch.tensor(start, dtype=torch.int32, device="cuda")
    status = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    # what a workspace may hold: not numbers, where nothing has written
    size = w12.load().w12_gdn_scan_workspace_bytes(n, R, H, D, mode)
    junk = torch.full((max(size, 1),), 255, dtype=torch.uint8, device="cuda")
    del junk
    out = torch.full((n, H, D), 5.0, dtype=BF, device="cuda")
    _, after = w12.w12_gdn_scan(*args, start=st, S_out=torch.empty_like(S), out=out, mode=mode, status=status)
    assert status.item() == 1
    kept = [r for r in range(R) if 0 <= start[r] <= start[r + 1] <= n]
    written = torch.zeros(n, dtype=torch.bool, device="cuda")
    done = 0
    for r in range(R):
        rows = slice(start[r], start[r + 1])
        if r in kept and start[r] < start[r + 1] and not torch.equal(after[r], S[r]):
            alone, S1 = w12.w12_gdn_scan(S[r:r + 1], *[x[rows] for x in args[1:]], S_out=torch.empty_like(S[:1]), mode=mode)
            assert torch.equal(after[r], S1[0])
            if not any(start[x] < start[r + 1] and start[r] < start[x + 1] for x in kept if x != r):  # rows of this one only
                assert torch.equal(out[rows], alone)
            written[rows] = True
            done += 1
        else:
            assert torch.equal(after[r], S[r])
            if mode == w12.W12_GDN_PATH:
                assert r not in kept or start[r] == start[r + 1]
    assert (out[~written] == 5).all()
    assert done or mode == w12.W12_GDN_WY
