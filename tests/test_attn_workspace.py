"""The tree attention's workspace in Python: who may make or grow it, and when."""
import threading
import time

import pytest
import torch

import lossless_bit_weight_02_gb300 as w12

CUDA = torch.device("cuda", 0)


@pytest.fixture
def capturing(monkeypatch):
    """The current stream is captured, as far as the binding can tell."""
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)


def test_not_grown_during_a_capture(capturing):
    ws = w12.AttnWorkspace("cpu")
    ws.device = CUDA
    with pytest.raises(RuntimeError, match="before the capture"):
        ws.ensure(ws.buf.numel() + 1)
    assert ws.ensure(ws.buf.numel()) is ws.buf  # what is there is used


def test_not_made_during_a_capture(capturing, monkeypatch):
    monkeypatch.setattr(w12, "_stream_of", lambda dev: 12345)
    monkeypatch.setattr(w12, "_ws_cache", {})
    for make in (lambda: w12.AttnWorkspace(CUDA), lambda: w12.default_attn_workspace(CUDA)):
        with pytest.raises(RuntimeError, match="before the capture"):
            make()
    assert not w12._ws_cache


def test_outgrown_buffers_stay():
    """A captured graph may hold the address of any buffer that the workspace has had; small steps of growth do not
    leave one behind each."""
    ws = w12.AttnWorkspace("cpu")
    had = {ws.buf.data_ptr()}
    for nbytes in range(300, 200000, 700):
        buf = ws.ensure(nbytes)
        assert buf.numel() >= nbytes and not buf.any()
        had.add(buf.data_ptr())
    assert {b.data_ptr() for b in ws._outgrown} | {ws.buf.data_ptr()} == had
    assert sum(b.numel() for b in ws._outgrown) < ws.buf.numel() < 2 * nbytes


class FakeLib:
    """The library's attention entry points, without a GPU: what would be launched is noted."""

    def __init__(self):
        self.calls = []

    def w12_tree_attn_workspace_bytes(self, n, R, q_heads, heads, dim):
        return 1000 + 10 * n * q_heads

    def w12_tree_attn(self, args, cache, ws, nbytes, stream):
        self.calls.append(w12._attn_args.unpack(args))
        return w12.W12_OK


@pytest.fixture
def fake(monkeypatch):
    """The binding over CPU tensors and a library that launches nothing."""
    lib = FakeLib()
    monkeypatch.setattr(w12, "_lib", lib)
    monkeypatch.setattr(w12, "_attn_bytes", {})
    monkeypatch.setattr(w12, "_ws_cache", {})
    monkeypatch.setattr(w12, "_current_device_of", lambda t, name: t.device)
    monkeypatch.setattr(w12, "_stream_of", lambda dev: 12345)
    return lib


class CpuCache(w12.KvCache):
    """A cache of CPU tensors."""

    def __init__(self, pages, page, heads, dim, pad=0):
        k = torch.zeros(pages, page, heads, dim + pad).bfloat16()[..., :dim]
        self.k, self.v, self.device = k, k.clone(), k.device
        self.page_tokens, self.heads, self.dim = page, heads, dim
        self._c, self._at = None, 0
        self._sizes = (*k.shape, *k.stride())


def host_case(**change):
    i32 = torch.int32
    c = dict(q=torch.zeros(6, 4, 64).bfloat16(), k=torch.zeros(6, 2, 64).bfloat16(), v=torch.zeros(6, 2, 64).bfloat16(),
             cache=CpuCache(8, 16, 2, 64), block_table=torch.zeros(3, 4, dtype=i32), ctx_len=torch.zeros(3, dtype=i32),
             parent=torch.zeros(6, dtype=i32), req=torch.zeros(6, dtype=i32), window=7)
    return {**c, **change}


def test_a_plan_is_used_again_for_its_own_tree_only(fake, monkeypatch):
    """Layers of one step share a plan; after a call with anything else that a plan depends on, it is refused."""
    c = host_case()
    run = lambda ws, reuse, **change: w12.w12_tree_attn(**{**c, **change}, workspace=ws, reuse_plan=reuse)  # noqa: E731
    ws = w12.AttnWorkspace("cpu")
    ws.ensure(1 << 16)  # large enough, but no plan was ever made in it
    with pytest.raises(ValueError, match="reuse_plan"):
        run(ws, True)
    run(ws, False)
    layer = dict(q=c["q"] + 1, k=c["k"] + 1, v=c["v"] + 1, cache=CpuCache(8, 16, 2, 64), scale=0.5, softcap=3.0, max_ctas=2)
    for _ in range(2):
        run(ws, True, **layer)
    assert [a[-1] for a in fake.calls] == [0, 1, 1]
    copies = {name: c[name].clone() for name in ("parent", "req", "ctx_len", "block_table")}
    run(ws, True, **copies)  # what they hold counts, not where it lies
    fake.calls.pop()
    for other in (dict(window=0), dict(window=8), dict(block_table=c["block_table"][:, :3]), dict(cache=CpuCache(9, 16, 2, 64)),
                  dict(cache=CpuCache(8, 8, 2, 64)), dict(cache=CpuCache(8, 16, 2, 64, 8)),
                  dict(q=torch.zeros(6, 8, 64).bfloat16()),
                  dict(cache=CpuCache(8, 16, 1, 64), k=c["k"][:, :1].contiguous(), v=c["v"][:, :1].contiguous()),
                  dict(q=c["q"][:5], k=c["k"][:5], v=c["v"][:5], parent=c["parent"][:5], req=c["req"][:5]),
                  dict(block_table=c["block_table"][:2], ctx_len=c["ctx_len"][:2])):
        with pytest.raises(ValueError, match="reuse_plan"):
            run(ws, True, **other)
        run(ws, True)  # (a refused call launched nothing: the plan still stands)
        run(ws, False, **other)  # another call between two layers
        with pytest.raises(ValueError, match="reuse_plan"):
            run(ws, True)
        run(ws, False)
    fake.calls.clear()
    fake.w12_tree_attn = lambda *a: w12.W12_ERR_CUDA
    with pytest.raises(w12.W12Error):
        run(ws, False)
    del fake.w12_tree_attn
    with pytest.raises(ValueError, match="reuse_plan"):  # no telling what that call has left
        run(ws, True)
    run(ws, False)
    with monkeypatch.context() as m:  # a captured step: planned and used again in the graph's replays, not outside
        m.setattr(w12, "_capturing", lambda dev: True)
        run(ws, False)
        run(ws, True)
    with pytest.raises(ValueError, match="captured"):
        run(ws, True)
    run(ws, False)
    run(ws, True)
    ws.ensure(2 * ws.buf.numel())  # a new buffer: no plan in it
    with pytest.raises(ValueError, match="reuse_plan"):
        run(ws, True)
    assert [a[-1] for a in fake.calls] == [0, 0, 1, 0, 1]


def test_a_workspace_elsewhere_is_refused(fake):
    """Its address would be handed to kernels of the tensors' device."""
    ws = w12.AttnWorkspace("meta")
    with pytest.raises(ValueError, match="workspace is on"):
        w12.w12_tree_attn(**host_case(), workspace=ws)
    assert not fake.calls


def in_threads(count, work):
    """work(i) in `count` threads at once; what they return."""
    got, failed, start = [None] * count, [], threading.Barrier(count)

    def body(i):
        try:
            start.wait(10)
            got[i] = work(i)
        except BaseException as e:  # noqa: BLE001 (handed to the caller)
            failed.append(e)

    threads = [threading.Thread(target=body, args=(i,)) for i in range(count)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not failed and not any(t.is_alive() for t in threads), failed
    return got


def test_calls_on_one_workspace_take_turns(fake):
    """A call's launches follow one another on the stream: no other thread's come between them, and none sees a
    buffer that another is about to replace."""
    inside, overlaps = [], []

    def call(args, cache, ws, nbytes, stream):
        inside.append(ws)
        time.sleep(0.002)
        overlaps.append(len(inside) > 1)
        inside.pop()
        return w12.W12_OK

    fake.w12_tree_attn = call
    ws = w12.AttnWorkspace("cpu")
    cases = [host_case(), host_case(q=torch.zeros(6, 40, 64).bfloat16())]
    in_threads(2, lambda i: [w12.w12_tree_attn(**cases[i], workspace=ws) for _ in range(20)])
    assert len(overlaps) == 40 and not any(overlaps)


def test_threads_have_default_workspaces_of_their_own(fake):
    """Two threads on one stream, each with the layers of its own step."""
    cases = [host_case(), host_case(window=3)]

    def steps(i):
        for _ in range(50):
            for layer in range(4):
                w12.w12_tree_attn(**cases[i], reuse_plan=layer > 0)
        return w12.default_attn_workspace("cpu")

    a, b = in_threads(2, steps)
    assert a is not b and len(fake.calls) == 400


def decode_case(n, seed, heads=2, dim=64, page=16):
    """Arguments of a call: n requests of one node, or of a chain of 40 nodes where n is 1."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    count = 40 if n == 1 else n
    kc, vc = torch.randn(2, 4 * n, page, heads, dim, generator=g, device="cuda").bfloat16()
    q, k, v = (torch.randn(count, h, dim, generator=g, device="cuda").bfloat16() for h in (2 * heads, heads, heads))
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(q=q, k=k, v=v, cache=w12.KvCache(kc, vc), block_table=torch.arange(4 * n, **i32).view(n, 4),
                ctx_len=torch.arange(n, **i32) % 64 + 1, parent=torch.arange(count, **i32) - 1 if n == 1 else None,
                req=None if n == 1 else torch.arange(n, **i32))


@pytest.mark.gpu
def test_two_graphs_on_one_stream(w12lib):
    """The default workspace of a captured stream: refused where the capture would have to make it, used where a
    call before the capture has, and right whichever graph is replayed first."""
    small, large = decode_case(5, 1), decode_case(1, 2)
    want = [w12lib.w12_tree_attn(**c) for c in (small, large)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with pytest.raises(RuntimeError, match="before the capture"):
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=s):
            w12lib.w12_tree_attn(**small)
    with torch.cuda.stream(s):
        for c in (large, small):
            w12lib.w12_tree_attn(**c)
    s.synchronize()
    graphs, outs = [], []
    for c in (small, large):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            outs.append(w12lib.w12_tree_attn(**c))
    for first in (1, 0):
        for i in (first, 1 - first, first):
            outs[i].zero_()
            graphs[i].replay()
            torch.cuda.synchronize()
            assert torch.equal(outs[i], want[i])
    with torch.cuda.stream(s):
        assert w12lib.default_attn_workspace(CUDA).status() == w12lib.W12_OK


@pytest.mark.gpu
def test_capture_with_a_workspace_that_is_too_small(w12lib):
    small, large = decode_case(5, 1), decode_case(1, 2)
    ws = w12lib.AttnWorkspace("cuda")
    want = w12lib.w12_tree_attn(**small, workspace=ws)
    assert ws.buf.numel() < w12lib._attn_workspace_bytes(40, 1, 4, 2, 64)
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="before the capture"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            w12lib.w12_tree_attn(**large, workspace=ws)
    assert torch.equal(w12lib.w12_tree_attn(**small, workspace=ws), want)


@pytest.mark.gpu
def test_a_graph_outlives_its_workspaces_growth(w12lib):
    """A decode call is captured, then a larger call on the workspace makes it grow: the graph's replays still have
    their own memory, whatever is allocated afterwards."""
    small, large = decode_case(5, 1), decode_case(1, 2)
    ws = w12lib.AttnWorkspace("cuda")
    want = w12lib.w12_tree_attn(**small, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = w12lib.w12_tree_attn(**small, workspace=ws)
    held = ws.buf.data_ptr(), ws.buf.numel()
    w12lib.w12_tree_attn(**large, workspace=ws)
    torch.cuda.synchronize()
    assert ws.buf.data_ptr() != held[0]
    others = [torch.full((held[1],), 7, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert all(o.data_ptr() + o.numel() <= held[0] or o.data_ptr() >= held[0] + held[1] for o in others)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and all((o == 7).all() for o in others)


@pytest.mark.gpu
def test_another_call_between_two_layers(w12lib):
    """A call of fewer nodes between two layers of a step: its plan is not taken for the step's, and the step's
    result is right once it is planned again."""
    small, large = decode_case(5, 1), decode_case(1, 2)
    ws = w12lib.AttnWorkspace("cuda")
    want = w12lib.w12_tree_attn(**large, workspace=ws)
    assert torch.equal(w12lib.w12_tree_attn(**large, workspace=ws, reuse_plan=True), want)
    w12lib.w12_tree_attn(**small, workspace=ws)
    with pytest.raises(ValueError, match="reuse_plan"):
        w12lib.w12_tree_attn(**large, workspace=ws, reuse_plan=True)
    assert torch.equal(w12lib.w12_tree_attn(**large, workspace=ws), want)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):  # a step of two layers
        outs = [w12lib.w12_tree_attn(**large, workspace=ws, reuse_plan=i > 0) for i in range(2)]
    with pytest.raises(ValueError, match="captured"):
        w12lib.w12_tree_attn(**large, workspace=ws, reuse_plan=True)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


@pytest.mark.gpu
def test_two_threads_on_one_stream(w12lib):
    """Steps of three layers, planned and used again, from two threads on one stream: each gets its own results."""
    cases = [decode_case(5, 1), decode_case(1, 2)]
    want = [w12lib.w12_tree_attn(**c) for c in cases]
    torch.cuda.synchronize()
    shared = w12lib.AttnWorkspace("cuda")

    def steps(i):
        outs = [w12lib.w12_tree_attn(**cases[i], reuse_plan=layer > 0) for _ in range(60) for layer in range(3)]
        outs += [w12lib.w12_tree_attn(**cases[i], workspace=shared) for _ in range(60)]
        torch.cuda.synchronize()
        return all(torch.equal(o, want[i]) for o in outs)

    assert in_threads(2, steps) == [True, True]
    assert shared.status() == w12lib.W12_OK


@pytest.mark.gpu
def test_a_workspace_in_host_memory_is_refused(w12lib):
    with pytest.raises(ValueError, match="workspace is on"):
        w12lib.w12_tree_attn(**decode_case(5, 1), workspace=w12lib.AttnWorkspace("cpu"))
