"""The tree attention's workspace in Python: who may make or grow it, and when."""
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
