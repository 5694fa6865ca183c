"""The example's verify step: every operator's output in its place, against
the 64-bit formula of its own inputs, and the accepted nodes in the cache."""
import os
import sys

import pytest
import torch

import layer_ref as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


def test_verify_step(w12lib, monkeypatch):
    import verify_layer as ex
    seen = []

    def record(name):
        f = getattr(w12lib, name)

        def g(*args, **kw):
            args = tuple(a.clone() if isinstance(a, torch.Tensor) else a for a in args)
            out = f(*args, **{**kw, **({"q_out": None, "k_out": None} if name == "w12_rope_append" else {})})
            seen.append((name, args, kw, out))
            if name == "w12_rope_append":  # as the call in place
                kw["q_out"].copy_(out[0]), kw["k_out"].copy_(out[1])
                return kw["q_out"], kw["k_out"]
            return out
        return g

    layers, step, x = ex.setup(2, 3, 60, 300, 512, 1024, 10, 2, 128, 16)
    plain, _ = ex.verify(layers, x, step)
    for name in ("w12_rmsnorm", "w12_rope_append", "w12_tree_attn", "w12_gemm"):
        monkeypatch.setattr(ex.w12, name, record(name))
    y, kv = ex.verify(layers, x, step)
    monkeypatch.undo()
    assert torch.equal(y, plain) and step["workspace"].status() == w12lib.W12_OK
    assert [s[0] for s in seen] == 2 * ["w12_rmsnorm", "w12_gemm", "w12_rope_append", "w12_tree_attn", "w12_gemm",
                                        "w12_rmsnorm", "w12_gemm", "w12_gemm"]
    for name, args, kw, out in seen:
        if name == "w12_rmsnorm":
            h, t = ref.rmsnorm(args[0], args[1], 1e-6, kw["residual"])
            assert ((out["y"].double() - t).abs() <= (ref.BF + ref.FP) * t.abs()).all()
            if "h" in out:
                assert ((out["h"].double() - h).abs() <= (ref.BF + ref.FP) * h.abs()).all()
        elif name == "w12_rope_append":
            for i, norm in ((0, kw["q_norm"]), (1, kw["k_norm"])):
                z, mag = ref.rope(args[i], args[2][None], args[3], [0] * 64, False, norm, 1e-6)
                assert ((out[i].double() - z).abs() <= (ref.BF + ref.FP) * z.abs() + 4e-6 * mag).all()
        elif name == "w12_tree_attn":
            q, k, v, cache, table, ctx, parent, req = args
            o, mag = ref.tree_attn(q, k, v, cache.k, cache.v, table, ctx, parent, req)
            assert ref.attn_failures(out, o, mag) == 0

    path, before = ex.best_path(step), step["ctx"].clone()
    ex.accept(layers, kv, path, step, 16)
    req, depth = step["req"][path].long(), step["depth"][path]
    for r in range(3):
        assert step["ctx"][r] == before[r] + (depth[req == r].max() if (req == r).any() else 0)
    for layer, (k, v) in zip(layers, kv):
        for i in path.tolist():
            r, t = int(step["req"][i]), int(before[step["req"][i]] + step["depth"][i] - 1)
            at = int(step["table"][r, t // 16])
            assert torch.equal(layer.cache.k[at, t % 16], k[i]) and torch.equal(layer.cache.v[at, t % 16], v[i])
    # decoding over the longer cache: a first-level node under the accepted path sees what the path's own child saw
    leaf = int(path[0])
    last = [i for i in path.tolist() if int(step["req"][i]) == int(step["req"][leaf])][-1]
    layer, (k, v) = layers[0], kv[0]
    q = torch.randn(1, 10, 128, device="cuda").bfloat16()
    r = step["req"][last:last + 1]
    o = w12lib.w12_tree_attn(q, k[last:last + 1], v[last:last + 1], layer.cache, step["table"], step["ctx"], None, r)
    x, mag = ref.tree_attn(q, k[last:last + 1], v[last:last + 1], layer.cache.k, layer.cache.v, step["table"],
                           step["ctx"], None, r)
    assert ref.attn_failures(o, x, mag) == 0


def test_the_example_runs(w12lib, capsys, monkeypatch):
    import verify_layer as ex
    monkeypatch.setattr(sys, "argv", ["verify_layer.py", "--layers", "1", "--requests", "2", "--nodes", "24", "--ctx", "200"])
    ex.main()
    assert "accepted" in capsys.readouterr().out
