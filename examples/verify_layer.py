"""A verify step of decoder layers whose weights are W12: drafted trees are
selected, every layer computes all their nodes at once over a paged cache, and
the accepted nodes' keys and values are appended to it.

    norm -> QKV GEMM -> rotary -> tree attention -> O GEMM -> residual + norm
         -> gate/up GEMM (SiLU fused) -> down GEMM -> next layer's residual + norm

Run:  python examples/verify_layer.py [--layers 4] [--requests 8] [--nodes 128] [--ctx 4096]
(random weights and cache; prints the time of a step)."""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import lossless_bit_weight_02_gb300 as w12  # noqa: E402


class Layer:
    """One decoder layer: W12 weights, norms, and its part of the paged cache."""

    def __init__(self, hidden, mlp, q_heads, heads, dim, pages, page_tokens, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(N, K):
            return w12.w12_encode((torch.randn(N, K, generator=g, device="cuda") * K ** -0.5).bfloat16())

        self.q_heads, self.heads, self.dim = q_heads, heads, dim
        self.qkv = weight((q_heads + 2 * heads) * dim, hidden)
        self.o = weight(hidden, q_heads * dim)
        self.gate_up = weight(2 * mlp, hidden)  # gate and up rows in turn, 8 of each (W12_GEMM_SILU_MUL)
        self.down = weight(hidden, mlp)
        self.norm_attn, self.norm_mlp = ((1 + 0.1 * torch.randn(2, hidden, generator=g, device="cuda")).bfloat16())
        self.norm_q, self.norm_k = ((1 + 0.1 * torch.randn(2, dim, generator=g, device="cuda")).bfloat16())
        k, v = torch.randn(2, pages, page_tokens, heads, dim, generator=g, device="cuda").bfloat16()
        self.cache = w12.KvCache(k, v)

    def verify(self, x, residual, step, first):
        """(what this layer adds, the residual stream before it, the nodes' keys, their values)."""
        n, D = x.shape[0], self.dim
        r = w12.w12_rmsnorm(x, self.norm_attn, residual=residual)
        h = r.get("h", x)  # the first layer has nothing to add yet
        qkv = w12.w12_gemm(r["y"], self.qkv)
        wq, wk = self.q_heads * D, self.heads * D
        q, k, v = (t.view(n, -1, D) for t in (qkv[:, :wq], qkv[:, wq:wq + wk], qkv[:, wq + wk:]))
        q, k = w12.w12_rope_append(q, k, step["pos"], step["inv_freq"], q_norm=self.norm_q, k_norm=self.norm_k,
                                   q_out=q, k_out=k)  # in place
        # the tree, the lengths and the pages are the same in every layer: analysed once
        a = w12.w12_tree_attn(q, k, v, self.cache, step["table"], step["ctx"], step["parent"], step["req"],
                              workspace=step["workspace"], reuse_plan=not first)
        r = w12.w12_rmsnorm(w12.w12_gemm(a.view(n, wq), self.o), self.norm_mlp, residual=h)
        m = w12.w12_gemm(r["y"], self.gate_up, opts=w12.make_opts(flags=w12.W12_GEMM_SILU_MUL))
        return w12.w12_gemm(m, self.down), r["h"], k, v


def make_step(log_probs, budget, ctx, table, rot, workspace):
    """The nodes of a verify step and what every layer needs of them."""
    sel = w12.w12_tree_select(log_probs, budget=budget, shared=True)
    n = int(sel["count"][0])
    req, depth, parent = (sel[name][:n].contiguous() for name in ("req", "depth", "parent"))
    inv_freq = 10000.0 ** (-torch.arange(rot // 2, device="cuda", dtype=torch.float32) / (rot // 2))
    return {"n": n, "req": req, "parent": parent, "depth": depth, "ctx": ctx, "table": table, "inv_freq": inv_freq,
            "pos": ctx[req.long()] + depth - 1, "workspace": workspace}


def verify(layers, x, step):
    """All layers over the step's nodes: (hidden states, every layer's keys and values)."""
    residual, kv = None, []
    for i, layer in enumerate(layers):
        x, residual, k, v = layer.verify(x, residual, step, i == 0)
        kv.append((k, v))
    return x + residual, kv


def accept(layers, kv, nodes, step, page_tokens):
    """Append the accepted nodes (their indices, root first in every request) and lengthen the requests."""
    req, depth = step["req"][nodes].long(), step["depth"][nodes].long()
    pos = step["ctx"][req].long() + depth - 1
    slots = step["table"][req, pos // page_tokens].long() * page_tokens + pos % page_tokens
    for layer, (k, v) in zip(layers, kv):
        w12.w12_kv_append(k[nodes], v[nodes], layer.cache, slots)
    step["ctx"].scatter_reduce_(0, req, (pos + 1).int(), "amax")


def setup(layers=4, requests=8, nodes=128, ctx=4096, hidden=5120, mlp=17408, q_heads=40, heads=8, dim=128,
          page_tokens=64, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    width = (ctx + 64 + page_tokens - 1) // page_tokens
    table = torch.randperm(requests * width, generator=g, device="cuda").view(requests, width).int()
    lens = torch.randint(ctx // 2, ctx + 1, (requests,), generator=g, device="cuda", dtype=torch.int32)
    stack = [Layer(hidden, mlp, q_heads, heads, dim, requests * width, page_tokens, seed + 1 + i) for i in range(layers)]
    lp = torch.randn(requests, 16, 8, generator=g, device="cuda").mul(2).log_softmax(-1)
    step = make_step(lp, nodes, lens, table, dim, w12.AttnWorkspace("cuda"))
    x = torch.randn(step["n"], hidden, generator=g, device="cuda").bfloat16()
    return stack, step, x


def best_path(step):
    """The deepest path of every request, as a verifier might accept it (node indices, roots first)."""
    parent, depth, req = (step[name].tolist() for name in ("parent", "depth", "req"))
    deepest = {}
    for i, r in enumerate(req):
        if r not in deepest or depth[i] > depth[deepest[r]]:
            deepest[r] = i
    path = []
    for i in deepest.values():
        line = []
        while i >= 0:
            line.append(i)
            i = parent[i]
        path += line[::-1]
    return torch.tensor(path, device="cuda")


def main():
    p = argparse.ArgumentParser()
    for name, value in (("layers", 4), ("requests", 8), ("nodes", 128), ("ctx", 4096)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    layers, step, x = setup(a.layers, a.requests, a.nodes, a.ctx)
    for _ in range(3):
        verify(layers, x, step)
    assert step["workspace"].status() == w12.W12_OK
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(10):
        y, kv = verify(layers, x, step)
    end.record()
    end.synchronize()
    path = best_path(step)
    before = step["ctx"].tolist()
    accept(layers, kv, path, step, layers[0].cache.page_tokens)
    print(f"{a.layers} layers, {step['n']} nodes of {a.requests} requests: {begin.elapsed_time(end) * 100:.0f} us a step")
    print(f"accepted {len(path)} nodes: cached tokens {before} -> {step['ctx'].tolist()}")


if __name__ == "__main__":
    main()
