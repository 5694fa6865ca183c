"""Plain 64-bit references of the operators between a layer's GEMMs (norm,
rotary positions + cache write, tree attention), and the error bounds that the
kernels' arithmetic allows.

Bounds, from the arithmetic alone:
  BF16 has 8 significant bits, so rounding moves a value by at most 2^-8 of it;
  FP32 steps before that add a few 2^-24, taken here as 2^-16 in all.
  e4m3 has 4 significant bits (at most 2^-4 of the value, or half its smallest
  step, 2^-10).
  Attention rounds every weight to BF16 before the product with V: at most
  2^-8 of sum_j p_j |v_j| / sum_j p_j; scores and exponentials in FP32 add less
  than 2^-10 of the same sum for scores of a few units.
"""
import math

import torch

BF = 2.0 ** -8
FP = 2.0 ** -16


def rmsnorm(x, w, eps, residual=None):
    h = x.double()
    if residual is not None:
        h = h + residual.double()
    t = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * w.double()
    return h, t


def group_scales(t):
    """max |t| / 448 over every 128 columns."""
    return torch.stack([t[:, k:k + 128].abs().amax(1) for k in range(0, t.shape[1], 128)], 1) / 448.0


def rope(x, pos, inv_freq, axis, interleaved, norm=None, eps=0.0):
    """(rotated x, the sum of magnitudes that each result is made of); x [n, heads, dim], pos [axes, n]."""
    z = x.double()
    if norm is not None:
        z = z / torch.sqrt((z * z).mean(-1, keepdim=True) + eps) * norm.double()
    y, mag = z.clone(), z.abs().clone()
    half = inv_freq.shape[0]
    for j in range(half):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        turn = pos[axis[j]].double() * inv_freq[j].double()
        c, s = turn.cos()[:, None], turn.sin()[:, None]
        y[..., a] = z[..., a] * c - z[..., b] * s
        y[..., b] = z[..., b] * c + z[..., a] * s
        mag[..., a] = mag[..., b] = z[..., a].abs() + z[..., b].abs()
    return y, mag


def tree_attn(q, k, v, kc, vc, table, ctx_len, parent, req, scale=0.0, softcap=0.0, window=0):
    """(o, sum_j p_j |v_j| / sum_j p_j); kc, vc [pages, page, heads, dim].  One row at a time over what it sees."""
    n, Hq, D = q.shape
    H, page = kc.shape[2], kc.shape[1]
    G = Hq // H
    scale = scale or 1.0 / math.sqrt(D)
    par = parent.tolist() if parent is not None else [-1] * n
    rq = req.tolist() if req is not None else [0] * n
    out = torch.zeros(n, Hq, D, dtype=torch.float64, device=q.device)
    mag = torch.zeros_like(out)
    depth = {}
    for i in range(n):
        line, at = [], i
        while at >= 0:
            line.append(at)
            at = par[at]
        depth[i] = len(line)
        L = int(ctx_len[rq[i]])
        pos = L + len(line) - 1
        first = max(0, pos - window + 1) if window else 0
        if window:
            line = line[:window]
        tok = torch.arange(first, max(first, L), device=q.device)
        at = table[rq[i]].long()[tok // page]
        rows = torch.tensor(line, device=q.device)
        K = torch.cat((kc[at, tok % page], k[rows])).double()  # [keys, H, D]
        V = torch.cat((vc[at, tok % page], v[rows])).double()
        x = torch.einsum("hgd,khd->hgk", q[i].double().view(H, G, D), K) * scale
        if softcap:
            x = softcap * torch.tanh(x / softcap)
        p = torch.softmax(x, -1)
        out[i] = torch.einsum("hgk,khd->hgd", p, V).reshape(Hq, D)
        mag[i] = torch.einsum("hgk,khd->hgd", p, V.abs()).reshape(Hq, D)
    return out, mag


def attn_failures(o, want, mag):
    """Entries of o beyond the bound."""
    tol = (BF + 2.0 ** -10) * mag + (BF + FP) * want.abs() + 1e-30
    return ((o.double() - want).abs() > tol).sum().item()
