"""Plain 64-bit references of the operators that end a verify step: acceptance
of drafted nodes, and the gated delta rule over sequences.

Bounds, from the arithmetic alone.
  Acceptance is a comparison: u q(y) < p(y), or which p(t) / e(t) is larger.
  The kernel's p carries the rounding of (x - max) / T (2^-23 of a magnitude
  that is below 32 wherever a decision can hang on it), of its exponential and
  of the sums: less than 2^-17 of p in all.  The reference returns the smallest
  relative margin of a request's decisions; where it is above MARGIN the
  outcome has to be the same.  Subtracting q from p can leave little of both, so
  margins there are taken relative to p before the subtraction.
  The scan token by token makes, per token, two dot products of D terms and an
  update of each entry: the error grows by at most (2 D + 8) 2^-24 of the sums of magnitudes
  (the recurrence on absolute values, `scan` returns them), T tokens' at most T
  times that; in chunks the operands of the products are sums of two BF16
  numbers (2^-17 of each) besides.
"""
import torch

MARGIN = 2.0 ** -14


def softmax64(x, T):
    x = x.double() / T
    top = x.max()
    if torch.isinf(top):
        p = (x == top).double()
    else:
        p = torch.exp(x - top)
    return p / p.sum()


def accept(logits, token, parent, req, R, temperature, uniform, noise, draft=None, draft_row=None, row=None,
           root_row=None, max_depth=16):
    """Per request (nodes, next token, margin); plain Python over plain lists."""
    n = len(token)
    out = []
    for r in range(R):
        kids = {}
        for i in range(n):
            if (req[i] if req is not None else 0) == r:
                kids.setdefault(parent[i], []).append(i)
        T = float(temperature[r])
        place, path, margin = -1, [], 1.0
        while True:
            at = (root_row[r] if root_row is not None else n + r) if place < 0 else (row[place] if row is not None else place)
            x = logits[at]
            below = kids.get(place, []) if len(path) < max_depth else []
            if T == 0:
                top = int((x == x.max()).nonzero()[0, 0])
                took = next((i for i in below if token[i] == top), None)
                if took is None:
                    nxt = top
                    break
                place = took
                path.append(took)
                continue
            p = softmax64(x, T)
            took, scale = None, 1.0
            for i in below:
                y = token[i]
                qy = float(draft[draft_row[i]][y]) if draft is not None else 1.0
                left, right = float(uniform[i]) * qy, float(p[y])
                ref = max(left, right, 1e-300)
                margin = min(margin, abs(left - right) / max(ref, float(p.max()) * 1e-6 * (draft is not None)) * scale)
                if left < right:
                    took = i
                    break
                rest = (p - draft[draft_row[i]].double()).clamp(min=0) if draft is not None else p.clone()
                if draft is None:
                    rest[y] = 0
                total = float(rest.sum())
                if total > 0:
                    scale *= total
                    p = rest / total
            if took is None:
                score = p / noise[r].double()
                best, second = torch.topk(score, 2).values.tolist() if len(score) > 1 else (1.0, 0.0)
                margin = min(margin, (best - second) / best * scale if best > 0 else 0.0)
                nxt = int(score.argmax())
                break
            place = took
            path.append(took)
        out.append((path, nxt, margin))
    return out


def scan(S, q, k, v, alpha, beta, seqs):
    """The rule token by token in 64 bits.  seqs: per request the list of its rows.  Returns (o {row: [H, D]}, S, and
    the same of the absolute values)."""
    H, Hk = S.shape[1], k.shape[1]
    heads = torch.arange(H, device=S.device) // (H // Hk)
    S = S.double().clone()
    A = S.abs()
    o, oa = {}, {}
    for r, rows in enumerate(seqs):
        for i in rows:
            kk, vv = k[i][heads].double(), v[i].double()
            a, b = alpha[i].double()[:, None, None], beta[i].double()[:, None]
            now = S[r] * a
            f = b * (vv - (now * kk[:, None, :]).sum(-1))
            S[r] = now + f[..., None] * kk[:, None, :]
            na = A[r] * a
            fa = b.abs() * (vv.abs() + (na * kk.abs()[:, None, :]).sum(-1))
            A[r] = na + fa[..., None] * kk.abs()[:, None, :]
            if q is not None:
                qq = q[i][heads].double()
                o[i] = (S[r] * qq[:, None, :]).sum(-1)
                oa[i] = (A[r] * qq.abs()[:, None, :]).sum(-1)
    return o, S, oa, A
