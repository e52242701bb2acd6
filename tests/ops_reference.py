"""Float64 definitions of the operators around the layer, for the tests."""
import math

import torch

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
U = 2.0 ** -24  # half a step of FP32


def layer_norm(x, w, b, eps):
    x = x.double()
    mu = x.mean(1)
    xc = x - mu[:, None]
    rstd = (xc.square().mean(1) + eps).rsqrt()
    xh = xc * rstd[:, None]
    y = xh if w is None else xh * w.double()
    return (y if b is None else y + b.double()), mu, rstd, xh


def layer_norm_backward(dy, x, mean, rstd, w):
    dy, x, rs = dy.double(), x.double(), rstd.double()[:, None]
    xh = (x - mean.double()[:, None]) * rs
    g = dy if w is None else dy * w.double()
    dx = rs * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0), xh, g


def scores(r, score):
    r = r.double()
    r = torch.where(r > -math.inf, r, -math.inf)  # a NaN counts as masked
    if score == "sigmoid":
        return r.sigmoid()
    m = r.max(1, keepdim=True).values
    e = torch.exp(r - torch.where(m.isinf(), 0.0, m))
    e = torch.where(m == math.inf, (r == math.inf).double(), e)
    z = e.sum(1, keepdim=True)
    return e / torch.where(z == 0, 1.0, z)


def group_route(r, K, G, TG, bias, score, rank, renorm, scale):
    """idx and w in float64, row by row in plain Python loops over sorted lists."""
    s = scores(r, score).cpu()
    c = s if bias is None else s + bias.double().cpu()
    T, E = s.shape
    rd = r.double().cpu()
    ok = (rd > -math.inf) & (c > -math.inf)
    n = E // G
    idx = torch.full((T, K), -1, dtype=torch.int32)
    w = torch.zeros(T, K, dtype=torch.float64)
    sl, cl, okl = s.tolist(), c.tolist(), ok.tolist()
    for t in range(T):
        groups = []
        for g in range(G):
            best = sorted((cl[t][e] for e in range(g * n, g * n + n) if okl[t][e]), reverse=True)[:rank]
            groups.append(sum(best) if best else -math.inf)
        keep = set(sorted(range(G), key=lambda g: (-groups[g], g))[:TG])
        pick = sorted((e for e in range(E) if okl[t][e] and e // n in keep), key=lambda e: (-cl[t][e], e))[:K]
        sel = [sl[t][e] for e in pick]
        if renorm:
            # scores below float64's range share by their logits
            z = sum(sel)
            if z == 0 and sel:
                top = max(float(rd[t, e]) for e in pick)
                sel = [math.exp(float(rd[t, e]) - top) for e in pick]
                z = sum(sel)
            sel = [v / z for v in sel] if sel else sel
        for k, e in enumerate(pick):
            idx[t, k] = e
            w[t, k] = scale * sel[k]
    return idx, w


def group_weights(r, idx, score, renorm, scale):
    """w as a differentiable function of the float64 logits r, the selection fixed."""
    there = (idx >= 0).double()
    if renorm and score == "softmax":
        # the softmax over all experts' normaliser cancels: a softmax over the selected
        # (written out, so that the others' gradient is zero and not float64's residue)
        at = torch.where(idx >= 0, r.gather(1, idx.long().clamp(min=0)), -math.inf)
        e = torch.exp(at - at.max(1, keepdim=True).values.clamp(min=-1e300).detach())
        return scale * e / e.sum(1, keepdim=True).clamp(min=1e-300)
    s = torch.sigmoid(r) if score == "sigmoid" else torch.softmax(r, 1)
    sel = s.gather(1, idx.long().clamp(min=0)) * there
    if renorm:
        sel = sel / sel.sum(1, keepdim=True).clamp(min=1e-300)
    return scale * sel


def quantize_rows(x):
    xf = x.float()
    bad = ~xf.isfinite().all(1)
    scale = torch.where(bad, math.nan, (xf.abs().amax(1).double() / 127).float())  # rounded once
    ok = scale > 0
    q = torch.where(ok[:, None], torch.round(xf.double() / torch.where(ok, scale, 1.0).double()[:, None]), 0.0)
    return q.clamp(-127, 127).to(torch.int8), scale


def matmul_int8(a, sa, b, sb, splits, rows, swiglu):
    """Float64 output, with |gate| where swiglu (for the tolerance)."""
    a, b = a.cpu().double(), b.cpu().double()
    sa, sb = sa.cpu().double(), sb.cpu().double()
    M = splits[-1]
    pick = torch.arange(M) if rows is None else rows.cpu().long()[:M]
    E, N, _ = b.shape
    y = torch.zeros(M, N, dtype=torch.float64)
    for e in range(E):
        lo, hi = splits[e], splits[e + 1]
        if hi > lo:
            y[lo:hi] = (a[pick[lo:hi]] @ b[e].T) * sa[pick[lo:hi], None] * sb[e]
    if not swiglu:
        return y, None
    g, u = y[:, :N // 2], y[:, N // 2:]
    return g * torch.sigmoid(g) * u, g.abs()
