"""Float64 definitions of the norms on both sides of a block and of the low-rank
adapters, with bounds of what FP32 arithmetic may be off by.

Bounds count half steps of FP32 (U): a sum of d terms runs in chains of at most
16 (rows past the registers: d / 1024) and a tree of 10, k = 26 + d / 1024 steps."""
import torch

from tests.ops_reference import HALF, U

TINY = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}  # half of the smallest subnormal


def store(v, dtype):
    """What rounding once to dtype may add."""
    return HALF[dtype] * v.abs() + TINY[dtype]


def stats_of(v, layer, eps):
    mu = v.mean(1, keepdim=True) if layer else torch.zeros_like(v[:, :1])
    return mu, ((v - mu).square().mean(1, keepdim=True) + eps).rsqrt()


def stats_error(v, mu, r, e, k, layer):
    """Errors of the mean and, relatively, of r, of values that are off by e."""
    em = e.mean(1, keepdim=True) + U * (2 * mu.abs() + k / r) if layer else torch.zeros_like(mu)
    return em, U * (k + 8) + r * e.square().mean(1, keepdim=True).sqrt()


def norm_error(v, mu, r, e, w, b, n, k, layer):
    """Of n = (v - mu) r w + b."""
    em, er = stats_error(v, mu, r, e, k, layer)
    xh = (v - mu) * r
    return w.abs() * (r * (e + em) + xh.abs() * (er + 6 * U)) + U * (b.abs() + n.abs())


def block_norm(x, y, gate, alpha, wp, bp, w, b, layer, post, norm, eps):
    """dict of value, bound: x (x') and n before rounding, stats [4, R] (with means)."""
    dt = x.dtype
    k = 26 + x.shape[1] / 1024
    one, zero = torch.ones(1, dtype=torch.float64, device=x.device), torch.zeros(1, dtype=torch.float64, device=x.device)
    v, e = x.double(), torch.zeros_like(x, dtype=torch.float64)
    R = x.shape[0]
    st = [zero.expand(R), one.expand(R), zero.expand(R), one.expand(R)]
    se = [torch.zeros_like(s) for s in st]
    out = {}
    if y is not None:
        z = y.double()
        ez = torch.zeros_like(z)
        if post:
            mu, r = stats_of(z, layer, eps)
            W, B = one if wp is None else wp.double(), zero if bp is None else bp.double()
            n = (z - mu) * r * W + B
            em, er = stats_error(z, mu, r, ez, k, layer)
            st[0], st[1], se[0], se[1] = mu[:, 0], r[:, 0], em[:, 0], (er * r)[:, 0]
            ez = norm_error(z, mu, r, ez, W, B, n, k, layer)
            z = n
        g = one if gate is None else gate.double()
        al = float(torch.tensor(alpha, dtype=torch.float32))
        v = al * x.double() + g * z
        e = g.abs() * ez + U * (2 * (g * z).abs() + (al * x.double()).abs() + v.abs())
        out["x"] = (v, e + store(v, dt))
    if norm:
        mu, r = stats_of(v, layer, eps)
        W, B = one if w is None else w.double(), zero if b is None else b.double()
        n = (v - mu) * r * W + B
        em, er = stats_error(v, mu, r, e, k, layer)
        st[2], st[3], se[2], se[3] = mu[:, 0], r[:, 0], em[:, 0], (er * r)[:, 0]
        en = norm_error(v, mu, r, e, W, B, n, k, layer)
        out["n"] = (n, en + store(n, dt))
    out["stats"] = (torch.stack(st), torch.stack(se))
    if not layer:
        out["stats"] = tuple(t[1::2] for t in out["stats"])
    return out


def block_norm_backward(x, stats, y, dn, dx, gate, alpha, wp, bp, w, layer, post):
    """dict of value, bound."""
    dt = x.dtype
    n, d = x.shape
    k = 26 + d / 1024
    chain = min(n, n / 16 + 60) + 8  # the longest chain of a column's sum
    st = stats.double()[:, :, None]
    ym, yr, xm, xr = st if layer else (0 * st[0], st[0], 0 * st[0], st[1])
    one, zero = torch.ones(1, dtype=torch.float64, device=x.device), torch.zeros(1, dtype=torch.float64, device=x.device)
    out = {}

    def mean(v):
        return v.mean(1, keepdim=True)

    t = torch.zeros_like(x, dtype=torch.float64) if dx is None else dx.double()
    et = U * t.abs()
    if dn is not None:
        dnd = dn.double()
        xh = (x.double() - xm) * xr
        h = dnd * (one if w is None else w.double())
        t = t + xr * (h - (mean(h) if layer else 0) - xh * mean(h * xh))
        et = et + U * (t.abs() + xr * (k + 14) * (h.abs() + mean(h.abs()) + xh.abs() * mean((h * xh).abs())))
        out["dweight"] = ((dnd * xh).sum(0), U * (chain + 4) * (dnd * xh).abs().sum(0))
        if layer:
            out["dbias"] = (dnd.sum(0), U * chain * dnd.abs().sum(0))
    al = float(torch.tensor(alpha, dtype=torch.float32)) if y is not None else 1.0
    out["dx"] = (al * t, abs(al) * et + U * (al * t).abs() + store(al * t, dt))
    if y is None:
        return out
    z = yh = y.double()
    ez = torch.zeros_like(z)
    W, B = one if wp is None else wp.double(), zero if bp is None else bp.double()
    if post:
        yh = (z - ym) * yr
        z = yh * W + B
        ez = U * (4 * (yh * W).abs() + 2 * B.abs() + z.abs())
    g = one if gate is None else gate.double()
    s1 = (t * yh, et * yh.abs() + 4 * U * (t * yh).abs())
    if gate is not None and gate.dim() == 2:
        v = t * z
        out["dgate"] = (v, et * z.abs() + ez * t.abs() + U * v.abs() + store(v, dt))
    elif gate is not None:
        bound = s1[1] * W.abs() + et * B.abs() + U * (chain + 6) * ((t * yh * W).abs() + (t * B).abs())
        out["dgate"] = ((t * z).sum(0), bound.sum(0))
    kk, ek = t * g, g.abs() * et + U * (t * g).abs()
    if post:
        out["dpost_weight"] = ((kk * yh).sum(0), (ek * yh.abs() + U * (chain + 6) * (kk * yh).abs()).sum(0))
        if layer:
            out["dpost_bias"] = (kk.sum(0), (ek + U * (chain + 2) * kk.abs()).sum(0))
        ek = ek * W.abs() + U * (kk * W).abs()
        kk = kk * W
        dy = yr * (kk - (mean(kk) if layer else 0) - yh * mean(kk * yh))
        ek = yr * (ek + mean(ek) + yh.abs() * mean(ek * yh.abs()) +
                   U * (k + 14) * (kk.abs() + mean(kk.abs()) + yh.abs() * mean((kk * yh).abs())))
        kk = dy
    out["dy"] = (kk, ek + store(kk, dt))
    return out


def adapter_add(base, x, a, b, offsets, rows, scale, out_dtype, parts=3):
    """Value and bound of the adapters' sum, row by row of a group. FP32 chains of a product of K
    terms are at most K long, whatever adds them; the inner values v are held in `parts` pieces of 8
    bits at least, which together leave 2^-8 parts of them."""
    T, N = x.shape[0], b.shape[1]
    val = torch.zeros(T, N, dtype=torch.float64, device=x.device) if base is None else base.double().clone()
    err = U * val.abs()
    off = [min(max(o, 0), T) for o in offsets.tolist()]
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        at = torch.arange(lo, hi, device=x.device) if rows is None else rows[lo:hi].long()
        if not len(at):
            continue
        s = 1.0 if scale is None else float(scale[e])
        A, B, X = a[e].double(), b[e].double(), x[at].double()
        v = s * (X @ A.T)
        ev = U * (sum_steps(A.shape[1]) + 4) * abs(s) * (X.abs() @ A.abs().T) + 2.0 ** (-8 * parts) * v.abs()
        delta = v @ B.T
        val[at] += delta
        err[at] += ev @ B.abs().T + U * (sum_steps(A.shape[0] * parts) + 2) * (v.abs() @ B.abs().T)
    return val, err + U * val.abs() + store(val, out_dtype)


def sum_steps(K):
    """Roundings that a term of a sum of K passes: chains of any order, tensor cores' included, whose sums of
    up to 16 terms drop what lies 2^-24 below the largest."""
    return K + 32
