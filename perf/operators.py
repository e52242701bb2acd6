"""Cases of the operators around the routed experts: layer norm (forward and
backward), group-limited routing (forward and backward) and the 8-bit expert
products with scales per token and channel.

``run`` computes a case in plain torch operations, or, with ``own`` true, by the
calls a user makes of the framework. ``exact`` gives the operators' definitions in
64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-5
# The listed cases' largest work, by which drawn cases are bounded.
MAX_ELEMENTS = 16384 * 2048
MAX_INT8_OPS = 131072 * 2816 * 2048
MAX_INT8_WEIGHTS = 256 * 4096 * 4096


def listed():
    return [
        # the norm in front of a decode step of 128 tokens at model width 4096
        {"name": "ln_decode", "op": "ln", "R": 128, "d": 4096, "dtype": "bf16", "pad": 0},
        # the norm in front of a prefill batch (16384 tokens, width 2048)
        {"name": "ln_prefill", "op": "ln", "R": 16384, "d": 2048, "dtype": "bf16", "pad": 0},
        # the same norm's backward in a training step (8192 tokens, width 4096)
        {"name": "ln_bwd_train", "op": "ln_bwd", "R": 8192, "d": 4096, "dtype": "bf16", "pad": 0},
        # a ragged FP32 batch on rows cut out of a wider buffer, at an odd width
        {"name": "ln_bwd_ragged", "op": "ln_bwd", "R": 5003, "d": 1411, "dtype": "f32", "pad": 5},
        # routing of a decode step: 256 experts in 8 groups, balance bias
        {"name": "route_decode", "op": "route", "T": 128, "E": 256, "K": 8, "G": 8, "TG": 4, "score": "sigmoid",
         "rank": 2, "renorm": True, "bias": True, "dtype": "f32", "empty": 0.0},
        # routing of a prefill batch padded to its length (5 % of the tokens route nowhere)
        {"name": "route_prefill", "op": "route", "T": 16384, "E": 256, "K": 8, "G": 8, "TG": 4, "score": "sigmoid",
         "rank": 2, "renorm": True, "bias": True, "dtype": "f32", "empty": 0.05},
        # softmax routing over an odd batch of BF16 logits, groups of 16, no bias, raw weights
        {"name": "route_ragged", "op": "route", "T": 10007, "E": 96, "K": 5, "G": 6, "TG": 2, "score": "softmax",
         "rank": 1, "renorm": False, "bias": False, "dtype": "bf16", "empty": 0.0},
        # the routing's gradient in a training step: raw softmax weights reach every logit
        {"name": "route_bwd_train", "op": "route_bwd", "T": 16384, "E": 256, "K": 8, "G": 8, "TG": 4,
         "score": "softmax", "rank": 2, "renorm": False, "bias": False, "dtype": "f32", "empty": 0.05},
        # one token through a dense 8-bit projection: the smallest call of a decode loop
        {"name": "int8_token", "op": "int8", "T": 1, "E": 1, "top": 1, "K": 4096, "N": 2048, "swiglu": False,
         "skew": 0.0, "dtype": "bf16", "out": "bf16"},
        # decode: 128 tokens on 8 of 256 experts, gate and up with the SwiGLU epilogue
        {"name": "int8_decode", "op": "int8", "T": 128, "E": 256, "top": 8, "K": 4096, "N": 4096, "swiglu": True,
         "skew": 0.0, "dtype": "bf16", "out": "bf16"},
        # a small layer's down product: 4096 tokens on 2 of 4 experts, FP32 output
        {"name": "int8_small_down", "op": "int8", "T": 4096, "E": 4, "top": 2, "K": 2048, "N": 768, "swiglu": False,
         "skew": 0.0, "dtype": "bf16", "out": "f32"},
        # prefill: 16384 tokens on 8 of 64 unevenly loaded experts, gate and up
        {"name": "int8_prefill", "op": "int8", "T": 16384, "E": 64, "top": 8, "K": 2048, "N": 2816, "swiglu": True,
         "skew": 1.1, "dtype": "bf16", "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ln", "ln_bwd", "route", "route_bwd", "int8", "int8"])
    if op in ("ln", "ln_bwd"):
        d = _log(rng, 16, 8192)
        if rng.random() < 0.7:
            d = max(16, d // 16 * 16)  # model widths; the others stay odd
        return {"op": op, "R": _log(rng, 1, max(1, MAX_ELEMENTS // d // (1 if op == "ln" else 2))), "d": d,
                "dtype": rng.choice(["f32", "bf16", "bf16", "f16"]), "pad": rng.choice([0, 0, 0, 3, 8])}
    if op in ("route", "route_bwd"):
        G = rng.choice([1, 2, 4, 5, 8, 16])
        E = G * rng.randint(4 if G > 1 else 8, 256 // G)
        TG = rng.randint(1, G)
        K = rng.randint(1, min(16, E // G * TG))
        return {"op": op, "T": _log(rng, 1, MAX_ELEMENTS // 8 // 256), "E": E, "K": K, "G": G, "TG": TG,
                "score": rng.choice(["sigmoid", "softmax"]), "rank": rng.choice([1, 2]),
                "renorm": K > 1 and rng.random() < 0.6, "bias": rng.random() < 0.6,
                "dtype": rng.choice(["f32", "f32", "bf16", "f16"]), "empty": rng.choice([0.0, 0.0, 0.1])}
    E = rng.choice([1, 1, 4, 8, 32, 64, 128])
    top = min(E, rng.choice([1, 2, 4, 8]))
    K = _log(rng, 64, 4096) // 16 * 16
    swiglu = rng.random() < 0.5
    N = _log(rng, 32, min(4096, MAX_INT8_WEIGHTS // 4 // E // K))
    N = N // 2 * 2 if swiglu else N
    T = _log(rng, 1, max(1, min(16384, MAX_INT8_OPS // top // N // K)))
    return {"op": op, "T": T, "E": E, "top": top, "K": K, "N": N, "swiglu": swiglu,
            "skew": rng.choice([0.0, 1.1]), "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]),
            "out": rng.choice(["bf16", "bf16", "f32"])}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rows(t, pad):
    """The same rows as a cut of a buffer that is `pad` columns wider."""
    if pad == 0:
        return t
    wide = torch.zeros(t.shape[0], t.shape[1] + pad, dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    dt = DTYPES[c["dtype"]]
    if c["op"] in ("ln", "ln_bwd"):
        R, d = c["R"], c["d"]
        # a residual stream: channel scales and offsets differ, a few channels are large
        ch = torch.exp(0.5 * _randn(g, d)) * (1 + 15 * (torch.rand(d, generator=g, device="cuda") < 0.005))
        x = (_randn(g, R, d) * ch + 0.3 * _randn(g, d)).to(dt)
        s = {"case": c, "x": _rows(x, c["pad"]), "w": 1 + 0.1 * _randn(g, d), "b": 0.1 * _randn(g, d)}
        if c["op"] == "ln_bwd":
            s["dy"] = _rows(_randn(g, R, d).to(dt), c["pad"])
            xd = x.double()  # the forward's saved statistics
            mu = xd.mean(1)
            s["mean"] = mu.float()
            s["rstd"] = (1 / torch.sqrt(((xd - mu[:, None]) ** 2).mean(1) + EPS)).float()
        return s
    if c["op"] in ("route", "route_bwd"):
        T, E, K = c["T"], c["E"], c["K"]
        r = (_randn(g, T, E) + 0.3 * _randn(g, E)).to(dt)
        if c["empty"]:  # padding tokens: every expert masked
            r[torch.rand(T, generator=g, device="cuda") < c["empty"]] = -math.inf
        s = {"case": c, "r": r, "bias": 0.05 * _randn(g, E) if c["bias"] else None}
        if c["op"] == "route_bwd":
            s["dw"] = _randn(g, T, K)
            s["idx"] = _exact_route(c, r, s["bias"])[0].to(torch.int32)
        return s
    T, E, top, K, N = c["T"], c["E"], c["top"], c["K"], c["N"]
    s = {"case": c, "x": (_randn(g, T, K) * torch.exp(0.3 * _randn(g, K))).to(dt)}
    q = torch.empty(E, N, K, dtype=torch.int8, device="cuda")
    for e in range(E):  # per-channel quantised normal weights: the largest of a channel at 127
        q[e] = (_randn(g, N, K) * 35).round_().clamp_(-127, 127).to(torch.int8)
    s["b"] = q
    s["b_scale"] = (0.5 + torch.rand(E, N, generator=g, device="cuda")) / (35 * math.sqrt(K))
    s["offsets"] = s["rows"] = None
    s["splits"] = [0, T]
    if E > 1:
        score = _randn(g, T, E) - c["skew"] * torch.log(1.0 + torch.randperm(E, generator=g, device="cuda"))
        flat = score.topk(top, dim=1).indices.reshape(-1)
        order = torch.argsort(flat, stable=True)
        s["rows"] = (order // top).to(torch.int32)
        counts = torch.bincount(flat, minlength=E)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["splits"] = s["offsets"].tolist()  # what the plain form walks over
    return s


# ---- plain forms -----------------------------------------------------------

def _plain_ln(s):
    x = s["x"].float()
    mu = x.mean(1, keepdim=True)
    xc = x - mu
    rstd = 1 / torch.sqrt((xc * xc).mean(1, keepdim=True) + EPS)
    y = xc * rstd * s["w"] + s["b"]
    return {"y": y.to(s["x"].dtype), "mean": mu[:, 0], "rstd": rstd[:, 0]}


def _plain_ln_bwd(s):
    x, dy = s["x"].float(), s["dy"].float()
    rstd = s["rstd"][:, None]
    xh = (x - s["mean"][:, None]) * rstd
    gy = dy * s["w"]
    dx = rstd * (gy - gy.mean(1, keepdim=True) - xh * (gy * xh).mean(1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xh).sum(0), "dbias": dy.sum(0)}


def _plain_scores(c, r, wide):
    """Scores in 64 bits where they decide the order of near ties, else in 32."""
    r = r.to(torch.float64 if wide else torch.float32)
    if c["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-r))
    m = r.max(1, keepdim=True).values
    e = torch.exp(r - torch.where(m == -math.inf, torch.zeros_like(m), m))
    z = e.sum(1, keepdim=True)
    return e / torch.where(z == 0, torch.ones_like(z), z)


def _first_max(v):
    """The index of each row's maximum, the lowest of equal ones."""
    n = v.shape[1]
    at = torch.arange(n, device=v.device)
    return torch.where(v == v.max(1, keepdim=True).values, at, n).min(1).values


def _plain_route(s):
    c, r = s["case"], s["r"]
    T, E, K, G = c["T"], c["E"], c["K"], c["G"]
    sc = _plain_scores(c, r, True)
    ch = sc if s["bias"] is None else sc + s["bias"].double()
    lowest = torch.tensor(-math.inf, dtype=ch.dtype, device=ch.device)
    ch = torch.where(r > -math.inf, ch, lowest)
    if G > 1:
        gr = ch.view(T, G, E // G)
        best = gr.max(2).values
        if c["rank"] == 2 and E // G > 1:
            second = _drop(gr.reshape(T * G, E // G), _first_max(gr.reshape(T * G, E // G)), lowest)
            second = second.max(1).values.view(T, G)
            best = torch.where(second == -math.inf, best, best + second)
        keep = torch.zeros(T, G, dtype=torch.bool, device=r.device)
        for _ in range(c["TG"]):
            j = _first_max(best)
            keep.scatter_(1, j[:, None], True)
            best = _drop(best, j, lowest)
        ch = torch.where(keep.repeat_interleave(E // G, 1), ch, lowest)
    idx = torch.empty(T, K, dtype=torch.int64, device=r.device)
    for k in range(K):
        j = _first_max(ch)
        idx[:, k] = torch.where(ch.gather(1, j[:, None])[:, 0] == -math.inf, -1, j)
        ch = _drop(ch, j, lowest)
    w = torch.where(idx < 0, 0.0, sc.gather(1, idx.clamp(min=0)))
    if c["renorm"]:
        z = w.sum(1, keepdim=True)
        w = w / torch.where(z == 0, torch.ones_like(z), z)
    return {"idx": idx.to(torch.int32), "w": (2.5 * w).float()}


def _drop(v, j, lowest):
    v = v.clone()
    v.scatter_(1, j[:, None], lowest.item())
    return v


def _plain_route_bwd(s):
    c, idx = s["case"], s["idx"].long()
    sc = _plain_scores(c, s["r"], False)
    there = idx >= 0
    sel = torch.where(there, sc.gather(1, idx.clamp(min=0)), 0.0)
    u = torch.where(there, 2.5 * s["dw"], 0.0)
    if c["renorm"]:
        z = sel.sum(1, keepdim=True)
        z = torch.where(z == 0, torch.ones_like(z), z)
        u = torch.where(there, (u - (u * sel / z).sum(1, keepdim=True)) / z, 0.0)
    full = torch.zeros_like(sc).scatter_add_(1, idx.clamp(min=0), u)
    if c["score"] == "sigmoid":
        d = full * sc * (1 - sc)
    else:
        d = sc * (full - (u * sel).sum(1, keepdim=True))
    return {"dlogits": d.to(s["r"].dtype)}


def _plain_quantize(x):
    xf = x.float()
    scale = (xf.abs().amax(1).double() / 127).float()  # torch divides by a plain number through its reciprocal
    div = torch.where(scale == 0, torch.ones_like(scale), scale)
    # the quotient in 64 bits: 32 would move values next to a half step
    return (xf.double() / div.double()[:, None]).round().clamp(-127, 127).to(torch.int8), scale


def _plain_int8(s):
    c = s["case"]
    q, scale = _plain_quantize(s["x"])
    out = []
    for e in range(c["E"]):
        lo, hi = s["splits"][e], s["splits"][e + 1]
        if lo == hi:
            continue
        at = slice(lo, hi) if s["rows"] is None else s["rows"][lo:hi].long()
        p = q[at].float() @ s["b"][e].float().t()
        p = p * scale[at][:, None] * s["b_scale"][e]
        if c["swiglu"]:
            a, u = p[:, :c["N"] // 2], p[:, c["N"] // 2:]
            p = a / (1 + torch.exp(-a)) * u
        out.append(p.to(DTYPES[c["out"]]))
    return {"q": q, "scale": scale, "out": torch.cat(out)}


_PLAIN = {"ln": _plain_ln, "ln_bwd": _plain_ln_bwd, "route": _plain_route, "route_bwd": _plain_route_bwd,
          "int8": _plain_int8}


def run(state):
    c = state["case"]
    if not own:
        return _PLAIN[c["op"]](state)
    from mixture_experts_ffn_fp32_gb300 import api
    if c["op"] == "ln":
        return api.layer_norm(state["x"], state["w"], state["b"], eps=EPS)
    if c["op"] == "ln_bwd":
        return api.layer_norm_backward(state["dy"], state["x"], state["mean"], state["rstd"], state["w"])
    if c["op"] == "route":
        return api.group_route(state["r"], c["K"], n_groups=c["G"], topk_groups=c["TG"], bias=state["bias"],
                               score=c["score"], group_rank=c["rank"], renormalize=c["renorm"], scale=2.5)
    if c["op"] == "route_bwd":
        return {"dlogits": api.group_route_backward(state["dw"], state["idx"], state["r"], score=c["score"],
                                                    renormalize=c["renorm"], scale=2.5)}
    qx = api.quantize_rows(state["x"])
    out = api.matmul_int8(qx["q"], qx["scale"], state["b"], state["b_scale"], offsets=state["offsets"],
                          rows=state["rows"], swiglu=c["swiglu"], out_dtype=c["out"])
    return {"q": qx["q"], "scale": qx["scale"], "out": out}


def work(case):
    c = case
    z = SIZE[c["dtype"]]
    if c["op"] == "ln":
        n = c["R"] * c["d"]
        return {"bytes": 2 * n * z + 8 * c["d"] + 8 * c["R"], "flops": 8 * n}
    if c["op"] == "ln_bwd":
        n = c["R"] * c["d"]
        return {"bytes": 3 * n * z + 12 * c["d"] + 8 * c["R"], "flops": 14 * n}
    if c["op"] == "route":
        n = c["T"] * c["E"]
        return {"bytes": n * z + (4 * c["E"] if c["bias"] else 0) + 8 * c["T"] * c["K"], "flops": 10 * n}
    if c["op"] == "route_bwd":
        n = c["T"] * c["E"]
        read = n if c["score"] == "softmax" else c["T"] * c["K"]  # sigmoid: the selected logits alone
        return {"bytes": (n + read) * z + 8 * c["T"] * c["K"], "flops": 8 * n}
    M = c["T"] * c["top"]
    used = c["E"] * (1 - (1 - 1 / c["E"]) ** M) if c["E"] > 1 else 1  # experts that receive rows
    no = c["N"] // 2 if c["swiglu"] else c["N"]
    return {"bytes": c["T"] * c["K"] * (z + 1) + 4 * c["T"] + used * c["N"] * (c["K"] + 4) + 4 * M
            + M * no * SIZE[c["out"]], "flops": 2 * M * c["N"] * c["K"]}


# ---- definitions in 64 bits, apart from the plain forms ---------------------

def _exact_route(c, r, bias):
    """Selected ids (-1: none) and the selected scores: a stable sort of the choices."""
    rd = r.double()
    ok = rd > -math.inf
    if c["score"] == "sigmoid":
        sc = torch.sigmoid(rd)
    else:
        sc = torch.nan_to_num(torch.softmax(rd, 1), nan=0.0)
    ch = sc + (0 if bias is None else bias.double())
    ch = ch.masked_fill(~ok, -math.inf)
    T, E, G, n = c["T"], c["E"], c["G"], c["E"] // c["G"]
    if G > 1:
        top = ch.view(T, G, n).sort(dim=2, descending=True, stable=True).values[:, :, :min(c["rank"], n)]
        none = top[:, :, 0] == -math.inf
        group = top.masked_fill(top == -math.inf, 0.0).sum(2).masked_fill(none, -math.inf)
        order = group.sort(dim=1, descending=True, stable=True).indices
        rank = torch.empty_like(order).scatter_(1, order, torch.arange(G, device=r.device).expand(T, G).contiguous())
        ch = ch.masked_fill((rank >= c["TG"]).repeat_interleave(n, 1), -math.inf)
    val, idx = ch.sort(dim=1, descending=True, stable=True)
    val, idx = val[:, :c["K"]], idx[:, :c["K"]]
    none = val == -math.inf
    return idx.masked_fill(none, -1), sc.gather(1, idx).masked_fill(none, 0.0)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "ln":
        x = s["x"].double()
        var, mu = torch.var_mean(x, 1, correction=0)
        rstd = (var + EPS) ** -0.5
        return {"y": torch.addcmul(s["b"].double(), (x - mu[:, None]) * rstd[:, None], s["w"].double()),
                "mean": mu, "rstd": rstd}
    if c["op"] == "ln_bwd":
        x, dy, w = s["x"].double(), s["dy"].double(), s["w"].double()
        k = s["rstd"].double()[:, None]
        xh = (x - s["mean"].double()[:, None]) * k
        d = c["d"]
        m1 = (dy @ w)[:, None] / d
        m2 = torch.einsum("rd,rd,d->r", dy, xh, w)[:, None] / d
        return {"dx": k * (dy * w - m1 - m2 * xh), "dweight": torch.einsum("rd,rd->d", dy, xh),
                "dbias": dy.sum(0)}
    if c["op"] == "route":
        idx, sel = _exact_route(c, s["r"], s["bias"])
        if c["renorm"]:
            sel = sel / sel.sum(1, keepdim=True).clamp(min=1e-300)
        return {"idx": idx.to(torch.int32), "w": 2.5 * sel}
    if c["op"] == "route_bwd":
        # each weight's derivative by each selected score, then the scores' by the logits
        T, E, K = c["T"], c["E"], c["K"]
        idx = s["idx"].long()
        r = s["r"].double()
        there = (idx >= 0).double()
        sc = torch.sigmoid(r) if c["score"] == "sigmoid" else torch.nan_to_num(torch.softmax(r, 1), nan=0.0)
        sel = sc.gather(1, idx.clamp(min=0)) * there
        dw = 2.5 * s["dw"].double() * there
        if c["renorm"]:
            z = sel.sum(1, keepdim=True).clamp(min=1e-300)
            dw = (dw / z - (dw * sel).sum(1, keepdim=True) / z ** 2) * there
        full = torch.zeros(T, E, dtype=torch.float64, device=r.device)
        full.scatter_add_(1, idx.clamp(min=0), dw)
        if c["score"] == "sigmoid":
            return {"dlogits": full * sc * torch.sigmoid(-r)}
        return {"dlogits": sc * full - sc * (sc * full).sum(1, keepdim=True)}
    x = s["x"].double()
    sd = x.abs().max(1).values / 127
    s32 = sd.float().double()  # the step that the stored scale stands for
    q = torch.where(s32[:, None] > 0, torch.round(x / s32[:, None].clamp(min=1e-300)), 0.0).clamp(-127, 127)
    lens = [b - a for a, b in zip(s["splits"], s["splits"][1:])]
    no = c["N"] // 2 if c["swiglu"] else c["N"]
    out = torch.empty(sum(lens), no, dtype=torch.float64, device=x.device)
    at = 0
    for e, n in enumerate(lens):
        if n == 0:
            continue
        pick = torch.arange(at, at + n, device=x.device) if s["rows"] is None else s["rows"][at:at + n].long()
        p = torch.einsum("mk,nk->mn", q[pick], s["b"][e].double())
        p *= s32[pick][:, None] * s["b_scale"][e].double()[None, :]
        if c["swiglu"]:
            p = p[:, :no] * torch.sigmoid(p[:, :no]) * p[:, no:]
        out[at:at + n] = p
        at += n
    return {"q": q.to(torch.int8), "scale": sd, "out": out}
