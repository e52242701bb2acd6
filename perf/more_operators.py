"""Cases of the operators on both sides of a block: the norms before and after it
fused with its gate and residual scale (forward and backward), and the low-rank
adapters of many requests beside a shared projection.

``run`` computes a case in plain torch operations, or, with ``own`` true, by the
calls a user makes of the framework. ``exact`` gives the operators' definitions in
64 bits.

    z  = Norm(y; wp, bp) or y,  x' = alpha x + g z,  n = Norm(x'; w, b)
    out[t] = base[t] + scale_e (x[t] A_e^T) B_e^T,  e the adapter of row t
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-5
# The listed cases' largest work, by which drawn cases are bounded.
MAX_ELEMENTS = 16384 * 2048
MAX_ADAPTER_ELEMENTS = 16384 * (2048 + 2816)
MAX_ADAPTER_MACS = 8192 * 64 * (4096 + 4096)
MAX_ADAPTER_WEIGHTS = 128 * 64 * (4096 + 4096)


def listed():
    return [
        # between the blocks of a decode step of 128 tokens at model width 4096
        {"name": "norm_decode", "op": "norm", "R": 128, "d": 4096, "dtype": "bf16", "pad": 0, "kind": "rms",
         "post": True, "gate": "none", "alpha": 1.0, "next": True},
        # a prefill batch (16384 tokens, width 2048), a gate per channel
        {"name": "norm_prefill", "op": "norm", "R": 16384, "d": 2048, "dtype": "bf16", "pad": 0, "kind": "rms",
         "post": True, "gate": "channel", "alpha": 1.0, "next": True},
        # FP32 rows of an odd width cut out of wider buffers, a gate per element, residual scale
        {"name": "norm_ragged", "op": "norm", "R": 5003, "d": 1411, "dtype": "f32", "pad": 5, "kind": "layer",
         "post": True, "gate": "element", "alpha": 1.7, "next": True},
        # the backward in a training step (8192 tokens, width 4096), a gate per channel
        {"name": "norm_bwd_train", "op": "norm_bwd", "R": 8192, "d": 4096, "dtype": "bf16", "pad": 0, "kind": "rms",
         "post": True, "gate": "channel", "alpha": 1.0, "next": True},
        # layer norms with biases and a gate per element
        {"name": "norm_bwd_gated", "op": "norm_bwd", "R": 4096, "d": 768, "dtype": "f16", "pad": 0, "kind": "layer",
         "post": True, "gate": "element", "alpha": 0.8, "next": True},
        # one token of one request: the smallest call of a decode loop
        {"name": "adapter_token", "op": "adapter", "T": 1, "d": 4096, "N": 2048, "r": 16, "E": 8, "requests": 1,
         "none": 0.0, "dtype": "bf16", "out": "bf16"},
        # decode: 128 requests of a token each on 64 adapters, some without one
        {"name": "adapter_decode", "op": "adapter", "T": 128, "d": 4096, "N": 4096, "r": 16, "E": 64,
         "requests": 128, "none": 0.1, "dtype": "bf16", "out": "bf16"},
        # decode of many requests on as many larger adapters
        {"name": "adapter_decode_wide", "op": "adapter", "T": 256, "d": 4096, "N": 4096, "r": 64, "E": 128,
         "requests": 256, "none": 0.0, "dtype": "bf16", "out": "f32"},
        # a prefill batch of 40 packed prompts beside a gate/up projection
        {"name": "adapter_prefill", "op": "adapter", "T": 16384, "d": 2048, "N": 2816, "r": 16, "E": 16,
         "requests": 40, "none": 0.1, "dtype": "bf16", "out": "bf16"},
        # few long prompts on large adapters
        {"name": "adapter_prefill_wide", "op": "adapter", "T": 8192, "d": 4096, "N": 4096, "r": 64, "E": 4,
         "requests": 6, "none": 0.0, "dtype": "bf16", "out": "bf16"},
        # an odd batch, widths and rank, FP16
        {"name": "adapter_ragged", "op": "adapter", "T": 3001, "d": 1411, "N": 1003, "r": 12, "E": 37,
         "requests": 211, "none": 0.2, "dtype": "f16", "out": "f16"},
        # an FP32 layer's projection
        {"name": "adapter_f32", "op": "adapter", "T": 4096, "d": 768, "N": 2048, "r": 8, "E": 8, "requests": 19,
         "none": 0.0, "dtype": "f32", "out": "f32"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    d = _log(rng, lo, hi)
    return max(lo, d // 16 * 16) if rng.random() < 0.7 else d  # model widths; the others stay odd


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "norm_bwd", "adapter", "adapter", "adapter", "adapter"])
    if op != "adapter":
        d = _width(rng, 16, 8192)
        post = rng.random() < 0.7
        nxt = rng.random() < 0.85
        return {"op": op, "R": _log(rng, 1, max(1, MAX_ELEMENTS // d // (1 if op == "norm" else 2))), "d": d,
                "dtype": rng.choice(["f32", "bf16", "bf16", "f16"]), "pad": rng.choice([0, 0, 0, 3, 8]),
                "kind": rng.choice(["rms", "rms", "layer"]), "post": post,
                "gate": rng.choice(["none", "channel", "element"]), "alpha": rng.choice([1.0, 1.0, 1.7]), "next": nxt}
    d, N = _width(rng, 64, 8192), _width(rng, 32, 8192)
    r = rng.choice([4, 8, 8, 16, 16, 16, 24, 32, 64, 128])
    E = _log(rng, 1, max(1, min(256, MAX_ADAPTER_WEIGHTS // r // (d + N))))
    T = _log(rng, 1, max(1, min(16384, MAX_ADAPTER_ELEMENTS // (d + N), MAX_ADAPTER_MACS // r // (d + N))))
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    return {"op": op, "T": T, "d": d, "N": N, "r": r, "E": E, "requests": _log(rng, 1, T),
            "none": rng.choice([0.0, 0.1, 0.4]), "dtype": dtype,
            "out": "f32" if dtype == "f32" else rng.choice([dtype, dtype, "f32"])}


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
    if c["op"] == "adapter":
        return _prepare_adapter(c, g, dt)
    R, d, layer = c["R"], c["d"], c["kind"] == "layer"
    # a residual stream: channel scales and offsets differ, a few channels are large
    ch = torch.exp(0.5 * _randn(g, d)) * (1 + 15 * (torch.rand(d, generator=g, device="cuda") < 0.005))
    s = {"case": c, "x": _rows((_randn(g, R, d) * ch + 0.3 * _randn(g, d)).to(dt), c["pad"])}
    s["y"] = _rows((_randn(g, R, d) * torch.exp(0.3 * _randn(g, d)) + 0.1).to(dt), c["pad"])
    s["w"] = 1 + 0.1 * _randn(g, d) if c["next"] else None
    s["b"] = 0.1 * _randn(g, d) if c["next"] and layer else None
    s["wp"] = 0.5 + 0.1 * _randn(g, d) if c["post"] else None
    s["bp"] = 0.1 * _randn(g, d) if c["post"] and layer else None
    s["gate"] = None
    if c["gate"] == "channel":
        s["gate"] = 0.3 + 0.1 * _randn(g, d)
    elif c["gate"] == "element":
        s["gate"] = _rows(torch.sigmoid(_randn(g, R, d)).to(dt), c["pad"])
    if c["op"] == "norm_bwd":
        # what the forward left: the new stream in place of the old one, and the statistics
        f = _exact_norm(c, s)
        s["x"] = _rows(f["x"].to(dt), c["pad"])
        s["stats"] = f["stats"].float()
        s["dn"] = _rows(_randn(g, R, d).to(dt), c["pad"]) if c["next"] else None
        s["dx"] = _rows((0.5 * _randn(g, R, d)).to(dt), c["pad"])
    return s


def _prepare_adapter(c, g, dt):
    T, d, N, r, E = c["T"], c["d"], c["N"], c["r"], c["E"]
    s = {"case": c, "x": (_randn(g, T, d) * torch.exp(0.3 * _randn(g, d))).to(dt),
         "a": (_randn(g, E, r, d) / math.sqrt(d)).to(dt), "b": (_randn(g, E, N, r) / math.sqrt(r)).to(dt),
         "scale": 0.25 + torch.rand(E, generator=g, device="cuda"), "base": _randn(g, T, N).to(DTYPES[c["out"]])}
    # requests lie one behind the other; each brings an adapter, or none (E)
    cuts = torch.randperm(T - 1, generator=g, device="cuda")[:c["requests"] - 1].sort().values + 1
    request = torch.searchsorted(cuts, torch.arange(T, device="cuda"), right=True)
    which = torch.randint(E, (c["requests"],), generator=g, device="cuda")
    which[torch.rand(c["requests"], generator=g, device="cuda") < c["none"]] = E
    ids = which[request]
    s["rows"] = torch.argsort(ids, stable=True).to(torch.int32)
    counts = torch.bincount(ids, minlength=E + 1)[:E]
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    s["splits"] = s["offsets"].tolist()  # what the plain form walks over
    return s


# ---- plain forms -----------------------------------------------------------

def _plain_stats(v, layer):
    m = v.mean(1, keepdim=True) if layer else torch.zeros_like(v[:, :1])
    vc = v - m if layer else v
    return m, 1 / torch.sqrt((vc * vc).mean(1, keepdim=True) + EPS)


def _plain_norm(s):
    c = s["case"]
    layer = c["kind"] == "layer"
    x, z = s["x"].float(), s["y"].float()
    one, zero = torch.ones_like(x[:, :1]), torch.zeros_like(x[:, :1])
    stats = {"ym": zero, "yr": one, "xm": zero, "xr": one}
    if c["post"]:
        stats["ym"], stats["yr"] = _plain_stats(z, layer)
        z = (z - stats["ym"]) * stats["yr"] * s["wp"]
        if layer:
            z = z + s["bp"]
    if s["gate"] is not None:
        z = z * s["gate"].float()
    v = c["alpha"] * x + z
    out = {"x": v.to(s["x"].dtype)}
    if c["next"]:
        stats["xm"], stats["xr"] = _plain_stats(v, layer)
        n = (v - stats["xm"]) * stats["xr"] * s["w"]
        if layer:
            n = n + s["b"]
        out["n"] = n.to(s["x"].dtype)
    keys = ("ym", "yr", "xm", "xr") if layer else ("yr", "xr")
    out["stats"] = torch.cat([stats[k] for k in keys], 1).t().contiguous()
    return out


def _plain_norm_bwd(s):
    c = s["case"]
    layer = c["kind"] == "layer"
    dt = s["x"].dtype
    st = s["stats"][:, :, None]
    ym, yr, xm, xr = st if layer else (0.0, st[0], 0.0, st[1])
    out = {}
    t = s["dx"].float()
    if c["next"]:
        dn = s["dn"].float()
        xh = (s["x"].float() - xm) * xr
        h = dn * s["w"]
        m = h.mean(1, keepdim=True) if layer else 0.0
        t = t + xr * (h - m - xh * (h * xh).mean(1, keepdim=True))
        out["dweight"] = (dn * xh).sum(0)
        if layer:
            out["dbias"] = dn.sum(0)
    out["dx"] = (c["alpha"] * t).to(dt)
    yh = z = s["y"].float()
    if c["post"]:
        yh = (yh - ym) * yr
        z = yh * s["wp"]
        if layer:
            z = z + s["bp"]
    k = t
    if c["gate"] == "channel":
        out["dgate"] = (t * z).sum(0)
        k = t * s["gate"]
    elif c["gate"] == "element":
        out["dgate"] = (t * z).to(dt)
        k = t * s["gate"].float()
    if c["post"]:
        out["dpost_weight"] = (k * yh).sum(0)
        if layer:
            out["dpost_bias"] = k.sum(0)
        k = k * s["wp"]
        m = k.mean(1, keepdim=True) if layer else 0.0
        k = yr * (k - m - yh * (k * yh).mean(1, keepdim=True))
    out["dy"] = k.to(dt)
    return out


def _plain_adapter(s):
    c = s["case"]
    out = s["base"].float()
    out = out.clone() if out is s["base"] else out
    for e in range(c["E"]):
        lo, hi = s["splits"][e], s["splits"][e + 1]
        if lo == hi:
            continue
        at = s["rows"][lo:hi].long()
        v = (s["x"][at].float() @ s["a"][e].float().t()) * s["scale"][e]
        out[at] += v @ s["b"][e].float().t()
    return {"out": out.to(s["base"].dtype)}


_PLAIN = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "adapter": _plain_adapter}


def run(state):
    c = state["case"]
    if not own:
        return _PLAIN[c["op"]](state)
    from mixture_experts_ffn_fp32_gb300 import api
    s = state
    if c["op"] == "adapter":
        return {"out": api.adapter_add(s["base"], s["x"], s["a"], s["b"], s["offsets"], rows=s["rows"],
                                       scale=s["scale"])}
    if c["op"] == "norm":
        return api.block_norm(s["x"], s["y"], weight=s["w"], bias=s["b"], post_weight=s["wp"], post_bias=s["bp"],
                              gate=s["gate"], alpha=c["alpha"], kind=c["kind"], post=c["post"], norm=c["next"],
                              eps=EPS)
    return api.block_norm_backward(s["x"], s["stats"], y=s["y"], dn=s["dn"], dx=s["dx"], weight=s["w"],
                                   post_weight=s["wp"], post_bias=s["bp"], gate=s["gate"], alpha=c["alpha"],
                                   kind=c["kind"], post=c["post"])


def work(case):
    c = case
    z = SIZE[c["dtype"]]
    if c["op"] != "adapter":
        n, layer = c["R"] * c["d"], c["kind"] == "layer"
        element = 1 if c["gate"] == "element" else 0
        vectors = (1 + layer) * (c["post"] + c["next"]) + (c["gate"] == "channel")
        stats = 4 * c["R"] * (4 if layer else 2)
        if c["op"] == "norm":
            return {"bytes": (3 + c["next"] + element) * n * z + 4 * c["d"] * vectors + stats, "flops": 14 * n}
        return {"bytes": (4 + 2 * c["next"] + 2 * element) * n * z + 8 * c["d"] * vectors + stats, "flops": 28 * n}
    T, d, N, r, E = c["T"], c["d"], c["N"], c["r"], c["E"]
    there = T * (1 - c["none"])
    used = E * (1 - (1 - 1 / E) ** (c["requests"] * (1 - c["none"]))) if E > 1 else 1
    return {"bytes": there * d * z + 2 * T * N * SIZE[c["out"]] + used * r * (d + N) * z + 4 * T,
            "flops": 2 * there * r * (d + N)}


# ---- definitions in 64 bits, apart from the plain forms ---------------------

def _exact_stats(v, layer):
    if layer:
        var, mu = torch.var_mean(v, 1, correction=0)
    else:
        var, mu = torch.linalg.vecdot(v, v) / v.shape[1], torch.zeros_like(v[:, 0])
    return mu, (var + EPS) ** -0.5


def _exact_norm(c, s):
    layer = c["kind"] == "layer"
    x, y = s["x"].double(), s["y"].double()
    R = c["R"]
    stats = [y.new_zeros(R), y.new_ones(R), y.new_zeros(R), y.new_ones(R)]
    if c["post"]:
        stats[0], stats[1] = _exact_stats(y, layer)
        y = torch.einsum("rd,r,d->rd", y - stats[0][:, None], stats[1], s["wp"].double())
        y = y if s["bp"] is None else y + s["bp"].double()
    gate = torch.ones_like(x[:1]) if s["gate"] is None else s["gate"].double()
    out = {"x": torch.addcmul(c["alpha"] * x, gate.expand_as(x), y)}
    if c["next"]:
        stats[2], stats[3] = _exact_stats(out["x"], layer)
        n = torch.einsum("rd,r,d->rd", out["x"] - stats[2][:, None], stats[3], s["w"].double())
        out["n"] = n if s["b"] is None else n + s["b"].double()
    out["stats"] = torch.stack(stats if layer else stats[1::2])
    return out


def _exact_norm_bwd(c, s):
    """Each norm's rows by the projection that its Jacobian is."""
    layer, d = c["kind"] == "layer", c["d"]
    st = s["stats"].double()
    ym, yr, xm, xr = st if layer else (torch.zeros_like(st[0]), st[0], torch.zeros_like(st[0]), st[1])

    def through(h, vh, r):
        p = h - torch.einsum("rd,rd,re->re", h, vh, vh) / d
        return r[:, None] * (p - h.sum(1, keepdim=True) / d if layer else p)

    out, t = {}, s["dx"].double()
    if c["next"]:
        xh = torch.einsum("rd,r->rd", s["x"].double() - xm[:, None], xr)
        dn = s["dn"].double()
        t = t + through(torch.einsum("rd,d->rd", dn, s["w"].double()), xh, xr)
        out["dweight"] = torch.einsum("rd,rd->d", dn, xh)
        if layer:
            out["dbias"] = torch.einsum("rd->d", dn)
    out["dx"] = c["alpha"] * t
    y = s["y"].double()
    yh = torch.einsum("rd,r->rd", y - ym[:, None], yr) if c["post"] else y
    g = torch.ones_like(t[:1]) if s["gate"] is None else s["gate"].double()
    g = g.expand_as(t)
    if c["gate"] != "none":
        z = torch.addcmul(torch.zeros_like(yh) if s["bp"] is None else s["bp"].double().expand_as(yh), yh,
                          torch.ones_like(yh) if s["wp"] is None else s["wp"].double().expand_as(yh))
        out["dgate"] = torch.einsum("rd,rd->d", t, z) if c["gate"] == "channel" else t * z
    if c["post"]:
        out["dpost_weight"] = torch.einsum("rd,rd,rd->d", t, g, yh)
        if layer:
            out["dpost_bias"] = torch.einsum("rd,rd->d", t, g)
        out["dy"] = through(torch.einsum("rd,rd,d->rd", t, g, s["wp"].double()), yh, yr)
    else:
        out["dy"] = t * g
    return out


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "norm":
        return _exact_norm(c, s)
    if c["op"] == "norm_bwd":
        return _exact_norm_bwd(c, s)
    out = s["base"].double()
    x = s["x"].double()
    for e, (lo, hi) in enumerate(zip(s["splits"], s["splits"][1:])):
        if lo < hi:
            pick = s["rows"][lo:hi].long()
            inner = torch.einsum("td,kd->tk", x[pick], s["a"][e].double())
            out.index_add_(0, pick, torch.einsum("tk,nk->tn", inner, s["scale"][e].double() * s["b"][e].double()))
    return {"out": out}
