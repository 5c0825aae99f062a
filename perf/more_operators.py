"""Cases of the norm, of the 8-bit expert operators and of the layer for a few tokens, and each operator's plain form.

* ``norm``       r = h + delta (stored in 16 bits), v = r / sqrt(mean(r^2) + eps) * weight; v in 16 bits, or in e4m3 with a
                 scale for each 128 values of a row, or both;
* ``norm_grad``  the gradients of its 16-bit output: dh (the residual's own gradient added) and dweight;
* ``mm8``        y[r] = W[e(r)] x[r], rows grouped by expert (``offsets``), both in e4m3: a scale for each 128 values of a row of
                 x, and for each block of 128 x 128 of W;
* ``geglu8``     a[r] = GELU(g) * u with [g; u] = W[e(r)] x[r] in those types, a in e4m3 with a scale for each 128 values;
* ``layer``      a routed layer and its shared expert for up to 32 tokens: y[t] = sum_j gates[t, j] FFN(e(t, j), x[t]) +
                 FFN(shared, x[t]), weights in 16 bits or in e4m3 with block scales.

Where ``own`` is true the calls go to the library's kernels, else to elementary torch operations in 32 bits.
"""

import math

import torch

own = False

D, F, F_SHARED, E, TOP_K = 2816, 704, 2816, 128, 8   # this repository's full-shape layer
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn
EPS = 1e-6
TINY = 2.0 ** -100   # the smallest maximum that a scale is made for: a group of zeros has a scale too


# ---------------------------------------------------------------- cases

def listed():
    full = {"experts": E, "top_k": TOP_K, "spread": 0.5}
    norm = {"op": "norm", "d": D, "dtype": "bf16", "weight": True}
    layer = {"op": "layer", **full, "d": D, "f": F, "shared": F_SHARED}
    return [
        # between two layers of one request's decode step: the last layer's fp32 output is added, latency counts
        {"name": "norm, 1 token", **norm, "rows": 1, "delta": "f32", "out": "16"},
        # between two layers of a 4096-token prompt chunk: 8-bit rows for the products that follow
        {"name": "norm, 4096 tokens, 8 bits", **norm, "rows": 4096, "delta": "bf16", "out": "8"},
        # training backward of the same, 4096 tokens
        {"name": "norm gradient, 4096 tokens", "op": "norm_grad", "rows": 4096, "d": D, "dtype": "bf16", "weight": True,
         "residual": True},
        # training backward of a batch of short samples, whose length is odd
        {"name": "norm gradient, short", "op": "norm_grad", "rows": 601, "d": D, "dtype": "f16", "weight": True,
         "residual": False},
        # down projections of a decode batch of 32 requests, two rows per expert; fp32 for a 32-bit combine
        {"name": "8-bit down, 32 tokens", "op": "mm8", **full, "tokens": 32, "pad": 0, "n": D, "k": F, "out": "f32"},
        # down projections of a 4096-token prompt chunk: about 256 rows per expert, ragged
        {"name": "8-bit down, 4096 tokens", "op": "mm8", **full, "tokens": 4096, "pad": 0, "n": D, "k": F, "out": "bf16"},
        # the shared expert's gate/up projection of such a chunk: one group of all rows
        {"name": "8-bit shared, 4096 tokens", "op": "mm8", "experts": 1, "top_k": 1, "spread": 0.0, "tokens": 4096,
         "pad": 0, "n": 2 * F_SHARED, "k": D, "out": "bf16"},
        # gate/up and the gated product of a decode batch, in a buffer with room left at its end
        {"name": "8-bit gated, 33 tokens", "op": "geglu8", **full, "tokens": 33, "pad": 40, "n": F, "k": D, "tanh": False},
        # gate/up and the gated product of a 4096-token prompt chunk
        {"name": "8-bit gated, 4096 tokens", "op": "geglu8", **full, "tokens": 4096, "pad": 0, "n": F, "k": D, "tanh": True},
        # one decode step of one request, 16-bit experts
        {"name": "layer, 1 token", **layer, "tokens": 1, "dtype": "bf16", "weights": "16", "tanh": False},
        # the same with 8-bit experts
        {"name": "layer, 1 token, 8 bits", **layer, "tokens": 1, "dtype": "bf16", "weights": "8", "tanh": False},
        # seven requests, or seven drafted tokens of one
        {"name": "layer, 7 tokens", **layer, "tokens": 7, "dtype": "f16", "weights": "16", "tanh": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "mm8", "mm8", "geglu8", "layer", "layer"])
    dtype = rng.choice(["bf16", "f16"])
    if op in ("norm", "norm_grad"):
        case = {"op": op, "rows": _log(rng, 1, 8192), "d": 8 * _log(rng, 8, 704), "dtype": dtype,
                "weight": rng.random() < 0.7}
        if op == "norm":
            return {**case, "delta": rng.choice(["none", dtype, "f32"]), "out": rng.choice(["8", "16", "both"])}
        return {**case, "residual": rng.random() < 0.5}
    experts = _log(rng, 4, 128)
    case = {"op": op, "experts": experts, "top_k": min(experts, rng.randint(1, 8)), "spread": rng.choice([0.0, 0.5, 1.0])}
    if op == "layer":
        return {**case, "tokens": _log(rng, 1, 32), "d": 16 * _log(rng, 4, 176), "f": 16 * _log(rng, 4, 88),
                "shared": rng.choice([0, 16 * _log(rng, 4, 176)]), "dtype": dtype, "weights": rng.choice(["16", "8"]),
                "tanh": rng.random() < 0.5}
    case = {**case, "tokens": _log(rng, 1, 4096), "pad": rng.choice([0, 0, 33]), "k": 16 * _log(rng, 4, 176)}
    if op == "geglu8":
        return {**case, "n": 16 * _log(rng, 4, 44), "tanh": rng.random() < 0.5}
    if rng.random() < 0.25:   # one group
        case.update(experts=1, top_k=1)
    return {**case, "n": 8 * _log(rng, 8, 176), "out": rng.choice(["bf16", "f16", "f32"])}


# ---------------------------------------------------------------- inputs

def _randn(g, dtype, *shape, scale=1.0):
    return torch.randn(*shape, generator=g, device="cuda", dtype=DTYPES[dtype]) * scale


def _blocks(n):
    return (n + 127) // 128


def _weights8(g, *shape, scale):
    """e4m3 weights [..., n, k] and the scales of their blocks, from normal values."""
    *e, n, k = shape
    v = torch.randn(*e, 128 * _blocks(n), 128 * _blocks(k), generator=g, device="cuda").mul_(scale)
    v[..., n:, :] = 0
    v[..., k:] = 0
    v = v.view(*e, _blocks(n), 128, _blocks(k), 128)
    s = v.abs().amax((-3, -1)) / 448
    q = (v / s[..., :, None, :, None]).to(E4M3).view(*e, 128 * _blocks(n), 128 * _blocks(k))
    return q[..., :n, :k].contiguous(), s


def _rows8(v):
    """Rows in e4m3 and their scales, as the norm leaves them."""
    m, d = v.shape
    p = torch.nn.functional.pad(v, (0, -d % 128)).view(m, _blocks(d), 128)
    s = p.abs().amax(-1).clamp(min=TINY) / 448
    return (p / s[:, :, None]).view(m, -1)[:, :d].to(E4M3), s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c, op = dict(case), case["op"]
    if op in ("norm", "norm_grad"):
        m, d, dt = c["rows"], c["d"], c["dtype"]
        # a residual stream: channels of different size, a few of them large
        size = torch.exp(0.5 * torch.randn(d, generator=g, device="cuda"))
        c.update(h=(torch.randn(m, d, generator=g, device="cuda") * size).to(DTYPES[dt]),
                 w=(1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(DTYPES[dt]) if c["weight"] else None)
        zeros = lambda *shape, t: torch.zeros(*shape, dtype=t, device="cuda")  # noqa: E731
        if op == "norm_grad":
            c.update(dy=_randn(g, dt, m, d), dres=_randn(g, dt, m, d) if c["residual"] else None,
                     dh=zeros(m, d, t=DTYPES[dt]), dw=zeros(d, t=torch.float32) if c["weight"] else None,
                     workspace=zeros(4 * d * min(m, 512), t=torch.uint8))
            return c
        delta = None if c["delta"] == "none" else _randn(g, c["delta"], m, d, scale=0.3)
        c.update(delta=delta, r=None if delta is None else zeros(m, d, t=DTYPES[dt]),
                 y=zeros(m, d, t=DTYPES[dt]) if c["out"] != "8" else None,
                 y8=zeros(m, d, t=E4M3) if c["out"] != "16" else None,
                 s=zeros(m, _blocks(d), t=torch.float32) if c["out"] != "16" else None)
        return c
    # top-k of logits with a popularity of each expert, as a router leaves them
    e, t = c["experts"], c["tokens"]
    logits = torch.randn(t, e, generator=g, device="cuda")
    logits += c["spread"] * torch.randn(e, generator=g, device="cuda")
    top = logits.topk(c["top_k"])
    if op == "layer":
        d, f, fs, dt = c["d"], c["f"], c["shared"], c["dtype"]
        c.update(x=_randn(g, dt, t, d), ids=top.indices.int(), gates=torch.softmax(top.values, 1),
                 y=torch.zeros(t, d, dtype=DTYPES[dt], device="cuda"))
        sizes = {"gu": (e, 2 * f, d), "down": (e, d, f), "shared_gu": (2 * fs, d), "shared_down": (d, fs)}
        for name, shape in sizes.items():
            if not fs and name.startswith("shared"):
                c[name] = c[name + "_scale"] = None
            elif c["weights"] == "8":
                c[name], c[name + "_scale"] = _weights8(g, *shape, scale=shape[-1] ** -0.5)
            else:
                c[name], c[name + "_scale"] = _randn(g, dt, *shape, scale=shape[-1] ** -0.5), None
        c.update(workspace=torch.zeros(2 * t * (c["top_k"] * f + fs), dtype=torch.uint8, device="cuda"))
        return c
    n, k, m = c["n"], c["k"], t * c["top_k"] + c["pad"]
    counts = torch.bincount(top.indices.reshape(-1), minlength=e)
    offsets = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    c["x"], c["sx"] = _rows8(torch.randn(m, k, generator=g, device="cuda"))
    c["w"], c["sw"] = _weights8(g, e, 2 * n if op == "geglu8" else n, k, scale=k ** -0.5)
    c.update(offsets=offsets, most=int(counts.max()))
    if op == "mm8":
        c["y"] = torch.zeros(m, n, dtype=DTYPES[c["out"]], device="cuda")
    else:
        c.update(a=torch.zeros(m, n, dtype=E4M3, device="cuda"), sa=torch.zeros(m, _blocks(n), device="cuda"))
    return c


# ---------------------------------------------------------------- the plain forms

def _wide_rows(x, s):
    """Rows of e4m3 as the values they stand for."""
    return x.float() * s.repeat_interleave(128, -1)[:, :x.shape[1]]


def _wide_weights(w, s):
    n, k = w.shape[-2:]
    v = w.float()
    if s is not None:
        v = v * s.repeat_interleave(128, -2)[..., :n, :].repeat_interleave(128, -1)[..., :k]
    return v


def _products(s):
    """Row r's W[e(r)] x[r] in 32 bits; rows behind the last group: 0."""
    x, w, offsets = _wide_rows(s["x"], s["sx"]), _wide_weights(s["w"], s["sw"]), s["offsets"]
    r = torch.arange(x.shape[0], device="cuda")
    e = torch.searchsorted(offsets[1:], r.int(), right=True).clamp(max=w.shape[0] - 1)
    if x.shape[0] * w[0].numel() < 1 << 28:   # a few rows: each with its own expert's weights
        y = torch.bmm(w[e], x[:, :, None])[:, :, 0]
    else:                                     # each expert's rows as [experts, most rows of one]
        at = offsets[:-1, None].long() + torch.arange(s["most"], device="cuda")
        there = at < offsets[1:, None]
        y = torch.bmm(x[torch.where(there, at, 0)].masked_fill(~there[:, :, None], 0), w.transpose(1, 2))
        y = y[e, (r - offsets[e]).clamp(max=s["most"] - 1)]
    return torch.where((r < offsets[-1])[:, None], y, 0)


def _gelu(v, tanh):
    if tanh:
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))


def _plain(s):
    op = s["op"]
    if op in ("norm", "norm_grad"):
        dt = DTYPES[s["dtype"]]
        r = s["h"]
        if op == "norm" and s["delta"] is not None:
            r = (r.float() + s["delta"].float()).to(dt)
        v = r.float()
        rstd = torch.rsqrt(v.square().mean(1, keepdim=True) + EPS)
        v = v * rstd
        w = 1.0 if s["w"] is None else s["w"].float()
        if op == "norm":
            v = v * w
            y8 = _rows8(v) if s["y8"] is not None else (None, None)
            return {"r": r if s["delta"] is not None else None, "y": v.to(dt) if s["y"] is not None else None,
                    "y8": y8[0], "s": y8[1]}
        dy = s["dy"].float()
        dh = rstd * (dy * w - v * (dy * w * v).mean(1, keepdim=True))
        if s["dres"] is not None:
            dh = dh + s["dres"].float()
        return {"dh": dh.to(dt), "dw": None if s["w"] is None else (dy * v).sum(0)}
    if op == "mm8":
        return _products(s).to(DTYPES[s["out"]])
    if op == "geglu8":
        h, n = _products(s), s["n"]
        a, sa = _rows8(_gelu(h[:, :n], s["tanh"]) * h[:, n:])
        there = torch.arange(a.shape[0], device="cuda")[:, None] < s["offsets"][-1]
        return {"a": a, "sa": torch.where(there, sa, 0)}
    x, ids, f = s["x"].float(), s["ids"].long(), s["f"]
    t, k = ids.shape
    e = ids.reshape(-1)
    scale = lambda name: None if s[name + "_scale"] is None else s[name + "_scale"][e]  # noqa: E731
    gu = torch.bmm(_wide_weights(s["gu"][e], scale("gu")), x.repeat_interleave(k, 0)[:, :, None])[:, :, 0]
    a = _gelu(gu[:, :f], s["tanh"]) * gu[:, f:]
    y = torch.bmm(_wide_weights(s["down"][e], scale("down")), a[:, :, None]).view(t, k, -1)
    y = (y * s["gates"][:, :, None]).sum(1)
    if s["shared"]:
        gu = x @ _wide_weights(s["shared_gu"], s["shared_gu_scale"]).T
        a = _gelu(gu[:, :s["shared"]], s["tanh"]) * gu[:, s["shared"]:]
        y = y + a @ _wide_weights(s["shared_down"], s["shared_down_scale"]).T
    return y.to(DTYPES[s["dtype"]])


def run(state):
    if not own:
        return _plain(state)
    import bit_routed_expert_router_gb300 as moe
    s, op = state, state["op"]
    if op == "norm":
        moe.check(moe.moe_rmsnorm(s["h"], s["y"], s["y8"], s["s"], delta=s["delta"], h_out=s["r"], weight=s["w"], eps=EPS))
        return {"r": s["r"], "y": s["y"], "y8": s["y8"], "s": s["s"]}
    if op == "norm_grad":
        moe.check(moe.moe_rmsnorm_grad(s["h"], s["dy"], s["dh"], dres=s["dres"], weight=s["w"], dweight=s["dw"],
                                       workspace=s["workspace"], eps=EPS))
        return {"dh": s["dh"], "dw": s["dw"]}
    if op == "mm8":
        moe.check(moe.moe_grouped_mm8(s["x"], s["sx"], s["offsets"], s["w"], s["sw"], s["y"]))
        return s["y"]
    variant = moe.MOE_GELU_TANH if s["tanh"] else moe.MOE_GELU_ERF
    if op == "geglu8":
        moe.check(moe.moe_grouped_geglu8(s["x"], s["sx"], s["offsets"], s["w"], s["sw"], s["a"], s["sa"],
                                         gelu_variant=variant))
        return {"a": s["a"], "sa": s["sa"]}
    routed = (s["gu"], s["down"], s["gu_scale"], s["down_scale"])
    shared = (s["shared_gu"], s["shared_down"], s["shared_gu_scale"], s["shared_down_scale"]) if s["shared"] else None
    moe.check(moe.moe_token_layer(s["x"], s["ids"], s["gates"], routed, s["y"], s["workspace"], shared=shared,
                                  gelu_variant=variant))
    return s["y"]


# ---------------------------------------------------------------- what it costs, and what it gives

def work(case):
    c, op = case, case["op"]
    size = {"bf16": 2, "f16": 2, "f32": 4, "none": 0}
    if op in ("norm", "norm_grad"):
        n, b = c["rows"] * c["d"], size[c["dtype"]]
        if op == "norm":
            out = {"8": 1 + 4 / 128, "16": b, "both": b + 1 + 4 / 128}[c["out"]]
            delta = size[c["delta"]]
            return {"bytes": n * (b + delta + (b if delta else 0) + out), "flops": 6 * n}
        return {"bytes": n * b * (4 if c["residual"] else 3) + 4 * c["d"], "flops": 12 * n}
    e, rows = c["experts"], c["tokens"] * c["top_k"]
    active = e * (1 - (1 - c["top_k"] / e) ** c["tokens"])
    if op == "layer":
        t, d, f, fs = c["tokens"], c["d"], c["f"], c["shared"]
        w = 3 * d * (active * f + fs)
        return {"bytes": w * (2 if c["weights"] == "16" else 1 + 4 / 128 ** 2) + 4 * t * d + 8 * rows,
                "flops": 6 * d * (rows * f + t * fs)}
    n, k = c["n"], c["k"]
    if op == "geglu8":
        return {"bytes": active * 2 * n * k * (1 + 4 / 128 ** 2) + rows * (k + n) * (1 + 4 / 128), "flops": 4 * rows * n * k}
    return {"bytes": active * n * k * (1 + 4 / 128 ** 2) + rows * k * (1 + 4 / 128) + size[c["out"]] * rows * n,
            "flops": 2 * rows * n * k}


def exact(case, seed):
    """The definitions in 64 bits, row group by row group and token by token."""
    s = prepare(case, seed)
    op = s["op"]

    def gelu(v):
        if s["tanh"]:
            return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v))
        return v * torch.special.ndtr(v)

    def quantised(v):
        q, scales = torch.zeros_like(v), []
        for lo in range(0, v.shape[1], 128):
            part = v[:, lo:lo + 128]
            scales.append(part.abs().amax(1).clamp(min=TINY) / 448)
            q[:, lo:lo + 128] = (part / scales[-1][:, None]).to(E4M3).double()
        return q, torch.stack(scales, 1)

    def stands_for(w, scale):
        """A matrix of e4m3 with its blocks' scales, or of 16 bits."""
        if scale is None:
            return w.double()
        at = [torch.arange(n, device="cuda") // 128 for n in w.shape]
        return w.double() * scale.double()[at[0]][:, at[1]]

    if op == "norm":
        total = s["h"].double() if s["delta"] is None else s["h"].double() + s["delta"].double()
        r = total.to(DTYPES[s["dtype"]]).double()   # the stored sum is what is normalised
        v = r / (r.pow(2).mean(1, keepdim=True) + EPS).sqrt() * (1 if s["w"] is None else s["w"].double())
        q, scale = quantised(v) if s["y8"] is not None else (None, None)
        return {"r": None if s["delta"] is None else total, "y": None if s["y"] is None else v, "y8": q, "s": scale}
    if op == "norm_grad":
        h, w = s["h"].double().requires_grad_(), torch.ones(s["d"], device="cuda", dtype=torch.float64)
        if s["w"] is not None:
            w = s["w"].double()
        w.requires_grad_()
        y = h / (h.pow(2).mean(1, keepdim=True) + EPS).sqrt() * w
        dh, dw = torch.autograd.grad(y, (h, w), s["dy"].double())
        return {"dh": dh if s["dres"] is None else dh + s["dres"].double(), "dw": None if s["w"] is None else dw}
    if op == "layer":
        def ffn(x, gu, down, gu_scale, down_scale):
            f = gu.shape[0] // 2
            h = x @ stands_for(gu, gu_scale).T
            return (gelu(h[..., :f]) * h[..., f:]) @ stands_for(down, down_scale).T

        at = lambda v, i: None if v is None else v[i]  # noqa: E731
        y = torch.zeros(s["tokens"], s["d"], dtype=torch.float64, device="cuda")
        ids = s["ids"].tolist()
        for t, picked in enumerate(ids):
            for j, i in enumerate(picked):
                y[t] += s["gates"][t, j].double() * ffn(s["x"][t].double(), s["gu"][i], s["down"][i], at(s["gu_scale"], i),
                                                        at(s["down_scale"], i))
        if s["shared"]:
            y += ffn(s["x"].double(), s["shared_gu"], s["shared_down"], s["shared_gu_scale"], s["shared_down_scale"])
        return y
    ends, n = s["offsets"].tolist(), s["n"]
    m = s["x"].shape[0]
    y = torch.zeros(m, s["w"].shape[1], dtype=torch.float64, device="cuda")
    for i, (lo, hi) in enumerate(zip(ends, ends[1:])):
        if hi > lo:
            x = s["x"][lo:hi].double() * s["sx"][lo:hi].double().repeat_interleave(128, 1)[:, :s["k"]]
            y[lo:hi] = x @ stands_for(s["w"][i], s["sw"][i]).T
    if op == "mm8":
        return y
    a, sa = torch.zeros(m, n, dtype=torch.float64, device="cuda"), torch.zeros(m, _blocks(n), dtype=torch.float64, device="cuda")
    a[:ends[-1]], sa[:ends[-1]] = quantised(gelu(y[:ends[-1], :n]) * y[:ends[-1], n:])
    return {"a": a, "sa": sa}
