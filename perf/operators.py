"""Cases of the 16-bit expert operators: what is measured, and each operator's plain form.

The operators work on rows that are grouped by expert (``offsets[e]`` ..
``offsets[e + 1]`` are the rows of expert ``e``), the way a routed layer leaves
them after its top-k:

* ``mm``          y[r] = W[e(r)] x[r], or with ``transpose`` the input gradient W[e(r)]^T dy[r];
* ``wgrad``       dW[e] = sum over the rows of e of dy[r] x[r]^T;
* ``geglu``       a[r] = GELU(g) * u with [g; u] = W[e(r)] x[r], and h = [g, u] where a backward pass follows;
* ``geglu_grad``  dh from h and da;
* ``lora``        y[t] = W x[t] + s[i] B[i] (A[i] x[t]) with i = ids[t], the adapter of the row's request.

Where ``own`` is true the calls go to the library's kernels, else to elementary
torch operations in 32 bits.
"""

import math

import torch

own = False

D, F, F_SHARED, E, TOP_K = 2816, 704, 2816, 128, 8   # this repository's full-shape layer
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    full = {"experts": E, "top_k": TOP_K, "spread": 0.5, "pad": 0}
    return [
        # one decode step of one request: eight experts' down projections, weights read once, latency counts
        {"name": "down, 1 token", "op": "mm", **full, "tokens": 1, "n": D, "k": F, "transpose": False,
         "dtype": "bf16", "out": "bf16"},
        # a decode batch of 32 requests, two rows per expert; 32-bit outputs for a 32-bit combine
        {"name": "down, 32 tokens", "op": "mm", **full, "tokens": 32, "n": D, "k": F, "transpose": False,
         "dtype": "f16", "out": "f32"},
        # prefill of a 4096-token chunk: about 256 rows per expert, ragged
        {"name": "down, 4096 tokens", "op": "mm", **full, "tokens": 4096, "n": D, "k": F, "transpose": False,
         "dtype": "bf16", "out": "bf16"},
        # backward of the gate/up projection: the gradient that leaves the layer
        {"name": "gate/up input gradient", "op": "mm", **full, "tokens": 4096, "n": 2 * F, "k": D,
         "transpose": True, "dtype": "bf16", "out": "bf16"},
        # backward of the gate/up projection: weight gradients kept in 32 bits for the optimiser
        {"name": "gate/up weight gradient", "op": "wgrad", **full, "tokens": 4096, "n": 2 * F, "k": D,
         "dtype": "bf16", "out": "f32"},
        # a small batch of short samples, skewed routing, in a buffer with room left at its end: most experts get a
        # few rows, some none
        {"name": "down weight gradient, short", "op": "wgrad", **full, "spread": 1.0, "tokens": 75, "pad": 40,
         "n": D, "k": F, "dtype": "f16", "out": "f16"},
        # one decode step of one request: eight experts' gate/up projections and the gated product
        {"name": "gated, 1 token", "op": "geglu", **full, "tokens": 1, "n": F, "k": D, "tanh": False,
         "keep": False, "dtype": "bf16"},
        # training forward of 4096 tokens: the gated product, and h for the backward pass
        {"name": "gated, 4096 tokens, h kept", "op": "geglu", **full, "tokens": 4096, "n": F, "k": D,
         "tanh": True, "keep": True, "dtype": "bf16"},
        # its backward pass
        {"name": "gated gradient, 4096 tokens", "op": "geglu_grad", "rows": 4096 * TOP_K, "pad": 0, "n": F,
         "tanh": True, "dtype": "bf16"},
        # the same for a short sample in a larger buffer
        {"name": "gated gradient, short", "op": "geglu_grad", "rows": 600, "pad": 424, "n": F, "tanh": False,
         "dtype": "f16"},
        # decode batch: 48 requests, 40 adapters loaded, some requests without one
        {"name": "adapters, 48 requests", "op": "lora", "tokens": 48, "runs": 48, "adapters": 40, "rank": 16,
         "n": 2 * F_SHARED, "k": D, "dtype": "bf16"},
        # a serving step that mixes the prompts of some requests with single tokens of others
        {"name": "adapters, mixed prompts", "op": "lora", "tokens": 4096, "runs": 100, "adapters": 24, "rank": 64,
         "n": F_SHARED, "k": D, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["mm", "mm", "mm", "wgrad", "geglu", "geglu_grad", "lora", "lora"])
    dtype = rng.choice(["bf16", "f16"])
    n, k = 8 * _log(rng, 8, 352), 8 * _log(rng, 8, 352)
    if op == "lora":
        tokens = _log(rng, 1, 4096)
        return {"op": op, "tokens": tokens, "runs": min(tokens, _log(rng, 1, 200)), "adapters": _log(rng, 1, 64),
                "rank": rng.choice([8, 16, 32, 64]), "n": n, "k": k, "dtype": dtype}
    if op == "geglu_grad":
        return {"op": op, "rows": _log(rng, 1, 32768), "pad": rng.choice([0, 0, 17]), "n": 8 * _log(rng, 8, 88),
                "tanh": rng.random() < 0.5, "dtype": dtype}
    experts = _log(rng, 4, 128)
    case = {"op": op, "experts": experts, "top_k": min(experts, rng.randint(1, 8)),
            "spread": rng.choice([0.0, 0.5, 1.0]), "pad": rng.choice([0, 0, 33]), "tokens": _log(rng, 1, 4096)}
    if op == "geglu":
        return {**case, "n": 16 * _log(rng, 4, 44), "k": k, "tanh": rng.random() < 0.5,
                "keep": rng.random() < 0.5, "dtype": dtype}
    n, k = (n, 8 * _log(rng, 8, 176)) if rng.random() < 0.5 else (8 * _log(rng, 8, 176), k)
    case = {**case, "n": n, "k": k, "dtype": dtype, "out": rng.choice([dtype, "f32"])}
    return {**case, "transpose": rng.random() < 0.4} if op == "mm" else case


# ---------------------------------------------------------------- inputs

def _randn(g, dtype, *shape, scale=1.0):
    return torch.randn(*shape, generator=g, device="cuda", dtype=DTYPES[dtype]) * scale


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c, dt, n, op = dict(case), case["dtype"], case["n"], case["op"]
    if op == "lora":
        t, k, r, na = c["tokens"], c["k"], c["rank"], c["adapters"]
        # the rows of a request stand together; each run has an adapter, or now and then none (-1)
        ends = torch.randperm(t, generator=g, device="cuda")[:c["runs"]].sort().values
        ends[0] = 0
        of_run = torch.randint(-1, na, (c["runs"],), generator=g, device="cuda", dtype=torch.int32)
        run_of = torch.searchsorted(ends, torch.arange(t, device="cuda"), right=True) - 1
        c.update(x=_randn(g, dt, t, k), w=_randn(g, dt, n, k, scale=k ** -0.5), ids=of_run[run_of],
                 a=_randn(g, dt, na, r, k, scale=k ** -0.5), b=_randn(g, dt, na, n, r, scale=0.25),
                 scale=torch.rand(na, generator=g, device="cuda") + 0.5,
                 y=torch.zeros(t, n, dtype=DTYPES[dt], device="cuda"),
                 workspace=torch.empty(4 * t * r, dtype=torch.uint8, device="cuda"))   # A x, four bytes a value
        return c
    if op == "geglu_grad":
        m = c["rows"] + c["pad"]
        c.update(h=_randn(g, dt, m, 2 * n, scale=1.5), da=_randn(g, dt, m, n),
                 n_rows=torch.tensor([c["rows"]], dtype=torch.int32, device="cuda"),
                 dh=torch.zeros(m, 2 * n, dtype=DTYPES[dt], device="cuda"))
        return c
    # top-k of logits with a popularity of each expert, as a router leaves them
    e, t, k = c["experts"], c["tokens"], c["k"]
    logits = torch.randn(t, e, generator=g, device="cuda")
    logits += c["spread"] * torch.randn(e, generator=g, device="cuda")
    counts = torch.bincount(logits.topk(c["top_k"]).indices.reshape(-1), minlength=e)
    offsets = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    m = t * c["top_k"] + c["pad"]
    c.update(offsets=offsets, most=int(counts.max()))
    if op == "mm":
        rows_in, rows_out = (n, k) if c["transpose"] else (k, n)
        c.update(x=_randn(g, dt, m, rows_in), w=_randn(g, dt, e, n, k, scale=rows_in ** -0.5),
                 y=torch.zeros(m, rows_out, dtype=DTYPES[c["out"]], device="cuda"))
    elif op == "wgrad":
        c.update(x=_randn(g, dt, m, k), dy=_randn(g, dt, m, n),
                 dw=torch.zeros(e, n, k, dtype=DTYPES[c["out"]], device="cuda"))
    else:
        c.update(x=_randn(g, dt, m, k), w=_randn(g, dt, e, 2 * n, k, scale=k ** -0.5),
                 a=torch.zeros(m, n, dtype=DTYPES[dt], device="cuda"),
                 h=torch.zeros(m, 2 * n, dtype=DTYPES[dt], device="cuda") if c["keep"] else None)
    return c


# ---------------------------------------------------------------- the plain forms

def _padded(s):
    """Each expert's row numbers as [experts, most rows of one], and which of them are its rows."""
    at = s["offsets"][:-1, None].long() + torch.arange(s["most"], device="cuda")
    there = at < s["offsets"][1:, None]
    return torch.where(there, at, 0), there


def _products(s, w):
    """Row r's W[e(r)] x[r] in 32 bits; rows behind the last group: 0."""
    x, offsets = s["x"], s["offsets"]
    r = torch.arange(x.shape[0], device="cuda")
    e = torch.searchsorted(offsets[1:], r.int(), right=True).clamp(max=w.shape[0] - 1)
    if x.shape[0] * w[0].numel() < 1 << 26:   # a few rows: each with its own expert's weights
        y = torch.bmm(w[e].float(), x.float()[:, :, None])[:, :, 0]
    else:
        at, there = _padded(s)
        y = torch.bmm(x[at].float().masked_fill(~there[:, :, None], 0), w.float().transpose(1, 2))
        y = y[e, (r - offsets[e]).clamp(max=s["most"] - 1)]
    return torch.where((r < offsets[-1])[:, None], y, 0)


def _gelu(v, tanh):
    if tanh:
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))


def _gelu_slope(v, tanh):
    if tanh:
        th = torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
        return 0.5 * (1 + th) + 0.5 * v * (1 - th * th) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * v * v)
    return 0.5 * (1 + torch.erf(v * math.sqrt(0.5))) + v * torch.exp(-0.5 * v * v) * math.sqrt(0.5 / math.pi)


def _plain(s):
    op, dt, n = s["op"], DTYPES[s["dtype"]], s["n"]
    if op == "mm":
        return _products(s, s["w"].transpose(1, 2) if s["transpose"] else s["w"]).to(DTYPES[s["out"]])
    if op == "wgrad":
        at, there = _padded(s)
        dy = s["dy"][at].float().masked_fill(~there[:, :, None], 0)
        x = s["x"][at].float().masked_fill(~there[:, :, None], 0)
        return torch.bmm(dy.transpose(1, 2), x).to(DTYPES[s["out"]])
    if op == "geglu":
        h = _products(s, s["w"])
        a = _gelu(h[:, :n], s["tanh"]) * h[:, n:]
        return (a.to(dt), h.to(dt)) if s["keep"] else a.to(dt)
    if op == "geglu_grad":
        g, u, da = s["h"][:, :n].float(), s["h"][:, n:].float(), s["da"].float()
        dh = torch.cat([da * u * _gelu_slope(g, s["tanh"]), da * _gelu(g, s["tanh"])], 1)
        return torch.where(torch.arange(dh.shape[0], device="cuda")[:, None] < s["n_rows"], dh, 0).to(dt)
    x, i = s["x"].float(), s["ids"].clamp(min=0).long()
    low = torch.bmm(s["a"][i].float(), x[:, :, None]) * torch.where(s["ids"] < 0, 0, s["scale"][i])[:, None, None]
    return (x @ s["w"].float().T + torch.bmm(s["b"][i].float(), low)[:, :, 0]).to(dt)


def run(state):
    if not own:
        return _plain(state)
    import bit_routed_expert_router_gb300 as moe
    s, op = state, state["op"]
    if op == "mm":
        moe.check(moe.moe_grouped_mm(s["x"], s["offsets"], s["w"], s["y"], transpose=s["transpose"]))
        return s["y"]
    if op == "wgrad":
        moe.check(moe.moe_grouped_wgrad(s["dy"], s["x"], s["offsets"], s["dw"]))
        return s["dw"]
    if op == "lora":
        moe.check(moe.moe_lora_mm(s["x"], s["w"], s["ids"], s["a"], s["b"], s["scale"], s["y"], s["workspace"]))
        return s["y"]
    variant = moe.MOE_GELU_TANH if s["tanh"] else moe.MOE_GELU_ERF
    if op == "geglu":
        moe.check(moe.moe_grouped_geglu(s["x"], s["offsets"], s["w"], s["a"], s["h"], gelu_variant=variant))
        return (s["a"], s["h"]) if s["keep"] else s["a"]
    moe.check(moe.moe_geglu_grad(s["h"], s["da"], s["dh"], s["n_rows"], gelu_variant=variant))
    return s["dh"]


# ---------------------------------------------------------------- what it costs, and what it gives

def work(case):
    c, n, op = case, case["n"], case["op"]
    size = {"bf16": 2, "f16": 2, "f32": 4}
    b = size[c["dtype"]]
    if op == "lora":
        t, k, r = c["tokens"], c["k"], c["rank"]
        # a run has one of the adapters with probability na / (na + 1)
        na = c["adapters"]
        used = na * (1 - (1 - 1 / (na + 1)) ** c["runs"])
        return {"bytes": b * (t * k + n * k + t * n + used * r * (n + k)) + 4 * (t + na),
                "flops": 2 * t * (n * k + r * (n + k) * na / (na + 1))}
    if op == "geglu_grad":
        return {"bytes": b * c["rows"] * 5 * n, "flops": 20 * c["rows"] * n}
    e, k, rows = c["experts"], c["k"], c["tokens"] * c["top_k"]
    active = e * (1 - (1 - c["top_k"] / e) ** c["tokens"])
    if op == "mm":
        into, out = (n, k) if c["transpose"] else (k, n)
        return {"bytes": b * (active * n * k + rows * into) + size[c["out"]] * rows * out, "flops": 2 * rows * n * k}
    if op == "wgrad":
        return {"bytes": b * rows * (n + k) + size[c["out"]] * e * n * k, "flops": 2 * rows * n * k}
    return {"bytes": b * (active * 2 * n * k + rows * k + rows * n * (3 if c["keep"] else 1)),
            "flops": 4 * rows * n * k}


def exact(case, seed):
    """The definitions in 64 bits, expert by expert and adapter by adapter."""
    s = prepare(case, seed)
    op, n = s["op"], s["n"]

    def gelu(v):
        if s["tanh"]:
            return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v))
        return v * torch.special.ndtr(v)

    if op == "lora":
        y = s["x"].double() @ s["w"].double().T
        for i in range(s["adapters"]):
            rows = (s["ids"] == i).nonzero()[:, 0]
            if len(rows):
                u = s["x"][rows].double() @ s["a"][i].double().T
                y[rows] += s["scale"][i].double() * (u @ s["b"][i].double().T)
        return y
    if op == "geglu_grad":
        rows = s["rows"]
        h = s["h"][:rows].double().requires_grad_()
        a = gelu(h[:, :n]) * h[:, n:]
        dh = torch.zeros(s["h"].shape, dtype=torch.float64, device="cuda")
        dh[:rows] = torch.autograd.grad(a, h, s["da"][:rows].double())[0]
        return dh
    ends = s["offsets"].tolist()
    m, x = s["x"].shape[0], s["x"]
    if op == "wgrad":
        return torch.stack([s["dy"][lo:hi].double().T @ x[lo:hi].double() for lo, hi in zip(ends, ends[1:])])
    w = s["w"].transpose(1, 2) if op == "mm" and s["transpose"] else s["w"]
    y = torch.zeros(m, w.shape[1], dtype=torch.float64, device="cuda")
    for i, (lo, hi) in enumerate(zip(ends, ends[1:])):
        if hi > lo:
            y[lo:hi] = x[lo:hi].double() @ w[i].double().T
    if op == "mm":
        return y
    a = gelu(y[:, :n]) * y[:, n:]
    return (a, y) if s["keep"] else a
