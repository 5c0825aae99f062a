"""What the tests of the 8-bit operators and of the layer for a few tokens share: inputs, and the operators in 64 bits."""

import math

import torch

import bit_routed_expert_router_gb300 as moe

BF16, F16, F32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def blocks(n):
    return (n + 127) // 128


def rand8(g, *shape):
    """e4m3 values of all sizes up to 448, of either sign, subnormal ones and zeros among them."""
    return (torch.randn(*shape, generator=g, device="cuda") * 60).clamp(-448, 448).to(E4M3)


def rand_scale(g, *shape):
    """Scales over a factor of 16."""
    return torch.exp2(4 * torch.rand(*shape, generator=g, device="cuda") - 12)


def wide_rows(x, sx):
    return x.double() * sx.double().repeat_interleave(128, -1)[..., :x.shape[-1]]


def wide_weights(w, sw):
    n, k = w.shape[-2:]
    return w.double() * sw.double().repeat_interleave(128, -2)[..., :n, :].repeat_interleave(128, -1)[..., :k]


def gelu(v, variant):
    if variant == moe.MOE_GELU_TANH:
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v))
    return v * torch.special.ndtr(v)


def offsets_of(counts, first=0):
    o = torch.zeros(len(counts) + 1, dtype=torch.int32)
    o[1:] = torch.tensor(counts).cumsum(0)
    return (o + first).cuda()


def products(x, w, offsets):
    """Row r's w[e] x[r] and the sum of the products' magnitudes, in 64 bits; zeros for rows of no group."""
    m, n = x.shape[0], w.shape[1]
    y, size = torch.zeros(m, n, dtype=torch.float64, device="cuda"), torch.zeros(m, n, dtype=torch.float64, device="cuda")
    ends = offsets.tolist()
    for e, (lo, hi) in enumerate(zip(ends, ends[1:])):
        if hi > lo:
            y[lo:hi], size[lo:hi] = x[lo:hi] @ w[e].T, x[lo:hi].abs() @ w[e].abs().T
    return y, size
