"""GELU far below zero, where it is a small difference from zero: its share of
the value counts, not of the gate.

fp32's own errors for -9 <= g <= -3, relative to the value.  erf form: the
exponential is off by 2 + 1.2 x 40.5 units of 2^-23, and its argument's two
roundings are stretched by 40.5; the fitted ratio by 1e-6 at most with its
roundings; the slope Phi + g p is at least 8 / 9 of g p.  With a few products
1.3e-5.  tanh form: the exponential of at most 67
has 2 + 1.2 x 67 units and an argument of five roundings times 67: 3.0e-5, and as
much for its slope, small (1 + g big s'), whose bracket is far from 0.  2^-14 is
6.1e-5."""

import pytest
import torch

import bit_routed_expert_router_gb300 as moe

from test_gpu_grouped import BF16, F16, offsets_of, ok

pytestmark = pytest.mark.gpu

BELOW = 2 ** -14


def gates(dtype):
    return -3 - 6 * torch.arange(64, device="cuda").div(63).to(dtype)


def exact(g, variant):
    """GELU without cancellation, differentiable."""
    if variant == moe.MOE_GELU_TANH:
        return g * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (g + 0.044715 * g ** 3))
    return 0.5 * g * torch.special.erfc(-g * 0.5 ** 0.5)


def check(got, want):
    half = torch.finfo(got.dtype).eps / 2
    least = torch.finfo(got.dtype).smallest_normal * half   # below it half a step is absolute
    assert ((got.double() - want).abs() <= (half + (1 + half) * BELOW) * want.abs() + least).all()


@pytest.mark.parametrize("variant", [moe.MOE_GELU_ERF, moe.MOE_GELU_TANH])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("m", [3, 100])   # few rows, and many
def test_gated_products_of_small_values(m, dtype, variant):
    """One product each: g is a weight, u is 1."""
    g, f = gates(dtype), 64
    w = torch.zeros(1, 2 * f, 8, dtype=dtype, device="cuda")
    w[0, :f, 0], w[0, f:, 1] = g, 1
    x = torch.zeros(m, 8, dtype=dtype, device="cuda")
    x[:, :2] = 1
    a = torch.empty(m, f, dtype=dtype, device="cuda")
    ok(moe.moe_grouped_geglu(x, offsets_of([m]), w, a, gelu_variant=variant))
    check(a, exact(g.double(), variant).expand(m, f))


@pytest.mark.parametrize("variant", [moe.MOE_GELU_ERF, moe.MOE_GELU_TANH])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_gated_gradients_of_small_values(dtype, variant):
    g = gates(dtype)
    h, da = torch.cat([g, torch.ones_like(g)])[None], torch.ones(1, 64, dtype=dtype, device="cuda")
    dh = torch.empty(1, 128, dtype=dtype, device="cuda")
    ok(moe.moe_geglu_grad(h, da, dh, gelu_variant=variant))
    gd = g.double().requires_grad_()
    value = exact(gd, variant)
    check(dh[0, :64], torch.autograd.grad(value.sum(), gd)[0])
    check(dh[0, 64:], value.detach())
