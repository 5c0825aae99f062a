"""Adapters whose values lie far from one: the same answers from few rows and
from many.  Whole numbers times powers of two, so that every product and every
partial sum is exact and the outputs equal the exact sum rounded once."""

import pytest
import torch

import bit_routed_expert_router_gb300 as moe

from test_gpu_grouped import BF16, F16, gen, lora_case, lora_reference, ok

pytestmark = pytest.mark.gpu

ROWS = [(40, 24), (128, 64), (300, 128), (900, 24)]   # rows and rank: each kernel of either half


def run(x, w, ids, a, b, scale):
    t, rank = x.shape[0], a.shape[1]
    y = torch.empty(t, w.shape[0], dtype=x.dtype, device="cuda")
    ok(moe.moe_lora_mm(x, w, ids, a, b, scale, y, torch.empty(4 * t * rank, dtype=torch.uint8, device="cuda")))
    return y


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("e,be", [(-30, 13), (-13, 13), (12, -12)])
@pytest.mark.parametrize("t,rank", ROWS)
def test_small_and_large_values_between_the_halves(t, rank, e, be, dtype):
    """s A x in steps of 2^-30, far below fp16's smallest, or past its largest: only its product with B has to fit."""
    x, w, ids, a, b, scale = lora_case(t, t, 264, 200, 5, rank, dtype, "any")
    scale, b, w = torch.full_like(scale, 2.0 ** e), b * 2 ** be, w * 2.0 ** (e + be)
    u = max(float((x.double() @ a[i].double().T).abs().max()) for i in range(5))
    assert u < 2 ** 16   # 16 bits are handed on
    assert torch.equal(run(x, w, ids, a, b, scale), lora_reference(x, w, ids, a, b, scale).to(dtype))


@pytest.mark.parametrize("t,rank", ROWS)
def test_every_bit_of_b_counts(t, rank):
    """fp16 values of B with all of their 11 bits, and s A x of at most 8."""
    x, w, ids, a, b, scale = lora_case(t + 1, t, 136, 200, 4, rank, F16, "any")
    g = gen(t)
    a = a * (torch.rand(a.shape, generator=g, device="cuda") < 0.1)
    b = torch.randint(-2047, 2048, b.shape, generator=g, device="cuda").to(F16)
    scale = torch.full_like(scale, 2.0 ** -6)
    assert max(float((x.double() @ a[i].double().T).abs().max()) for i in range(4)) < 2 ** 8
    assert torch.equal(run(x, w, ids, a, b, scale), lora_reference(x, w, ids, a, b, scale).to(F16))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("t,rank", ROWS)
def test_infinities_of_b_are_infinite(t, rank, dtype):
    """What 64-bit arithmetic makes of them: an infinity with the sign of its value of A x, NaN where that is 0 or where
    both signs meet; on every kernel, and nothing in other rows and features."""
    x, w, ids, a, b, scale = lora_case(t + 2, t, 136, 200, 4, rank, dtype, "any")
    b[3, 17, 5], b[3, 100, rank - 1], b[1, 30], b[2, 7, 3] = float("inf"), float("-inf"), float("-inf"), float("nan")
    y = run(x, w, ids, a, b, scale)
    u = torch.einsum("tk,trk->tr", x.double(), a[ids.clamp(min=0).long()].double()) * scale[ids.clamp(min=0).long(), None]
    term = (u[:, None, :] * b[ids.clamp(min=0).long()].double()).sum(2)
    want = (x.double() @ w.double().T + torch.where((ids < 0)[:, None], 0, term)).to(dtype)
    assert want.isinf().any() and want.isnan().any()
    assert torch.equal(y.isnan(), want.isnan())
    assert torch.equal(y.nan_to_num(nan=0.0, posinf=float("inf"), neginf=float("-inf")),
                       want.nan_to_num(nan=0.0, posinf=float("inf"), neginf=float("-inf")))
