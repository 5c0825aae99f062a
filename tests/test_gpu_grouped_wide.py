"""The persistent kernel where its tiles are 256 columns wide: more tiles than
one round of the pairs of CTAs (at most 152 SMs), several to a pair.  Whole
numbers, as in test_gpu_grouped.py: exact up to the outputs' rounding."""

import math

import pytest
import torch

import bit_routed_expert_router_gb300 as moe

from test_gpu_grouped import BF16, F16, F32, SENTINEL, buffer, gelu, gen, ints, lora_case, lora_reference, offsets_of, ok, products

pytestmark = pytest.mark.gpu

PAIRS = 76
BORDERS = [255, 256, 257, 513, 0, 1, 1000, 31, 511]


def tiles_of_128(counts, feat, width):
    return sum(-(-c // 128) for c in counts) * -(-feat // width)


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (F16, F32), (F16, F16)])
@pytest.mark.parametrize("n,k", [(264, 328), (520, 200), (328, 1000)])
def test_products(n, k, dtype, out, transpose):
    counts, behind = BORDERS * 6, 9
    into, to = (n, k) if transpose else (k, n)
    assert tiles_of_128(counts, to, 256) > PAIRS
    g, m = gen(n), sum(counts) + behind
    x, w = ints(g, dtype, m, into), ints(g, dtype, len(counts), n, k)
    x[m - behind:] = math.nan
    whole, y = buffer(out, m, to)
    ok(moe.moe_grouped_mm(x, offsets_of(counts), w, y, transpose=transpose))
    assert torch.equal(y, products(x, counts, w.transpose(1, 2) if transpose else w).to(out))
    assert (whole[:, to:] == SENTINEL).all()


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("variant", [moe.MOE_GELU_ERF, moe.MOE_GELU_TANH])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("f,k", [(304, 136), (704, 72)])
def test_gated_products(f, k, dtype, variant, keep):
    """The tolerance of a: its GELU is within a few units of 2^-23 of the gate (2^-19), then one rounding."""
    counts, behind = BORDERS * 5, 9
    assert tiles_of_128(counts, f, 128) > PAIRS
    g, m = gen(f), sum(counts) + behind
    x, w = ints(g, dtype, m, k, top=1), ints(g, dtype, len(counts), 2 * f, k) / 8
    whole_a, a = buffer(dtype, m, f)
    whole_h, h = buffer(dtype, m, 2 * f)
    ok(moe.moe_grouped_geglu(x, offsets_of(counts), w, a, h if keep else None, gelu_variant=variant))
    ref = products(x, counts, w)
    rows = slice(0, m - behind)
    gate, up = ref[rows, :f], ref[rows, f:]
    want, half = gelu(gate, variant) * up, torch.finfo(dtype).eps / 2
    bound = half * want.abs() + (1 + half) * 2 ** -19 * (gate * up).abs() + torch.finfo(dtype).smallest_normal * half
    assert ((a[rows].double() - want).abs() <= bound).all()
    assert (whole_a[:, f:] == SENTINEL).all() and (whole_a[m - behind:] == SENTINEL).all()
    if keep:
        assert torch.equal(h[rows], ref[rows].to(dtype))
        assert (whole_h[m - behind:] == SENTINEL).all()
    assert (whole_h[:, 2 * f if keep else 0:] == SENTINEL).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("order", ["runs", "any"])
@pytest.mark.parametrize("t,n,k,N,rank", [(5000, 520, 136, 37, 72), (5001, 776, 520, 300, 128), (20000, 264, 72, 90, 40)])
def test_adapters(t, n, k, N, rank, order, dtype):
    assert tiles_of_128([t], n, 256) > PAIRS
    x, w, ids, a, b, scale = lora_case(t, t, n, k, N, rank, dtype, order)
    whole, y = buffer(dtype, t, n)
    ok(moe.moe_lora_mm(x, w, ids, a, b, scale, y, torch.empty(4 * t * rank, dtype=torch.uint8, device="cuda")))
    assert torch.equal(y, lora_reference(x, w, ids, a, b, scale).to(dtype))
    assert (whole[:, n:] == SENTINEL).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("order", ["runs", "any"])
def test_broken_adapters_in_tile_after_tile(order, dtype):
    """About 18 tiles a pair, more than the marks of a tile's broken values are taken in turn."""
    t, n, k, N, rank = 60000, 1288, 72, 25, 72
    assert tiles_of_128([t], n, 256) > 2 * 16 * PAIRS
    x, w, ids, a, b, scale = lora_case(1, t, n, k, N, rank, dtype, order)
    a[3], b[7], b[11, 700, 66], b[20, 3, 1] = math.nan, math.inf, math.nan, -math.inf
    y = torch.empty(t, n, dtype=dtype, device="cuda")
    ok(moe.moe_lora_mm(x, w, ids, a, b, scale, y, torch.empty(4 * t * rank, dtype=torch.uint8, device="cuda")))
    a[3], b[7], b[11, 700, 66], b[20, 3, 1] = 0, 0, 0, 0
    want = lora_reference(x, w, ids, a, b, scale).to(dtype)
    bad = torch.zeros(t, n, dtype=torch.bool, device="cuda")
    bad[(ids == 3) | (ids == 7)] = True
    bad[ids == 11, 700] = True
    bad[ids == 20, 3] = True
    assert not y[bad].isfinite().any()
    assert torch.equal(y[~bad], want[~bad])
