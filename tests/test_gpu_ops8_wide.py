"""The norm, the 8-bit products and the layer for a few tokens at offsets past 32 bits: rows far apart, many weights."""

import pytest
import torch

import bit_routed_expert_router_gb300 as moe
from ops8_reference import BF16, E4M3, F16, F32, blocks, gen, products, rand8, rand_scale, wide_rows, wide_weights
from test_gpu_grouped8 import case, close, close_gated
from test_gpu_norm import near16, near8, near_grads, normed
from test_gpu_token_layer import call as layer_call, case as layer_case, check as layer_check, weights as layer_weights

pytestmark = pytest.mark.gpu

FAR = (1 << 31) + 4096   # values from a row to the next


def apart(rows, cols, dtype, ld=FAR):
    """Rows `ld` values apart, in memory of their own."""
    return torch.empty((rows - 1) * ld + cols, dtype=dtype, device="cuda").as_strided((rows, cols), (ld, 1))


def spread(v):
    far = apart(*v.shape, v.dtype)
    (far.view(torch.uint8) if v.dtype == E4M3 else far).copy_(v.view(torch.uint8) if v.dtype == E4M3 else v)
    return far


def test_norm_and_its_gradient():
    g = gen(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    h, delta, w = r(3, 264).to(BF16), r(3, 264), r(264).to(BF16)
    far, y8, s = spread(h), apart(3, 264, E4M3), torch.empty(3, 3, device="cuda")
    moe.check(moe.moe_rmsnorm(far, far, weight=w))
    near16(far, normed(h, w), BF16)
    far.copy_(h)
    moe.check(moe.moe_rmsnorm(far, None, y8, s, delta=spread(delta), h_out=far, weight=w))
    assert torch.equal(far, (h.float() + delta).to(BF16))
    near8(y8, s, normed(far, w))
    h, dy, dw, ws = far.clone(), r(3, 264).to(BF16), torch.empty(264, device="cuda"), torch.empty(4 * 264 * 3, dtype=torch.uint8, device="cuda")
    moe.check(moe.moe_rmsnorm_grad(far, spread(dy), far, dres=spread(dy), weight=w, dweight=dw, workspace=ws))
    near_grads(h, dy, dy, w, far, dw)


@pytest.mark.parametrize("out", [BF16, F32])
def test_products_of_rows_far_apart(out):
    x, sx, off, w, sw = case([1, 2], 264, 272)
    y = apart(3, 264, out, FAR // 2)
    moe.check(moe.moe_grouped_mm8(spread(x), sx, off, w, sw, y))
    close(y, *products(wide_rows(x, sx), wide_weights(w, sw), off), 272)
    x, sx, off, w, sw = case([40, 3], 264, 272)
    y = apart(43, 264, out, 1 << 27)   # a tile's rows stored as one
    moe.check(moe.moe_grouped_mm8(x, sx, off, w, sw, y))
    close(y, *products(wide_rows(x, sx), wide_weights(w, sw), off), 272)


def test_gated_products_of_rows_far_apart():
    x, sx, off, w, sw = case([1, 2], 2 * 144, 272)
    sx *= 2.0 ** -10
    a, sa = apart(3, 144, E4M3), torch.empty(3, 2, device="cuda")
    moe.check(moe.moe_grouped_geglu8(spread(x), sx, off, w, sw, a, sa))
    close_gated(a, sa, x, sx, off, w, sw, 144, moe.MOE_GELU_ERF)


def test_weights_past_32_bits():
    """The last of 40 experts of 64 MiB."""
    E, n, k, m = 40, 8192, 8192, 5
    g = gen(4)
    x, sx, sw = rand8(g, m, k), rand_scale(g, m, blocks(k)), rand_scale(g, E, blocks(n), blocks(k))
    w = torch.empty(E, n, k, dtype=E4M3, device="cuda")
    w[-1].view(torch.uint8).copy_(rand8(g, n, k).view(torch.uint8))
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[-1] = m
    y = torch.empty(m, n, device="cuda")
    moe.check(moe.moe_grouped_mm8(x, sx, off, w, sw, y))
    close(y, *products(wide_rows(x, sx), wide_weights(w[-1:], sw[-1:]), off[-2:]), k)


@pytest.mark.parametrize("eight", [False, True])
def test_layer_of_many_weights(eight):
    """Experts of 8 and 4 Mi values, 2^31 of them and more; the last ones are picked."""
    t, k, E, d, f = 2, 2, 530, 2048, 2048
    g = gen(5)
    x, ids, gates = torch.randn(t, d, generator=g, device="cuda").to(F16), [[E - 1, E - 2], [E - 2, 3]], torch.rand(t, k, device="cuda")
    some = layer_weights(g, F16, eight, (3,), d, f)
    at = [3, E - 2, E - 1]
    routed = []
    for v in some:
        all_ = torch.empty(E, *v.shape[1:], dtype=v.dtype, device="cuda")
        for i, e in enumerate(at):
            all_[e].view(torch.uint8).copy_(v[i].view(torch.uint8))
        routed.append(all_)
    y = layer_call(x, torch.tensor(ids, dtype=torch.int32, device="cuda"), gates, routed, None)
    layer_check(y, x, torch.tensor([[2, 1], [1, 0]], dtype=torch.int32, device="cuda"), gates, some, None, moe.MOE_GELU_ERF)


def test_layer_of_rows_far_apart():
    x, ids, gates, routed, shared = layer_case(3, 2, 8, 272, 80, 48)
    y = apart(3, 272, F32, FAR // 2)
    layer_call(spread(x), ids, gates, routed, shared, y=y)
    layer_check(y, x, ids, gates, routed, shared, moe.MOE_GELU_ERF)
