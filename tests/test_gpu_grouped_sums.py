"""Long sums of the 16-bit operators: products of one sign, where an
accumulator that truncates falls short by a share that grows with the length.

What is allowed.  A k16 step on the tensor cores was measured to lose 2.3 units
of 2^-23 of its accumulator; 4 are allowed, of an accumulator that is half of
its last value on average.  16-bit outputs are summed in pieces of 256 such
steps, each added with a rounding of 2^-24.  With s the sum of these the fp32
value lies between ref (1 - s) and ref (1 + s), and rounding never turns an order
round: the output lies between those two as the output's type rounds them."""

import pytest
import torch

import bit_routed_expert_router_gb300 as moe

from test_gpu_grouped import BF16, F16, gen, offsets_of, ok

pytestmark = pytest.mark.gpu

PIECE, UNIT = 4096, 2 ** -23


def positive(g, dtype, rows, cols, length):
    """Values around length^-0.5, up to twice that in the last column: sums of `length` products are around 1."""
    v = torch.rand(rows, cols, generator=g, device="cuda").add_(0.5).mul_(length ** -0.5)
    return v.mul_(torch.linspace(1, 2, cols, device="cuda")).to(dtype)


def check(y, ref, length, more=0.0):
    s = min(length, PIECE) / 16 * 4 * UNIT / 2 + -(-length // PIECE) * 2 ** -24 + more
    assert (y >= (ref * (1 - s)).to(y.dtype)).all() and (y <= (ref * (1 + s)).to(y.dtype)).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("m", [2 ** 16 + 5, 2 ** 20, 2 ** 24])
def test_weight_gradients_of_long_groups(m, dtype):
    g, n, k = gen(1), 72, 40
    dy, x = positive(g, dtype, m, n, m), positive(g, dtype, m, k, m)
    dw = torch.empty(3, n, k, dtype=dtype, device="cuda")
    counts = [m // 4 - 3, 0, m - m // 4]
    ok(moe.moe_grouped_wgrad(dy, x, offsets_of(counts), dw))
    assert (dw[1] == 0).all()
    for e, (lo, hi) in ((0, (0, counts[0])), (2, (counts[0], m - 3))):
        ref = sum(a.double().T @ b.double() for a, b in zip(dy[lo:hi].split(2 ** 20), x[lo:hi].split(2 ** 20)))
        check(dw[e], ref, hi - lo)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("m", [9, 300])   # few rows, and many
@pytest.mark.parametrize("transpose", [False, True])
def test_long_products(transpose, m, dtype):
    """As many products a row as allowed."""
    g, out, red = gen(2), 264, 65536
    x = positive(g, dtype, m, red, red)
    w = positive(g, dtype, *((red, out) if transpose else (out, red)), red)[None]
    y = torch.empty(m, out, dtype=dtype, device="cuda")
    ok(moe.moe_grouped_mm(x, offsets_of([m]), w, y, transpose=transpose))
    check(y, x.double() @ (w[0].double() if transpose else w[0].double().T), red)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("m", [9, 300])
def test_long_gated_products(m, dtype):
    """Through h, which is the sums themselves; a follows from the same fp32 values: GELU of a gate near 1 passes on 1.3 of
    a relative error at most, and its own arithmetic is far below either."""
    g, f, k = gen(3), 144, 65536
    x, w = positive(g, dtype, m, k, k), positive(g, dtype, 2 * f, k, k)[None]
    a, h = torch.empty(m, f, dtype=dtype, device="cuda"), torch.empty(m, 2 * f, dtype=dtype, device="cuda")
    ok(moe.moe_grouped_geglu(x, offsets_of([m]), w, a, h))
    ref = x.double() @ w[0].double().T
    check(h, ref, k)
    sums = PIECE / 16 * 4 * UNIT / 2 + 17 * 2 ** -24
    check(a, torch.nn.functional.gelu(ref[:, :f]) * ref[:, f:], k, more=2 * sums)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("t", [9, 300, 900])   # both kernels of either half
def test_long_products_with_adapters(t, dtype):
    """W x and the adapter's term about as large.  Both of the term's sums count, and A x handed on with 16 bits, and the
    product with B of parts of them (2^-15)."""
    g, n, k, N, rank = gen(4), 200, 65536, 3, 40
    x, w = positive(g, dtype, t, k, k), positive(g, dtype, n, k, k)
    a = positive(g, dtype, N * rank, k, k).reshape(N, rank, k)
    b, scale = positive(g, dtype, N * n, rank, rank ** 2).reshape(N, n, rank), torch.ones(N, device="cuda")
    ids = torch.randint(-1, N, (t,), generator=g, device="cuda", dtype=torch.int32)
    y = torch.empty(t, n, dtype=dtype, device="cuda")
    ok(moe.moe_lora_mm(x, w, ids, a, b, scale, y, torch.empty(4 * t * rank, dtype=torch.uint8, device="cuda")))
    ref = x.double() @ w.double().T
    for i in range(N):
        r = (ids == i).nonzero()[:, 0]
        ref[r] += (x[r].double() @ a[i].double().T) @ b[i].double().T
    check(y, ref, k, more=PIECE / 16 * 4 * UNIT / 2 + 2 ** -15)


def check32(y, ref, length):
    """32-bit outputs: pieces of 24 k16 steps, and no further rounding."""
    s = min(length, 384) / 16 * 4 * UNIT / 2 + -(-length // 384) * 2 ** -24
    assert ((y.double() - ref).abs() <= s * ref).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("m", [9, 300])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("red", [200, 2816, 65536])
def test_products_in_32_bits(red, transpose, m, dtype):
    g, out = gen(5), 264
    x = positive(g, dtype, m, red, red)
    w = positive(g, dtype, *((red, out) if transpose else (out, red)), red)[None]
    y = torch.empty(m, out, device="cuda")
    ok(moe.moe_grouped_mm(x, offsets_of([m]), w, y, transpose=transpose))
    check32(y, x.double() @ (w[0].double() if transpose else w[0].double().T), red)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("m", [400, 3001, 2 ** 20])
def test_weight_gradients_in_32_bits(m, dtype):
    g, n, k = gen(6), 72, 40
    dy, x = positive(g, dtype, m, n, m), positive(g, dtype, m, k, m)
    dw = torch.empty(1, n, k, device="cuda")
    ok(moe.moe_grouped_wgrad(dy, x, offsets_of([m]), dw))
    check32(dw[0], dy.double().T @ x.double(), m)
