"""The 16-bit operators against their definitions in 64 bits.

Most cases use small whole numbers: every product and every partial sum is
then exact in fp32 (below 2^24), in any order, so the result has to equal the
exact sum rounded once to the output's type: no tolerance at all.
"""

import math

import pytest
import torch

import bit_routed_expert_router_gb300 as moe

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
SENTINEL = 7.0

# rows of each expert: both kernels (at most 4 rows an expert on average, and more), empty experts, single rows, the
# borders of the 16-, 32-, 64- and 256-row tiles
FEW = [[1], [0, 1, 0, 1], [3, 0, 2], [16, 0, 0, 0, 0], [0] * 40 + [130, 1] + [0] * 8, [64] + [0] * 15,
       [65] + [0] * 20 + [7], [1] * 70, [8, 1, 0, 3, 2, 5, 4, 4]]
MANY = [[5], [31, 33, 32, 0], [255, 0, 256, 257, 1], [513, 64], [0, 0, 300], [40] * 37, [1000, 3, 0, 17, 129]]
SIDES = [(8, 8), (72, 136), (136, 72), (264, 328), (512, 64), (704, 1000)]


def ints(g, dtype, *shape, top=2):
    return torch.randint(-top, top + 1, shape, generator=g, device="cuda").to(dtype)


def gen(seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def offsets_of(counts, before=0):
    off = torch.tensor([0] + counts).cumsum(0) + before
    return off.to(torch.int32).cuda()


def buffer(dtype, rows, cols, pad=8):
    """An output in a larger buffer, everything at the sentinel: (whole buffer, view)."""
    whole = torch.full((rows, cols + pad), SENTINEL, dtype=dtype, device="cuda")
    return whole, whole[:, :cols]


def products(x, counts, w, before=0):
    """W[e] x[r] in 64 bits; rows outside the groups keep the sentinel."""
    y = torch.full((x.shape[0], w.shape[1]), SENTINEL, dtype=torch.float64, device="cuda")
    lo = before
    for e, c in enumerate(counts):
        y[lo:lo + c] = x[lo:lo + c].double() @ w[e].double().T
        lo += c
    return y


def ok(status):
    moe.check(status)
    moe.check(moe.moe_grouped_sync())


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (F16, F32), (F16, F16), (BF16, F32)])
@pytest.mark.parametrize("i,counts", list(enumerate(FEW + MANY)))
def test_products(i, counts, dtype, out, transpose):
    n, k = SIDES[i % len(SIDES)]
    g, E, before, behind = gen(i), len(counts), i % 3, 5
    m = before + sum(counts) + behind
    into, to = (n, k) if transpose else (k, n)
    x = ints(g, dtype, m, into + 8)[:, :into]
    x[:before] = x[m - behind:] = math.nan   # rows outside the groups may hold anything
    w = ints(g, dtype, E, n, k)
    whole, y = buffer(out, m, to)
    ok(moe.moe_grouped_mm(x, offsets_of(counts, before), w, y, transpose=transpose))
    want = products(x, counts, w.transpose(1, 2) if transpose else w, before).to(out)
    assert torch.equal(y, want)
    assert (whole[:, to:] == SENTINEL).all()


@pytest.mark.parametrize("dtype,out", [(BF16, F32), (F16, F16), (BF16, BF16)])
@pytest.mark.parametrize("i,counts", list(enumerate(FEW + MANY)))
def test_weight_gradients(i, counts, dtype, out):
    n, k = SIDES[i % len(SIDES)]
    g, E, before, behind = gen(i), len(counts), i % 3, 70
    m = before + sum(counts) + behind
    x, dy = ints(g, dtype, m, k + 8)[:, :k], ints(g, dtype, m, n)
    x[:before] = x[m - behind:] = math.nan
    dy[:before] = dy[m - behind:] = math.inf
    dw = torch.full((E + 1, n, k), SENTINEL, dtype=out, device="cuda")
    ok(moe.moe_grouped_wgrad(dy, x, offsets_of(counts, before), dw[:E]))
    lo = before
    for e, c in enumerate(counts):
        want = dy[lo:lo + c].double().T @ x[lo:lo + c].double()
        assert torch.equal(dw[e], want.to(out)), e
        lo += c
    assert (dw[E] == SENTINEL).all()


@pytest.mark.parametrize("rows", [3000, 20000])
def test_as_many_experts_as_allowed(rows):
    g, E = gen(15), 1024
    counts = torch.bincount(torch.randint(0, E, (rows,), generator=g, device="cuda") ** 2 // E, minlength=E).tolist()
    x, dy, w, off = ints(g, F16, rows, 72), ints(g, F16, rows, 40), ints(g, F16, E, 40, 72), offsets_of(counts)
    y, dw = torch.empty(rows, 40, dtype=F16, device="cuda"), torch.empty(E, 40, 72, dtype=F16, device="cuda")
    ok(moe.moe_grouped_mm(x, off, w, y))
    ok(moe.moe_grouped_wgrad(dy, x, off, dw))
    e_of = torch.repeat_interleave(torch.arange(E, device="cuda"), torch.tensor(counts, device="cuda"))
    assert torch.equal(y, torch.bmm(w[e_of].double(), x[:, :, None].double())[:, :, 0].to(F16))
    outer = torch.zeros(E, 40, 72, dtype=torch.float64, device="cuda")
    outer.index_add_(0, e_of, dy[:, :, None].double() * x[:, None, :].double())
    assert torch.equal(dw, outer.to(F16))


def test_long_weight_gradients():
    """Groups of hundreds of rows: the reduction goes in pieces."""
    g, counts, n, k = gen(4), [1000, 385, 0, 384, 2600], 264, 328
    x, dy, off = ints(g, BF16, sum(counts), k), ints(g, BF16, sum(counts), n), offsets_of(counts)
    dw = torch.full((5, n, k), SENTINEL, dtype=F32, device="cuda")
    ok(moe.moe_grouped_wgrad(dy, x, off, dw))
    lo = 0
    for e, c in enumerate(counts):
        assert torch.equal(dw[e], (dy[lo:lo + c].double().T @ x[lo:lo + c].double()).float()), e
        lo += c


def test_full_shape_products():
    """The repository's full layer: 128 experts, 32,768 rows, whole-number inputs."""
    g, E, n, k = gen(3), 128, 1408, 2816
    counts = torch.bincount(torch.randint(0, E, (32768,), generator=g, device="cuda"), minlength=E).tolist()
    off = offsets_of(counts)
    x, w, dy = ints(g, BF16, 32768, k), ints(g, BF16, E, n, k), ints(g, BF16, 32768, n)
    y = torch.empty(32768, n, dtype=F32, device="cuda")
    dx = torch.empty(32768, k, dtype=BF16, device="cuda")
    dw = torch.empty(E, n, k, dtype=F32, device="cuda")
    ok(moe.moe_grouped_mm(x, off, w, y))
    ok(moe.moe_grouped_mm(dy, off, w, dx, transpose=True))
    ok(moe.moe_grouped_wgrad(dy, x, off, dw))
    lo = 0
    for e, c in enumerate(counts):
        s = slice(lo, lo + c)
        assert torch.equal(y[s], x[s].float() @ w[e].float().T), e   # exact in fp32 too
        assert torch.equal(dx[s], (dy[s].float() @ w[e].float()).to(BF16)), e
        assert torch.equal(dw[e], dy[s].float().T @ x[s].float()), e
        lo += c


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("k", [200, 1000, 2816])
@pytest.mark.parametrize("counts", [[2, 0, 3], [50, 31, 0, 64], [150, 31, 0, 300]])
def test_products_of_real_values(dtype, counts, k):
    """Normal inputs, 32-bit outputs.  A k16 step adds 16 products to the accumulator with at most 17 roundings or
    truncations of 2^-23 of the largest magnitude that occurs, which sum |x w| bounds; an accumulator takes at most 24
    steps (32 where the reduction is no longer than 512), and the pieces are added with one rounding each."""
    g, n = gen(5), 264
    m = sum(counts)
    x = torch.randn(m, k, generator=g, device="cuda").to(dtype)
    w = (torch.randn(len(counts), n, k, generator=g, device="cuda") / k ** 0.5).to(dtype)
    y = torch.empty(m, n, dtype=F32, device="cuda")
    ok(moe.moe_grouped_mm(x, offsets_of(counts), w, y))
    ref, mag = products(x, counts, w), products(x.abs(), counts, w.abs())
    assert ((y - ref).abs() <= ((min(k / 16 + 1, 24) if k > 512 else k / 16 + 1) * 17 + k / 384 + 8) * 2 ** -23 * mag).all()


def test_a_group_keeps_its_nan():
    """NaN and infinities in one expert's rows or weights reach no other expert."""
    g, n, k, counts = gen(6), 136, 200, [37, 20, 41]
    x, dy, w = ints(g, BF16, 98, k), ints(g, BF16, 98, n), ints(g, BF16, 3, n, k)
    x[37:57], dy[37:57], w[1] = math.nan, math.inf, math.nan
    off = offsets_of(counts)
    y, dw = torch.empty(98, n, dtype=F32, device="cuda"), torch.empty(3, n, k, dtype=F32, device="cuda")
    ok(moe.moe_grouped_mm(x, off, w, y))
    ok(moe.moe_grouped_wgrad(dy, x, off, dw))
    assert y[37:57].isnan().all() and dw[1].isnan().all()
    rows = torch.cat([torch.arange(37), torch.arange(57, 98)]).cuda()
    assert torch.equal(y[rows], products(x, counts, w)[rows].float())
    for e, s in ((0, slice(0, 37)), (2, slice(57, 98))):
        assert torch.equal(dw[e], (dy[s].double().T @ x[s].double()).float())


@pytest.mark.parametrize("m", [40, 300])
def test_offsets_out_of_range_stay_inside_the_tensors(m):
    """Undefined outputs, but nothing outside the given rows is touched (the kernels clamp every offset)."""
    g, n, k = gen(7), 72, 136
    x, dy, w = ints(g, BF16, m, k), ints(g, BF16, m, n), ints(g, BF16, 3, n, k)
    for bad in ([-5, 10, 900, 2000], [30, 10, 35, 0], [m + 10, m + 20, m + 30, m + 40], [0, m, 0, m], [m, 0, m, 0],
                [-2 ** 31, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        whole = torch.full((m + 600, n), SENTINEL, dtype=BF16, device="cuda")
        ok(moe.moe_grouped_mm(x, off, w, whole[300:300 + m]))
        assert (whole[:300] == SENTINEL).all() and (whole[300 + m:] == SENTINEL).all()
        dw = torch.full((5, n, k), SENTINEL, dtype=F32, device="cuda")
        ok(moe.moe_grouped_wgrad(dy, x, off, dw[1:4]))
        assert (dw[0] == SENTINEL).all() and (dw[4] == SENTINEL).all()


# ---------------------------------------------------------------- the gated product

def gelu(v, variant):
    if variant == moe.MOE_GELU_TANH:
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("variant", [moe.MOE_GELU_ERF, moe.MOE_GELU_TANH])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("i,counts", list(enumerate(FEW + MANY)))
def test_gated_products(i, counts, dtype, variant, keep):
    """Whole-number x and weights in eighths, so g and u are exact.  Then a = g / 2 * (1 + erf) * u in fp32: erff is
    within 2 ulp and tanhf within 2 ulp of a value up to 1, its argument within 4 roundings (a slope of at most 1),
    so 1 + (..) is off by at most 8 * 2^-24 * 2 and the products by a rounding each: 2^-19 of |g u| covers it."""
    f, k = [(16, 8), (48, 136), (144, 72), (272, 328), (704, 200)][i % 5]
    g, E, before, behind = gen(i), len(counts), i % 3, 5
    m = before + sum(counts) + behind
    x = ints(g, dtype, m, k, top=1)
    w = ints(g, dtype, E, 2 * f, k) / 8
    whole_a, a = buffer(dtype, m, f)
    whole_h, h = buffer(dtype, m, 2 * f)
    ok(moe.moe_grouped_geglu(x, offsets_of(counts, before), w, a, h if keep else None, gelu_variant=variant))
    ref = products(x, counts, w, before)
    rows = slice(before, m - behind)
    gate, up = ref[rows, :f], ref[rows, f:]
    want = gelu(gate, variant) * up
    half = torch.finfo(dtype).eps / 2
    # below the smallest normal number a step is absolute
    bound = half * want.abs() + (1 + half) * 2 ** -19 * (gate * up).abs() + torch.finfo(dtype).smallest_normal * half
    assert ((a[rows].double() - want).abs() <= bound).all()
    assert (whole_a[:, f:] == SENTINEL).all() and (whole_a[:before] == SENTINEL).all()
    assert (whole_a[m - behind:] == SENTINEL).all()
    if keep:
        assert torch.equal(h[rows], ref[rows].to(dtype))
        assert (whole_h[:, 2 * f:] == SENTINEL).all() and (whole_h[m - behind:] == SENTINEL).all()
    else:
        assert (whole_h == SENTINEL).all()


def exact_gated_grad(h, da, variant):
    f = da.shape[1]
    h = h.double().requires_grad_()
    return torch.autograd.grad(gelu(h[:, :f], variant) * h[:, f:], h, da.double())[0]


@pytest.mark.parametrize("variant", [moe.MOE_GELU_ERF, moe.MOE_GELU_TANH])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("m,f,rows", [(1, 8, None), (1, 704, 1), (37, 104, 20), (513, 64, 0), (300, 88, None),
                                      (64, 200, 999), (2000, 704, None)])
def test_gated_gradient(m, f, rows, dtype, variant):
    """The slope's terms: (1 + erf) / 2 is off by at most 4 * 2^-24, g p(g) (at most 1/4) by the exponential's 2 ulp
    and three roundings; tanh: 1 - t^2 by 4 * 2^-23 times g s' / 2, which 1 - t^2 keeps below 1.3 where it matters
    and |g s'| / 2 below 50 for |g| <= 8: 2^-17 of |da u|, and 2^-19 of |da g|, cover them."""
    g = gen(m)
    h = torch.randn(m, 2 * f, generator=g, device="cuda").mul(1.5).clamp(-8, 8).to(dtype)
    da = torch.randn(m, f, generator=g, device="cuda").to(dtype)
    whole, dh = buffer(dtype, m, 2 * f)
    n_rows = None if rows is None else torch.tensor([rows], dtype=torch.int32, device="cuda")
    ok(moe.moe_geglu_grad(h, da, dh, n_rows, gelu_variant=variant))
    done = m if rows is None else min(rows, m)
    want = exact_gated_grad(h[:done], da[:done], variant)
    hd, dd = h[:done].double(), da[:done].double()
    slack = torch.cat([2 ** -17 * (dd * hd[:, f:]).abs(), 2 ** -19 * (dd * hd[:, :f]).abs()], 1)
    half = torch.finfo(dtype).eps / 2
    bound = half * want.abs() + (1 + half) * slack + torch.finfo(dtype).smallest_normal * half
    assert ((dh[:done].double() - want).abs() <= bound).all()
    assert (whole[done:] == SENTINEL).all() and (whole[:, 2 * f:] == SENTINEL).all()


@pytest.mark.parametrize("variant", [moe.MOE_GELU_ERF, moe.MOE_GELU_TANH])
def test_gated_gradient_of_extremes(variant):
    """Far from zero GELU is 0 or the identity: no NaN where the value itself has none."""
    gate = torch.tensor([-3e4, -100.0, -12.0, -0.0, 0.0, 12.0, 100.0, 3e4], device="cuda")
    h = torch.cat([gate, torch.ones(8, device="cuda")])[None].to(F16)
    da, dh = torch.ones(1, 8, dtype=F16, device="cuda"), torch.empty(1, 16, dtype=F16, device="cuda")
    ok(moe.moe_geglu_grad(h, da, dh, gelu_variant=variant))
    want = torch.tensor([0, 0, 0, 0.5, 0.5, 1, 1, 1], dtype=F16, device="cuda")
    assert torch.equal(dh[0, :8], want)
    assert torch.equal(dh[0, 8:], torch.where(gate < 0, 0, gate).to(F16))


def test_gated_gradient_in_place():
    g = gen(1)
    h, da = torch.randn(50, 400, generator=g, device="cuda").to(BF16), torch.randn(50, 200, device="cuda").to(BF16)
    dh = torch.empty_like(h)
    ok(moe.moe_geglu_grad(h, da, dh))
    ok(moe.moe_geglu_grad(h, da, h))
    assert torch.equal(h, dh)


# ---------------------------------------------------------------- adapters

def lora_reference(x, w, ids, a, b, scale):
    y = x.double() @ w.double().T
    for i in range(a.shape[0]):
        r = (ids == i).nonzero()[:, 0]
        y[r] += scale[i].double() * (x[r].double() @ a[i].double().T) @ b[i].double().T
    return y


def lora_case(seed, t, n, k, N, rank, dtype, order, top=2):
    g = gen(seed)
    x, w = ints(g, dtype, t, k + 8, top=top)[:, :k], ints(g, dtype, n, k, top=top)
    # few non-zero values in A: A x stays below 2^16 (16 bits are handed on) and every sum below 2^24
    a = ints(g, dtype, N, rank, k) * (torch.rand(N, rank, k, generator=g, device="cuda") < 0.1)
    b = ints(g, dtype, N, n, rank)
    scale = torch.tensor([0.5, 1.0, 2.0], device="cuda")[torch.arange(N, device="cuda") % 3].contiguous()
    ids = torch.randint(-1, N, (t,), generator=g, device="cuda", dtype=torch.int32)
    if order == "runs":
        ids = ids.sort().values
    elif order == "none":
        ids.fill_(-1)
    elif order == "one":
        ids.fill_(N - 1)
    elif order == "wild" and t > 2:   # numbers that are no adapter's
        ids[0], ids[t // 2], ids[t - 1] = N, 2 ** 31 - 1, -2 ** 31
    return x, w, ids, a, b, scale


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("t,n,k,N,rank,order", [
    (1, 8, 8, 1, 8, "one"), (1, 264, 1000, 3, 16, "runs"), (2, 136, 72, 5, 24, "any"), (7, 72, 328, 2, 64, "wild"),
    (33, 200, 512, 40, 8, "any"), (64, 704, 200, 7, 128, "any"), (64, 136, 136, 64, 40, "none"),
    (65, 264, 136, 9, 16, "any"), (127, 40, 64, 3, 32, "wild"), (300, 328, 520, 4, 64, "runs"),
    (513, 1000, 264, 100, 8, "any"), (1000, 136, 1000, 1, 128, "one"), (600, 520, 72, 300, 16, "any"),
    (2100, 520, 328, 12, 64, "runs"), (66000, 72, 64, 5, 8, "runs")])
def test_adapters(t, n, k, N, rank, order, dtype):
    x, w, ids, a, b, scale = lora_case(t, t, n, k, N, rank, dtype, order)
    whole, y = buffer(dtype, t, n)
    workspace = torch.full((4 * t * rank,), 255, dtype=torch.uint8, device="cuda")   # NaN, whatever the type
    ok(moe.moe_lora_mm(x, w, ids, a, b, scale, y, workspace))
    assert torch.equal(y, lora_reference(x, w, ids, a, b, scale).to(dtype))
    assert (whole[:, n:] == SENTINEL).all()


@pytest.mark.parametrize("t", [40, 200])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_adapters_of_real_values(t, dtype):
    """The sums' fp32 errors as in test_products_of_real_values, A x and B's sum among them; A x handed on as two
    bf16 values (half a step of the second: 2^-17); and one rounding."""
    g, n, k, N, rank = gen(t), 328, 1000, 5, 64
    x = torch.randn(t, k, generator=g, device="cuda").to(dtype)
    w = (torch.randn(n, k, generator=g, device="cuda") / k ** 0.5).to(dtype)
    a = (torch.randn(N, rank, k, generator=g, device="cuda") / k ** 0.5).to(dtype)
    b = (torch.randn(N, n, rank, generator=g, device="cuda") / 4).to(dtype)
    scale = torch.rand(N, generator=g, device="cuda") + 0.5
    ids = torch.randint(-1, N, (t,), generator=g, device="cuda", dtype=torch.int32)
    y = torch.empty(t, n, dtype=dtype, device="cuda")
    ok(moe.moe_lora_mm(x, w, ids, a, b, scale, y, torch.empty(4 * t * rank, dtype=torch.uint8, device="cuda")))
    ref = lora_reference(x, w, ids, a, b, scale)
    mag = lora_reference(x.abs(), w.abs(), ids, a.abs(), b.abs(), scale)
    err = (y.double() - ref).abs()
    assert (err <= torch.finfo(dtype).eps / 2 * ref.abs() + 1.01 * ((k / 16 + rank + 8) * 17 * 2 ** -23 + 2 ** -17) * mag).all()


@pytest.mark.parametrize("t", [30, 150, 700])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_a_broken_adapter_stays_with_its_requests(t, dtype):
    x, w, ids, a, b, scale = lora_case(9, t, 136, 200, 5, 16, dtype, "any")
    ws = torch.empty(4 * t * 16, dtype=torch.uint8, device="cuda")
    y = torch.empty(t, 136, dtype=dtype, device="cuda")
    a[1], b[2], b[3, 17, 5] = math.nan, math.inf, -math.inf   # all of A, all of B, one value of B
    ok(moe.moe_lora_mm(x, w, ids, a, b, scale, y, ws))
    a[1], b[2], b[3, 17, 5] = 0, 0, 0
    want = lora_reference(x, w, ids, a, b, scale).to(dtype)
    fine = (ids != 1) & (ids != 2) & (ids != 3)
    assert torch.equal(y[fine], want[fine])
    assert not y[(ids == 1) | (ids == 2)].isfinite().any()
    third = ids == 3
    assert not y[third, 17].isfinite().any()
    others = torch.arange(136, device="cuda") != 17
    assert torch.equal(y[third][:, others], want[third][:, others])


@pytest.mark.parametrize("t", [40, 900])
def test_rows_that_are_not_finite_stay_alone(t):
    x, w, ids, a, b, scale = lora_case(10, t, 264, 200, 3, 24, BF16, "any")
    x[3], x[t - 1, 7] = math.nan, math.inf
    y = torch.empty(t, 264, dtype=BF16, device="cuda")
    ok(moe.moe_lora_mm(x, w, ids, a, b, scale, y, torch.empty(4 * t * 24, dtype=torch.uint8, device="cuda")))
    fine = torch.ones(t, dtype=torch.bool, device="cuda")
    fine[3] = fine[t - 1] = False
    assert torch.equal(y[fine], lora_reference(x, w, ids, a, b, scale).to(BF16)[fine])
    assert y[3].isnan().all()


# ---------------------------------------------------------------- streams, graphs, devices

def test_captured_and_replayed_with_new_groups():
    """The offsets are read on the device: a captured call follows them, and the rows' values."""
    g, E, n, k, m = gen(11), 9, 136, 200, 600
    x, w = ints(g, BF16, m, k), ints(g, BF16, E, 2 * n, k)
    w2 = ints(g, BF16, E, k, n)
    off = offsets_of([10] * E)
    a, h = torch.empty(m, n, dtype=BF16, device="cuda"), torch.empty(m, 2 * n, dtype=BF16, device="cuda")
    y, dw = torch.empty(m, k, dtype=F32, device="cuda"), torch.empty(E, k, n, dtype=F32, device="cuda")
    n = 128
    w, a, h, w2, dw = w[:, :2 * n].contiguous(), a[:, :n], h[:, :2 * n], w2[:, :, :n].contiguous(), dw[:, :, :n].contiguous()

    def step():
        moe.check(moe.moe_grouped_geglu(x, off, w, a, h))
        moe.check(moe.moe_grouped_mm(a, off, w2, y))
        moe.check(moe.moe_grouped_wgrad(x, a, off, dw))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for counts in ([0, 300, 1, 2, 0, 0, 290, 7, 0], [60] * 9, [0] * 8 + [3]):
        off.copy_(offsets_of(counts))
        x.copy_(ints(g, BF16, m, k))
        y.fill_(SENTINEL)
        graph.replay()
        ok(moe.MOE_OK)
        rows = sum(counts)
        got_y, got_dw, got_a = y.clone(), dw.clone(), a[:rows].clone()
        assert torch.equal(h[:rows], products(x, counts, w)[:rows].to(BF16))
        ref = products(a, counts, w2)
        assert ((got_y[:rows] - ref[:rows]).abs() <= 20 * 17 * 2 ** -23 * products(a.abs(), counts, w2.abs())[:rows]).all()
        assert (got_y[rows:] == SENTINEL).all()
        step()
        ok(moe.MOE_OK)
        assert torch.equal(y, got_y) and torch.equal(dw, got_dw) and torch.equal(a[:rows], got_a)


def test_calls_on_two_streams_at_once():
    g, n, k, E = gen(12), 264, 520, 6
    counts = [70, 0, 129, 300, 1, 40]
    off, w = offsets_of(counts), ints(g, F16, E, n, k)
    xs = [ints(g, F16, sum(counts), k) for _ in range(8)]
    lx, lw, ids, la, lb, scale = lora_case(13, 48, n, k, 5, 16, F16, "any")
    ys = [torch.empty(sum(counts), n, dtype=F32, device="cuda") for _ in xs]
    ls = [torch.empty(48, n, dtype=F16, device="cuda") for _ in xs]
    ws = [torch.empty(4 * 48 * 16, dtype=torch.uint8, device="cuda") for _ in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i, x in enumerate(xs):
        s = streams[i % 2]
        moe.check(moe.moe_grouped_mm(x, off, w, ys[i], stream=s))
        moe.check(moe.moe_lora_mm(lx, lw, ids, la, lb, scale, ls[i], ws[i], stream=s))
    for s in streams:
        moe.check(moe.moe_grouped_sync(s))
    want = lora_reference(lx, lw, ids, la, lb, scale).to(F16)
    for x, y, l in zip(xs, ys, ls):
        assert torch.equal(y, products(x, counts, w).float())
        assert torch.equal(l, want)


def test_one_workspace_for_calls_in_a_row():
    """Calls in one stream may share a workspace and feed each other without waiting."""
    x, w, ids, a, b, scale = lora_case(14, 48, 200, 200, 6, 16, BF16, "any", top=1)
    ws = torch.empty(4 * 48 * 16, dtype=torch.uint8, device="cuda")
    want, outs, cur = x, [], x
    for i in range(4):
        y = torch.empty(48, 200, dtype=BF16, device="cuda")
        moe.check(moe.moe_lora_mm(cur, w, ids, a, b, scale, y, ws))
        outs.append(y)
        cur = y.clamp(-2, 2)
    ok(moe.MOE_OK)
    for y in outs:
        assert torch.equal(y, lora_reference(want, w, ids, a, b, scale).to(BF16))
        want = y.clamp(-2, 2)


def test_no_rows():
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    x, dy = torch.empty(0, 64, dtype=BF16, device="cuda"), torch.empty(0, 32, dtype=BF16, device="cuda")
    dw = torch.full((3, 32, 64), SENTINEL, dtype=BF16, device="cuda")
    w = torch.zeros_like(dw)
    ok(moe.moe_grouped_mm(x, off, w, dy))
    ok(moe.moe_grouped_wgrad(dy, x, off, dw))
    assert (dw == 0).all()
    dw.fill_(SENTINEL)
    x, dy = torch.full((70, 64), math.nan, dtype=BF16, device="cuda"), torch.full((70, 32), math.nan, dtype=BF16, device="cuda")
    y = torch.full((70, 32), SENTINEL, dtype=BF16, device="cuda")
    ok(moe.moe_grouped_mm(x, off, w, y))
    ok(moe.moe_grouped_wgrad(dy, x, off, dw))
    assert (dw == 0).all() and (y == SENTINEL).all()


@pytest.mark.parametrize("transpose", [False, True])
def test_as_many_rows_as_allowed(transpose):
    m = 2 ** 24
    g = gen(20)
    counts = [5, 2 ** 23 - 3, 2 ** 23 - 4]   # two rows behind them
    x, w = ints(g, BF16, m, 8), ints(g, BF16, 3, 8, 8)
    y = torch.full((m, 8), SENTINEL, dtype=F32, device="cuda")
    ok(moe.moe_grouped_mm(x, offsets_of(counts), w, y, transpose=transpose))
    assert torch.equal(y, products(x, counts, w.transpose(1, 2) if transpose else w).float())


@pytest.mark.parametrize("out", [F32, BF16])
def test_weight_gradients_of_as_many_rows_as_allowed(out):
    m = 2 ** 24
    g = gen(21)
    x, dy = ints(g, BF16, m, 8, top=1), ints(g, BF16, m, 16, top=1)   # every partial sum is below 2^24
    dw = torch.full((2, 16, 8), SENTINEL, dtype=out, device="cuda")
    ok(moe.moe_grouped_wgrad(dy, x, offsets_of([2 ** 23 - 5, 2 ** 23]), dw))
    want = [dy[lo:hi].double().T @ x[lo:hi].double() for lo, hi in ((0, 2 ** 23 - 5), (2 ** 23 - 5, m - 5))]
    assert torch.equal(dw, torch.stack(want).to(out))


def test_adapters_of_many_rows():
    """More blocks of rows than a launch has in any dimension but its first."""
    t = 64 * 65535 + 7
    x, w, ids, a, b, scale = lora_case(22, t, 8, 8, 3, 8, BF16, "any")
    y = torch.full((t, 8), SENTINEL, dtype=BF16, device="cuda")
    ok(moe.moe_lora_mm(x, w, ids, a, b, scale, y, torch.empty(4 * t * 8, dtype=torch.uint8, device="cuda")))
    assert torch.equal(y, lora_reference(x, w, ids, a, b, scale).to(BF16))


@pytest.mark.parametrize("m", [1, 2])
def test_a_row_of_a_wider_tensor(m):
    """The distance of a lone row to the next means nothing: it need not be a multiple of 8."""
    g = gen(23)
    x, w = ints(g, BF16, m, 75 if m == 1 else 80)[:, :72], ints(g, BF16, 1, 40, 72)
    y = torch.full((m, 45 if m == 1 else 48), SENTINEL, dtype=BF16, device="cuda")
    ok(moe.moe_grouped_mm(x, offsets_of([m]), w, y[:, :40]))
    assert torch.equal(y[:, :40], products(x, [m], w).to(BF16)) and (y[:, 40:] == SENTINEL).all()


@pytest.mark.parametrize("captured", [False, True])
def test_many_weight_gradients_on_two_streams_at_once(captured):
    """More tiles than run at once, in launches that share the device: every tile is done, and done once."""
    g, n, k, E = gen(24), 520, 264, 60
    counts = [(7 * e) % 90 for e in range(E)]
    off, m = offsets_of(counts), sum(counts)
    x, dy = ints(g, BF16, m, k), ints(g, BF16, m, n)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.full((E, n, k), SENTINEL, dtype=out, device="cuda") for out in (F32, BF16, F32)] for _ in streams]
    graphs = []
    torch.cuda.synchronize()

    def calls(i):
        for dw in outs[i]:
            moe.check(moe.moe_grouped_wgrad(dy, x, off, dw))

    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            calls(i)
        if captured:
            s.synchronize()
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[i]):
                calls(i)
    torch.cuda.synchronize()
    for repeat in range(4):
        x.copy_(ints(g, BF16, m, k))
        torch.cuda.synchronize()
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                graphs[i].replay() if captured else calls(i)
        for s in streams:
            moe.check(moe.moe_grouped_sync(s))
        lo, want = 0, []
        for c in counts:
            want.append(dy[lo:lo + c].double().T @ x[lo:lo + c].double())
            lo += c
        for dw in outs[0] + outs[1]:
            assert torch.equal(dw, torch.stack(want).to(dw.dtype))
