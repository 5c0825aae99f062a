"""The norm and its gradient against the formulas in 64 bits."""

import pytest
import torch

import bit_routed_expert_router_gb300 as moe

pytestmark = pytest.mark.gpu

BF16, F16, F32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
SHAPES = [(1, 8), (1, 2816), (3, 136), (17, 120), (2, 128), (600, 704), (33, 8200), (5, 16384), (1025, 264)]
# fp32 roundings on the way to a value: a row's sum takes at most 16 products a thread, 5 steps of a warp and 32 warps, each
# half a step of 2^-23 of a sum of squares, which the root halves; the root, the quotient and the products add five.  32 in all.
ROUNDED = 32 * 2.0 ** -24


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rand(g, dtype, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def half_step(dtype):
    """Relative to a value, and the least one (half a step of the subnormal values)."""
    return torch.finfo(dtype).eps / 2, torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def normed(r, w, eps=1e-6):
    v = r.double()
    v = v / (v.square().mean(1, keepdim=True) + eps).sqrt()
    return v if w is None else v * w.double()


def near16(got, want, dtype):
    rel, least = half_step(dtype)
    assert torch.all((got.double() - want).abs() <= want.abs() * (rel + 2 * ROUNDED) + least)


def groups(v):
    return torch.nn.functional.pad(v, (0, -v.shape[1] % 128)).view(v.shape[0], -1, 128)


def near8(q, s, want):
    """e4m3 rows and their scales against the values: half a step of e4m3 (2^-4 of a value, 2^-10 of the scale at least)."""
    top = groups(want).abs().amax(-1).clamp(min=2.0 ** -100)
    assert torch.all((s.double() - top / 448).abs() <= 4 * ROUNDED * top / 448)
    value = q.double() * s.double().repeat_interleave(128, 1)[:, :want.shape[1]]
    wide = s.double().repeat_interleave(128, 1)[:, :want.shape[1]]
    assert torch.all((value - want).abs() <= want.abs() * (2.0 ** -4 + 8 * ROUNDED) + wide * 2.0 ** -10)
    # and the rounding is to the nearest: the quotient that was rounded is off by 4 ROUNDED of itself at most, so the value
    # taken is at most twice that further away than the one nearest to the exact quotient
    exact = want / wide
    nearest = exact.float().clamp(-448, 448).to(E4M3).double()
    assert torch.all((q.double() - exact).abs() <= (nearest - exact).abs() + 8 * ROUNDED * exact.abs())


def call(h, delta, w, out, inplace=False, eps=1e-6):
    m, d = h.shape
    dev = h.device
    y = torch.empty(m, d, dtype=h.dtype, device=dev) if out != "8" else None
    y8 = torch.empty(m, d, dtype=E4M3, device=dev) if out != "16" else None
    s = torch.empty(m, (d + 127) // 128, device=dev) if out != "16" else None
    r = None if delta is None else h if inplace else torch.empty_like(h)
    moe.check(moe.moe_rmsnorm(h, y, y8, s, delta=delta, h_out=r, weight=w, eps=eps))
    return r, y, y8, s


@pytest.mark.parametrize("m,d", SHAPES)
@pytest.mark.parametrize("dtype,delta,weight,out", [(BF16, None, True, "both"), (F16, F16, False, "both"), (BF16, F32, True, "8"),
                                                    (F16, F32, True, "16"), (BF16, BF16, False, "16"), (F16, None, False, "8")])
def test_norm(m, d, dtype, delta, weight, out):
    g = gen(m + d)
    h = rand(g, dtype, m, d, scale=3)
    dl = None if delta is None else rand(g, delta, m, d)
    w = rand(g, dtype, d) if weight else None
    r, y, y8, s = call(h, dl, w, out)
    if dl is not None:
        assert torch.equal(r, (h.float() + dl.float()).to(dtype))
    want = normed(h if r is None else r, w)
    if y is not None:
        near16(y, want, dtype)
    if y8 is not None:
        near8(y8, s, want)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_strided_rows_and_outputs_in_place(dtype):
    g = gen(3)
    wide = rand(g, dtype, 9, 1000)
    h, delta, w = wide[:, 8:528], rand(g, F32, 9, 1024)[:, 4:524], rand(g, dtype, 520)
    before, sum_ = wide.clone(), (h.float() + delta.float()).to(dtype)
    buf8 = torch.full((9, 1024), 1.0, device="cuda").to(E4M3)
    s = torch.empty(9, 5, device="cuda")
    moe.check(moe.moe_rmsnorm(h, None, buf8[:, 16:536], s, delta=delta, h_out=h, weight=w))
    assert torch.equal(h, sum_)
    assert torch.equal(wide[:, :8], before[:, :8]) and torch.equal(wide[:, 528:], before[:, 528:])
    assert torch.all(buf8[:, :16].float() == 1) and torch.all(buf8[:, 536:].float() == 1)
    near8(buf8[:, 16:536], s, normed(sum_, w))
    moe.check(moe.moe_rmsnorm(h, h, weight=w))
    near16(h, normed(sum_, w), dtype)


def test_zeros_large_small_and_non_finite_values():
    h = torch.zeros(6, 256, dtype=BF16, device="cuda")
    h[1] = 1e18                       # squares add up to 2.6e38, inside fp32
    h[2] = 1e-30                      # nothing but eps in the mean
    h[3, 5], h[3, 6] = float("inf"), 2.0
    h[4, 200], h[4, 0] = float("nan"), 1.0
    h[5, :] = torch.linspace(-4, 4, 256)
    _, y, y8, s = call(h, None, None, "both")
    near16(y[[0, 1, 2, 5]], normed(h[[0, 1, 2, 5]], None), BF16)
    near8(y8[[0, 1, 2, 5]], s[[0, 1, 2, 5]], normed(h[[0, 1, 2, 5]], None))
    assert torch.all(s[0] == 2.0 ** -100 / 448) and torch.all(y8[0].float() == 0)
    # an infinity: 1 / sqrt(infinity) is 0, so NaN where it stands and 0 elsewhere
    assert torch.isnan(y[3, 5]) and torch.all(y[3, :5] == 0) and torch.all(y[3, 6:] == 0)
    assert torch.isnan(s[3, 0]) and torch.all(torch.isnan(y8[3, :128].float())) and torch.all(y8[3, 128:].float() == 0)
    assert torch.all(torch.isnan(y[4])) and torch.all(torch.isnan(s[4])) and torch.all(torch.isnan(y8[4].float()))


def test_an_infinite_weight_stays_in_its_block():
    h, w = torch.ones(2, 300, dtype=F16, device="cuda")[:, :296].contiguous(), torch.ones(296, dtype=F16, device="cuda")
    w[130] = float("inf")
    _, y, y8, s = call(h, None, w, "both")
    assert torch.all(torch.isinf(y[:, 130])) and torch.all(torch.isinf(s[:, 1])) and torch.all(torch.isnan(y8[:, 130].float()))
    rest = [i for i in range(128, 256) if i != 130]
    assert torch.all(y8[:, rest].float() == 0)
    assert torch.all(torch.isfinite(s[:, [0, 2]])) and torch.all(y8[:, :128].float() == 448) and torch.all(y8[:, 256:].float() == 448)


def grads(h, dy, dres, w, eps=1e-6):
    x = h.double().requires_grad_()
    wt = torch.ones(h.shape[1], dtype=torch.float64, device="cuda") if w is None else w.double()
    wt.requires_grad_()
    dh, dw = torch.autograd.grad(normed(x, wt, eps), (x, wt), dy.double())
    return dh if dres is None else dh + dres.double(), dw


def call_grad(h, dy, dres, w, dh=None):
    m, d = h.shape
    dh = torch.empty_like(h) if dh is None else dh
    dw = torch.empty(d, device="cuda") if w is not None else None
    ws = torch.empty(4 * d * min(m, 512), dtype=torch.uint8, device="cuda") if w is not None else None
    moe.check(moe.moe_rmsnorm_grad(h, dy, dh, dres=dres, weight=w, dweight=dw, workspace=ws))
    return dh, dw


def near_grads(h, dy, dres, w, dh, dw):
    want, want_w = grads(h, dy, dres, w)
    rstd = 1 / (h.double().square().mean(1, keepdim=True) + 1e-6).sqrt()
    gy, x = dy.double() * (1 if w is None else w.double()), h.double() * rstd
    # fp32 roundings of both terms' sizes, then the rounding of the output
    parts = rstd * (gy.abs() + x.abs() * (gy * x).abs().mean(1, keepdim=True)) + (0 if dres is None else dres.double().abs())
    rel, least = half_step(h.dtype)
    assert torch.all((dh.double() - want).abs() <= want.abs() * rel + 2 * ROUNDED * parts + least)
    if dw is not None:
        # m / 512 + 1 rows in one sum, 48 of those, and the roundings of a term
        n = (h.shape[0] / 512 + 50) * 2.0 ** -24 + 2 * ROUNDED
        assert torch.all((dw.double() - want_w).abs() <= n * (dy.double() * x).abs().sum(0))


@pytest.mark.parametrize("m,d", SHAPES)
@pytest.mark.parametrize("dtype,weight,residual", [(BF16, True, True), (F16, False, False), (F16, True, False), (BF16, False, True)])
def test_gradients(m, d, dtype, weight, residual):
    g = gen(2 * m + d)
    h, dy = rand(g, dtype, m, d, scale=2), rand(g, dtype, m, d)
    dres, w = rand(g, dtype, m, d) if residual else None, rand(g, dtype, d) if weight else None
    near_grads(h, dy, dres, w, *call_grad(h, dy, dres, w))


def test_gradients_strided_and_in_place():
    g = gen(11)
    wide = rand(g, BF16, 70, 1000)
    h, dy, dres, w = wide[:, 16:720], rand(g, BF16, 70, 704), rand(g, BF16, 70, 704), rand(g, BF16, 704)
    keep = dy.clone(), dres.clone(), h.clone()
    near_grads(h, *keep[:2], w, *call_grad(h, dy, dres, w, dh=dy))
    near_grads(h, *keep[:2], w, *call_grad(h, keep[0], dres, w, dh=dres))
    near_grads(keep[2], *keep[:2], w, *call_grad(h, *keep[:2], w, dh=h))


def test_gradients_against_differences():
    """The formula itself: central differences in 64 bits along a direction of both leaves."""
    g = gen(5)
    h, dy, w = (torch.randn(*s, generator=g, device="cuda", dtype=torch.float64) for s in [(4, 40), (4, 40), (40,)])
    dh, dw = grads(h, dy, None, w)
    a, b = torch.randn_like(h), torch.randn_like(w)
    f = lambda t: (normed(h.detach() + t * a, w.detach() + t * b) * dy).sum()  # noqa: E731
    slope = float((dh * a).sum() + (dw * b).sum())
    assert abs(float(f(1e-5) - f(-1e-5)) / 2e-5 - slope) <= 1e-7 * float((dh * a).abs().sum() + (dw * b).abs().sum())


def test_no_rows():
    h, dw = torch.empty(0, 64, dtype=BF16, device="cuda"), torch.ones(64, device="cuda")
    w = torch.ones(64, dtype=BF16, device="cuda")
    moe.check(moe.moe_rmsnorm(h, h, weight=w))
    moe.check(moe.moe_rmsnorm_grad(h, h, h, weight=w, dweight=dw, workspace=torch.empty(0, dtype=torch.uint8, device="cuda")))
    assert torch.all(dw == 0)


def test_in_a_graph_and_on_another_stream():
    g = gen(21)
    h, dy, w = rand(g, BF16, 700, 2816), rand(g, BF16, 700, 2816), rand(g, BF16, 2816)
    y8, s = torch.empty(700, 2816, dtype=E4M3, device="cuda"), torch.empty(700, 22, device="cuda")
    dh, dw = torch.empty_like(h), torch.empty(2816, device="cuda")
    ws = torch.empty(4 * 512 * 2816, dtype=torch.uint8, device="cuda")

    def both():
        moe.check(moe.moe_rmsnorm(h, None, y8, s, weight=w))
        moe.check(moe.moe_rmsnorm_grad(h, dy, dh, weight=w, dweight=dw, workspace=ws))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for seed in (1, 2):
        h.copy_(rand(gen(seed), BF16, 700, 2816))
        graph.replay()
        got = [t.clone() for t in (y8.view(torch.uint8), s, dh, dw)]
        both()
        for a, b in zip(got, (y8.view(torch.uint8), s, dh, dw)):
            assert torch.equal(a, b)


# the forms that the shapes above leave out: two rows a thread (many rows), and two words a thread of 288 to 512 in the gradient
MORE = [(2501, 2816), (10001, 264), (20001, 8), (2433, 4096), (40, 4104), (301, 5000), (9, 8192)]


@pytest.mark.parametrize("m,d", MORE)
@pytest.mark.parametrize("dtype,delta,out", [(BF16, F32, "both"), (F16, F16, "8"), (BF16, None, "16")])
def test_norm_of_many_and_of_long_rows(m, d, dtype, delta, out):
    g = gen(3 * m + d)
    h, w = rand(g, dtype, m, d, scale=3), rand(g, dtype, d)
    dl = None if delta is None else rand(g, delta, m, d)
    before = h.clone()
    r, y, y8, s = call(h, dl, w, out, inplace=True)
    if dl is not None:
        assert torch.equal(r, (before.float() + dl.float()).to(dtype))
    want = normed(h, w)
    if y is not None:
        near16(y, want, dtype)
    if y8 is not None:
        near8(y8, s, want)


@pytest.mark.parametrize("m,d", MORE)
@pytest.mark.parametrize("dtype,residual", [(BF16, True), (F16, False)])
def test_gradients_of_many_and_of_long_rows(m, d, dtype, residual):
    g = gen(5 * m + d)
    h, dy, w = rand(g, dtype, m, d, scale=2), rand(g, dtype, m, d), rand(g, dtype, d)
    dres = rand(g, dtype, m, d) if residual else None
    near_grads(h, dy, dres, w, *call_grad(h, dy, dres, w))


def test_calls_on_two_streams_at_once():
    """Workspaces of their own; the same inputs."""
    g = gen(41)
    h, dy, w = rand(g, BF16, 900, 1032), rand(g, BF16, 900, 1032), rand(g, BF16, 1032)
    want = call_grad(h, dy, None, w)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append([call_grad(h, dy, None, w) for _ in range(3)])
    torch.cuda.synchronize()
    for dh, dw in sum(got, []):
        assert torch.equal(dh, want[0]) and torch.equal(dw, want[1])


@pytest.mark.parametrize("size,weight,eps", [(1e-27, 1.0, 1e-30), (1e-20, 1e-7, 1e-30), (1.0, 1e26, 1e-6), (1e17, 1e-20, 0.0), (0.0, 1.0, 1e-30)])
def test_quotients_of_very_small_and_large_values(size, weight, eps):
    """Past where they come from the row and the weight alone."""
    g = gen(51)
    h, w = rand(g, BF16, 6, 400, scale=size), (1 + 0.2 * torch.randn(400, generator=g, device="cuda")).mul(weight).to(BF16)
    _, y, y8, s = call(h, None, w, "both", eps=eps)
    want = normed(h, w, eps)
    near16(y, want, BF16)
    near8(y8, s, want)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_quotients_are_rounded_to_the_nearest(dtype):
    """e4m3 values against quotients in 64 bits: off only where these lie next to a tie, by three roundings of fp32 at most
    (r w is exact, 448 / top takes two, the product one)."""
    h, w = rand(gen(61), dtype, 3000, 1024), rand(gen(62), dtype, 1024)
    _, _, y8, _ = call(h, None, w, "8")
    u = groups(h.double() * w.double())
    q = (u * 448 / u.abs().amax(-1, keepdim=True)).view(3000, 1024)
    got = y8.double()
    nearest = q.float().to(E4M3).double()
    assert torch.all((got - q).abs() <= (nearest - q).abs() + 3 * 2.0 ** -24 * 2 * q.abs())


@pytest.mark.parametrize("m", [5, 2500])   # one row a thread, and two
def test_rows_that_are_infinite_in_eight_bits(m):
    """Squares below fp32's range and eps = 0: r times an infinite quotient.  A block with a zero in it has a NaN, one
    without has infinities only, and the outputs agree."""
    h = torch.full((m, 2816), 1e-23, dtype=BF16, device="cuda")
    h[:, 200:210] = 0                  # block 1: infinities and NaN; block 2 none but NaN
    h[:, 256:384] = 0
    h[1] = 3.0                         # a row as others are
    _, y, y8, s = call(h, None, None, "both", eps=0.0)
    v = h.float() / h.float().square().mean(1, keepdim=True).sqrt()
    assert torch.equal(torch.isnan(y), torch.isnan(v)) and torch.equal(torch.isinf(y), torch.isinf(v))
    rest = [i for i in range(m) if i != 1]
    assert torch.all(torch.isnan(s[rest, 1:3])) and torch.all(torch.isinf(s[rest, :1])) and torch.all(torch.isinf(s[rest, 3:]))
    assert torch.all(torch.isnan(y8[rest].float()))
    near8(y8[1:2], s[1:2], normed(h[1:2], None))


@pytest.mark.parametrize("m", [6, 2500])
@pytest.mark.parametrize("size,weight,eps", [(1e17, 1e25, 1e-6), (1e17, 1e25, 0.0), (5e17, 2e21, 1e-6), (1e-20, 1e-24, 1e-30)])
def test_products_of_row_and_weight_past_fp32(m, size, weight, eps):
    """r w is above or below fp32's range, the normed value times the weight is not."""
    g = gen(71)
    h = (torch.randn(m, 400, generator=g, device="cuda").clamp(-3, 3) * size).to(BF16)
    w = (1 + 0.2 * torch.randn(400, generator=g, device="cuda")).mul(weight).to(BF16)
    _, y, y8, s = call(h, None, w, "both", eps=eps)
    want = normed(h, w, eps)
    near16(y, want, BF16)
    near8(y8, s, want)


def parts_of(m, d):
    """CTAs of the gradient's row kernel: each sums every parts-th row, and their sums are added 64 at a time."""
    words = d // 8
    warps = (words + 63) // 64 if words > 512 else (words + 31) // 32
    return min(m, 512, torch.cuda.get_device_properties(0).multi_processor_count * max(1, 32 // warps))


@pytest.mark.parametrize("m,d", [(20001, 264), (9000, 2816), (40000, 64), (3000, 8200), (700, 16384)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_weight_gradients_of_many_rows_of_one_sign(m, d, dtype):
    """dy x > 0: what long fp32 sums lose adds up.  A column takes ceil(m / parts) additions in a CTA, ceil(parts / 64) in a
    thread of the second kernel and 64 there, each half a step of a sum that is the whole one at most, and a term its own
    roundings (ROUNDED for 1 / sqrt, two products)."""
    g = gen(m + d)
    h, dy = (torch.rand(m, d, generator=g, device="cuda") + 0.5).to(dtype), (torch.rand(m, d, generator=g, device="cuda") + 0.5).to(dtype)
    w = rand(g, dtype, d)
    _, dw = call_grad(h, dy, None, w)
    x = normed(h, None)
    want = (dy.double() * x).sum(0)
    parts = parts_of(m, d)
    n = -(-m // parts) + -(-parts // 64) + 64
    assert torch.all((dw.double() - want).abs() <= (n * 2.0 ** -24 + ROUNDED + 2 * 2.0 ** -24) * want)


@pytest.mark.parametrize("m,d", [(7, 2816), (2500, 264), (40, 8200), (301, 16384)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_the_normed_rows_in_deltas_place(m, d, dtype):
    g = gen(91)
    h, delta, w = rand(g, dtype, m, d, scale=2), rand(g, dtype, m, d), rand(g, dtype, d)
    y, r, y8, s = torch.empty_like(h), torch.empty_like(h), torch.empty(m, d, dtype=E4M3, device="cuda"), torch.empty(m, (d + 127) // 128, device="cuda")
    moe.check(moe.moe_rmsnorm(h, y, y8, s, delta=delta, h_out=r, weight=w))
    y8b, sb = torch.empty_like(y8), torch.empty_like(s)
    moe.check(moe.moe_rmsnorm(h, delta, y8b, sb, delta=delta, h_out=h, weight=w))   # y in delta's place, h_out in h's
    assert torch.equal(delta, y) and torch.equal(h, r)
    assert torch.equal(y8.view(torch.uint8), y8b.view(torch.uint8)) and torch.equal(s, sb)
