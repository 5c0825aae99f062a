"""The layer for a few tokens against the formula in 64 bits."""

import pytest
import torch

import bit_routed_expert_router_gb300 as moe
from ops8_reference import BF16, E4M3, F16, F32, blocks, gelu, gen, rand8, rand_scale, wide_weights

pytestmark = pytest.mark.gpu


def weights(g, dtype, eight, lead, d, f):
    if not eight:
        r = lambda *s: (torch.randn(*s, generator=g, device="cuda") * s[-1] ** -0.5).to(dtype)  # noqa: E731
        return r(*lead, 2 * f, d), r(*lead, d, f)
    gu, down = rand8(g, *lead, 2 * f, d), rand8(g, *lead, d, f)
    # values of about 60 times 2^-10: weights of about the size that the fan-in wants
    su, sd = rand_scale(g, *lead, blocks(2 * f), blocks(d)) / d ** 0.5, rand_scale(g, *lead, blocks(d), blocks(f)) / f ** 0.5
    return gu, down, 8 * su, 8 * sd


def wide(w):
    return [t.double() for t in w[:2]] if len(w) == 2 else [wide_weights(w[0], w[2]), wide_weights(w[1], w[3])]


def case(t, k, E, d, f, fs, dtype=BF16, eight=False, seed=0):
    g = gen(seed + 1000 * t + d)
    x = torch.randn(t, d, generator=g, device="cuda").to(dtype)
    top = torch.randn(t, E, generator=g, device="cuda").topk(k)
    ids, gates = top.indices.int(), torch.softmax(top.values, 1)
    return x, ids, gates, weights(g, dtype, eight, (E,), d, f), weights(g, dtype, eight, (), d, fs) if fs else None


def call(x, ids, gates, routed, shared, variant=moe.MOE_GELU_ERF, out=None, y=None, stream=None):
    f, fs = routed[1].shape[-1], shared[1].shape[-1] if shared else 0
    ws = torch.empty(2 * x.shape[0] * (ids.shape[1] * f + fs), dtype=torch.uint8, device="cuda")
    y = torch.full(x.shape, 7.0, dtype=out or x.dtype, device="cuda") if y is None else y
    moe.check(moe.moe_token_layer(x, ids, gates, routed, y, ws, shared=shared, gelu_variant=variant, stream=stream))
    return y


def check(y, x, ids, gates, routed, shared, variant):
    """Error: the rounding of each a to 16 bits and the fp32 sums before it, carried through the down product's magnitudes,
    then the output's rounding."""
    half = torch.finfo(x.dtype).eps / 2
    tiny = torch.finfo(x.dtype).smallest_normal * half
    d = x.shape[1]
    want, bound = torch.zeros(x.shape, dtype=torch.float64, device="cuda"), torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    E = routed[0].shape[0]

    def add(t, gate, gu, down):
        f = down.shape[1]
        xt = x[t].double()
        h, size = gu @ xt, gu.abs() @ xt.abs()
        # the tensor cores truncate, the partial sums round: at most 2^-23 of the magnitudes a product, in fp32
        e32 = (d + 64) * 2.0 ** -23
        g, u, eg, eu = h[:f], h[f:], e32 * size[:f], e32 * size[f:]
        a = gate * gelu(g, variant) * u
        ea = abs(gate) * (1.13 * eg * (u.abs() + eu) + gelu(g, variant).abs() * eu) + 2.0 ** -18 * a.abs()
        ea = ea + half * (a.abs() + ea) + tiny
        want[t] += down @ a
        bound[t] += down.abs() @ (ea + (f + 64) * 2.0 ** -23 * (a.abs() + ea))

    rw, sw = wide(routed), wide(shared) if shared else None
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if 0 <= e < E:
                add(t, float(gates[t, j]), rw[0][e], rw[1][e])
        if shared:
            add(t, 1.0, *sw)
    # the sums over the experts take a rounding for each of them
    bound += (ids.shape[1] + 2) * 2.0 ** -23 * (want.abs() + bound)
    if y.dtype != F32:
        out = torch.finfo(y.dtype).eps / 2
        bound += out * (want.abs() + bound) + torch.finfo(y.dtype).smallest_normal * out
    err = (y.double() - want).abs()
    assert torch.all(err <= bound), float((err / bound).max())
    # and as a whole: independent roundings do not add up as their bound does
    assert (y.double() - want).norm() <= 4 * half * want.norm()


@pytest.mark.parametrize("t,k,E,d,f,fs", [(1, 1, 1, 16, 16, 0), (1, 2, 8, 256, 128, 128), (3, 2, 5, 144, 176, 48), (7, 8, 16, 272, 80, 0),
                                          (8, 4, 12, 528, 144, 272), (9, 3, 9, 400, 304, 16), (17, 5, 40, 656, 96, 128),
                                          (32, 8, 32, 1040, 208, 512), (31, 32, 64, 128, 64, 64), (1, 8, 128, 2816, 704, 2816)])
@pytest.mark.parametrize("dtype,eight,variant", [(BF16, False, moe.MOE_GELU_ERF), (F16, False, moe.MOE_GELU_TANH),
                                                 (BF16, True, moe.MOE_GELU_TANH), (F16, True, moe.MOE_GELU_ERF)])
def test_layer(t, k, E, d, f, fs, dtype, eight, variant):
    args = case(t, k, E, d, f, fs, dtype, eight)
    for out in (dtype, F32):
        check(call(*args, variant=variant, out=out), *args, variant)


@pytest.mark.parametrize("eight", [False, True])
def test_every_token_at_one_expert_and_repeated_ids(eight):
    x, ids, gates, routed, shared = case(32, 4, 6, 320, 112, 64, BF16, eight)
    ids[:] = 5
    gates = torch.rand(32, 4, generator=gen(3), device="cuda")
    check(call(x, ids, gates, routed, shared), x, ids, gates, routed, shared, moe.MOE_GELU_ERF)


@pytest.mark.parametrize("eight", [False, True])
def test_ids_outside_add_nothing(eight):
    x, ids, gates, routed, shared = case(5, 3, 6, 320, 112, 64, F16, eight)
    ids[0] = -1
    ids[1, 1], ids[2, 0], ids[3, 2] = 6, 1 << 30, -(1 << 31)
    check(call(x, ids, gates, routed, shared), x, ids, gates, routed, shared, moe.MOE_GELU_ERF)
    ids[:] = -1
    check(call(x, ids, gates, routed, shared), x, ids, gates, routed, shared, moe.MOE_GELU_ERF)
    assert torch.all(call(x, ids, gates, routed, None) == 0)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("t", [4, 20])
def test_non_finite_weights_reach_their_own_tokens(eight, t):
    x, ids, gates, routed, shared = case(t, 2, 8, 320, 112, 64, BF16, eight)
    ids[:, 0], ids[:, 1] = 1, 2
    ids[1, 0], ids[3, 1] = 7, 7
    clean = call(x, ids, gates, routed, shared)
    for which, spot in ((0, (7, 5, 9)), (1, (7, 300, 100))):
        bad = [w.clone() for w in routed]
        if eight:
            bad[which].view(torch.uint8)[spot] = 0x7F   # NaN
        else:
            bad[which][spot] = float("inf")
        y = call(x, ids, gates, tuple(bad), shared)
        hit = torch.zeros(t, dtype=torch.bool, device="cuda")
        hit[1] = hit[3] = True
        assert torch.equal(y[~hit], clean[~hit])
        if which == 0:      # a feature of a: every output that weighs it
            assert torch.all(~torch.isfinite(y[hit]))
        else:
            assert torch.all(~torch.isfinite(y[hit, 300]))
            y[:, 300] = clean[:, 300]
            assert torch.equal(y, clean)


def test_non_finite_tokens_stay_tokens():
    args = case(12, 3, 8, 272, 96, 80, BF16)
    clean = call(*args)
    x = args[0].clone()
    x[4, 7] = float("nan")
    y = call(x, *args[1:])
    assert torch.all(torch.isnan(y[4]))
    y[4] = clean[4]
    assert torch.equal(y, clean)


def test_strided_rows_leave_the_rest():
    x, ids, gates, routed, shared = case(6, 2, 4, 256, 64, 64, BF16)
    wide_x = torch.randn(6, 512, device="cuda").to(BF16)
    wide_x[:, 64:320] = x
    y = torch.full((6, 400), 7.0, dtype=F32, device="cuda")
    call(wide_x[:, 64:320], ids, gates, routed, shared, y=y[:, 8:264])
    check(y[:, 8:264], x, ids, gates, routed, shared, moe.MOE_GELU_ERF)
    assert torch.all(y[:, :8] == 7) and torch.all(y[:, 264:] == 7)


@pytest.mark.parametrize("eight", [False, True])
def test_in_a_graph_with_new_tokens(eight):
    x, ids, gates, routed, shared = case(3, 4, 16, 512, 256, 384, F16, eight)
    y, ws = torch.empty_like(x), torch.empty(2 * 3 * (4 * 256 + 384), dtype=torch.uint8, device="cuda")

    def step():
        moe.check(moe.moe_token_layer(x, ids, gates, routed, y, ws, shared=shared))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
        step()
    for seed in (1, 2):
        other = case(3, 4, 16, 512, 256, 384, F16, False, seed=seed)
        x.copy_(other[0]), ids.copy_(other[1]), gates.copy_(other[2])
        graph.replay()
        got = y.clone()
        step()
        assert torch.equal(got, y)
        check(y, x, ids, gates, routed, shared, moe.MOE_GELU_ERF)


def test_two_streams_at_once():
    """A workspace each."""
    args = [case(5, 4, 16, 512, 256, 384, BF16, seed=s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in args]
    torch.cuda.synchronize()
    ys = [torch.empty_like(a[0]) for a in args]
    ws = [torch.empty(2 * 5 * (4 * 256 + 384), dtype=torch.uint8, device="cuda") for _ in args]
    for _ in range(10):
        for a, y, w, s in zip(args, ys, ws, streams):
            moe.check(moe.moe_token_layer(*a[:4], y, w, shared=a[4], stream=s))
    torch.cuda.synchronize()
    for a, y in zip(args, ys):
        check(y, *a, moe.MOE_GELU_ERF)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("t,d,f,fs", [(1, 512, 1024, 2048), (3, 256, 2048, 0), (32, 1024, 512, 1024), (2, 16, 4096, 16)])
def test_narrow_outputs_and_long_reductions(t, d, f, fs, eight):
    """Outputs whose reduction is split over a cluster of two to eight CTAs."""
    args = case(t, 4, 12, d, f, fs, BF16, eight)
    check(call(*args), *args, moe.MOE_GELU_ERF)


def test_the_most_pairs_and_experts():
    """32 tokens that name 32 experts each, of 1024."""
    args = case(32, 32, 1024, 64, 32, 48, F16)
    check(call(*args), *args, moe.MOE_GELU_ERF)


def formula(x, ids, gates, routed, shared, variant):
    rw, sw = wide(routed), wide(shared) if shared else None

    def ffn(xt, gu, down):
        h = gu @ xt
        f = down.shape[1]
        return down @ (gelu(h[:f], variant) * h[f:])

    y = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if 0 <= e < rw[0].shape[0]:
                y[t] += gates[t, j].double() * ffn(x[t].double(), rw[0][e], rw[1][e])
        if shared:
            y[t] += ffn(x[t].double(), *sw)
    return y


def between(dtype):
    """What lies between the two products is off by half a step of its type at most (packed fp16: 2^-13 of the largest of its
    eight features, of sqrt(8) times their root mean square, which is less).  The down product spreads these errors as it
    spreads the values (Gaussian weights, hundreds of outputs: within a quarter); those of the fp32 sums are a hundredth of
    them."""
    assert 2.0 ** -13 * 8 ** 0.5 < torch.finfo(dtype).eps / 2
    return 1.25 * torch.finfo(dtype).eps / 2


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("size,gate", [(1000.0, 1.0), (1000.0, 1e-4), (1.0, 1e-6), (0.01, 1.0), (1e-4, 1e-3), (30.0, 1e4)])
def test_values_between_the_products_past_16_bits(size, gate, dtype, eight):
    """GELU(g) u and its product with the gate from 1e-12 to 1e6."""
    x, ids, gates, routed, shared = case(5, 3, 6, 272, 304, 272, dtype, eight, seed=81)
    x, gates = (x.float() * size).to(dtype), gates * gate
    for sh in (shared, None):
        want = formula(x, ids, gates, routed, sh, moe.MOE_GELU_ERF)
        y = call(x, ids, gates, routed, sh, out=F32)
        err = (y.double() - want).norm(dim=1) / want.norm(dim=1)
        assert torch.all(err <= between(dtype)), float(err.max())


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_small_features_beside_large_ones(dtype, eight):
    """Features of very different size, blocks of eight one after the other; outputs that weigh the small ones only."""
    t, d, f = 4, 256, 432
    x, ids, gates, routed, _ = case(t, 2, 4, d, f, 0, dtype, False, seed=82)
    gu, down = routed[0].clone(), routed[1].clone()
    small = torch.arange(f, device="cuda") // 8 % 2 == 1
    gu[:, :f][:, small] *= 2.0 ** -6       # g and u: GELU(g) u is about 2^-12 of the others
    gu[:, f:][:, small] *= 2.0 ** -6
    down[:, :64, ~small] = 0               # the first outputs see the small features only
    down[:, 64:128] = 0
    down[:, 64:128, 8:16] = 1              # the next ones eight of them
    if eight:
        one = lambda n, k: torch.ones(4, blocks(n), blocks(k), device="cuda")  # noqa: E731
        routed = ((gu.float() * 64).to(E4M3), down.to(E4M3), one(2 * f, d) / 64, one(d, f))
    else:
        routed = gu, down
    want = formula(x, ids, gates, routed, None, moe.MOE_GELU_ERF)
    y = call(x, ids, gates, routed, None, out=F32)
    for lo, hi in ((0, 64), (64, 65), (128, 256)):
        err, size = (y.double() - want)[:, lo:hi].norm(dim=1), want[:, lo:hi].norm(dim=1)
        if lo == 64:   # one sum of eight values, which may cancel: the bound is of their magnitudes
            size = size.clamp(min=float(want[:, 64].abs().mean()))
            err = err / 8 ** 0.5
        assert torch.all(err <= 2 * between(dtype) * size), float((err / size).max())


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_infinities_keep_their_signs(dtype, eight):
    """An infinite token value, and one that only the product makes infinite: infinities where the formula has them."""
    x, ids, gates, routed, _ = case(6, 2, 4, 256, 64, 0, dtype, eight, seed=83)
    x[2, 7] = float("inf")
    if not eight:
        routed[0][1, 64 + 9, 5] = float("-inf")
        routed[1][:, 100, 9] = 0     # no weight there: NaN
    y = call(x, ids, gates, routed, None, out=F32)
    want = formula(x, ids, gates, routed, None, moe.MOE_GELU_ERF)
    assert torch.equal(torch.isfinite(y), torch.isfinite(want))
    inf = torch.isinf(want)
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    assert torch.equal(y[inf], want[inf].float())


@pytest.mark.parametrize("t", [2, 8, 9, 32])
@pytest.mark.parametrize("dtype,eight", [(BF16, False), (F16, False), (BF16, True), (F16, True)])
def test_full_shape_layers_of_more_tokens(t, dtype, eight):
    args = case(t, 8, 128, 2816, 704, 2816, dtype, eight, seed=84)
    want = formula(*args, moe.MOE_GELU_ERF)
    err = (call(*args, out=F32).double() - want).norm(dim=1) / want.norm(dim=1)
    assert torch.all(err <= between(dtype)), float(err.max())
    half = torch.finfo(dtype).eps / 2
    y = call(*args)
    assert torch.all((y.double() - want).norm(dim=1) <= (half + between(dtype)) * want.norm(dim=1))


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("t", [1, 12])
def test_rows_of_plain_and_packed_values(t, eight):
    """fp16: blocks of eight features inside and outside of the type's range side by side, other ones for each token; the rows
    that need no packing are bit for bit what they are alone."""
    d, f, fs = 256, 432, 400
    x, ids, gates, routed, shared = case(t, 2, 4, d, f, fs, F16, eight, seed=85)
    x[1::3] *= 300.0
    x[2::3] *= 0.004
    want = formula(x, ids, gates, routed, shared, moe.MOE_GELU_TANH)
    y = call(x, ids, gates, routed, shared, out=F32, variant=moe.MOE_GELU_TANH)
    err = (y.double() - want).norm(dim=1) / want.norm(dim=1)
    assert torch.all(err <= between(F16)), float(err.max())
    alone = call(x[::3].contiguous(), ids[::3].contiguous(), gates[::3].contiguous(), routed, shared, out=F32, variant=moe.MOE_GELU_TANH)
    assert (y[::3] - alone).norm() <= 1e-5 * alone.norm()   # (chunks may end elsewhere)


@pytest.mark.parametrize("eight", [False, True])
def test_the_largest_and_smallest_fp32_values(eight):
    """GELU(g) u up to 1e33 and down to 1e-25 in one call, by way of the router's tokens and the weights' scales; features that
    are zero beside them."""
    d, f = 128, 80
    x, ids, gates, routed, _ = case(3, 1, 3, d, f, 0, F16, True, seed=86)
    ids[:, 0] = torch.arange(3)
    gates[:] = 1
    gu, down, su, sd = routed
    gu.view(torch.uint8)[:, 32:48] = 0
    su[0] *= 1e16
    su[1] *= 1e-12
    sd[0] *= 1e-16
    if not eight:   # fp16 weights hold no such scales: as large as they come
        wide_gu = wide_weights(gu, su)
        wide_gu[0] *= 1e4 / wide_gu[0].abs().max()
        wide_gu[1] *= 1e-4 / wide_gu[1].abs().max()
        routed = wide_gu.to(F16), wide_weights(down, sd.clamp(min=sd[1:].min())).to(F16)
    want = formula(x, ids, gates, routed, None, moe.MOE_GELU_ERF)
    y = call(x, ids, gates, routed, None, out=F32)
    err = (y.double() - want).norm(dim=1) / want.norm(dim=1)
    assert torch.all(err <= between(F16)), float(err.max())


@pytest.mark.parametrize("t,k,E,d,f,fs", [(1, 2, 8, 256, 704, 0), (3, 3, 12, 512, 304, 528), (20, 4, 6, 528, 400, 272)])
@pytest.mark.parametrize("size", [1.0, 300.0, 1e4, 0.003])
def test_bf16_layers_of_8_bit_experts_hold_fp16_between(t, k, E, d, f, fs, size):
    """e4m3 weights are exact in fp16 too: what lies between the products is off by an eighth of what bf16 would be, at any
    size."""
    x, ids, gates, routed, shared = case(t, k, E, d, f, fs, BF16, True, seed=87)
    x = (x.float() * size).to(BF16)
    want = formula(x, ids, gates, routed, shared, moe.MOE_GELU_TANH)
    y = call(x, ids, gates, routed, shared, variant=moe.MOE_GELU_TANH, out=F32)
    err = (y.double() - want).norm(dim=1) / want.norm(dim=1)
    assert torch.all(err <= between(F16)), float(err.max())
