"""The 8-bit grouped products against the formulas in 64 bits."""

import pytest
import torch

import bit_routed_expert_router_gb300 as moe
from ops8_reference import (BF16, E4M3, F16, F32, blocks, gelu, gen, offsets_of, products, rand8, rand_scale, wide_rows,
                            wide_weights)

pytestmark = pytest.mark.gpu

# (rows of each expert, n, k): one row, no rows, odd sizes, a block that ends early on either side, several tiles
CASES = [([1], 8, 16), ([0, 3, 0, 1], 136, 144), ([5, 0, 17, 2], 704, 2816), ([300, 0, 1, 257], 264, 400), ([33] * 8, 128, 128),
         ([0, 0, 0], 64, 64), ([513], 1000, 1104), ([2] * 100 + [0] * 28, 192, 256), ([700, 90], 2816, 704)]


def rounding(k):
    """Relative to the sum of the products' magnitudes.  A block of 128 products is summed by the tensor cores, whose additions
    truncate: at most 128 of 2^-23 of what is summed so far (the products are exact); the blocks in fp32, each with a rounding
    of its scale and its product; the fp32 sum of the blocks takes one each."""
    return (128 * 2 + 3 + blocks(k)) * 2.0 ** -24


def close(got, want, size, k):
    rel = torch.finfo(got.dtype).eps / 2 if got.dtype != F32 else 0
    least = torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps / 2
    err = (got.double() - want).abs()
    assert torch.all(err <= want.abs() * rel + (1 + rel) * rounding(k) * size + least), float((err / size.clamp(min=1e-30)).max())


def case(counts, n, k, seed=0, pad=0, first=0):
    g = gen(seed)
    m = sum(counts) + pad + first
    x, sx = rand8(g, m, k), rand_scale(g, m, blocks(k))
    w, sw = rand8(g, len(counts), n, k), rand_scale(g, len(counts), blocks(n), blocks(k))
    return x, sx, offsets_of(counts, first), w, sw


@pytest.mark.parametrize("counts,n,k", CASES)
@pytest.mark.parametrize("out", [BF16, F16, F32])
def test_products(counts, n, k, out):
    x, sx, off, w, sw = case(counts, n, k, seed=n + k)
    if out is F16:
        sx = sx * 2.0 ** -8   # inside its range
    y = torch.full((x.shape[0], n), 7.0, dtype=out, device="cuda")
    moe.check(moe.moe_grouped_mm8(x, sx, off, w, sw, y))
    moe.check(moe.moe_grouped_sync())
    want, size = products(wide_rows(x, sx), wide_weights(w, sw), off)
    close(y, want, size, k)


def close_gated(a, sa, x, sx, off, w, sw, f, variant):
    """The 8-bit output: half a step of e4m3 past the error of the fp32 value, which moves with g and u."""
    k = x.shape[1]
    h, size = products(wide_rows(x, sx), wide_weights(w, sw), off)
    g, u, eg, eu = h[:, :f], h[:, f:], rounding(k) * size[:, :f], rounding(k) * size[:, f:]
    v = gelu(g, variant) * u
    # |GELU'| is at most 1.13; GELU itself is good to 2^-19 of its value
    err = 1.13 * eg * (u.abs() + eu) + (gelu(g, variant).abs()) * eu + 2.0 ** -18 * v.abs()
    pad = lambda t: torch.nn.functional.pad(t, (0, -f % 128)).view(t.shape[0], blocks(f), 128)  # noqa: E731
    top, top_err = pad(v).abs().amax(-1).clamp(min=2.0 ** -100), pad(err).amax(-1)
    lo, hi = int(off[0]), int(off[-1])
    assert torch.all((sa.double() - top / 448).abs()[lo:hi] <= (top_err / 448 + 2.0 ** -22 * top / 448)[lo:hi])
    wide = sa.double().repeat_interleave(128, 1)[:, :f]
    got = a.double() * wide
    # a value past 448 scales (the largest's own error) is 448: its error is counted in err
    bound = v.abs() * (2.0 ** -4 + 2.0 ** -20) + wide * 2.0 ** -10 + 1.1 * err
    assert torch.all((got - v).abs()[lo:hi] <= bound[lo:hi])


@pytest.mark.parametrize("counts,f,k", [([1], 16, 16), ([0, 3, 0, 1], 144, 272), ([5, 0, 17, 2], 704, 2816), ([300, 0, 1, 257], 176, 400),
                                        ([33] * 8, 128, 128), ([513], 416, 1104), ([2] * 100 + [0] * 28, 96, 256), ([0, 0], 64, 64)])
@pytest.mark.parametrize("variant", [moe.MOE_GELU_ERF, moe.MOE_GELU_TANH])
def test_gated(counts, f, k, variant):
    x, sx, off, w, sw = case(counts, 2 * f, k, seed=f + k)
    sx = sx * 2.0 ** -6 * k ** -0.5
    m = x.shape[0]
    a, sa = torch.zeros(m, f, device="cuda").to(E4M3), torch.zeros(m, blocks(f), device="cuda")
    moe.check(moe.moe_grouped_geglu8(x, sx, off, w, sw, a, sa, gelu_variant=variant))
    moe.check(moe.moe_grouped_sync())
    close_gated(a, sa, x, sx, off, w, sw, f, variant)


@pytest.mark.parametrize("n", [264, 6600])   # few tiles, and many
def test_rows_of_no_group_and_strides(n):
    counts, k = [40, 0, 9], 272
    x, sx, off, w, sw = case(counts, n, k, pad=13, first=5)
    wide_x = torch.zeros(x.shape[0], 512, device="cuda").to(E4M3)
    wide_x[:, 32:32 + k] = x
    y = torch.full((x.shape[0], n + 136), 7.0, dtype=BF16, device="cuda")
    moe.check(moe.moe_grouped_mm8(wide_x[:, 32:32 + k], sx, off, w, sw, y[:, 8:8 + n]))
    want, size = products(wide_rows(x, sx), wide_weights(w, sw), off)
    close(y[5:54, 8:8 + n], want[5:54], size[5:54], k)
    y[5:54, 8:8 + n] = 7
    assert torch.all(y == 7)
    f = 128 + 4 * 16
    w, sw = rand8(gen(1), 3, 2 * f, k), rand_scale(gen(2), 3, 3, 3)
    a, sa = torch.ones(x.shape[0], 256, device="cuda").to(E4M3), torch.ones(x.shape[0], 2, device="cuda")
    moe.check(moe.moe_grouped_geglu8(wide_x[:, 32:32 + k], sx, off, w, sw, a[:, 16:16 + f], sa))
    close_gated(a[:, 16:16 + f], sa, x, sx, off, w, sw, f, moe.MOE_GELU_ERF)
    assert torch.all(sa[:5] == 1) and torch.all(sa[54:] == 1) and torch.all(a[:, :16].float() == 1)
    assert torch.all(a[:5].float() == 1) and torch.all(a[54:].float() == 1) and torch.all(a[:, 16 + f:].float() == 1)


@pytest.mark.parametrize("n", [160, 6504])   # few tiles, and many
def test_non_finite_rows_stay_rows(n):
    counts, k = [20, 30, 10], 384
    x, sx, off, w, sw = case(counts, n, k, pad=4)
    clean = torch.empty(x.shape[0], n, device="cuda")
    moe.check(moe.moe_grouped_mm8(x, sx, off, w, sw, clean))
    bad, bad_s = x.clone(), sx.clone()
    bad.view(torch.uint8)[7, 200] = 0x7F            # NaN
    bad_s[33, 1] = float("nan")
    bad.view(torch.uint8)[60:] = 0x7F               # rows behind the last group
    bad_s[60:] = float("nan")
    y = torch.empty(x.shape[0], n, device="cuda")
    moe.check(moe.moe_grouped_mm8(bad, bad_s, off, w, sw, y))
    assert torch.all(torch.isnan(y[[7, 33]]))
    keep = [r for r in range(60) if r not in (7, 33)]
    assert torch.equal(y[keep], clean[keep])
    # an expert's NaN weight: its feature, in its rows
    bad_w = w.clone()
    bad_w.view(torch.uint8)[1, 130, 3] = 0xFF
    moe.check(moe.moe_grouped_mm8(x, sx, off, bad_w, sw, y))
    assert torch.all(torch.isnan(y[20:50, 130]))
    y[20:50, 130] = clean[20:50, 130]
    assert torch.equal(y[:60], clean[:60])


def test_long_reductions_of_one_sign():
    """65,536 products of one sign: what truncating sums would lose shows."""
    g = gen(9)
    x, w = rand8(g, 40, 65536).float().abs().to(E4M3), rand8(g, 1, 72, 65536).float().abs().to(E4M3)
    sx, sw = torch.ones(40, 512, device="cuda"), torch.ones(1, 1, 512, device="cuda")
    y, off = torch.empty(40, 72, device="cuda"), offsets_of([40])
    moe.check(moe.moe_grouped_mm8(x, sx, off, w, sw, y))
    want = x.double() @ w[0].double().T
    # 512 blocks summed one after the other in fp32, half a step each, and what a block's 128 truncated additions lose
    assert torch.all((y.double() - want).abs() <= (512 + 3 + 256) * 2.0 ** -24 * want)


@pytest.mark.parametrize("n", [64, 6600])   # few tiles, and many
def test_offsets_out_of_order_stay_inside(n):
    """Undefined outputs, but only inside the tensors: what surrounds them is as it was."""
    x, sx, _, w, sw = case([16, 16, 16], n, 64)
    buf = torch.full((48 + 200, n), 3.0, device="cuda")
    for off in ([0, 40, 10, 48], [-5, 16, 100, 1 << 30], [48, 30, 20, 0], [10, 10, 10, 10]):
        buf.fill_(3.0)
        moe.check(moe.moe_grouped_mm8(x, sx, torch.tensor(off, dtype=torch.int32, device="cuda"), w, sw, buf[100:148]))
        moe.check(moe.moe_grouped_sync())
        assert torch.all(buf[:100] == 3) and torch.all(buf[148:] == 3)


def test_in_a_graph_and_on_another_stream():
    counts, f, k = [70, 0, 31, 155], 256, 512
    x, sx, off, w, sw = case(counts, 2 * f, k)
    sx *= 2.0 ** -9
    m = x.shape[0]
    w2, sw2 = rand8(gen(4), 4, 264, f), rand_scale(gen(5), 4, 3, 2)
    a, sa, y = torch.zeros(m, f, device="cuda").to(E4M3), torch.zeros(m, 2, device="cuda"), torch.zeros(m, 264, device="cuda")

    def both():
        moe.check(moe.moe_grouped_geglu8(x, sx, off, w, sw, a, sa))
        moe.check(moe.moe_grouped_mm8(a, sa, off, w2, sw2, y))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for n, counts in enumerate(([10, 200, 0, 46], [0, 0, 256, 0])):
        off.copy_(offsets_of(counts))
        x.copy_(rand8(gen(50 + n), m, k))
        a.zero_(), y.zero_()
        graph.replay()
        got = a.clone(), sa.clone(), y.clone()
        both()
        moe.check(moe.moe_grouped_sync())
        assert torch.equal(got[0].view(torch.uint8), a.view(torch.uint8)) and torch.equal(got[1], sa) and torch.equal(got[2], y)
        want, size = products(wide_rows(a, sa), wide_weights(w2, sw2), off)
        close(y, want, size, f)


def test_two_streams_at_once():
    args = [case([60, 80], 512, 1024, seed=s) for s in (1, 2)]
    ys = [torch.empty(140, 512, device="cuda") for _ in args]
    streams = [torch.cuda.Stream() for _ in args]
    torch.cuda.synchronize()
    for _ in range(5):
        for (x, sx, off, w, sw), y, s in zip(args, ys, streams):
            moe.check(moe.moe_grouped_mm8(x, sx, off, w, sw, y, stream=s))
    for s in streams:
        moe.check(moe.moe_grouped_sync(s))
    for (x, sx, off, w, sw), y in zip(args, ys):
        want, size = products(wide_rows(x, sx), wide_weights(w, sw), off)
        close(y, want, size, 1024)


def test_the_most_experts():
    counts = [i % 3 for i in range(1024)]
    x, sx, off, w, sw = case(counts, 72, 80)
    y = torch.empty(x.shape[0], 72, device="cuda")
    moe.check(moe.moe_grouped_mm8(x, sx, off, w, sw, y))
    want, size = products(wide_rows(x, sx), wide_weights(w, sw), off)
    close(y, want, size, 80)


def test_no_group_has_rows():
    x, sx, off, w, sw = case([0, 0, 0], 128, 144, pad=9, first=4)
    y = torch.full((13, 128), 7.0, device="cuda")
    a, sa = torch.ones(13, 64, device="cuda").to(E4M3), torch.ones(13, 1, device="cuda")
    moe.check(moe.moe_grouped_mm8(x, sx, off, w, sw, y))
    moe.check(moe.moe_grouped_geglu8(x, sx, off, w, sw, a, sa))
    moe.check(moe.moe_grouped_sync())
    assert torch.all(y == 7) and torch.all(a.float() == 1) and torch.all(sa == 1)


@pytest.mark.parametrize("out", [BF16, F32])
def test_many_experts_with_whole_and_ragged_tiles(out):
    """1024 experts leave one output buffer a warp; whole blocks of 32 rows and what is left of them in turn."""
    counts = [0] * 1024
    for i, c in enumerate((32, 33, 64, 127, 128, 129, 160, 1, 256, 31)):
        counts[100 * i + 7] = c
    x, sx, off, w, sw = case(counts, 136, 272, pad=3)
    y = torch.full((x.shape[0], 144), 7.0, dtype=out, device="cuda")
    moe.check(moe.moe_grouped_mm8(x, sx, off, w, sw, y[:, :136]))
    want, size = products(wide_rows(x, sx), wide_weights(w, sw), off)
    close(y[:-3, :136], want[:-3], size[:-3], 272)
    y[:-3, :136] = 7
    assert torch.all(y == 7)


def test_the_same_rows_alone_and_in_a_batch():
    """A row's sums do not depend on the rows and groups around it: bit for bit."""
    counts, n, k = [130, 0, 257, 3], 264, 400
    x, sx, off, w, sw = case(counts, n, k)
    y, one = torch.empty(390, n, device="cuda"), torch.empty(1, n, device="cuda")
    moe.check(moe.moe_grouped_mm8(x, sx, off, w, sw, y))
    for r, e in ((0, 0), (129, 0), (130, 2), (386, 2), (388, 3)):
        moe.check(moe.moe_grouped_mm8(x[r:r + 1], sx[r:r + 1], offsets_of([1]), w[e:e + 1], sw[e:e + 1], one))
        assert torch.equal(one[0], y[r])


@pytest.mark.parametrize("out", [BF16, F16, F32])
@pytest.mark.parametrize("counts,n,k", [([1], 20008, 144), ([300, 0, 1, 257], 2840, 400), ([513, 40], 5000, 272), ([33] * 8, 5384, 128)])
def test_products_of_many_tiles(counts, n, k, out):
    """More tiles than multiprocessors, of 256 features, the last ones ragged."""
    x, sx, off, w, sw = case(counts, n, k, seed=n + k)
    sx = sx * 2.0 ** -8
    y = torch.full((x.shape[0], n), 7.0, dtype=out, device="cuda")
    moe.check(moe.moe_grouped_mm8(x, sx, off, w, sw, y))
    close(y, *products(wide_rows(x, sx), wide_weights(w, sw), off), k)


def test_few_and_many_tiles_give_the_same_sums():
    """An expert's first features alone, and among many: bit for bit."""
    x, sx, off, w, sw = case([100, 60], 6528, 656)
    y, few = torch.empty(160, 6528, device="cuda"), torch.empty(160, 256, device="cuda")
    moe.check(moe.moe_grouped_mm8(x, sx, off, w, sw, y))
    moe.check(moe.moe_grouped_mm8(x, sx, off, w.view(torch.uint8)[:, :256].contiguous().view(E4M3), sw[:, :2].contiguous(), few))
    assert torch.equal(few, y[:, :256])


@pytest.mark.parametrize("variant", [moe.MOE_GELU_ERF, moe.MOE_GELU_TANH])
@pytest.mark.parametrize("f", [176, 304, 128])
@pytest.mark.parametrize("k", [384, 272])
def test_non_finite_values_stay_in_their_blocks_when_gated(f, k, variant):
    """A NaN or an infinity in a row, in a gate or up row of an expert, in a scale on either side of where the up rows pass
    from one block of scales to the next: the blocks that the formula says, everything else bit for bit as without."""
    counts = [20, 33, 150]
    x, sx, off, w, sw = case(counts, 2 * f, k, seed=f + k)
    sx = sx * 2.0 ** -6 * k ** -0.5
    m, expert = x.shape[0], torch.arange(3, device="cuda").repeat_interleave(torch.tensor(counts, device="cuda"))
    pad = lambda t: torch.nn.functional.pad(t, (0, -f % 128)).view(m, blocks(f), 128)  # noqa: E731

    def run(x, sx, w, sw):
        a, sa = torch.zeros(m, f, device="cuda").to(E4M3), torch.zeros(m, blocks(f), device="cuda")
        moe.check(moe.moe_grouped_geglu8(x, sx, off, w, sw, a, sa, gelu_variant=variant))
        return a, sa

    def spoil(which, at, value):
        v = [x.clone(), sx.clone(), w.clone(), sw.clone()]
        (v[which].view(torch.uint8) if v[which].dtype == E4M3 else v[which])[at] = value
        return v

    clean_a, clean_s = run(x, sx, w, sw)
    nan, inf = float("nan"), float("inf")
    up = blocks(2 * f) - 1
    cases = [(0, (25, 130), 0x7F), (1, (40, 1), nan), (2, (1, 40, 3), 0xFF), (2, (1, f + 100, 200), 0x7F),
             (3, (2, f // 128, 1), nan), (3, (2, up, 0), nan), (3, (2, up, 2), inf), (3, (0, up - 1, 1), inf), (1, (60, 2), inf)]
    for which, at, value in cases:
        bad = spoil(which, at, value)
        a, sa = run(*bad)
        h = torch.zeros(m, 2 * f, dtype=torch.float64, device="cuda")
        for b in range(blocks(k)):   # the factors of a block's sum, not of its products: infinity times 0 is NaN
            part = slice(128 * b, min(128 * b + 128, k))
            sums = torch.einsum("rk,rnk->rn", bad[0][:, part].double(), bad[2].double()[expert][:, :, part])
            h += bad[1][:, b, None].double() * bad[3].double()[expert][:, :, b].repeat_interleave(128, 1)[:, :2 * f] * sums
        v = gelu(h[:, :f], variant) * h[:, f:]
        has_nan, has_inf = pad(torch.isnan(v)).any(-1), pad(torch.isinf(v)).any(-1)
        assert has_nan.any() or has_inf.any()
        hit = has_nan | has_inf
        wide = lambda t: t.repeat_interleave(128, 1)[:, :f]  # noqa: E731
        assert torch.all(torch.isnan(sa[has_nan])) and torch.all(torch.isnan(a.float()[wide(has_nan)]))
        only = has_inf & ~has_nan
        assert torch.all(torch.isinf(sa[only]))
        spot = wide(only) & torch.isinf(v)
        assert torch.all(torch.isnan(a.float()[spot])) and torch.all(a.float()[wide(only) & ~spot] == 0)
        assert torch.equal(sa[~hit], clean_s[~hit])
        assert torch.equal(a.view(torch.uint8)[wide(~hit)], clean_a.view(torch.uint8)[wide(~hit)])
