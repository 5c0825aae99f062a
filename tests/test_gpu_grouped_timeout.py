"""Waits of the 16-bit operators that run out.  A hook stops the threads that
load operands after the first load of each CTA and shortens the limit of the
bounded waits: everything that waits for what was not loaded gives up, the
kernels return, and the host reads MOE_ETIMEOUT.  Nothing faults, nothing outside
the outputs is touched, and the next calls are right."""

import pytest
import torch

import bit_routed_expert_router_gb300 as moe

from test_gpu_grouped import BF16, F16, F32, SENTINEL, gen, ints, lora_case, lora_reference, offsets_of, ok, products

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def told():
    """Every stream that asks is told of a timeout: after these tests all that others may be given have been."""
    yield
    for s in [None] + [torch.cuda.Stream() for _ in range(64)]:
        moe.moe_grouped_sync(s)


class Stalled:
    """Calls inside load one stage a CTA and wait 0.1 ms."""

    def __enter__(self):
        moe.check(moe.moe_test_hook(None, moe.HOOK_SPIN_LIMIT, 200_000))
        moe.check(moe.moe_test_hook(None, moe.HOOK_STOP_LOADS, 1))

    def __exit__(self, *exc):
        moe.check(moe.moe_test_hook(None, moe.HOOK_SPIN_LIMIT, 0))
        moe.check(moe.moe_test_hook(None, moe.HOOK_STOP_LOADS, 0))


def guarded(dtype, *shape):
    """An output between two blocks of sentinels."""
    n = 1
    for s in shape:
        n *= s
    whole = torch.full((n + 2048,), SENTINEL, dtype=dtype, device="cuda")
    return whole, whole[1024:1024 + n].view(*shape)


def run_out(call, *outs):
    with Stalled():
        moe.check(call())
        assert moe.moe_grouped_sync() == moe.MOE_ETIMEOUT
    for whole in outs:
        assert (whole[:1024] == SENTINEL).all() and (whole[-1024:] == SENTINEL).all()
    assert moe.moe_grouped_sync() == moe.MOE_OK
    ok(call())


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("counts,out", [([9, 0, 14], BF16), ([300, 0, 1100], BF16), ([300, 0, 1100], F32)])
def test_products(counts, out, transpose):
    g, n, k = gen(1), 1000, 1032
    x, w = ints(g, BF16, sum(counts), n if transpose else k), ints(g, BF16, 3, n, k)
    whole, y = guarded(out, sum(counts), k if transpose else n)
    off = offsets_of(counts)
    run_out(lambda: moe.moe_grouped_mm(x, off, w, y, transpose=transpose), whole)
    assert torch.equal(y, products(x, counts, w.transpose(1, 2) if transpose else w).to(out))


@pytest.mark.parametrize("out", [F16, F32])
@pytest.mark.parametrize("E", [3, 100])   # 100: more tiles than pairs of CTAs
def test_weight_gradients(E, out):
    g, n, k = gen(2), 520, 264
    counts = [129 + e % 7 for e in range(E)]
    x, dy, off = ints(g, F16, sum(counts), k), ints(g, F16, sum(counts), n), offsets_of(counts)
    whole, dw = guarded(out, E, n, k)
    run_out(lambda: moe.moe_grouped_wgrad(dy, x, off, dw), whole)
    lo = 0
    for e, c in enumerate(counts):
        assert torch.equal(dw[e], (dy[lo:lo + c].double().T @ x[lo:lo + c].double()).to(out))
        lo += c


@pytest.mark.parametrize("counts", [[9, 0, 14], [300, 0, 1100]])
def test_gated_products(counts):
    g, f, k = gen(3), 304, 1032
    x, w, off = ints(g, BF16, sum(counts), k, top=1), ints(g, BF16, 3, 2 * f, k), offsets_of(counts)
    whole_a, a = guarded(BF16, sum(counts), f)
    whole_h, h = guarded(BF16, sum(counts), 2 * f)
    run_out(lambda: moe.moe_grouped_geglu(x, off, w, a, h), whole_a, whole_h)
    assert torch.equal(h, products(x, counts, w).to(BF16))


@pytest.mark.parametrize("t,rank", [(40, 16), (128, 64), (700, 72), (5000, 128)])
def test_adapters(t, rank):
    x, w, ids, a, b, scale = lora_case(4, t, 520, 1032, 5, rank, BF16, "any")
    whole, y = guarded(BF16, t, 520)
    ws = torch.empty(4 * t * rank, dtype=torch.uint8, device="cuda")
    run_out(lambda: moe.moe_lora_mm(x, w, ids, a, b, scale, y, ws), whole)
    assert torch.equal(y, lora_reference(x, w, ids, a, b, scale).to(BF16))


@pytest.mark.parametrize("captured", [False, True])
def test_one_callers_timeout_is_not_anothers(captured):
    """A launch that gave up on one stream: calls of another stream that follow do all of their work, and both streams
    are told of it."""
    g, n, k, E = gen(5), 520, 264, 100
    counts = [129 + e % 7 for e in range(E)]
    x, dy, off = ints(g, BF16, sum(counts), k), ints(g, BF16, sum(counts), n), offsets_of(counts)
    dws = [torch.full((E, n, k), SENTINEL, dtype=F32, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    want, lo = [], 0
    for c in counts:
        want.append(dy[lo:lo + c].double().T @ x[lo:lo + c].double())
        lo += c
    want = torch.stack(want).float()

    def call(i):
        moe.check(moe.moe_grouped_wgrad(dy, x, off, dws[i], stream=streams[i]))

    call(1)
    for s in streams:
        moe.moe_grouped_sync(s)   # whatever earlier launches left
    graph = torch.cuda.CUDAGraph()
    if captured:
        with torch.cuda.graph(graph, stream=streams[1]):
            call(1)
    for repeat in range(2):
        dws[1].fill_(SENTINEL)
        torch.cuda.synchronize()
        with Stalled():
            call(0)
        streams[0].synchronize()
        if captured:
            with torch.cuda.stream(streams[1]):
                graph.replay()
        else:
            call(1)
        assert moe.moe_grouped_sync(streams[1]) == moe.MOE_ETIMEOUT
        assert torch.equal(dws[1], want)
        assert moe.moe_grouped_sync(streams[0]) == moe.MOE_ETIMEOUT
        assert [moe.moe_grouped_sync(s) for s in streams] == [moe.MOE_OK] * 2
        call(0)
        moe.check(moe.moe_grouped_sync(streams[0]))
        assert torch.equal(dws[0], want)
    assert moe.moe_grouped_sync() == moe.MOE_ETIMEOUT   # and this one
    assert moe.moe_grouped_sync() == moe.MOE_OK


def test_no_sync_in_a_capture():
    """Refused, and the capture goes on."""
    g = gen(6)
    x, w, y = ints(g, BF16, 40, 64), ints(g, BF16, 1, 72, 64), torch.empty(40, 72, dtype=BF16, device="cuda")
    off = offsets_of([40])
    ok(moe.moe_grouped_mm(x, off, w, y))
    y.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.check(moe.moe_grouped_mm(x, off, w, y))
        assert moe.moe_grouped_sync() == moe.MOE_EINVAL
    graph.replay()
    ok(moe.MOE_OK)
    assert torch.equal(y, products(x, [40], w).to(BF16))
