"""Waits of the 8-bit products and of the layer for a few tokens that run out: as for the 16-bit operators, the kernels
return, nothing outside the outputs is touched, the host reads MOE_ETIMEOUT, and the next calls are right."""

import time

import pytest
import torch

import bit_routed_expert_router_gb300 as moe
from ops8_reference import BF16, E4M3, F16, F32, blocks, products, wide_rows, wide_weights
from test_gpu_grouped8 import case, close, close_gated
from test_gpu_grouped_timeout import Stalled
from test_gpu_token_layer import case as layer_case, check as layer_check

pytestmark = pytest.mark.gpu

GUARD = 4096


@pytest.fixture(scope="module", autouse=True)
def told():
    """Every stream that asks is told of a timeout: after these tests all that others may be given have been."""
    yield
    for s in [None] + [torch.cuda.Stream() for _ in range(64)]:
        moe.moe_grouped_sync(s)


def guarded(dtype, *shape):
    """An output between two blocks of bytes that must stay."""
    size = torch.empty(*shape, dtype=dtype).nbytes
    whole = torch.full((size + 2 * GUARD,), 0x35, dtype=torch.uint8, device="cuda")
    return whole, whole[GUARD:GUARD + size].view(dtype).view(*shape)


def run_out(call, *outs):
    with Stalled():
        moe.check(call())
        assert moe.moe_grouped_sync() == moe.MOE_ETIMEOUT
    for whole in outs:
        assert torch.all(whole[:GUARD] == 0x35) and torch.all(whole[-GUARD:] == 0x35)
    assert moe.moe_grouped_sync() == moe.MOE_OK
    moe.check(call())
    moe.check(moe.moe_grouped_sync())


@pytest.mark.parametrize("counts,out,n", [([9, 0, 14], BF16, 1000), ([300, 0, 1100], F16, 1000), ([300, 0, 1100], F32, 1000),
                                          ([9, 0, 14], BF16, 6600), ([300, 0, 1100], F16, 2104), ([300, 0, 1100], F32, 2104)])
def test_products(counts, out, n):
    """Few tiles, and many."""
    k = 1040
    x, sx, off, w, sw = case(counts, n, k)
    sx *= 2.0 ** -8
    whole, y = guarded(out, sum(counts), n)
    run_out(lambda: moe.moe_grouped_mm8(x, sx, off, w, sw, y), whole)
    close(y, *products(wide_rows(x, sx), wide_weights(w, sw), off), k)


@pytest.mark.parametrize("counts", [[9, 0, 14], [300, 0, 1100]])
def test_gated_products(counts):
    f, k = 304, 1040
    x, sx, off, w, sw = case(counts, 2 * f, k)
    sx *= 2.0 ** -6 * k ** -0.5
    whole_a, a = guarded(E4M3, sum(counts), f)
    whole_s, sa = guarded(F32, sum(counts), blocks(f))
    run_out(lambda: moe.moe_grouped_geglu8(x, sx, off, w, sw, a, sa), whole_a, whole_s)
    close_gated(a, sa, x, sx, off, w, sw, f, moe.MOE_GELU_ERF)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("t", [1, 20])
def test_token_layer(t, eight):
    """2,080 values: three chunks or more of each unit of the first kernel."""
    x, ids, gates, routed, shared = layer_case(t, 4, 12, 2080, 304, 528, BF16, eight)
    whole_w, ws = guarded(torch.uint8, 2 * t * (4 * 304 + 528))
    whole_y, y = guarded(F32, t, 2080)
    run_out(lambda: moe.moe_token_layer(x, ids, gates, routed, y, ws, shared=shared), whole_w, whole_y)
    layer_check(y, x, ids, gates, routed, shared, moe.MOE_GELU_ERF)


def test_one_operators_timeout_is_told_once():
    """Counts of three kinds of kernels, one report each time."""
    x, sx, off, w, sw = case([200, 300], 512, 1024)
    y = torch.empty(500, 512, device="cuda")
    largs = layer_case(2, 2, 8, 2080, 304, 0)
    ws, ly = torch.empty(2 * 2 * 2 * 304, dtype=torch.uint8, device="cuda"), torch.empty_like(largs[0])
    with Stalled():
        moe.check(moe.moe_grouped_mm8(x, sx, off, w, sw, y))
        moe.check(moe.moe_token_layer(*largs[:4], ly, ws))
    assert moe.moe_grouped_sync() == moe.MOE_ETIMEOUT
    assert moe.moe_grouped_sync() == moe.MOE_OK


def test_asking_is_one_copy():
    """Whatever kinds of kernels report: about as long as one blocking copy of four bytes, not as several."""
    one = torch.ones(1, dtype=torch.int32, device="cuda")

    def shortest(f):
        best = 1.0
        for _ in range(20):
            start = time.perf_counter()
            for _ in range(50):
                f()
            best = min(best, (time.perf_counter() - start) / 50)
        return best

    shortest(moe.moe_grouped_sync)
    assert shortest(moe.moe_grouped_sync) <= 1.8 * shortest(one.cpu)


@pytest.mark.parametrize("captured", [False, True])
def test_a_launch_gives_up_once(captured):
    """The second kernel's 4,096 CTAs start in more than ten waves, of which the first gives up; each wave that did so by
    itself would hold its memories for 10 ms."""
    t, k, E, d, f = 32, 8, 64, 65536, 16
    x, ids, gates, routed, _ = layer_case(t, k, E, d, f, 0)
    whole_w, ws = guarded(torch.uint8, 2 * t * k * f)
    whole_y, y = guarded(BF16, t, d)

    def call():
        moe.check(moe.moe_token_layer(x, ids, gates, routed, y, ws))

    call()
    torch.cuda.synchronize()
    want = y.clone()
    moe.moe_grouped_sync()
    graph = torch.cuda.CUDAGraph()
    with Stalled():
        if captured:
            with torch.cuda.graph(graph):
                call()
        for _ in range(2):   # the replays of a graph's node are one launch to the kernels: the second does nothing
            start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            start.record()
            graph.replay() if captured else call()
            end.record()
            torch.cuda.synchronize()
            assert start.elapsed_time(end) < 60
            if not captured:
                assert moe.moe_grouped_sync() == moe.MOE_ETIMEOUT
    if captured:
        assert moe.moe_grouped_sync() == moe.MOE_ETIMEOUT
    assert moe.moe_grouped_sync() == moe.MOE_OK
    for whole in (whole_w, whole_y):
        assert torch.all(whole[:GUARD] == 0x35) and torch.all(whole[-GUARD:] == 0x35)
    call()
    moe.check(moe.moe_grouped_sync())
    assert torch.equal(y, want)
