"""Argument checks of the norm, the 8-bit operators and the layer for a few tokens, on a machine without a GPU: every
refusal comes before any CUDA work, so made-up addresses are enough."""

import pytest
import torch

import bit_routed_expert_router_gb300 as moe
from bit_routed_expert_router_gb300 import build as moe_build

P = 1 << 20   # an aligned address that nothing reads
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.lib()


NORM = dict(dtype=moe.MOE_BF16, h=P, ldh=264, delta=P, ldd=264, delta_dtype=moe.MOE_F32, weight=P, eps=1e-6, m=4, d=264,
            h_out=P, ldo=264, y=P, ldy=264, y8=P, ldy8=264, scale=P, stream=None)
NGRAD = dict(dtype=moe.MOE_F16, h=P, ldh=264, dy=P, lddy=264, dres=P, lddres=264, weight=P, eps=1e-6, m=4, d=264, dh=P,
             lddh=264, dweight=P, workspace=P, workspace_bytes=4 * 4 * 264, stream=None)

MM8 = dict(x=P, ldx=64, sx=P, m=4, offsets=P, n_experts=2, w=P, sw=P, n=32, k=64, y=P, ldy=32, out_dtype=moe.MOE_F32, stream=None)
GEGLU8 = dict(gelu_variant=0, x=P, ldx=64, sx=P, m=4, offsets=P, n_experts=2, w=P, sw=P, f=32, k=64, a=P, lda=32, sa=P, stream=None)
FFN8, FFN16 = moe.MoeFfnWeights(P, P, P, P), moe.MoeFfnWeights(P, P, None, None)   # one with scales, one without
LAYER = dict(dtype=moe.MOE_BF16, gelu_variant=1, x=P, ldx=64, t=4, ids=P, gates=P, top_k=2, n_experts=8, routed=FFN16, shared=FFN16,
             d=64, f=32, f_shared=48, y=P, ldy=64, out_dtype=moe.MOE_F32, workspace=P, workspace_bytes=2 * 4 * (2 * 32 + 48), stream=None)

COMMON = [dict(dtype=moe.MOE_F32), dict(dtype=5), dict(h=None), dict(h=P + 8), dict(ldh=256), dict(ldh=268), dict(weight=P + 2),
          dict(eps=-1e-6), dict(eps=INF), dict(eps=NAN), dict(m=-1), dict(m=(1 << 24) + 1), dict(d=0), dict(d=260), dict(d=16392)]
BAD = (
    [("moe_rmsnorm", NORM, b) for b in COMMON + [
        dict(delta=P + 4), dict(ldd=260), dict(ldd=266), dict(delta_dtype=moe.MOE_F16), dict(delta_dtype=4), dict(delta=None),
        dict(h_out=None), dict(h_out=P + 2), dict(ldo=256), dict(y=None, y8=None, scale=None), dict(y=P + 8), dict(ldy=260),
        dict(y8=P + 4), dict(ldy8=256), dict(ldy8=268), dict(scale=None), dict(scale=P + 2), dict(y8=None)]] +
    [("moe_rmsnorm_grad", NGRAD, b) for b in COMMON + [
        dict(dy=None), dict(dy=P + 4), dict(lddy=256), dict(dres=P + 8), dict(lddres=260), dict(dh=None), dict(lddh=256),
        dict(dweight=P + 4), dict(weight=None), dict(workspace=None), dict(workspace=P + 8),
        dict(workspace_bytes=4 * 4 * 264 - 1)]] +
    [(name, good, b) for name, good in (("moe_grouped_mm8", MM8), ("moe_grouped_geglu8", GEGLU8)) for b in [
        dict(x=None), dict(x=P + 8), dict(ldx=48), dict(ldx=72), dict(sx=None), dict(sx=P + 2), dict(m=-1),
        dict(m=(1 << 24) + 1), dict(offsets=None), dict(offsets=P + 1), dict(n_experts=0), dict(n_experts=1025), dict(w=None),
        dict(w=P + 8), dict(sw=None), dict(sw=P + 1), dict(k=0), dict(k=72), dict(k=65552)]] +
    [("moe_grouped_mm8", MM8, b) for b in [
        dict(n=0), dict(n=20), dict(n=65544), dict(y=None), dict(y=P + 8), dict(ldy=24), dict(ldy=36), dict(out_dtype=3)]] +
    [("moe_grouped_geglu8", GEGLU8, b) for b in [
        dict(gelu_variant=2), dict(f=0), dict(f=24), dict(f=32784), dict(a=None), dict(a=P + 8), dict(lda=16), dict(lda=40),
        dict(sa=None), dict(sa=P + 2)]] +
    [("moe_token_layer", LAYER, b) for b in [
        dict(dtype=moe.MOE_F32), dict(gelu_variant=-1), dict(x=None), dict(x=P + 2), dict(ldx=56), dict(ldx=68), dict(t=-1),
        dict(t=33), dict(ids=None), dict(ids=P + 2), dict(gates=None), dict(gates=P + 1), dict(top_k=0), dict(top_k=33),
        dict(n_experts=0), dict(n_experts=1025), dict(routed=None), dict(routed=FFN8), dict(shared=FFN8), dict(shared=None),
        dict(routed=moe.MoeFfnWeights(P, None, None, None)), dict(routed=moe.MoeFfnWeights(P + 8, P, None, None)),
        dict(shared=moe.MoeFfnWeights(P, P, None, P)), dict(d=0), dict(d=72), dict(d=65552), dict(f=8), dict(f=40),
        dict(f=32784), dict(f_shared=0), dict(f_shared=40), dict(y=None), dict(y=P + 8), dict(ldy=56), dict(ldy=65),
        dict(out_dtype=moe.MOE_F16), dict(workspace=None), dict(workspace=P + 8),
        dict(workspace_bytes=2 * 4 * (2 * 32 + 48) - 1)]])


@pytest.mark.parametrize("name,good,bad", BAD, ids=[f"{n}-{b}" for n, _, b in BAD])
def test_bad_arguments_are_refused_before_cuda(lib, name, good, bad):
    assert getattr(lib, name)(*{**good, **bad}.values()) == moe.MOE_EINVAL


@pytest.mark.parametrize("name,good,none", [("moe_rmsnorm", NORM, dict(m=0)),
                                            ("moe_rmsnorm_grad", NGRAD, dict(m=0, dweight=None)),
                                            ("moe_grouped_mm8", MM8, dict(m=0)), ("moe_grouped_geglu8", GEGLU8, dict(m=0)),
                                            ("moe_token_layer", LAYER, dict(t=0))])
def test_no_rows_is_no_work(lib, name, good, none):
    assert getattr(lib, name)(*{**good, **none}.values()) == moe.MOE_OK


def test_the_binding_refuses_norms_that_do_not_fit(lib):
    bf, e4 = torch.bfloat16, torch.float8_e4m3fn
    h, y, y8, s, w = (torch.zeros(4, 264, dtype=bf), torch.zeros(4, 264, dtype=bf), torch.zeros(4, 264, dtype=e4),
                      torch.zeros(4, 3), torch.zeros(264, dtype=bf))
    bad = [((h, y[:3]), {}), ((h, y.half()), {}), ((h, y, y8), {}), ((h, y, None, s), {}), ((h, y, y8, s[:, :2]), {}),
           ((h, y, y8.view(torch.uint8), s), {}), ((h, y), dict(delta=y)), ((h, y), dict(h_out=y)),
           ((h, y), dict(delta=y.double(), h_out=y)), ((h, y), dict(weight=w.float())), ((h, y), dict(weight=w[:8])),
           ((h[0], y[0]), {}), ((h.t(), y.t()), {}), ((h, y), {})]   # the last: host tensors
    for a, k in bad:
        assert moe.moe_rmsnorm(*a, **k) == moe.MOE_EINVAL
    dw, ws = torch.zeros(264), torch.zeros(4 * 4 * 264, dtype=torch.uint8)
    bad = [((h, y[:3], y), {}), ((h, y, y.half()), {}), ((h, y, y), dict(dres=y.float())), ((h, y, y), dict(weight=w[:8])),
           ((h, y, y), dict(weight=w, dweight=dw.double(), workspace=ws)), ((h, y, y), dict(weight=w, dweight=dw, workspace=ws[::2])),
           ((h, y, y), dict(weight=w, dweight=dw, workspace=ws))]
    for a, k in bad:
        assert moe.moe_rmsnorm_grad(*a, **k) == moe.MOE_EINVAL


def test_the_binding_refuses_products_that_do_not_fit(lib):
    e4 = torch.float8_e4m3fn
    x, sx, off, w, sw = (torch.zeros(4, 144, dtype=e4), torch.zeros(4, 2), torch.zeros(3, dtype=torch.int32),
                         torch.zeros(2, 264, 144, dtype=e4), torch.zeros(2, 3, 2))
    y, a, sa = torch.zeros(4, 264), torch.zeros(4, 132, dtype=e4), torch.zeros(4, 2)
    good = (x, sx, off, w, sw)
    swaps = [(0, x[:, :128]), (0, x.view(torch.uint8)), (0, x.t().contiguous().t()), (1, sx[:, :1]), (1, sx.double()),
             (1, sx.t().contiguous().t()), (2, off[:2]), (2, off.long()), (3, w[0]), (3, w.view(torch.uint8)), (3, w.transpose(1, 2)),
             (4, sw[:, :2]), (4, sw.half()), (None, None)]   # the last: host tensors
    for at, v in swaps:
        args = list(good)
        if at is not None:
            args[at] = v
        assert moe.moe_grouped_mm8(*args, y) == moe.MOE_EINVAL
        assert moe.moe_grouped_geglu8(*args, a, sa) == moe.MOE_EINVAL
    for bad in (y[:3], y[:, :256], y.double(), y.t().contiguous().t()):
        assert moe.moe_grouped_mm8(*good, bad) == moe.MOE_EINVAL
    for b in ((a[:, :128], sa), (a, sa[:, :1]), (a.float(), sa), (a, sa.double())):
        assert moe.moe_grouped_geglu8(*good, *b) == moe.MOE_EINVAL


def test_the_binding_refuses_layers_that_do_not_fit(lib):
    bf, e4 = torch.bfloat16, torch.float8_e4m3fn
    z = lambda *s, t=bf: torch.zeros(*s, dtype=t)  # noqa: E731
    x, ids, gates, y, ws = z(3, 64), z(3, 2, t=torch.int32), z(3, 2, t=torch.float32), z(3, 64), z(2000, t=torch.uint8)
    routed, shared = (z(4, 64, 64), z(4, 64, 32)), (z(96, 64), z(64, 48))
    routed8 = (z(4, 64, 64, t=e4), z(4, 64, 32, t=e4), z(4, 1, 1, t=torch.float32), z(4, 1, 1, t=torch.float32))
    good = dict(x=x, ids=ids, gates=gates, routed=routed, y=y, workspace=ws, shared=shared)
    bad = [dict(x=x[0]), dict(x=x.half()), dict(ids=ids.long()), dict(ids=ids[:2]), dict(gates=gates[:, :1]), dict(gates=gates.half()),
           dict(routed=(z(4, 60, 64), z(4, 64, 32))), dict(routed=(z(4, 64, 64), z(3, 64, 32))), dict(routed=(z(64, 64), z(64, 32))),
           dict(routed=routed8[:2]), dict(routed=(*routed8[:3], None)), dict(routed=(*routed, None, routed8[3])),
           dict(routed=(*routed8[:3], z(4, 1, 2, t=torch.float32))), dict(shared=(z(96, 64).t(), z(64, 48))), dict(shared=(z(96, 60), z(60, 48))),
           dict(y=y[:2]), dict(y=y.t().contiguous().t()), dict(workspace=ws[::2]), {}]   # the last: host tensors
    for b in bad:
        assert moe.moe_token_layer(**{**good, **b}) == moe.MOE_EINVAL
