"""The 16-bit operators' argument checks, on a machine without a GPU: every
refusal comes before any CUDA work, so made-up addresses are enough."""

import pytest
import torch

import bit_routed_expert_router_gb300 as moe
from bit_routed_expert_router_gb300 import build as moe_build

P = 1 << 20   # an aligned address that nothing reads


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.lib()


MM = dict(dtype=moe.MOE_BF16, transpose=0, x=P, ldx=64, m=4, offsets=P, n_experts=2, w=P, n=32, k=64, y=P, ldy=32,
          out_dtype=moe.MOE_F32, stream=None)
WGRAD = dict(dtype=moe.MOE_F16, dy=P, lddy=32, x=P, ldx=64, m=4, offsets=P, n_experts=2, n=32, k=64, dw=P,
             out_dtype=moe.MOE_F16, stream=None)
GEGLU = dict(dtype=moe.MOE_BF16, gelu_variant=0, x=P, ldx=64, m=4, offsets=P, n_experts=2, w=P, f=32, k=64, a=P, lda=32,
             h=P, ldh=64, stream=None)
GRAD = dict(dtype=moe.MOE_BF16, gelu_variant=1, h=P, ldh=64, da=P, ldda=32, m=4, f=32, n_rows=None, dh=P, lddh=64,
            stream=None)
LORA = dict(dtype=moe.MOE_BF16, x=P, ldx=64, t=4, w=P, n=32, k=64, ids=P, a=P, b=P, scale=P, n_adapters=2, rank=16,
            y=P, ldy=32, workspace=P, workspace_bytes=4 * 4 * 16, stream=None)

SIDES = [dict(n=0), dict(n=12), dict(k=-8), dict(k=65544)]
GROUPS = [dict(dtype=moe.MOE_F32), dict(dtype=7), dict(m=-1), dict(m=(1 << 24) + 1), dict(offsets=None),
          dict(offsets=P + 2), dict(n_experts=0), dict(n_experts=1025)]
X = [dict(x=None), dict(x=P + 8), dict(ldx=56), dict(ldx=68)]
BAD = (
    [("moe_grouped_mm", MM, b) for b in SIDES + GROUPS + X + [
        dict(w=None), dict(w=P + 2), dict(y=None), dict(y=P + 4), dict(ldy=24), dict(ldy=36), dict(transpose=2),
        dict(out_dtype=moe.MOE_F16), dict(out_dtype=3), dict(transpose=1)]] +
    [("moe_grouped_wgrad", WGRAD, b) for b in SIDES + GROUPS + X + [
        dict(dy=None), dict(dy=P + 8), dict(lddy=16), dict(lddy=33), dict(dw=None), dict(dw=P + 8),
        dict(out_dtype=moe.MOE_BF16)]] +
    [("moe_grouped_geglu", GEGLU, b) for b in SIDES[2:] + GROUPS + X + [
        dict(f=0), dict(f=24), dict(f=32784), dict(gelu_variant=2), dict(w=None), dict(a=None), dict(lda=24),
        dict(lda=33), dict(h=P + 8), dict(ldh=56), dict(ldh=65)]] +
    [("moe_geglu_grad", GRAD, b) for b in [
        dict(dtype=moe.MOE_F32), dict(gelu_variant=-1), dict(m=-1), dict(m=(1 << 24) + 1), dict(f=4), dict(f=0),
        dict(f=32776), dict(n_rows=P + 1), dict(h=None), dict(ldh=56), dict(da=None), dict(ldda=24), dict(dh=None),
        dict(lddh=60), dict(dh=P + 8)]] +
    [("moe_lora_mm", LORA, b) for b in SIDES + X + [
        dict(dtype=moe.MOE_F32), dict(t=-1), dict(t=(1 << 24) + 1), dict(w=None), dict(a=None), dict(b=None),
        dict(a=P + 8), dict(b=P + 8), dict(ids=None), dict(ids=P + 1), dict(scale=None), dict(n_adapters=0),
        dict(rank=0), dict(rank=12), dict(rank=136), dict(y=None), dict(ldy=24), dict(workspace=None),
        dict(workspace=P + 8), dict(workspace_bytes=255)]])


@pytest.mark.parametrize("name,good,bad", BAD, ids=[f"{n}-{b}" for n, _, b in BAD])
def test_bad_arguments_are_refused_before_cuda(lib, name, good, bad):
    assert getattr(lib, name)(*{**good, **bad}.values()) == moe.MOE_EINVAL


@pytest.mark.parametrize("name,good,none", [("moe_grouped_mm", MM, "m"), ("moe_grouped_geglu", GEGLU, "m"),
                                            ("moe_geglu_grad", GRAD, "m"), ("moe_lora_mm", LORA, "t")])
def test_no_rows_is_no_work(lib, name, good, none):
    assert getattr(lib, name)(*{**good, none: 0}.values()) == moe.MOE_OK


def _tensors():
    bf = torch.bfloat16
    return dict(x=torch.zeros(4, 64, dtype=bf), w=torch.zeros(2, 32, 64, dtype=bf), y=torch.zeros(4, 32, dtype=bf),
                offsets=torch.zeros(3, dtype=torch.int32))


def test_the_binding_refuses_tensors_that_do_not_fit(lib):
    t = _tensors()
    x, w, y, off = t["x"], t["w"], t["y"], t["offsets"]
    bad = [(x[:, :56], off, w, y), (x, off[:2], w, y), (x, off.long(), w, y), (x, off, w.half(), y),
           (x, off, w, y[:3]), (x, off, w, y[:, :24]), (x.t().contiguous().t(), off, w, y),
           (x, off, w.transpose(1, 2), y), (x, off, w[0], y), (x, off, w, y.double()), (x, off, w, y.half())]
    for a in bad:
        assert moe.moe_grouped_mm(*a) == moe.MOE_EINVAL
    assert moe.moe_grouped_mm(x, off, w, y) == moe.MOE_EINVAL   # host tensors
    assert moe.moe_grouped_wgrad(y, x, off, torch.zeros(2, 64, 32, dtype=x.dtype)) == moe.MOE_EINVAL
    assert moe.moe_grouped_wgrad(y[:3], x, off, torch.zeros_like(w)) == moe.MOE_EINVAL
    a, h = torch.zeros(4, 16, dtype=x.dtype), torch.zeros(4, 32, dtype=x.dtype)
    assert moe.moe_grouped_geglu(x, off, w, y) == moe.MOE_EINVAL
    assert moe.moe_grouped_geglu(x, off, w, a, h[:, :16]) == moe.MOE_EINVAL
    assert moe.moe_geglu_grad(h, a, a) == moe.MOE_EINVAL
    assert moe.moe_geglu_grad(h, a, h.clone(), n_rows=torch.zeros(1)) == moe.MOE_EINVAL
    A, B = torch.zeros(3, 8, 64, dtype=x.dtype), torch.zeros(3, 32, 8, dtype=x.dtype)
    s, ids, ws = torch.ones(3), torch.zeros(4, dtype=torch.int32), torch.zeros(4 * 4 * 8, dtype=torch.uint8)
    for a in [(x, w[0], ids.long(), A, B, s, y, ws), (x, w[0], ids, A, B[:2], s, y, ws),
              (x, w[0], ids[:3], A, B, s, y, ws), (x, w[0], ids, A, B, s.double(), y, ws),
              (x, w[0], ids, A.transpose(1, 2), B, s, y, ws), (x, w[0], ids, A, B, s, y, ws)]:
        assert moe.moe_lora_mm(*a) == moe.MOE_EINVAL
