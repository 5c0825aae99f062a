"""The 16-bit operators as they would be used together: one routed layer with
16-bit experts and a shared projection with adapters, forward, backward and
token by token."""

import pytest
import torch

import bit_routed_expert_router_gb300 as moe

from test_gpu_grouped import BF16, F16, F32, gelu, gen, lora_reference

pytestmark = pytest.mark.gpu

D, F, E, K = 256, 128, 8, 2


def rand(g, dtype, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def route(h, router_w):
    """The library's router: ids and gates of each token."""
    T = h.shape[0]
    cfg = moe.make_config(D, F, F, E, K)
    ids = torch.empty(T, K, dtype=torch.int32, device="cuda")
    gates = torch.empty(T, K, dtype=F32, device="cuda")
    moe.check(moe.moe_route_noalloc(cfg, router_w, h, T, None, ids, gates))
    return ids, gates


def group(ids):
    """(token, k) pairs by expert: their order, where each pair went, and the row ranges.  No host synchronisation."""
    flat = ids.reshape(-1).long()
    order = flat.argsort(stable=True)
    where = torch.empty_like(order)
    where[order] = torch.arange(order.numel(), device="cuda")
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.zeros(E, dtype=torch.long, device="cuda").scatter_add_(0, flat, torch.ones_like(flat)).cumsum(0)
    return order, where, offsets


def layer(h, router_w, w_gu, w_down, shared, adapters, workspace):
    """h [T, D] -> (y [T, D] fp32, what the backward pass needs)."""
    T = h.shape[0]
    ids, gates = route(h, router_w)
    order, where, offsets = group(ids)
    x = h[order // K]
    a = torch.empty(T * K, F, dtype=h.dtype, device="cuda")
    hid = torch.empty(T * K, 2 * F, dtype=h.dtype, device="cuda")
    out = torch.empty(T * K, D, dtype=F32, device="cuda")
    ys = torch.empty(T, D, dtype=h.dtype, device="cuda")
    moe.check(moe.moe_grouped_geglu(x, offsets, w_gu, a, hid))
    moe.check(moe.moe_grouped_mm(a, offsets, w_down, out))
    moe.check(moe.moe_lora_mm(h, shared, *adapters, ys, workspace))
    y = (out[where].reshape(T, K, D) * gates[:, :, None]).sum(1) + ys.float()
    return y, (ids, gates, order, where, offsets, x, a, hid)


def reference(h, ids, gates, w_gu, w_down, shared, adapters):
    """The same layer in 64 bits, from the definitions (differentiable)."""
    y = lora_reference(h, shared, adapters[0], *adapters[1:]) if not h.requires_grad else 0
    routed = []
    for t in range(h.shape[0]):
        s = 0
        for j in range(K):
            e = int(ids[t, j])
            gu = w_gu[e] @ h[t]
            s = s + gates[t, j].double() * (w_down[e] @ (gelu(gu[:F], moe.MOE_GELU_ERF) * gu[F:]))
        routed.append(s)
    return torch.stack(routed) + y


def case(T, dtype, seed=0):
    g = gen(seed)
    h = rand(g, dtype, T, D)
    router_w = rand(g, F16, E, D, scale=D ** -0.5)
    w_gu, w_down = rand(g, dtype, E, 2 * F, D, scale=D ** -0.5), rand(g, dtype, E, D, F, scale=F ** -0.5)
    shared = rand(g, dtype, D, D, scale=D ** -0.5)
    adapters = (torch.randint(-1, 3, (T,), generator=g, device="cuda", dtype=torch.int32),
                rand(g, dtype, 3, 16, D, scale=D ** -0.5), rand(g, dtype, 3, D, 16, scale=0.25),
                torch.rand(3, generator=g, device="cuda") + 0.5)
    return h, router_w, w_gu, w_down, shared, adapters, torch.empty(4 * T * 16, dtype=torch.uint8, device="cuda")


def near(got, want, roundings, dtype=BF16):
    """Every tensor on the way that is rounded to 16 bits moves by half a step of each value at most, so by that
    share of its norm; a Gaussian matrix stretches a direction by at most about 3 times the mean one."""
    rel = (got.double() - want).norm() / want.norm()
    assert rel <= 3 * roundings * torch.finfo(dtype).eps / 2, float(rel)


@pytest.mark.parametrize("T", [1, 3, 40])
def test_forward(T):
    args = case(T, BF16, T)
    y, (ids, gates, *_) = layer(*args)
    moe.check(moe.moe_grouped_sync())
    h, _, w_gu, w_down, shared, adapters, _ = args
    want = reference(h.double(), ids, gates, w_gu.double(), w_down.double(), shared.double(), adapters)
    near(y, want, 2)   # a, and the shared output


def test_tokens_one_by_one_are_the_batch():
    """A token's output does not depend on its batch beyond the order of fp32 sums: one token at a time and all at
    once round the same values, up to a step of bf16 where the sum lies next to a border."""
    h, router_w, w_gu, w_down, shared, adapters, ws = case(24, BF16, 5)
    y, _ = layer(h, router_w, w_gu, w_down, shared, adapters, ws)
    for t in range(24):
        one, _ = layer(h[t:t + 1], router_w, w_gu, w_down, shared, (adapters[0][t:t + 1], *adapters[1:]), ws)
        near(one, y[t:t + 1].double(), 2)
    moe.check(moe.moe_grouped_sync())


def backward(dy, gates, order, offsets, x, a, hid, w_gu, w_down, dtype):
    """Gradients of sum(dy * routed output): of the rows' inputs and of both weights (gates held)."""
    g = (dy[order // K] * gates.reshape(-1)[order][:, None]).to(dtype)
    m = g.shape[0]
    da, dhid = torch.empty(m, F, dtype=dtype, device="cuda"), torch.empty(m, 2 * F, dtype=dtype, device="cuda")
    dx = torch.empty(m, D, dtype=F32, device="cuda")
    dw_down, dw_gu = torch.empty(E, D, F, dtype=F32, device="cuda"), torch.empty(E, 2 * F, D, dtype=F32, device="cuda")
    moe.check(moe.moe_grouped_mm(g, offsets, w_down, da, transpose=True))
    moe.check(moe.moe_grouped_wgrad(g, a, offsets, dw_down))
    moe.check(moe.moe_geglu_grad(hid, da, dhid, offsets[E:]))
    moe.check(moe.moe_grouped_mm(dhid, offsets, w_gu, dx, transpose=True))
    moe.check(moe.moe_grouped_wgrad(dhid, x, offsets, dw_gu))
    return dx, dw_gu, dw_down


def test_training_step_against_the_formula_and_differences():
    T = 48
    h, router_w, w_gu, w_down, shared, adapters, ws = case(T, BF16, 8)
    dy = rand(gen(9), F32, T, D)
    y, (ids, gates, order, where, offsets, x, a, hid) = layer(h, router_w, w_gu, w_down, shared, adapters, ws)
    dx, dw_gu, dw_down = backward(dy, gates, order, offsets, x, a, hid, w_gu, w_down, BF16)
    moe.check(moe.moe_grouped_sync())
    dh = torch.zeros(T, D, dtype=torch.float64, device="cuda").index_add_(0, order // K, dx.double())

    leaves = [v.double().requires_grad_() for v in (h, w_gu, w_down)]
    loss = (reference(leaves[0], ids, gates, leaves[1], leaves[2], None, None) * dy.double()).sum()
    grads = torch.autograd.grad(loss, leaves)
    near(dh, grads[0], 4)       # g, da, hid, dhid
    near(dw_gu, grads[1], 4)
    near(dw_down, grads[2], 2)  # g, a

    # the formula itself, by central differences in 64 bits along a direction of all three
    step, dirs = 1e-5, [torch.randn(v.shape, generator=gen(10 + i), device="cuda", dtype=torch.float64)
                        for i, v in enumerate(leaves)]
    with torch.no_grad():
        at = []
        for s in (step, -step):
            moved = [v + s * d for v, d in zip(leaves, dirs)]
            moved[0].requires_grad_()   # routed part only, as above
            at.append((reference(moved[0], ids, gates, *moved[1:], None, None) * dy.double()).sum())
    slope = float(sum((g * d).sum() for g, d in zip(grads, dirs)))
    assert abs(float(at[0] - at[1]) / (2 * step) - slope) <= 1e-6 * sum(float((g * d).abs().sum()) for g, d in zip(grads, dirs))


def test_training_step_in_a_graph():
    """Forward and backward captured together and replayed on new tokens: bit for bit the eager calls."""
    T = 64
    h, router_w, w_gu, w_down, shared, adapters, ws = case(T, F16, 11)
    dy = rand(gen(12), F32, T, D)
    ids, gates = route(h, router_w)
    order, where, offsets = group(ids)
    x = h[order // K].contiguous()
    a, hid = torch.empty(T * K, F, dtype=F16, device="cuda"), torch.empty(T * K, 2 * F, dtype=F16, device="cuda")

    def step():
        moe.check(moe.moe_grouped_geglu(x, offsets, w_gu, a, hid))
        return backward(dy, gates, order, offsets, x, a, hid, w_gu, w_down, F16)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in (1, 2):
        h = rand(gen(seed), F16, T, D)
        i, gt = route(h, router_w)
        o, _, off = group(i)
        gates.copy_(gt), order.copy_(o), offsets.copy_(off), x.copy_(h[o // K])
        graph.replay()
        got = [v.clone() for v in outs]
        want = step()
        moe.check(moe.moe_grouped_sync())
        for u, v in zip(got, want):
            assert torch.equal(u, v)
