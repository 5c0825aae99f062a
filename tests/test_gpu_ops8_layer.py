"""The norm, the 8-bit operators and the layer for a few tokens as they would be used together: the routed layer of a
block from its residual stream to the next block's, for many tokens (rows grouped by expert) and for a few, and the norm's
part of a training step."""

import os
import subprocess
import sys

import pytest
import torch

import bit_routed_expert_router_gb300 as moe
from ops8_reference import BF16, E4M3, F16, F32, blocks, gelu, gen, rand8, rand_scale, wide_weights
from test_gpu_grouped8 import rounding
from test_gpu_norm import ROUNDED, half_step, near16, near_grads, normed

pytestmark = pytest.mark.gpu

D, F, FS, E, K = 320, 176, 272, 12, 3
ERF = moe.MOE_GELU_ERF


def empty(*shape, dtype=F32):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def weights(seed, dtype=BF16):
    """The norms' weights, the router's, and the experts' and the shared expert's in e4m3 with their scales."""
    g = gen(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    eight = lambda lead, n, k: (rand8(g, *lead, n, k), 8 * rand_scale(g, *lead, blocks(n), blocks(k)) / k ** 0.5)  # noqa: E731
    ffn = lambda lead, f: [v for pair in zip(eight(lead, 2 * f, D), eight(lead, D, f)) for v in pair]  # noqa: E731
    norms = [(1 + 0.1 * r(D)).to(dtype) for _ in range(2)]
    return norms, (r(E, D) * D ** -0.5).to(F16), ffn((E,), F), ffn((), FS)


def route(x, router_w):
    t = x.shape[0]
    ids, gates = empty(t, K, dtype=torch.int32), empty(t, K)
    moe.check(moe.moe_route_noalloc(moe.make_config(D, F, FS, E, K), router_w, x, t, None, ids, gates))
    return ids, gates


def block_of_rows(h, delta, norms, router_w, routed, shared):
    """(r, x, ids, gates, y, next r, next x): rows grouped by expert, in 8 bits all the way."""
    t = h.shape[0]
    r, x, x8, s = torch.empty_like(h), torch.empty_like(h), empty(t, D, dtype=E4M3), empty(t, blocks(D))
    moe.check(moe.moe_rmsnorm(h, x, x8, s, delta=delta, h_out=r, weight=norms[0]))
    ids, gates = route(x, router_w)
    flat = ids.reshape(-1).long()
    order = flat.argsort(stable=True)
    where = torch.empty_like(order)
    where[order] = torch.arange(order.numel(), device="cuda")
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.zeros(E, dtype=torch.long, device="cuda").scatter_add_(0, flat, torch.ones_like(flat)).cumsum(0)

    def ffn(x8, s, offsets, gate_up, down, gate_up_scale, down_scale):
        m, f = x8.shape[0], down.shape[-1]
        a, sa, y = empty(m, f, dtype=E4M3), empty(m, blocks(f)), empty(m, D)
        moe.check(moe.moe_grouped_geglu8(x8, s, offsets, gate_up, gate_up_scale, a, sa))
        moe.check(moe.moe_grouped_mm8(a, sa, offsets, down, down_scale, y))
        return y

    rows = x8.view(torch.uint8)[order // K].view(E4M3)
    y = ffn(rows, s[order // K], offsets, *routed)[where].reshape(t, K, D) * gates[:, :, None]
    whole = torch.zeros(2, dtype=torch.int32, device="cuda")
    whole[1:] = t
    y = y.sum(1) + ffn(x8, s, whole, *(w[None] for w in shared))
    r2, x2 = torch.empty_like(h), torch.empty_like(h)
    moe.check(moe.moe_rmsnorm(r, x2, delta=y, h_out=r2, weight=norms[1]))
    return r, x, ids, gates, y, r2, x2


def block_of_tokens(h, delta, norms, router_w, routed, shared):
    """The same of up to 32 tokens: nothing to group."""
    t = h.shape[0]
    r, x, y, ws = torch.empty_like(h), torch.empty_like(h), empty(t, D), empty(2 * t * (K * F + FS), dtype=torch.uint8)
    moe.check(moe.moe_rmsnorm(h, x, delta=delta, h_out=r, weight=norms[0]))
    ids, gates = route(x, router_w)
    moe.check(moe.moe_token_layer(x, ids, gates, routed, y, ws, shared=shared))
    r2, x2 = torch.empty_like(h), torch.empty_like(h)
    moe.check(moe.moe_rmsnorm(r, x2, delta=y, h_out=r2, weight=norms[1]))
    return r, x, ids, gates, y, r2, x2


def step8(v, ev):
    """Error of values v, known up to ev, in 8 bits: half a step of e4m3, of the scale where the values are subnormal."""
    m, n = v.shape
    top = torch.nn.functional.pad(v.abs() + ev, (0, -n % 128)).view(m, -1, 128).amax(-1).clamp(min=2.0 ** -100)
    return ev + (v.abs() + ev) * (2.0 ** -4 + 2.0 ** -18) + top.repeat_interleave(128, 1)[:, :n] / 448 * (2.0 ** -10 + 2.0 ** -18)


def step16(v, ev, dtype=BF16):
    rel, least = half_step(dtype)
    return ev + (v.abs() + ev) * rel + least


def expect(h, delta, out, norms, routed, shared, step):
    """What a block gives from its formulas in 64 bits, with a bound carried along: `step` is the rounding of the products'
    inputs.  The stored residual rows are exact, the routing is the library's own."""
    r, x, ids, gates, y, r2, x2 = out
    assert torch.equal(r, (h.float() + delta.float()).to(h.dtype))
    v = normed(r, norms[0])
    near16(x, v, h.dtype)
    ex = step(v, 2 * ROUNDED * v.abs())
    want, bound = torch.zeros_like(v), torch.zeros_like(v)

    def product(v, ev, w):
        return v @ w.T, ev @ w.abs().T + rounding(w.shape[1]) * ((v.abs() + ev) @ w.abs().T)

    def add(t, gate, gate_up, down):
        hid, eh = product(v[t], ex[t], gate_up)
        f = down.shape[-1]
        g, u, eg, eu = hid[:, :f], hid[:, f:], eh[:, :f], eh[:, f:]
        a = gelu(g, ERF) * u
        ea = step(a, 1.13 * eg * (u.abs() + eu) + gelu(g, ERF).abs() * eu + 2.0 ** -18 * a.abs())
        o, eo = product(a, ea, down)
        want[t] += gate * o
        bound[t] += gate * (eo + (K + 4) * 2.0 ** -24 * (o.abs() + eo))

    wide = lambda w: (wide_weights(w[0], w[2]), wide_weights(w[1], w[3]))  # noqa: E731
    rw = wide(routed)
    for e in range(E):
        for j in range(K):
            t = (ids[:, j] == e).nonzero()[:, 0]
            if t.numel():
                add(t, gates[t, j].double()[:, None], rw[0][e], rw[1][e])
    add(torch.arange(h.shape[0], device="cuda"), 1.0, *wide(shared))
    assert torch.all((y.double() - want).abs() <= bound)
    # and as a whole: independent roundings do not add up as their bounds do (three of half a step, stretched threefold)
    half = 2.0 ** -4 if step is step8 else 2.0 ** -8
    assert (y.double() - want).norm() <= 9 * half * want.norm()
    assert torch.equal(r2, (r.float() + y).to(h.dtype))
    near16(x2, normed(r2, norms[1]), h.dtype)


@pytest.mark.parametrize("t", [1, 5, 32, 64])
@pytest.mark.parametrize("delta", [BF16, F32])
def test_a_block(t, delta):
    w = weights(t)
    g = gen(100 + t)
    h, dl = torch.randn(t, D, generator=g, device="cuda").to(BF16), torch.randn(t, D, generator=g, device="cuda").to(delta)
    expect(h, dl, block_of_rows(h, dl, *w), w[0], *w[2:], step8)
    if t <= 32:
        expect(h, dl, block_of_tokens(h, dl, *w), w[0], *w[2:], step16)
    moe.check(moe.moe_grouped_sync())


@pytest.mark.parametrize("block,t", [(block_of_rows, 48), (block_of_tokens, 4)])
def test_a_block_in_a_graph(block, t):
    """Captured as a whole and replayed on new tokens: bit for bit the eager calls."""
    w = weights(7)
    h, dl = torch.randn(t, D, device="cuda").to(BF16), torch.randn(t, D, device="cuda")
    block(h, dl, *w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = block(h, dl, *w)
    for seed in (1, 2):
        g = gen(seed)
        h.copy_(torch.randn(t, D, generator=g, device="cuda")), dl.copy_(torch.randn(t, D, generator=g, device="cuda"))
        graph.replay()
        got = [v.clone() for v in outs]
        want = block(h, dl, *w)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        expect(h, dl, want, w[0], *w[2:], step8 if block is block_of_rows else step16)
    moe.check(moe.moe_grouped_sync())


def test_two_graphs_of_one_workspace_in_turn():
    """A workspace holds nothing between calls: graphs that share it and run one after the other stay right."""
    w, t = weights(8), 3
    x = [torch.randn(t, D, generator=gen(s), device="cuda").to(BF16) for s in (1, 2)]
    ys, ws = [torch.empty_like(v) for v in x], empty(2 * t * (K * F + FS), dtype=torch.uint8)
    picked = [route(v, w[1]) for v in x]
    graphs = [torch.cuda.CUDAGraph() for _ in x]

    def call(i):
        moe.check(moe.moe_token_layer(x[i], *picked[i], w[2], ys[i], ws, shared=w[3]))

    call(0), call(1)
    want = [y.clone() for y in ys]
    torch.cuda.synchronize()
    for i, graph in enumerate(graphs):
        with torch.cuda.graph(graph):
            call(i)
    for _ in range(3):
        for y in ys:
            y.zero_()
        ws.fill_(0xFF)
        for graph in graphs:
            graph.replay()
        for y, v in zip(ys, want):
            assert torch.equal(y, v)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_the_norm_in_a_training_step(dtype):
    """Forward and backward through norm and gated products, in 16 bits: the norm's gradients of what the products hand
    back, and the residual's gradient past them."""
    g = gen(31)
    counts = [40, 0, 70]
    m, n = sum(counts), len(counts)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    h, dy, w = r(m, D).to(dtype), r(m, D).to(dtype), (1 + 0.1 * r(D)).to(dtype)
    gu, down = (r(n, 2 * F, D) * D ** -0.5).to(dtype), (r(n, D, F) * F ** -0.5).to(dtype)
    off = torch.tensor([0, 40, 40, 110], dtype=torch.int32, device="cuda")
    new = lambda *s: empty(*s, dtype=dtype)  # noqa: E731
    x, a, hid, da, dhid, dx, dh = new(m, D), new(m, F), new(m, 2 * F), new(m, F), new(m, 2 * F), new(m, D), new(m, D)
    dw, ws = empty(D), empty(4 * D * m, dtype=torch.uint8)

    def step():
        moe.check(moe.moe_rmsnorm(h, x, weight=w))
        moe.check(moe.moe_grouped_geglu(x, off, gu, a, hid))
        moe.check(moe.moe_grouped_mm(dy, off, down, da, transpose=True))
        moe.check(moe.moe_geglu_grad(hid, da, dhid))
        moe.check(moe.moe_grouped_mm(dhid, off, gu, dx, transpose=True))
        moe.check(moe.moe_rmsnorm_grad(h, dx, dh, dres=dy, weight=w, dweight=dw, workspace=ws))

    step()
    moe.check(moe.moe_grouped_sync())
    near_grads(h, dx, dy, w, dh, dw)
    # the whole step against the formula's gradients: x, hid, da, dhid, dx are rounded on the way (and dh at its end), each
    # by half a step of its norm at most, which a Gaussian matrix stretches by about 3 at most
    hl, wl = h.double().requires_grad_(), w.double().requires_grad_()
    xl = normed(hl, wl)
    out = []
    for e, (lo, hi) in enumerate(zip([0, 40, 40], [40, 40, 110])):
        v = xl[lo:hi] @ gu[e].double().T
        out.append((gelu(v[:, :F], ERF) * v[:, F:]) @ down[e].double().T)
    want = torch.autograd.grad(((torch.cat(out) + hl) * dy.double()).sum(), (hl, wl))
    for got, v in zip((dh, dw), want):
        assert (got.double() - v).norm() <= 3 * 6 * torch.finfo(dtype).eps / 2 * v.norm()
    # captured, on new rows
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    h.copy_(r(m, D))
    dh.zero_(), dw.zero_()
    graph.replay()
    got = dh.clone(), dw.clone()
    step()
    assert torch.equal(got[0], dh) and torch.equal(got[1], dw)


FIRST = """
import torch, bit_routed_expert_router_gb300 as moe
n = lambda *s, t=torch.float32: torch.ones(*s, device="cuda").to(t)
E4, BF = torch.float8_e4m3fn, torch.bfloat16
h, x8, s, a, sa, y = n(4, 128, t=BF), n(4, 128, t=E4), n(4, 1), n(4, 64, t=E4), n(4, 1), n(4, 128, t=BF)
gu, down, sgu, sd = n(2, 128, 128, t=E4), n(2, 128, 64, t=E4), n(2, 1, 1) / 128, n(2, 1, 1) / 64
off, ids, gates = torch.tensor([0, 1, 4], dtype=torch.int32, device="cuda"), n(4, 1, t=torch.int32), n(4, 1)
ws, dh, dw, w, wg = n(4 * 2 * 64, t=torch.uint8), n(4, 128, t=BF), n(128), n(128, t=BF), n(4 * 4 * 128, t=torch.uint8)
z = torch.empty_like(y)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    moe.check(moe.moe_rmsnorm(h, None, x8, s, weight=w))
    moe.check(moe.moe_grouped_geglu8(x8, s, off, gu, sgu, a, sa))
    moe.check(moe.moe_grouped_mm8(a, sa, off, down, sd, y))
    moe.check(moe.moe_token_layer(h, ids, gates, (gu, down, sgu, sd), z, ws))
    moe.check(moe.moe_rmsnorm_grad(h, y, dh, weight=w, dweight=dw, workspace=wg))
graph.replay()
moe.check(moe.moe_grouped_sync())
# every product is one or GELU(1) = 0.8413: rounded to e4m3 it is the block's largest, and exact but for the scale
for v in (y, z):
    assert torch.all((v.float() - 0.8413).abs() <= 0.01), v
assert torch.all(dw != 1)
"""


def test_the_first_calls_of_a_process_in_a_capture():
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                                       os.environ.get("PYTHONPATH", "")]))
    done = subprocess.run([sys.executable, "-c", FIRST], env=env, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


@pytest.mark.parametrize("t", [1, 20])
def test_the_layer_in_place_of_its_tokens(t):
    w = weights(9)
    x, ws = torch.randn(t, D, generator=gen(3), device="cuda").to(BF16), empty(2 * t * (K * F + FS), dtype=torch.uint8)
    ids, gates = route(x, w[1])
    y = torch.empty_like(x)
    moe.check(moe.moe_token_layer(x, ids, gates, w[2], y, ws, shared=w[3]))
    moe.check(moe.moe_token_layer(x, ids, gates, w[2], x, ws, shared=w[3]))
    assert torch.equal(x, y)
