"""Python binding of libmoe (routed mixture-of-experts FFN on one GB300).

A thin ctypes layer over the C ABI declared in ``include/moe.h``: every
function below has the C entry point's name and only marshals arguments
(torch tensors -> device pointers, streams -> ``cudaStream_t``).  All
arithmetic runs in the library's CUDA kernels; there is no CPU fallback, and
loading fails loudly if ``libmoe.so`` has not been built.
"""

from __future__ import annotations

import ctypes as C
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libmoe.so")

MOE_OK, MOE_EINVAL, MOE_ENOMEM, MOE_ECUDA, MOE_ESTATE, MOE_ETIMEOUT, MOE_EDOMAIN, MOE_EIO = range(8)
MOE_RESIDENT_HBM, MOE_HOST_POOL, MOE_FILE_POOL = 0, 1, 2
MOE_FILE_DIRECT = 1
MOE_STAGING_HOST, MOE_STAGING_DEVICE, MOE_STAGING_FUSED = 0, 1, 2
MOE_CACHE_LRU, MOE_CACHE_LFU = 0, 1
MOE_GELU_ERF, MOE_GELU_TANH = 0, 1
MOE_BF16, MOE_F16, MOE_F32 = 0, 1, 2
HOOK_FAIL_NEXT_COPY, HOOK_WAIT_LIMIT_US, HOOK_PDL, HOOK_PERSISTENT, HOOK_TIMELINE, HOOK_FREE_BYTES = 1, 2, 3, 4, 5, 6
HOOK_PREFILL_TC = 7
HOOK_CLUSTER = 9
HOOK_SPIN_LIMIT = 10      # bounded waits of the persistent decode kernels (no context: of the operators): cycles
HOOK_AT_REST = 11         # MOE_OK when the persistent kernels' launch words are back at rest
HOOK_WAIT_DIAG = 12       # the clustered kernel's first wait that ran out (site << 16 | CTA) into a host uint32
HOOK_SMALL_BATCH = 13     # small-batch grouped GEMVs (calls of at most 32 tokens) on / off
HOOK_STOP_LOADS = 15      # no context: loads after which the operators' loading threads stop (<= 0: never)
HOOK_TOKEN_LOOP = 14      # decode steps of 2 to 4 tokens: one clustered-kernel launch per token on / off


class MoeConfig(C.Structure):
    _fields_ = [("d", C.c_int32), ("f", C.c_int32), ("f_shared", C.c_int32), ("n_experts", C.c_int32),
                ("top_k", C.c_int32), ("group", C.c_int32), ("n_layers", C.c_int32),
                ("gelu_variant", C.c_int32), ("prenorm", C.c_int32), ("max_tokens", C.c_int32),
                ("norm_eps", C.c_float)]


class MoeExpertWeights(C.Structure):
    _fields_ = [("gate_q", C.c_void_p), ("gate_sb", C.c_void_p), ("up_q", C.c_void_p),
                ("up_sb", C.c_void_p), ("down_q", C.c_void_p), ("down_sb", C.c_void_p)]


class MoeFfnWeights(C.Structure):
    _fields_ = [("gate_up", C.c_void_p), ("down", C.c_void_p), ("gate_up_scale", C.c_void_p), ("down_scale", C.c_void_p)]


class MoeTraceRec(C.Structure):
    _fields_ = [("token", C.c_int32), ("layer", C.c_int32), ("k_pos", C.c_int32), ("expert", C.c_int32),
                ("hit", C.c_int32), ("slot", C.c_int32), ("evicted", C.c_int32)]


class MoeStats(C.Structure):
    _fields_ = [(n, C.c_int64) for n in ("steps", "hits", "misses", "staged_bytes", "n_slots",
                                          "expert_bytes", "shared_bytes", "device_bytes",
                                          "host_pool_bytes", "file_read_bytes", "host_tier_hits",
                                          "host_tier_bytes")]


class MoeKernelTime(C.Structure):
    _fields_ = [("launches", C.c_int64), ("total_ms", C.c_double)]


N_KERNEL_KINDS = 8
KERNEL_KINDS = {0: "router_topk_plan", 1: "gateup_gelu_gemv", 2: "down_combine_gemv", 3: "decode_persistent",
                4: "prefill_route_group", 5: "prefill_tcgen05_gemm", 6: "prefill_combine", 7: "small_batch_gemv"}


class MoeError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{status_name(status)}: {message}")
        self.status = status


_lib = None

# name -> (restype, argtypes)
_SIGS = {
    "moe_create": (C.c_int, [C.POINTER(MoeConfig), C.c_int, C.POINTER(C.c_void_p)]),
    "moe_init_layer": (C.c_int, [C.c_void_p, C.c_int, C.c_void_p, C.POINTER(MoeExpertWeights),
                                 C.POINTER(MoeExpertWeights), C.c_int]),
    "moe_set_slots": (C.c_int, [C.c_void_p, C.c_int]),
    "moe_set_cache_policy": (C.c_int, [C.c_void_p, C.c_int]),
    "moe_set_expert_file": (C.c_int, [C.c_void_p, C.c_char_p, C.c_int, C.c_uint64, C.c_int]),
    "moe_set_file_cache": (C.c_int, [C.c_void_p, C.c_int]),
    "moe_set_staging": (C.c_int, [C.c_void_p, C.c_int]),
    "moe_pread_parallel": (C.c_int, [C.c_char_p, C.c_uint64, C.c_uint64, C.c_void_p, C.c_int, C.c_uint64]),
    "moe_host_read_rate": (C.c_int, [C.c_void_p, C.c_uint64, C.c_int, C.c_void_p, C.POINTER(C.c_double)]),
    "moe_decode_step": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_void_p,
                                  C.c_void_p, C.POINTER(MoeTraceRec), C.c_int, C.POINTER(C.c_int),
                                  C.c_void_p]),
    "moe_prefill": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_void_p,
                              C.c_void_p, C.c_void_p]),
    "moe_set_debug": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int]),
    "moe_set_debug_logits": (C.c_int, [C.c_void_p, C.c_void_p]),
    "moe_sync": (C.c_int, [C.c_void_p, C.c_void_p]),
    "moe_get_stats": (C.c_int, [C.c_void_p, C.POINTER(MoeStats)]),
    "moe_get_cache_state": (C.c_int, [C.c_void_p, C.c_int, C.c_void_p, C.c_void_p]),
    "moe_reset_cache": (C.c_int, [C.c_void_p]),
    "moe_expert_bytes": (C.c_int64, [C.POINTER(MoeConfig)]),
    "moe_shared_bytes": (C.c_int64, [C.POINTER(MoeConfig)]),
    "moe_test_hook": (C.c_int, [C.c_void_p, C.c_int, C.c_int64]),
    "moe_route_noalloc": (C.c_int, [C.POINTER(MoeConfig), C.c_void_p, C.c_void_p, C.c_int, C.c_void_p,
                                    C.c_void_p, C.c_void_p, C.c_void_p]),
    "moe_grouped_mm": (C.c_int, [C.c_int, C.c_int, C.c_void_p, C.c_int64, C.c_int, C.c_void_p, C.c_int, C.c_void_p,
                                 C.c_int, C.c_int, C.c_void_p, C.c_int64, C.c_int, C.c_void_p]),
    "moe_grouped_wgrad": (C.c_int, [C.c_int, C.c_void_p, C.c_int64, C.c_void_p, C.c_int64, C.c_int, C.c_void_p,
                                    C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_int, C.c_void_p]),
    "moe_grouped_geglu": (C.c_int, [C.c_int, C.c_int, C.c_void_p, C.c_int64, C.c_int, C.c_void_p, C.c_int, C.c_void_p,
                                    C.c_int, C.c_int, C.c_void_p, C.c_int64, C.c_void_p, C.c_int64, C.c_void_p]),
    "moe_geglu_grad": (C.c_int, [C.c_int, C.c_int, C.c_void_p, C.c_int64, C.c_void_p, C.c_int64, C.c_int, C.c_int,
                                 C.c_void_p, C.c_void_p, C.c_int64, C.c_void_p]),
    "moe_lora_mm": (C.c_int, [C.c_int, C.c_void_p, C.c_int64, C.c_int, C.c_void_p, C.c_int, C.c_int, C.c_void_p,
                              C.c_void_p, C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_void_p, C.c_int64, C.c_void_p,
                              C.c_uint64, C.c_void_p]),
    "moe_rmsnorm": (C.c_int, [C.c_int, C.c_void_p, C.c_int64, C.c_void_p, C.c_int64, C.c_int, C.c_void_p, C.c_float,
                              C.c_int, C.c_int, C.c_void_p, C.c_int64, C.c_void_p, C.c_int64, C.c_void_p, C.c_int64,
                              C.c_void_p, C.c_void_p]),
    "moe_rmsnorm_grad": (C.c_int, [C.c_int, C.c_void_p, C.c_int64, C.c_void_p, C.c_int64, C.c_void_p, C.c_int64,
                                   C.c_void_p, C.c_float, C.c_int, C.c_int, C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p,
                                   C.c_uint64, C.c_void_p]),
    "moe_grouped_mm8": (C.c_int, [C.c_void_p, C.c_int64, C.c_void_p, C.c_int, C.c_void_p, C.c_int, C.c_void_p, C.c_void_p,
                                  C.c_int, C.c_int, C.c_void_p, C.c_int64, C.c_int, C.c_void_p]),
    "moe_grouped_geglu8": (C.c_int, [C.c_int, C.c_void_p, C.c_int64, C.c_void_p, C.c_int, C.c_void_p, C.c_int, C.c_void_p,
                                     C.c_void_p, C.c_int, C.c_int, C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p]),
    "moe_token_layer": (C.c_int, [C.c_int, C.c_int, C.c_void_p, C.c_int64, C.c_int, C.c_void_p, C.c_void_p, C.c_int, C.c_int,
                                  C.POINTER(MoeFfnWeights), C.POINTER(MoeFfnWeights), C.c_int, C.c_int, C.c_int, C.c_void_p,
                                  C.c_int64, C.c_int, C.c_void_p, C.c_uint64, C.c_void_p]),
    "moe_grouped_sync": (C.c_int, [C.c_void_p]),
    "moe_profile": (C.c_int, [C.c_void_p, C.c_int]),
    "moe_get_profile": (C.c_int, [C.c_void_p, C.POINTER(MoeKernelTime), C.c_int]),
    "moe_status_string": (C.c_char_p, [C.c_int]),
    "moe_last_error": (C.c_char_p, [C.c_void_p]),
    "moe_destroy": (None, [C.c_void_p]),
}


def lib():
    """Load libmoe.so (built by ``build.build()``); raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libmoe.so not built ({LIB_PATH}); run __graft_entry__.build()")
        L = C.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def moe_status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


def status_name(status: int) -> str:
    try:
        return moe_status_string(status)
    except Exception:  # pragma: no cover
        return f"status {status}"


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def check(status: int, ctx=None) -> None:
    """Raise MoeError for a non-OK status, with the context's last message."""
    if status != MOE_OK:
        msg = moe_last_error(ctx) if ctx is not None else ""
        raise MoeError(status, msg)


# ---------------------------------------------------------------- C entry points

def make_config(d, f, f_shared, n_experts, top_k, n_layers=1, group=64, gelu_variant=MOE_GELU_ERF,
                prenorm=0, max_tokens=32, norm_eps=1e-6) -> MoeConfig:
    return MoeConfig(d, f, f_shared, n_experts, top_k, group, n_layers, gelu_variant, prenorm, max_tokens,
                     norm_eps)


def moe_create(cfg: MoeConfig, device: int = 0):
    """Returns (status, ctx handle or None)."""
    h = C.c_void_p()
    st = lib().moe_create(C.byref(cfg), device, C.byref(h))
    return st, (h.value if st == MOE_OK else None)


def expert_weights(d: dict, index=None) -> MoeExpertWeights:
    """Marshal one expert's canonical tensors (``index`` selects from stacked [E, ...] tensors)."""
    def p(name):
        t = d[name] if index is None else d[name][index]
        return _ptr(t)
    return MoeExpertWeights(p("gate_q"), p("gate_sb"), p("up_q"), p("up_sb"), p("down_q"), p("down_sb"))


def moe_init_layer(ctx, layer: int, router_w, experts: dict, shared: dict, residency=MOE_RESIDENT_HBM) -> int:
    """router_w fp16 [E, d]; experts: stacked canonical tensors [E, ...]; shared: canonical tensors."""
    E = router_w.shape[0]
    for t in list(experts.values()) + list(shared.values()) + [router_w]:
        assert t.is_contiguous(), "weights must be contiguous"
    arr = (MoeExpertWeights * E)(*[expert_weights(experts, e) for e in range(E)])
    sw = expert_weights(shared)
    return lib().moe_init_layer(ctx, layer, _ptr(router_w), arr, C.byref(sw), residency)


def moe_set_slots(ctx, n_slots: int) -> int:
    return lib().moe_set_slots(ctx, n_slots)


def moe_set_cache_policy(ctx, policy: int) -> int:
    return lib().moe_set_cache_policy(ctx, policy)


def moe_set_expert_file(ctx, path, n_threads: int = 8, chunk_bytes: int = 0, flags: int = 0) -> int:
    return lib().moe_set_expert_file(ctx, None if path is None else os.fsencode(path), n_threads, chunk_bytes,
                                     flags)


def moe_set_staging(ctx, mode: int) -> int:
    return lib().moe_set_staging(ctx, mode)


def moe_set_file_cache(ctx, n_host: int) -> int:
    return lib().moe_set_file_cache(ctx, n_host)


def moe_host_read_rate(host_buf, nbytes: int, reps: int = 5, stream=None):
    """(status, GB/s): plain-load read rate of pinned host memory from every SM."""
    out = C.c_double(0.0)
    st = lib().moe_host_read_rate(_ptr(host_buf), nbytes, reps, _stream(stream), C.byref(out))
    return st, out.value


def moe_pread_parallel(path, offset: int, nbytes: int, dst, n_threads: int = 8, chunk_bytes: int = 0) -> int:
    """Read [offset, offset + nbytes) of `path` into `dst` (a writable buffer:
    a numpy array or a pinned host tensor)."""
    return lib().moe_pread_parallel(None if path is None else os.fsencode(path), offset, nbytes, _ptr(dst),
                                    n_threads, chunk_bytes)


def moe_decode_step(ctx, h_in, B: int, layer_begin: int, layer_end: int, logit_bias=None, h_out=None,
                    y_last=None, trace=None, stream=None):
    """Returns (status, n_trace).  ``trace`` is a ctypes array of MoeTraceRec or None."""
    n = C.c_int(0)
    cap = len(trace) if trace is not None else 0
    st = lib().moe_decode_step(ctx, _ptr(h_in), B, layer_begin, layer_end, _ptr(logit_bias), _ptr(h_out),
                               _ptr(y_last), trace, cap, C.byref(n), _stream(stream))
    return st, n.value


def moe_prefill(ctx, h, T: int, layer_begin: int, layer_end: int, logit_bias=None, h_out=None, y_last=None,
                stream=None) -> int:
    return lib().moe_prefill(ctx, _ptr(h), T, layer_begin, layer_end, _ptr(logit_bias), _ptr(h_out),
                             _ptr(y_last), _stream(stream))


def moe_set_debug(ctx, x_layers=None, ids=None, gates=None, y_layers=None, max_layers: int = 0) -> int:
    return lib().moe_set_debug(ctx, _ptr(x_layers), _ptr(ids), _ptr(gates), _ptr(y_layers), max_layers)


def moe_set_debug_logits(ctx, logits=None) -> int:
    return lib().moe_set_debug_logits(ctx, _ptr(logits))


def moe_sync(ctx, stream=None) -> int:
    return lib().moe_sync(ctx, _stream(stream))


def moe_get_stats(ctx):
    s = MoeStats()
    st = lib().moe_get_stats(ctx, C.byref(s))
    return st, s


def moe_get_cache_state(ctx, layer: int, n_slots: int):
    import numpy as np
    eos = np.zeros(n_slots, dtype=np.int32)
    lu = np.zeros(n_slots, dtype=np.int64)
    st = lib().moe_get_cache_state(ctx, layer, eos.ctypes.data, lu.ctypes.data)
    return st, eos, lu


def moe_reset_cache(ctx) -> int:
    return lib().moe_reset_cache(ctx)


def moe_expert_bytes(cfg: MoeConfig) -> int:
    return lib().moe_expert_bytes(C.byref(cfg))


def moe_shared_bytes(cfg: MoeConfig) -> int:
    return lib().moe_shared_bytes(C.byref(cfg))


def moe_test_hook(ctx, hook: int, value: int) -> int:
    return lib().moe_test_hook(ctx, hook, value)


ROUTE_NOALLOC_MAX_B = 64


def moe_route_noalloc(cfg: MoeConfig, router_w, h, B: int, logit_bias, ids, gates, stream=None) -> int:
    """Routing without any device allocation (see include/moe.h); every buffer is the caller's."""
    return lib().moe_route_noalloc(C.byref(cfg), _ptr(router_w), _ptr(h), B, _ptr(logit_bias), _ptr(ids),
                                   _ptr(gates), _stream(stream))


# ---------------------------------------------------------------- 16-bit operators (no context)
#
# Sizes, strides and types come from the tensors.  Tensors that do not fit together (shape, type, device, a last
# dimension that is not contiguous) return MOE_EINVAL like the library's own checks.  The call runs on the tensors'
# device, on `stream` or that device's current stream.

_DTYPE = _INT32 = _FLOAT32 = _E4M3 = _current_device = _raw_stream = _fn = None   # from torch and the library, on the first call


def _from_torch() -> None:
    global _DTYPE, _INT32, _FLOAT32, _E4M3, _current_device, _raw_stream, _fn
    import torch
    _fn = lib()
    _DTYPE = {torch.bfloat16: MOE_BF16, torch.float16: MOE_F16, torch.float32: MOE_F32}
    _INT32, _FLOAT32 = torch.int32, torch.float32
    # (without the check that CUDA has been initialised: whoever has tensors there has done so)
    _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    _E4M3 = torch.float8_e4m3fn
    # the stream's handle without the 3 us of a torch.cuda.Stream object: these calls start kernels of 10 us
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda device: torch.cuda.current_stream(device).cuda_stream)


# The checks are written out in each function and ask a tensor as little as they can: a call of a few microseconds on the
# GPU waits for the host (with helper functions for the checks they took 1 us longer).


def _whole(t, shape, dtype, dev: int) -> bool:
    """A contiguous tensor of this shape and type on device `dev`."""
    return t.shape == shape and t.dtype is dtype and t.is_contiguous() and t.get_device() == dev


def _call(fn, dev: int, stream, *args) -> int:
    if dev < 0:
        return MOE_EINVAL
    if stream is None:
        stream = _raw_stream(dev)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if dev == _current_device():
        return fn(*args, stream)
    import torch
    with torch.cuda.device(dev):
        return fn(*args, stream)


def moe_grouped_mm(x, offsets, w, y, transpose: bool = False, stream=None) -> int:
    """y[r] = w[e] x[r] (or w[e]^T x[r]) for the rows of each expert; w [E, n, k], offsets int32 [E + 1]."""
    if _DTYPE is None:
        _from_torch()
    sw, sx = w.shape, x.shape
    if len(sw) != 3 or len(sx) != 2:
        return MOE_EINVAL
    (E, n, k), m, dev, dt = sw, sx[0], w.get_device(), w.dtype
    into, out = (n, k) if transpose else (k, n)
    if sx[1] != into or y.shape != (m, out):
        return MOE_EINVAL
    # a row's values are contiguous; the row stride of a single row says nothing
    tx, ty = x.stride(), y.stride()
    if not (tx[1] == 1 and ty[1] == 1 and x.dtype is dt and w.is_contiguous() and x.get_device() == dev and
            y.get_device() == dev and _whole(offsets, (E + 1,), _INT32, dev)):
        return MOE_EINVAL
    return _call(_fn.moe_grouped_mm, dev, stream, _DTYPE.get(dt, -1), 1 if transpose else 0, x.data_ptr(),
                 tx[0] if m > 1 else into, m, offsets.data_ptr(), E, w.data_ptr(), n, k, y.data_ptr(),
                 ty[0] if m > 1 else out, _DTYPE.get(y.dtype, -1))


def moe_grouped_wgrad(dy, x, offsets, dw, stream=None) -> int:
    """dw[e] = sum over the rows of each expert of dy[r] x[r]^T; dw [E, n, k], all of it written."""
    if _DTYPE is None:
        _from_torch()
    sw, sx = dw.shape, x.shape
    if len(sw) != 3 or len(sx) != 2:
        return MOE_EINVAL
    (E, n, k), m, dev, dt = sw, sx[0], dw.get_device(), x.dtype
    if sx[1] != k or dy.shape != (m, n):
        return MOE_EINVAL
    tx, ty = x.stride(), dy.stride()
    if not (tx[1] == 1 and ty[1] == 1 and dy.dtype is dt and dw.is_contiguous() and x.get_device() == dev and
            dy.get_device() == dev and _whole(offsets, (E + 1,), _INT32, dev)):
        return MOE_EINVAL
    return _call(_fn.moe_grouped_wgrad, dev, stream, _DTYPE.get(dt, -1), dy.data_ptr(), ty[0] if m > 1 else n,
                 x.data_ptr(), tx[0] if m > 1 else k, m, offsets.data_ptr(), E, n, k, dw.data_ptr(),
                 _DTYPE.get(dw.dtype, -1))


def moe_grouped_geglu(x, offsets, w, a, h=None, gelu_variant: int = MOE_GELU_ERF, stream=None) -> int:
    """a[r] = GELU(g) u, [g, u] = w[e] x[r]; w [E, 2 f, k]; h [m, 2 f] (optional) receives [g, u]."""
    if _DTYPE is None:
        _from_torch()
    sw, sx = w.shape, x.shape
    if len(sw) != 3 or len(sx) != 2 or sw[1] % 2:
        return MOE_EINVAL
    (E, n, k), m, dev, dt = sw, sx[0], w.get_device(), w.dtype
    f = n // 2
    if sx[1] != k or a.shape != (m, f):
        return MOE_EINVAL
    tx, ta = x.stride(), a.stride()
    if not (tx[1] == 1 and ta[1] == 1 and x.dtype is dt and a.dtype is dt and w.is_contiguous() and
            x.get_device() == dev and a.get_device() == dev and _whole(offsets, (E + 1,), _INT32, dev)):
        return MOE_EINVAL
    ph = ldh = None
    if h is not None:
        if not (h.shape == (m, n) and h.stride(1) == 1 and h.dtype is dt and h.get_device() == dev):
            return MOE_EINVAL
        ph, ldh = h.data_ptr(), h.stride(0) if m > 1 else n
    return _call(_fn.moe_grouped_geglu, dev, stream, _DTYPE.get(dt, -1), gelu_variant, x.data_ptr(),
                 tx[0] if m > 1 else k, m, offsets.data_ptr(), E, w.data_ptr(), f, k, a.data_ptr(),
                 ta[0] if m > 1 else f, ph, ldh or 0)


def moe_geglu_grad(h, da, dh, n_rows=None, gelu_variant: int = MOE_GELU_ERF, stream=None) -> int:
    """dh = [da u GELU'(g), da GELU(g)] for h = [g, u]; n_rows: int32 tensor of one value, the rows to do."""
    if _DTYPE is None:
        _from_torch()
    sa = da.shape
    if len(sa) != 2:
        return MOE_EINVAL
    (m, f), dev, dt = sa, da.get_device(), da.dtype
    n = 2 * f
    if h.shape != (m, n) or dh.shape != (m, n):
        return MOE_EINVAL
    th, ta, td = h.stride(), da.stride(), dh.stride()
    if not (th[1] == 1 and ta[1] == 1 and td[1] == 1 and h.dtype is dt and dh.dtype is dt and h.get_device() == dev and
            dh.get_device() == dev):
        return MOE_EINVAL
    rows = None
    if n_rows is not None:
        if n_rows.numel() != 1 or n_rows.dtype is not _INT32 or n_rows.get_device() != dev:
            return MOE_EINVAL
        rows = n_rows.data_ptr()
    if m <= 1:
        th, ta, td = (n,), (f,), (n,)
    return _call(_fn.moe_geglu_grad, dev, stream, _DTYPE.get(dt, -1), gelu_variant, h.data_ptr(), th[0], da.data_ptr(),
                 ta[0], m, f, rows, dh.data_ptr(), td[0])


def moe_lora_mm(x, w, ids, a, b, scale, y, workspace, stream=None) -> int:
    """y[t] = w x[t] + scale[i] b[i] (a[i] x[t]), i = ids[t]; w [n, k], a [N, rank, k], b [N, n, rank], scale fp32
    [N], ids int32 [t] (-1: no adapter), workspace: a tensor of at least 4 * t * rank bytes."""
    if _DTYPE is None:
        _from_torch()
    sw, sx, sa = w.shape, x.shape, a.shape
    if len(sw) != 2 or len(sx) != 2 or len(sa) != 3:
        return MOE_EINVAL
    (n, k), (N, rank, _), t, dev, dt = sw, sa, sx[0], w.get_device(), w.dtype
    if sx[1] != k or y.shape != (t, n):
        return MOE_EINVAL
    tx, ty = x.stride(), y.stride()
    if not (tx[1] == 1 and ty[1] == 1 and x.dtype is dt and y.dtype is dt and w.is_contiguous() and
            x.get_device() == dev and y.get_device() == dev and _whole(a, (N, rank, k), dt, dev) and
            _whole(b, (N, n, rank), dt, dev) and _whole(scale, (N,), _FLOAT32, dev) and
            _whole(ids, (t,), _INT32, dev) and workspace.is_contiguous() and workspace.get_device() == dev):
        return MOE_EINVAL
    return _call(_fn.moe_lora_mm, dev, stream, _DTYPE.get(dt, -1), x.data_ptr(), tx[0] if t > 1 else k, t, w.data_ptr(),
                 n, k, ids.data_ptr(), a.data_ptr(), b.data_ptr(), scale.data_ptr(), N, rank, y.data_ptr(),
                 ty[0] if t > 1 else n, workspace.data_ptr(), workspace.nbytes)


def moe_grouped_sync(stream=None) -> int:
    return lib().moe_grouped_sync(_stream(stream))


# ---------------------------------------------------------------- norm and 8-bit operators (no context)
#
# As above; 8-bit tensors are torch.float8_e4m3fn, their scales contiguous float32.


def moe_rmsnorm(h, y=None, y8=None, scale=None, delta=None, h_out=None, weight=None, eps: float = 1e-6, stream=None) -> int:
    """h_out = h + delta, y = RMS norm of it times weight, in h's type; y8, scale: the same in e4m3 with a scale for each
    128 values ([m, ceil(d / 128)]).  delta comes with h_out; y or y8 (with scale), or both."""
    if _DTYPE is None:
        _from_torch()
    sh = h.shape
    if len(sh) != 2:
        return MOE_EINVAL
    (m, d), dev, dt, th = sh, h.get_device(), h.dtype, h.stride()
    if th[1] != 1 or (delta is None) != (h_out is None) or (y8 is None) != (scale is None):
        return MOE_EINVAL
    # a row's values are contiguous; the row stride of a single row says nothing
    one = m <= 1
    pd = po = py = p8 = ps = pw = None
    ldd = ldo = ldy = ld8 = dd = 0
    if delta is not None:
        td, to = delta.stride(), h_out.stride()
        if not (delta.shape == sh and h_out.shape == sh and td[1] == 1 and to[1] == 1 and h_out.dtype is dt and
                delta.get_device() == dev and h_out.get_device() == dev):
            return MOE_EINVAL
        pd, ldd, dd, po, ldo = delta.data_ptr(), d if one else td[0], _DTYPE.get(delta.dtype, -1), h_out.data_ptr(), d if one else to[0]
    if y is not None:
        ty = y.stride()
        if not (y.shape == sh and ty[1] == 1 and y.dtype is dt and y.get_device() == dev):
            return MOE_EINVAL
        py, ldy = y.data_ptr(), d if one else ty[0]
    if y8 is not None:
        t8 = y8.stride()
        if not (y8.shape == sh and t8[1] == 1 and y8.dtype is _E4M3 and y8.get_device() == dev and
                scale.shape == (m, (d + 127) // 128) and scale.dtype is _FLOAT32 and scale.is_contiguous() and
                scale.get_device() == dev):
            return MOE_EINVAL
        p8, ld8, ps = y8.data_ptr(), d if one else t8[0], scale.data_ptr()
    if weight is not None:
        if not (weight.shape == (d,) and weight.dtype is dt and weight.is_contiguous() and weight.get_device() == dev):
            return MOE_EINVAL
        pw = weight.data_ptr()
    return _call(_fn.moe_rmsnorm, dev, stream, _DTYPE.get(dt, -1), h.data_ptr(), d if one else th[0], pd, ldd, dd, pw, eps, m, d,
                 po, ldo, py, ldy, p8, ld8, ps)


def moe_rmsnorm_grad(h, dy, dh, dres=None, weight=None, dweight=None, workspace=None, eps: float = 1e-6, stream=None) -> int:
    """dh (dres added to it) and dweight (float32 [d]) of y = RMS norm of h times weight for the gradient dy; workspace: a
    tensor of at least 4 * d * min(m, 512) bytes, with dweight."""
    if _DTYPE is None:
        _from_torch()
    sh = h.shape
    if len(sh) != 2:
        return MOE_EINVAL
    (m, d), dev, dt, th, ty, to = sh, h.get_device(), h.dtype, h.stride(), dy.stride(), dh.stride()
    if not (dy.shape == sh and dh.shape == sh and th[1] == 1 and ty[1] == 1 and to[1] == 1 and dy.dtype is dt and
            dh.dtype is dt and dy.get_device() == dev and dh.get_device() == dev):
        return MOE_EINVAL
    one = m <= 1
    pr = pw = pdw = ws = None
    ldr = nws = 0
    if dres is not None:
        tr = dres.stride()
        if not (dres.shape == sh and tr[1] == 1 and dres.dtype is dt and dres.get_device() == dev):
            return MOE_EINVAL
        pr, ldr = dres.data_ptr(), d if one else tr[0]
    if weight is not None:
        if not (weight.shape == (d,) and weight.dtype is dt and weight.is_contiguous() and weight.get_device() == dev):
            return MOE_EINVAL
        pw = weight.data_ptr()
    if dweight is not None:
        if workspace is None or not (dweight.shape == (d,) and dweight.dtype is _FLOAT32 and dweight.is_contiguous() and
                                     dweight.get_device() == dev and workspace.is_contiguous() and
                                     workspace.get_device() == dev):
            return MOE_EINVAL
        pdw, ws, nws = dweight.data_ptr(), workspace.data_ptr(), workspace.nbytes
    return _call(_fn.moe_rmsnorm_grad, dev, stream, _DTYPE.get(dt, -1), h.data_ptr(), d if one else th[0], dy.data_ptr(),
                 d if one else ty[0], pr, ldr, pw, eps, m, d, dh.data_ptr(), d if one else to[0], pdw, ws, nws)


def moe_grouped_mm8(x, sx, offsets, w, sw, y, stream=None) -> int:
    """y[r] = w[e] x[r] for the rows of each expert, x [m, k] and w [E, n, k] in e4m3 with the scales sx [m, ceil(k / 128)]
    and sw [E, ceil(n / 128), ceil(k / 128)]; y in 16 or 32 bits."""
    if _DTYPE is None:
        _from_torch()
    sh, sm = w.shape, x.shape
    if len(sh) != 3 or len(sm) != 2:
        return MOE_EINVAL
    (E, n, k), m, dev = sh, sm[0], w.get_device()
    if sm[1] != k or y.shape != (m, n):
        return MOE_EINVAL
    tx, ty, kb = x.stride(), y.stride(), (k + 127) // 128
    if not (tx[1] == 1 and ty[1] == 1 and x.dtype is _E4M3 and x.get_device() == dev and y.get_device() == dev and
            w.dtype is _E4M3 and w.is_contiguous() and
            sx.shape == (m, kb) and sx.dtype is _FLOAT32 and sx.is_contiguous() and sx.get_device() == dev and
            sw.shape == (E, (n + 127) // 128, kb) and sw.dtype is _FLOAT32 and sw.is_contiguous() and sw.get_device() == dev and
            offsets.shape == (E + 1,) and offsets.dtype is _INT32 and offsets.is_contiguous() and offsets.get_device() == dev):
        return MOE_EINVAL
    return _call(_fn.moe_grouped_mm8, dev, stream, x.data_ptr(), tx[0] if m > 1 else k, sx.data_ptr(), m,
                 offsets.data_ptr(), E, w.data_ptr(), sw.data_ptr(), n, k, y.data_ptr(), ty[0] if m > 1 else n,
                 _DTYPE.get(y.dtype, -1))


def moe_grouped_geglu8(x, sx, offsets, w, sw, a, sa, gelu_variant: int = MOE_GELU_ERF, stream=None) -> int:
    """a[r] = GELU(g) u, [g, u] = w[e] x[r] in e4m3 as in moe_grouped_mm8, w [E, 2 f, k]; a [m, f] in e4m3 with the scales
    sa [m, ceil(f / 128)]."""
    if _DTYPE is None:
        _from_torch()
    sh, sm = w.shape, x.shape
    if len(sh) != 3 or len(sm) != 2 or sh[1] % 2:
        return MOE_EINVAL
    (E, n, k), m, dev = sh, sm[0], w.get_device()
    f = n // 2
    if sm[1] != k or a.shape != (m, f):
        return MOE_EINVAL
    tx, ta, kb = x.stride(), a.stride(), (k + 127) // 128
    if not (tx[1] == 1 and ta[1] == 1 and x.dtype is _E4M3 and a.dtype is _E4M3 and x.get_device() == dev and
            a.get_device() == dev and w.dtype is _E4M3 and w.is_contiguous() and
            sx.shape == (m, kb) and sx.dtype is _FLOAT32 and sx.is_contiguous() and sx.get_device() == dev and
            sw.shape == (E, (n + 127) // 128, kb) and sw.dtype is _FLOAT32 and sw.is_contiguous() and sw.get_device() == dev and
            sa.shape == (m, (f + 127) // 128) and sa.dtype is _FLOAT32 and sa.is_contiguous() and sa.get_device() == dev and
            offsets.shape == (E + 1,) and offsets.dtype is _INT32 and offsets.is_contiguous() and offsets.get_device() == dev):
        return MOE_EINVAL
    return _call(_fn.moe_grouped_geglu8, dev, stream, gelu_variant, x.data_ptr(), tx[0] if m > 1 else k, sx.data_ptr(), m,
                 offsets.data_ptr(), E, w.data_ptr(), sw.data_ptr(), f, k, a.data_ptr(), ta[0] if m > 1 else f,
                 sa.data_ptr())


def _ffn(weights, E: int, d: int, dt, dev: int):
    """(f, MoeFfnWeights) of (gate_up [2 f, d], down [d, f], and for e4m3 their scales; E >= 0: each of E experts), or None."""
    gate_up, down, *scales = weights
    su, f = gate_up.shape, down.shape[-1]
    pu = pd = None
    if len(scales) == 2 and scales[0] is not None:
        up, dn = scales
        db, hb, fb = (d + 127) // 128, (2 * f + 127) // 128, (f + 127) // 128
        if dn is None or not (
                up.shape == ((hb, db) if E < 0 else (E, hb, db)) and up.dtype is _FLOAT32 and up.is_contiguous() and
                up.get_device() == dev and dn.shape == ((db, fb) if E < 0 else (E, db, fb)) and dn.dtype is _FLOAT32 and
                dn.is_contiguous() and dn.get_device() == dev):
            return None
        dt, pu, pd = _E4M3, up.data_ptr(), dn.data_ptr()
    else:
        for t in scales:
            if t is not None:
                return None
    if not (su == ((2 * f, d) if E < 0 else (E, 2 * f, d)) and gate_up.dtype is dt and gate_up.is_contiguous() and
            gate_up.get_device() == dev and down.shape == ((d, f) if E < 0 else (E, d, f)) and down.dtype is dt and
            down.is_contiguous() and down.get_device() == dev):
        return None
    return f, MoeFfnWeights(gate_up.data_ptr(), down.data_ptr(), pu, pd)


def moe_token_layer(x, ids, gates, routed, y, workspace, shared=None, gelu_variant: int = MOE_GELU_ERF, stream=None) -> int:
    """y[t] = sum_j gates[t, j] FFN(routed[ids[t, j]], x[t]) + FFN(shared, x[t]) for up to 32 tokens.  routed: (gate_up
    [E, 2 f, d], down [E, d, f]) of x's type, or with their scales (gate_up, down, gate_up_scale, down_scale) in e4m3;
    shared: the same without E, or None; workspace: a tensor of at least 2 * t * (top_k * f + f_shared) bytes."""
    if _DTYPE is None:
        _from_torch()
    sx, si = x.shape, ids.shape
    if len(sx) != 2 or len(si) != 2 or routed[0].dim() != 3:
        return MOE_EINVAL
    (t, d), k, dev, dt, E = sx, si[1], x.get_device(), x.dtype, routed[0].shape[0]
    tx, ty = x.stride(), y.stride()
    if not (si[0] == t and y.shape == sx and tx[1] == 1 and ty[1] == 1 and y.get_device() == dev and
            ids.dtype is _INT32 and ids.is_contiguous() and ids.get_device() == dev and
            gates.shape == si and gates.dtype is _FLOAT32 and gates.is_contiguous() and gates.get_device() == dev and
            workspace.is_contiguous() and workspace.get_device() == dev):
        return MOE_EINVAL
    r, s = _ffn(routed, E, d, dt, dev), (0, None) if shared is None else _ffn(shared, -1, d, dt, dev)
    if r is None or s is None:
        return MOE_EINVAL
    return _call(_fn.moe_token_layer, dev, stream, _DTYPE.get(dt, -1), gelu_variant, x.data_ptr(), tx[0] if t > 1 else d, t,
                 ids.data_ptr(), gates.data_ptr(), k, E, C.byref(r[1]), None if s[1] is None else C.byref(s[1]), d, r[0], s[0],
                 y.data_ptr(), ty[0] if t > 1 else d, _DTYPE.get(y.dtype, -1), workspace.data_ptr(), workspace.nbytes)


def moe_profile(ctx, enable: bool) -> int:
    return lib().moe_profile(ctx, 1 if enable else 0)


def moe_get_profile(ctx):
    """Returns (status, list of (launches, total_ms) per kernel kind); resets the totals."""
    arr = (MoeKernelTime * N_KERNEL_KINDS)()
    st = lib().moe_get_profile(ctx, arr, N_KERNEL_KINDS)
    return st, [(a.launches, a.total_ms) for a in arr]


def moe_last_error(ctx) -> str:
    r = lib().moe_last_error(ctx)
    return r.decode() if r else ""


def moe_destroy(ctx) -> None:
    lib().moe_destroy(ctx)
