"""Thin ctypes binding of libstrata_moe.so (include/strata_moe.h).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  Functions take the C names; device buffers may be torch tensors
(their data_ptr is passed) or integer device addresses; streams may be
torch.cuda.Stream objects, raw handles, or None for the current torch stream.
The library must have been built (quantized_routed_expert_04_b200.build);
there is no fallback: a missing library raises.
"""
from __future__ import annotations

import ctypes
import enum
import os
import struct

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libstrata_moe.so")

_lib = None


class Status(enum.IntEnum):
    OK = 0
    INVALID_ARG = 1
    UNSUPPORTED = 2
    NOT_BOUND = 3
    SLOT_CONFLICT = 4
    TOO_MANY_EXPERTS = 5
    OOM = 6
    CUDA = 7
    DEVICE_STATUS = 8
    SCRATCH_LIMIT = 9
    RANGE = 10


class ArenaStats(ctypes.Structure):
    _fields_ = [("hits", ctypes.c_int), ("misses", ctypes.c_int), ("bytes", ctypes.c_size_t)]


class PrefillStats(ctypes.Structure):
    _fields_ = [("chunks", ctypes.c_int), ("passes", ctypes.c_int), ("hits", ctypes.c_int),
                ("misses", ctypes.c_int), ("bytes", ctypes.c_size_t)]


class StrataError(RuntimeError):
    def __init__(self, status, where=""):
        self.status = Status(status)
        super().__init__("%s: %s" % (where, _load().strata_status_str(int(status)).decode()))


def load_library():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libstrata_moe.so is not built (run python -m "
                               "quantized_routed_expert_04_b200.build)")
        lib = ctypes.CDLL(LIB_PATH)
        P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L, F = ctypes.c_longlong, ctypes.c_float
        sig = {
            "strata_moe_create": (I, [I, I, I, I, I, I, ctypes.POINTER(P)]),
            "strata_moe_destroy": (None, [P]),
            "strata_moe_expert_bytes": (Z, [I, I]),
            "strata_moe_expert_bytes_fmt": (Z, [I, I, I]),
            "strata_moe_set_format": (I, [P, I]),
            "strata_moe_set_router": (I, [P, P, P]),
            "strata_moe_bind_shared": (I, [P, I, P]),
            "strata_moe_set_routing": (I, [P, I, P, ctypes.c_float]),
            "strata_moe_bind_slot": (I, [P, I, I, P]),
            "strata_moe_slot_expert": (I, [P, I]),
            "strata_moe_reserve": (I, [P, I]),
            "strata_moe_route": (I, [P, P, I, P, P, P, P]),
            "strata_moe_forward": (I, [P, P, I, P, P]),
            "strata_moe_forward_routed": (I, [P, P, I, P, P, P, P]),
            "strata_moe_forward_noalloc": (I, [P, P, I, P, P]),
            "strata_moe_get_status": (I, [P, P]),
            "strata_moe_last_device_bits": (I, [P]),
            "strata_moe_profile": (I, [P, I]),
            "strata_moe_set_wait_limit": (I, [P, ctypes.c_ulonglong]),
            "strata_moe_profile_read": (I, [P, I, P, P]),
            "strata_rmsnorm": (I, [I, P, L, P, L, P, F, I, I, P, L, P, L, P, P, I, P]),
            "strata_rmsnorm_backward_workspace": (Z, [I, I]),
            "strata_rmsnorm_backward": (I, [I, P, L, P, F, P, L, P, L, I, I, P, L, P, P, Z, P]),
            "strata_moe_balance_workspace": (Z, [P, I, I]),
            "strata_moe_balance": (I, [P, P, P, I, P, I, P, F, P, P, P, P, Z, P]),
            "strata_moe_balance_backward": (I, [P, P, I, P, I, P, F, P, P, P, P, P]),
            "strata_moe_route_backward_workspace": (Z, [P, I]),
            "strata_moe_route_backward": (I, [P, P, I, P, P, P, P, P, P, P, P, Z, P]),
            "strata_packed_rmsnorm": (I, [P]),
            "strata_packed_rmsnorm_backward": (I, [P]),
            "strata_packed_balance": (I, [P]),
            "strata_packed_balance_backward": (I, [P]),
            "strata_packed_route_backward": (I, [P]),
            "strata_moe_forward_norm": (I, [P, P, P, P, F, I, P, P, P, P]),
            "strata_moe_forward_q8": (I, [P, P, P, I, I, P, P, P]),
            "strata_status_str": (ctypes.c_char_p, [I]),
            "strata_arena_create": (I, [P, P, P, ctypes.POINTER(P)]),
            "strata_arena_destroy": (None, [P]),
            "strata_arena_ensure": (I, [P, P, I, P, P, ctypes.POINTER(ArenaStats)]),
            "strata_arena_copy_ms": (I, [P, ctypes.POINTER(ctypes.c_float)]),
            "strata_arena_slot_of": (I, [P, I]),
            "strata_arena_prefill": (I, [P, P, I, I, P, P, P, ctypes.POINTER(PrefillStats)]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


_load = load_library


def _addr(buf):
    if buf is None:
        return None
    if isinstance(buf, int):
        return buf
    return buf.data_ptr()


_torch = None    # torch, imported on first use


def _get_torch():
    global _torch
    import torch
    _torch = torch
    return torch


def _stream(stream):
    if stream is None:
        # the raw handle of torch.cuda.current_stream() (building the Stream
        # object alone takes longer than a launch)
        t = _torch or _get_torch()
        return t._C._cuda_getCurrentRawStream(t.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(st, where):
    if st != 0:
        raise StrataError(st, where)


def strata_moe_create(hidden, inter, n_experts, top_k, n_shared, n_slots):
    h = ctypes.c_void_p()
    _check(_load().strata_moe_create(hidden, inter, n_experts, top_k, n_shared, n_slots,
                                     ctypes.byref(h)), "strata_moe_create")
    return h.value


def strata_moe_destroy(h):
    _load().strata_moe_destroy(h)


def strata_moe_expert_bytes(hidden, inter):
    return int(_load().strata_moe_expert_bytes(hidden, inter))


FORMAT_INT4, FORMAT_NVFP4 = 0, 1


def strata_moe_expert_bytes_fmt(hidden, inter, fmt):
    return int(_load().strata_moe_expert_bytes_fmt(hidden, inter, fmt))


def strata_moe_set_format(h, fmt):
    _check(_load().strata_moe_set_format(h, int(fmt)), "strata_moe_set_format")


def strata_moe_set_router(h, W, bias=None):
    _check(_load().strata_moe_set_router(h, _addr(W), _addr(bias)), "strata_moe_set_router")


ROUTE_SOFTMAX, ROUTE_SIGMOID = 0, 1


def strata_moe_set_routing(h, mode, corr=None, routed_scale=1.0):
    _check(_load().strata_moe_set_routing(h, int(mode), _addr(corr), float(routed_scale)),
           "strata_moe_set_routing")


def strata_moe_bind_shared(h, i, blob):
    _check(_load().strata_moe_bind_shared(h, i, _addr(blob)), "strata_moe_bind_shared")


def strata_moe_bind_slot(h, slot, expert_id, blob):
    _check(_load().strata_moe_bind_slot(h, slot, expert_id, _addr(blob)), "strata_moe_bind_slot")


def strata_moe_slot_expert(h, slot):
    return int(_load().strata_moe_slot_expert(h, slot))


def strata_moe_reserve(h, max_tokens):
    _check(_load().strata_moe_reserve(h, max_tokens), "strata_moe_reserve")


def strata_moe_route(h, x, n_tokens, logits, idx, w, stream=None):
    _check(_load().strata_moe_route(h, _addr(x), n_tokens, _addr(logits), _addr(idx), _addr(w),
                                    _stream(stream)), "strata_moe_route")


def strata_moe_forward(h, x, n_tokens, out, stream=None):
    _check(_load().strata_moe_forward(h, _addr(x), n_tokens, _addr(out), _stream(stream)),
           "strata_moe_forward")


def strata_moe_forward_routed(h, x, n_tokens, idx, w, out, stream=None):
    _check(_load().strata_moe_forward_routed(h, _addr(x), n_tokens, _addr(idx), _addr(w),
                                             _addr(out), _stream(stream)),
           "strata_moe_forward_routed")


def strata_moe_forward_noalloc(h, x, n_tokens, out, stream=None):
    _check(_load().strata_moe_forward_noalloc(h, _addr(x), n_tokens, _addr(out), _stream(stream)),
           "strata_moe_forward_noalloc")


NOALLOC_SCRATCH_BYTES = 16 << 20
NOALLOC_MAX_TOKENS = 64


def strata_moe_get_status(h, stream=None):
    """Synchronise and return (Status, raw device bits); does not raise."""
    st = _load().strata_moe_get_status(h, _stream(stream))
    return Status(st), int(_load().strata_moe_last_device_bits(h))


DEFAULT_WAIT_NS = 2_000_000_000


def strata_moe_set_wait_limit(h, ns):
    _check(_load().strata_moe_set_wait_limit(h, int(ns)), "strata_moe_set_wait_limit")


def strata_moe_profile(h, enable):
    _check(_load().strata_moe_profile(h, 1 if enable else 0), "strata_moe_profile")


PHASES = ("router", "topk", "bucket", "pack", "gate_up", "down", "combine", "gather", "fused")


def strata_moe_profile_read(h):
    """{phase: (launches, total ms)} since the last read."""
    n = len(PHASES)
    launches = (ctypes.c_int * n)()
    ms = (ctypes.c_double * n)()
    _check(_load().strata_moe_profile_read(h, n, launches, ms), "strata_moe_profile_read")
    return {PHASES[i]: (launches[i], ms[i]) for i in range(n)}


DTYPE_BF16, DTYPE_F16, DTYPE_F32 = 0, 1, 2
_dtypes = None   # torch dtype -> code


def _dtype(t):
    global _dtypes
    if _dtypes is None:
        torch = _get_torch()
        _dtypes = {torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16, torch.float32: DTYPE_F32}
    return _dtypes.get(t.dtype, -1)


def _refuse(where):
    raise StrataError(Status.INVALID_ARG, where)


# Operands of the calls that take torch tensors: their addresses (0: not given),
# once their sizes, types and device go together (dev: the device index of the
# first one).
def _rows(t, shape, dtype, dev, where):
    """(address, row stride) of a 2-D operand with unit column stride."""
    if t is None:
        return 0, 0
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        _refuse(where)
    ld, one = t.stride()
    if one != 1 and shape[1] > 1:
        _refuse(where)
    return t.data_ptr(), ld


# The types that an operand of a kind may have (torch's, known once a tensor has
# come).
_BF16, _F32, _I32, _BYTES, _E4M3 = [], [], [], [], []


def _of_kind(t, kind):
    if not _F32:
        torch = _get_torch()
        _BF16.append(torch.bfloat16)
        _I32.append(torch.int32)
        _BYTES.extend((torch.uint8, torch.bool, torch.int8))
        _E4M3.extend((torch.float8_e4m3fn, torch.uint8))
        _F32.append(torch.float32)
    return t.dtype in kind


def _flat(t, dev, nbytes, kind, where):
    """Address of a contiguous operand of nbytes bytes and of one of the kind's types."""
    if t is None:
        return 0
    if (t.nbytes != nbytes or t.get_device() != dev or not t.is_contiguous() or
            t.dtype not in kind and not _of_kind(t, kind)):
        _refuse(where)
    return t.data_ptr()


def _workspace(t, dev, where):
    """(address, bytes) of a workspace."""
    if t is None:
        return 0, 0
    if t.get_device() != dev or not t.is_contiguous():
        _refuse(where)
    return t.data_ptr(), t.nbytes


def _stream_on(stream, dev, where):
    """Handle of the stream of a call on device dev, which must be the current one."""
    t = _torch or _get_torch()
    if dev < 0 or dev != t.cuda.current_device():
        _refuse(where)
    return t._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


# The arguments of the calls below go to the library as one array of 8-byte
# words (csrc/packed.cu), which takes a third of the time of converting them
# one by one.
class _Packed:
    def __init__(self, name, words):
        self.name, self.pack, self.call = name, struct.Struct(words).pack, None

    def __call__(self, where, *words):
        call = self.call
        if call is None:
            call = self.call = getattr(_load(), self.name)
        st = call(self.pack(*words))
        if st != 0:
            raise StrataError(st, where)


_packed_rmsnorm = _Packed("strata_packed_rmsnorm", "=6qd10q")
_packed_rmsnorm_backward = _Packed("strata_packed_rmsnorm_backward", "=4qd12q")
_packed_balance = _Packed("strata_packed_balance", "=7qd6q")
_packed_balance_backward = _Packed("strata_packed_balance_backward", "=6qd5q")
_packed_route_backward = _Packed("strata_packed_route_backward", "=13q")


def strata_rmsnorm(x, residual, weight, eps, residual_out=None, out=None, out_q8=None, scales=None,
                   group=0, stream=None):
    """Rows are torch tensors [tokens][hidden] with unit column stride."""
    w = "strata_rmsnorm"
    shape, dt, dev = x.shape, x.dtype, x.get_device()
    if len(shape) != 2:
        _refuse(w)
    T, H = shape
    xa, ldx = _rows(x, shape, dt, dev, w)
    ra, ldr = _rows(residual, shape, dt, dev, w)
    roa, ldro = _rows(residual_out, shape, dt, dev, w)
    oa, ldo = _rows(out, shape, dt, dev, w)
    sa = qa = 0
    if out_q8 is not None:
        if group <= 0 or scales is None:
            _refuse(w)
        qa = _flat(out_q8, dev, T * H, _E4M3, w)
        sa = _flat(scales, dev, T * -(-H // group) * 4, _F32, w)
    wa = _flat(weight, dev, H * 4, _F32, w)
    _packed_rmsnorm(w, _dtype(x), xa, ldx, ra, ldr, wa, eps, T, H, roa, ldro, oa, ldo, qa, sa, group,
                    _stream_on(stream, dev, w))


def strata_rmsnorm_backward_workspace(n_tokens, hidden):
    return int(_load().strata_rmsnorm_backward_workspace(n_tokens, hidden))


def strata_rmsnorm_backward(h, weight, eps, dout, dsum, dx, dweight=None, workspace=None,
                            stream=None):
    w = "strata_rmsnorm_backward"
    shape, dt, dev = h.shape, h.dtype, h.get_device()
    if len(shape) != 2:
        _refuse(w)
    T, H = shape
    ha, ldh = _rows(h, shape, dt, dev, w)
    da, ldd = _rows(dout, shape, dt, dev, w)
    sa, lds = _rows(dsum, shape, dt, dev, w)
    xa, ldx = _rows(dx, shape, dt, dev, w)
    wa, dwa = _flat(weight, dev, H * 4, _F32, w), _flat(dweight, dev, H * 4, _F32, w)
    ws, nws = _workspace(workspace, dev, w)
    _packed_rmsnorm_backward(w, _dtype(h), ha, ldh, wa, eps, da, ldd, sa, lds, T, H, xa, ldx, dwa,
                             ws, nws, _stream_on(stream, dev, w))


def strata_moe_forward_norm(h, x, residual, weight, eps, n_tokens, residual_out, normed, out,
                            stream=None):
    _check(_load().strata_moe_forward_norm(h, _addr(x), _addr(residual), _addr(weight), eps,
                                           n_tokens, _addr(residual_out), _addr(normed),
                                           _addr(out), _stream(stream)), "strata_moe_forward_norm")


def strata_moe_forward_q8(h, x_q8, scales, group, n_tokens, x, out, stream=None):
    _check(_load().strata_moe_forward_q8(h, _addr(x_q8), _addr(scales), group, n_tokens, _addr(x),
                                         _addr(out), _stream(stream)), "strata_moe_forward_q8")


def strata_moe_balance_workspace(h, n_tokens, n_seq=1):
    return int(_load().strata_moe_balance_workspace(h, n_tokens, n_seq))


def strata_moe_balance(h, logits, idx, n_tokens, coef, counts, tokens, loss, workspace,
                       workspace_bytes, seq_off=None, n_seq=1, mask=None, stream=None):
    _check(_load().strata_moe_balance(h, _addr(logits), _addr(idx), n_tokens, _addr(seq_off),
                                      n_seq, _addr(mask), coef, _addr(counts), _addr(tokens),
                                      _addr(loss), _addr(workspace), workspace_bytes,
                                      _stream(stream)), "strata_moe_balance")


def strata_moe_balance_backward(h, logits, n_tokens, coef, counts, tokens, dlogits, dloss=None,
                                seq_off=None, n_seq=1, mask=None, stream=None):
    _check(_load().strata_moe_balance_backward(h, _addr(logits), n_tokens, _addr(seq_off), n_seq,
                                               _addr(mask), coef, _addr(counts), _addr(tokens),
                                               _addr(dloss), _addr(dlogits), _stream(stream)),
           "strata_moe_balance_backward")


def strata_moe_route_backward_workspace(h, n_tokens):
    return int(_load().strata_moe_route_backward_workspace(h, n_tokens))


def strata_moe_route_backward(h, x, n_tokens, logits, idx, dw, dlogits, dW, db, dx, workspace,
                              workspace_bytes, stream=None):
    _check(_load().strata_moe_route_backward(h, _addr(x), n_tokens, _addr(logits), _addr(idx),
                                             _addr(dw), _addr(dlogits), _addr(dW), _addr(db),
                                             _addr(dx), _addr(workspace), workspace_bytes,
                                             _stream(stream)), "strata_moe_route_backward")


def strata_status_str(st):
    return _load().strata_status_str(int(st)).decode()


def strata_arena_create(layer_h, host_pool, arena_dev):
    a = ctypes.c_void_p()
    _check(_load().strata_arena_create(layer_h, _addr(host_pool), _addr(arena_dev),
                                       ctypes.byref(a)), "strata_arena_create")
    return a.value


def strata_arena_destroy(a):
    _load().strata_arena_destroy(a)


def strata_arena_ensure(a, ids, stream=None, copy_stream=None):
    """ids: a sequence of expert ids (host).  Returns (hits, misses, bytes)."""
    import numpy as np
    arr = np.ascontiguousarray(np.asarray(ids, dtype=np.int32).reshape(-1))
    st = ArenaStats()
    _check(_load().strata_arena_ensure(a, arr.ctypes.data, int(arr.size), _stream(stream),
                                       _stream(copy_stream), ctypes.byref(st)),
           "strata_arena_ensure")
    return st.hits, st.misses, int(st.bytes)


def strata_arena_copy_ms(a):
    ms = ctypes.c_float()
    _check(_load().strata_arena_copy_ms(a, ctypes.byref(ms)), "strata_arena_copy_ms")
    return ms.value


def strata_arena_slot_of(a, expert_id):
    return int(_load().strata_arena_slot_of(a, expert_id))


def strata_arena_prefill(a, x, n_tokens, chunk_tokens, out, stream=None, copy_stream=None):
    """Chunked prefill through the arena; returns its stats as a dict."""
    st = PrefillStats()
    _check(_load().strata_arena_prefill(a, _addr(x), n_tokens, chunk_tokens, _addr(out),
                                        _stream(stream), _stream(copy_stream), ctypes.byref(st)),
           "strata_arena_prefill")
    return {"chunks": st.chunks, "passes": st.passes, "hits": st.hits, "misses": st.misses,
            "bytes": int(st.bytes)}


class Arena:
    """Owning wrapper of an expert arena over a StrataMoE layer."""

    def __init__(self, layer, host_pool, arena_dev):
        self.layer, self.host_pool, self.arena_dev = layer, host_pool, arena_dev
        self.a = strata_arena_create(layer.h, host_pool, arena_dev)

    def ensure(self, ids, stream=None, copy_stream=None):
        return strata_arena_ensure(self.a, ids, stream, copy_stream)

    def copy_ms(self):
        return strata_arena_copy_ms(self.a)

    def slot_of(self, expert_id):
        return strata_arena_slot_of(self.a, expert_id)

    def prefill(self, x, chunk_tokens, out, stream=None, copy_stream=None):
        return strata_arena_prefill(self.a, x, x.shape[0], chunk_tokens, out, stream, copy_stream)

    def close(self):
        if self.a:
            strata_arena_destroy(self.a)
            self.a = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class StrataMoE:
    """Owning wrapper: a layer handle plus convenience methods (same calls)."""

    def __init__(self, hidden, inter, n_experts, top_k, n_shared, n_slots):
        self.hidden, self.inter, self.n_experts = hidden, inter, n_experts
        self.top_k, self.n_shared, self.n_slots = top_k, n_shared, n_slots
        self.h = strata_moe_create(hidden, inter, n_experts, top_k, n_shared, n_slots)

    def close(self):
        if self.h:
            strata_moe_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def set_router(self, W, bias=None):
        strata_moe_set_router(self.h, W, bias)

    def set_format(self, fmt):
        strata_moe_set_format(self.h, fmt)

    def set_routing(self, mode, corr=None, routed_scale=1.0):
        strata_moe_set_routing(self.h, mode, corr, routed_scale)

    def bind_shared(self, i, blob):
        strata_moe_bind_shared(self.h, i, blob)

    def bind_slot(self, slot, expert_id, blob):
        strata_moe_bind_slot(self.h, slot, expert_id, blob)

    def reserve(self, max_tokens):
        strata_moe_reserve(self.h, max_tokens)

    def route(self, x, logits, idx, w, stream=None):
        strata_moe_route(self.h, x, x.shape[0], logits, idx, w, stream)

    def forward(self, x, out, stream=None):
        strata_moe_forward(self.h, x, x.shape[0], out, stream)

    def forward_routed(self, x, idx, w, out, stream=None):
        strata_moe_forward_routed(self.h, x, x.shape[0], idx, w, out, stream)

    def forward_noalloc(self, x, out, stream=None):
        strata_moe_forward_noalloc(self.h, x, x.shape[0], out, stream)

    # The calls below take torch tensors and check that their sizes go together
    # (StrataError, INVALID_ARG).
    def forward_norm(self, x, residual, weight, eps, residual_out, normed, out, stream=None):
        w = "strata_moe_forward_norm"
        T, dev = x.shape[0], x.get_device()
        n = T * self.hidden * 2
        a = [_flat(t, dev, n, _BF16, w) for t in (x, residual, residual_out, normed, out)]
        wa = _flat(weight, dev, self.hidden * 4, _F32, w)
        strata_moe_forward_norm(self.h, a[0], a[1], wa, eps, T, a[2], a[3], a[4],
                                _stream_on(stream, dev, w))

    def forward_q8(self, x_q8, scales, group, x, out, stream=None):
        w = "strata_moe_forward_q8"
        T, H, dev = x_q8.shape[0], self.hidden, x_q8.get_device()
        if group <= 0:
            _refuse(w)
        qa = _flat(x_q8, dev, T * H, _E4M3, w)
        sa = _flat(scales, dev, T * -(-H // group) * 4, _F32, w)
        xa, oa = _flat(x, dev, T * H * 2, _BF16, w), _flat(out, dev, T * H * 2, _BF16, w)
        strata_moe_forward_q8(self.h, qa, sa, group, T, xa, oa, _stream_on(stream, dev, w))

    # Training the router; `workspace` is a buffer of the size that the
    # *_workspace method gives, kept by the caller.
    def balance_workspace(self, n_tokens, n_seq=1):
        return strata_moe_balance_workspace(self.h, n_tokens, n_seq)

    def balance(self, logits, idx, coef, counts, tokens, loss, workspace, seq_off=None, mask=None,
                stream=None):
        w = "strata_moe_balance"
        T, E, dev = logits.shape[0], self.n_experts, logits.get_device()
        n_seq = 1 if seq_off is None else seq_off.numel() - 1
        la, ia = _flat(logits, dev, T * E * 4, _F32, w), _flat(idx, dev, T * self.top_k * 4, _I32, w)
        ca, ta = _flat(counts, dev, n_seq * E * 4, _I32, w), _flat(tokens, dev, n_seq * 4, _I32, w)
        sa, ma = _flat(seq_off, dev, n_seq * 4 + 4, _I32, w), _flat(mask, dev, T, _BYTES, w)
        loa = _flat(loss, dev, 4, _F32, w)
        ws, nws = _workspace(workspace, dev, w)
        _packed_balance(w, self.h or 0, la, ia, T, sa, n_seq, ma, coef, ca, ta, loa, ws, nws,
                        _stream_on(stream, dev, w))

    def balance_backward(self, logits, coef, counts, tokens, dlogits, dloss=None, seq_off=None,
                         mask=None, stream=None):
        w = "strata_moe_balance_backward"
        T, E, dev = logits.shape[0], self.n_experts, logits.get_device()
        n_seq = 1 if seq_off is None else seq_off.numel() - 1
        la, da = _flat(logits, dev, T * E * 4, _F32, w), _flat(dlogits, dev, T * E * 4, _F32, w)
        ca, ta = _flat(counts, dev, n_seq * E * 4, _I32, w), _flat(tokens, dev, n_seq * 4, _I32, w)
        sa, ma = _flat(seq_off, dev, n_seq * 4 + 4, _I32, w), _flat(mask, dev, T, _BYTES, w)
        dla = _flat(dloss, dev, 4, _F32, w)
        _packed_balance_backward(w, self.h or 0, la, T, sa, n_seq, ma, coef, ca, ta, dla, da,
                                 _stream_on(stream, dev, w))

    def route_backward_workspace(self, n_tokens):
        return strata_moe_route_backward_workspace(self.h, n_tokens)

    def route_backward(self, x, logits, idx, dw, dlogits, dW, db, dx, workspace, stream=None):
        w = "strata_moe_route_backward"
        T, dev = x.shape[0], x.get_device()
        E, k, H = self.n_experts, self.top_k, self.hidden
        xa, dxa = _flat(x, dev, T * H * 2, _BF16, w), _flat(dx, dev, T * H * 2, _BF16, w)
        la, dla = _flat(logits, dev, T * E * 4, _F32, w), _flat(dlogits, dev, T * E * 4, _F32, w)
        ia, dwa = _flat(idx, dev, T * k * 4, _I32, w), _flat(dw, dev, T * k * 4, _F32, w)
        dWa, dba = _flat(dW, dev, E * H * 4, _F32, w), _flat(db, dev, E * 4, _F32, w)
        ws, nws = _workspace(workspace, dev, w)
        _packed_route_backward(w, self.h or 0, xa, T, la, ia, dwa, dla, dWa, dba, dxa, ws, nws,
                               _stream_on(stream, dev, w))

    def status(self, stream=None):
        return strata_moe_get_status(self.h, stream)

    def set_wait_limit(self, ns):
        strata_moe_set_wait_limit(self.h, ns)
