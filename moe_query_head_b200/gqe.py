"""ctypes binding of the GQE C ABI (include/gqe.h): argument marshalling only.

Every function here has the name of the C entry point it calls and passes torch tensors'
device pointers and the current CUDA stream through unchanged; all computation happens in
libgqe.so's kernels. If the library is missing, importing this module raises: there is no
fallback path.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgqe.so")

GQE_OK, GQE_ERR_INVALID_ARG, GQE_ERR_UNSUPPORTED, GQE_ERR_WORKSPACE, GQE_ERR_CUDA, \
    GQE_ERR_TIMEOUT = range(6)
GQE_BF16, GQE_F32 = 0, 1
VARIANTS = {"gqe": 0, "weighted_concat": 1, "hard_concat": 2}
TENSORS = {"K": 0, "V": 1, "Q": 2, "Z": 3, "PSEL": 4, "W": 5, "LOGITS": 6}

EXPORTED = ("gqe_create", "gqe_forward", "gqe_get_routing", "gqe_get_tensor",
            "gqe_check_device_status", "gqe_set_spin_limit", "gqe_destroy", "gqe_status_str",
            "gqe_workspace_bytes", "gqe_kernel_launches", "gqe_set_stage_events",
            "gqe_stage_name", "gqe_route_static", "gqe_exp2_fma", "gqe_selftest_timeout",
            "gqe_decode", "gqe_enable_backward", "gqe_backward", "gqe_backward_launches",
            "gqe_set_group_range", "gqe_backward_begin", "gqe_backward_finish",
            "gqe_qk_norm_rope", "gqe_qk_norm_rope_workspace_bytes", "gqe_qk_norm_rope_backward",
            "gqe_qk_norm_rope_append", "gqe_attention_forward", "gqe_attention_workspace_bytes",
            "gqe_attention_backward", "gqe_attention_decode_workspace_bytes",
            "gqe_attention_decode", "gqe_check_op_status", "gqe_set_qk_transform",
            "gqe_set_scores")
GQE_NUM_STAGES = 6


class GQEError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {status_str(status)}")
        self.status = status


class Heads(ctypes.Structure):
    """gqe_heads: a [heads, tokens, d_h] tensor by its strides."""
    _fields_ = [("data", ctypes.c_void_p), ("heads", ctypes.c_int),
                ("head_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64)]


class QkTransform(ctypes.Structure):
    """gqe_qk_transform."""
    _fields_ = [("d_h", ctypes.c_int), ("dtype", ctypes.c_int), ("norm", ctypes.c_int),
                ("eps", ctypes.c_float), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p), ("rot_dim", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("inv_freq", ctypes.c_void_p)]


class Scores(ctypes.Structure):
    """gqe_scores."""
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("G", ctypes.c_int),
                ("k", ctypes.c_int), ("S", ctypes.c_int), ("d_h", ctypes.c_int),
                ("causal", ctypes.c_int), ("scale", ctypes.c_float), ("softcap", ctypes.c_float),
                ("slopes", ctypes.c_void_p), ("key_begin", ctypes.c_void_p),
                ("key_end", ctypes.c_void_p)]


def _load() -> ctypes.CDLL:
    if not os.path.exists(_LIB_PATH):
        raise ImportError(
            f"GQE CUDA library not built ({_LIB_PATH} missing); run "
            "`python -m moe_query_head_b200.build`")
    lib = ctypes.CDLL(_LIB_PATH)
    P, I, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    lib.gqe_create.argtypes = [ctypes.POINTER(P), I, I, I, I, I, I, I64]
    lib.gqe_create.restype = I
    lib.gqe_forward.argtypes = [P, P, I, I, P, P, P, P, P, P, I, I, I, I, I, I, P, P, P]
    lib.gqe_forward.restype = I
    lib.gqe_decode.argtypes = [P, P, I, P, P, I, P, P, P, P, P, P, P, I, I, I, I, I, P, P, P]
    lib.gqe_decode.restype = I
    lib.gqe_get_routing.argtypes = [P, P, P, P, P, P]
    lib.gqe_get_routing.restype = I
    lib.gqe_get_tensor.argtypes = [P, I, P, SZ, P]
    lib.gqe_get_tensor.restype = I
    lib.gqe_check_device_status.argtypes = [P, P]
    lib.gqe_check_device_status.restype = I
    lib.gqe_set_spin_limit.argtypes = [P, I64]
    lib.gqe_set_spin_limit.restype = I
    lib.gqe_destroy.argtypes = [P]
    lib.gqe_destroy.restype = None
    lib.gqe_status_str.argtypes = [I]
    lib.gqe_status_str.restype = ctypes.c_char_p
    lib.gqe_workspace_bytes.argtypes = [I, I, I, I, I, I, I64]
    lib.gqe_workspace_bytes.restype = I64
    lib.gqe_kernel_launches.argtypes = [P]
    lib.gqe_kernel_launches.restype = I
    lib.gqe_set_stage_events.argtypes = [P, ctypes.POINTER(P), I]
    lib.gqe_set_stage_events.restype = I
    lib.gqe_stage_name.argtypes = [I]
    lib.gqe_stage_name.restype = ctypes.c_char_p
    lib.gqe_route_static.argtypes = [P, I, I, I, I, P, P, P, P, P, P]
    lib.gqe_route_static.restype = I
    lib.gqe_exp2_fma.argtypes = [P, P, I, P]
    lib.gqe_exp2_fma.restype = I
    lib.gqe_selftest_timeout.argtypes = [P, ctypes.c_int64, P]
    lib.gqe_selftest_timeout.restype = I
    lib.gqe_set_group_range.argtypes = [P, I, I]
    lib.gqe_set_group_range.restype = I
    lib.gqe_enable_backward.argtypes = [P]
    lib.gqe_enable_backward.restype = I
    lib.gqe_backward.argtypes = [P, P, I, I, P, P, P, P, P, P, I, I, I, I, I, I, P,
                                 ctypes.c_float, P, P, P, P, P, P, P, P]
    lib.gqe_backward.restype = I
    lib.gqe_backward_begin.argtypes = [P, P, I, I, P, P, P, P, P, P, I, I, I, I, I, I, P, P, P]
    lib.gqe_backward_begin.restype = I
    lib.gqe_backward_finish.argtypes = [P, P, I, I, P, P, P, P, P, P, I, I, I, I, I, I, P,
                                        ctypes.c_float, P, P, P, P, P, P, P, P, P]
    lib.gqe_backward_finish.restype = I
    lib.gqe_backward_launches.argtypes = [P]
    lib.gqe_backward_launches.restype = I
    lib.gqe_qk_norm_rope.argtypes = [P, I, P, P, P, I, P, P, P]
    lib.gqe_qk_norm_rope.restype = I
    lib.gqe_qk_norm_rope_workspace_bytes.argtypes = [I]
    lib.gqe_qk_norm_rope_workspace_bytes.restype = I64
    lib.gqe_qk_norm_rope_backward.argtypes = [P, I, P, P, P, I, P, P, P, P, P, P, P, SZ, P]
    lib.gqe_qk_norm_rope_backward.restype = I
    lib.gqe_qk_norm_rope_append.argtypes = [P, I, P, P, P, P, I, P, P, P, P]
    lib.gqe_qk_norm_rope_append.restype = I
    lib.gqe_attention_forward.argtypes = [P, P, P, P, P, P, P]
    lib.gqe_attention_forward.restype = I
    lib.gqe_attention_workspace_bytes.argtypes = [P]
    lib.gqe_attention_workspace_bytes.restype = I64
    lib.gqe_attention_backward.argtypes = [P, P, P, P, P, P, P, P, P, P, P, SZ, P]
    lib.gqe_attention_backward.restype = I
    lib.gqe_attention_decode_workspace_bytes.argtypes = [P, I]
    lib.gqe_attention_decode_workspace_bytes.restype = I64
    lib.gqe_attention_decode.argtypes = [P, P, P, P, I, P, P, P, SZ, P]
    lib.gqe_attention_decode.restype = I
    lib.gqe_set_qk_transform.argtypes = [P, P, P, P, P]
    lib.gqe_set_qk_transform.restype = I
    lib.gqe_set_scores.argtypes = [P, ctypes.c_float, ctypes.c_float, P, P, P]
    lib.gqe_set_scores.restype = I
    lib.gqe_check_op_status.argtypes = [P]
    lib.gqe_check_op_status.restype = I
    return lib


lib = _load()


def status_str(status: int) -> str:
    return lib.gqe_status_str(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != GQE_OK:
        raise GQEError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def gqe_workspace_bytes(dim, N, G, k, d_h, dtype, max_tokens) -> int:
    return int(lib.gqe_workspace_bytes(dim, N, G, k, d_h, dtype, max_tokens))


# What has been set on each handle (by its address): its device, the number of its groups, and the
# sizes of the slopes, positions and intervals (gqe_set_scores, gqe_set_qk_transform), which the
# library reads without knowing them.
_set_on = {}


def _address(h):
    return getattr(h, "value", h)


def _check_sizes(h, where: str, tokens: int, k: int, shared: bool, names) -> None:
    """The tensors set on a handle have the sizes that this call reads."""
    on = _set_on.get(_address(h))
    if on is None or len(on) == 2:
        return
    want = dict.fromkeys(names, tokens)
    want["slopes"] = on["groups"] * k + shared
    for name, n in want.items():
        if on.get(name, n) != n:
            raise GQEError(GQE_ERR_INVALID_ARG, f"{where} ({name} of {on[name]} values, {n} are read)")


def gqe_create(dim, N, G, k, d_h, dtype, max_tokens) -> ctypes.c_void_p:
    h = ctypes.c_void_p()
    _check(lib.gqe_create(ctypes.byref(h), dim, N, G, k, d_h, dtype, max_tokens), "gqe_create")
    _set_on[h.value] = {"device": torch.cuda.current_device(), "groups": G}
    return h


def gqe_forward(h, x, B, T, W_r, W_q, W_k, W_v, W_shared, W_o, N, G, k, d_h, variant, causal,
                out, aux_loss=None, stream=None) -> None:
    _check_sizes(h, "gqe_forward", B * T, k, W_shared is not None,
                 ("positions", "key_begin", "key_end"))
    _check(lib.gqe_forward(h, _ptr(x), B, T, _ptr(W_r), _ptr(W_q), _ptr(W_k), _ptr(W_v),
                           _ptr(W_shared), _ptr(W_o), N, G, k, d_h, variant, causal, _ptr(out),
                           _ptr(aux_loss), _stream(stream)), "gqe_forward")


def gqe_decode(h, x, B, k_cache, v_cache, L_max, lengths, W_r, W_q, W_k, W_v, W_shared, W_o,
               N, G, k, d_h, variant, out, aux_loss=None, stream=None) -> None:
    """One generation step with a KV cache (see include/gqe.h); lengths is an int32 device
    tensor and is not modified."""
    _check_sizes(h, "gqe_decode", B, k, W_shared is not None, ("key_begin",))
    _check(lib.gqe_decode(h, _ptr(x), B, _ptr(k_cache), _ptr(v_cache), L_max, _ptr(lengths),
                          _ptr(W_r), _ptr(W_q), _ptr(W_k), _ptr(W_v), _ptr(W_shared), _ptr(W_o),
                          N, G, k, d_h, variant, _ptr(out), _ptr(aux_loss), _stream(stream)),
           "gqe_decode")


def gqe_set_group_range(h, g0: int, g1: int) -> None:
    """Restricts the handle to groups g0 .. g1-1 of the layer (see include/gqe.h)."""
    _check(lib.gqe_set_group_range(h, int(g0), int(g1)), "gqe_set_group_range")
    if _address(h) in _set_on:
        _set_on[_address(h)]["groups"] = int(g1) - int(g0)


def gqe_enable_backward(h) -> None:
    """Allocates the handle's backward workspace (see include/gqe.h)."""
    _check(lib.gqe_enable_backward(h), "gqe_enable_backward")


def gqe_backward(h, x, B, T, W_r, W_q, W_k, W_v, W_shared, W_o, N, G, k, d_h, variant, causal,
                 dy, aux_grad, dx, dW_r, dW_q, dW_k, dW_v, dW_shared, dW_o, stream=None) -> None:
    """Gradients of <dy, y> + aux_grad * aux_loss of the handle's last gqe_forward (same
    arguments); every gradient is a float32 device tensor (see include/gqe.h)."""
    _check(lib.gqe_backward(h, _ptr(x), B, T, _ptr(W_r), _ptr(W_q), _ptr(W_k), _ptr(W_v),
                            _ptr(W_shared), _ptr(W_o), N, G, k, d_h, variant, causal, _ptr(dy),
                            float(aux_grad), _ptr(dx), _ptr(dW_r), _ptr(dW_q), _ptr(dW_k),
                            _ptr(dW_v), _ptr(dW_shared), _ptr(dW_o), _stream(stream)),
           "gqe_backward")


def gqe_backward_begin(h, x, B, T, W_r, W_q, W_k, W_v, W_shared, W_o, N, G, k, d_h, variant,
                       causal, dy, slot_dot, stream=None) -> None:
    """Phase 1 of the backward of a handle's last gqe_forward: writes this handle's share of
    <dslot, slot> per token to slot_dot (float32 [B*T], device; see include/gqe.h)."""
    _check(lib.gqe_backward_begin(h, _ptr(x), B, T, _ptr(W_r), _ptr(W_q), _ptr(W_k), _ptr(W_v),
                                  _ptr(W_shared), _ptr(W_o), N, G, k, d_h, variant, causal,
                                  _ptr(dy), _ptr(slot_dot), _stream(stream)),
           "gqe_backward_begin")


def gqe_backward_finish(h, x, B, T, W_r, W_q, W_k, W_v, W_shared, W_o, N, G, k, d_h, variant,
                        causal, dy, aux_grad, slot_dot, dx, dW_r, dW_q, dW_k, dW_v, dW_shared,
                        dW_o, stream=None) -> None:
    """Phase 2: the gradients, given <dslot, slot> summed over the layer's group ranges."""
    _check(lib.gqe_backward_finish(h, _ptr(x), B, T, _ptr(W_r), _ptr(W_q), _ptr(W_k),
                                   _ptr(W_v), _ptr(W_shared), _ptr(W_o), N, G, k, d_h, variant,
                                   causal, _ptr(dy), float(aux_grad), _ptr(slot_dot), _ptr(dx),
                                   _ptr(dW_r), _ptr(dW_q), _ptr(dW_k), _ptr(dW_v),
                                   _ptr(dW_shared), _ptr(dW_o), _stream(stream)),
           "gqe_backward_finish")


def gqe_backward_launches(h) -> int:
    return int(lib.gqe_backward_launches(h))


def gqe_get_routing(h, sel=None, gates=None, counts=None, mean_prob=None, stream=None) -> None:
    _check(lib.gqe_get_routing(h, _ptr(sel), _ptr(gates), _ptr(counts), _ptr(mean_prob),
                               _stream(stream)), "gqe_get_routing")


def gqe_get_tensor(h, which: str, dst, stream=None) -> None:
    _check(lib.gqe_get_tensor(h, TENSORS[which], _ptr(dst), dst.numel() * dst.element_size(),
                              _stream(stream)), "gqe_get_tensor")


def gqe_check_device_status(h, stream=None) -> int:
    return int(lib.gqe_check_device_status(h, _stream(stream)))


def gqe_set_spin_limit(h, limit: int) -> None:
    _check(lib.gqe_set_spin_limit(h, int(limit)), "gqe_set_spin_limit")


def gqe_destroy(h) -> None:
    _set_on.pop(_address(h), None)
    lib.gqe_destroy(h)


def gqe_kernel_launches(h) -> int:
    return int(lib.gqe_kernel_launches(h))


def gqe_route_static(logits, M, N, G, k, sel, gates, counts, mean_prob, aux_loss=None,
                     stream=None) -> None:
    """Routing from precomputed logits with no device allocation (see include/gqe.h)."""
    _check(lib.gqe_route_static(_ptr(logits), M, N, G, k, _ptr(sel), _ptr(gates), _ptr(counts),
                                _ptr(mean_prob), _ptr(aux_loss), _stream(stream)),
           "gqe_route_static")


def gqe_selftest_timeout(h, spin: int, stream=None) -> None:
    """Makes one bounded device wait run out on purpose (see include/gqe.h)."""
    _check(lib.gqe_selftest_timeout(h, spin, _stream(stream)), "gqe_selftest_timeout")


def gqe_exp2_fma(inp, out, stream=None) -> None:
    """Diagnostic: the softmax's FMA-pipe exp2, elementwise (float32 device tensors)."""
    _check(lib.gqe_exp2_fma(_ptr(inp), _ptr(out), inp.numel(), _stream(stream)), "gqe_exp2_fma")


def gqe_stage_name(i: int):
    r = lib.gqe_stage_name(int(i))
    return None if r is None else r.decode()


def gqe_set_stage_events(h, events) -> None:
    """events: GQE_NUM_STAGES + 1 torch.cuda.Event(enable_timing=True) objects, each
    already recorded once (torch creates the underlying cudaEvent_t lazily), or None."""
    if not events:
        _check(lib.gqe_set_stage_events(h, None, 0), "gqe_set_stage_events")
        return
    arr = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
    _check(lib.gqe_set_stage_events(h, arr, len(events)), "gqe_set_stage_events")


# ----------------------------------------------------------------------------------------
# Operators on the layer's streams, without a handle. Tensors are [heads, tokens, d_h] views
# with dense rows (any head and token strides that are multiples of 16 bytes); sizes, types
# and devices are checked here, the rest by the library. Calls run on the tensors' device, on
# `stream` or that device's current stream. Their structs are packed as bytes, which costs the
# small calls (one new token per sequence) a third of what ctypes structures do.
# ----------------------------------------------------------------------------------------
_DTYPES = {torch.bfloat16: GQE_BF16, torch.float32: GQE_F32}
_pack_heads = struct.Struct("@Piqq").pack
_pack_transform = struct.Struct("@iiifPPiiP").pack
_pack_scores = struct.Struct("@iiiiiiiffPPP").pack
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _require(ok: bool, where: str) -> None:
    if not ok:
        raise GQEError(GQE_ERR_INVALID_ARG, where)


def _heads(t, shape, dtype, index, where: str) -> bytes:
    """The gqe_heads of a tensor of this shape, type and device with dense rows."""
    st = t.stride()
    if (t.shape != shape or t.dtype is not dtype or t.get_device() != index
            or (st[2] != 1 and t.numel())):
        raise GQEError(GQE_ERR_INVALID_ARG, where)
    return _pack_heads(t.data_ptr(), shape[0], st[0], st[1])


def _cache(t, shape, dtype, index, where: str) -> bytes:
    """The gqe_heads of a KV cache [G, B, L_max, d_h] with dense rows."""
    st = t.stride()
    if (t.shape != shape or t.dtype is not dtype or t.get_device() != index
            or (t.numel() and (st[3] != 1 or (shape[2] > 1 and st[2] != shape[3])))):
        raise GQEError(GQE_ERR_INVALID_ARG, where)
    return _pack_heads(t.data_ptr(), shape[0], st[0], st[1])


def _vector(t, n, dtype, index, where: str) -> int:
    """Address of a dense vector of n values; 0 (a null pointer) for None."""
    if t is None:
        return 0
    if (t.numel() != n or t.dtype is not dtype or t.get_device() != index
            or not t.is_contiguous()):
        raise GQEError(GQE_ERR_INVALID_ARG, where)
    return t.data_ptr()


def _device(t, where: str) -> int:
    """The index of a CUDA tensor's device."""
    index = t.get_device()
    if index < 0:
        raise GQEError(GQE_ERR_INVALID_ARG, where)
    return index


def _call(fn, index: int, stream, where: str, *args) -> None:
    """fn(*args, stream) with the tensors' device current."""
    raw = stream.cuda_stream if stream is not None else _raw_stream(index)
    if index == torch.cuda.current_device():
        status = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            status = fn(*args, raw)
    if status != GQE_OK:
        raise GQEError(status, where)


def _scratch(n: int, index: int, stream):
    """n bytes from torch's allocator, in order with the call's stream."""
    if stream is None:
        return torch.empty(n, dtype=torch.uint8, device=index)
    with torch.cuda.stream(stream):
        return torch.empty(n, dtype=torch.uint8, device=index)


def _room(workspace, size, index: int, stream, where: str):
    """Address, bytes and owner of a call's scratch: the caller's, or `size` new bytes."""
    if workspace is None:
        if not size > 0:
            return 0, 0, None
        workspace = _scratch(size, index, stream)
        return workspace.data_ptr(), size, workspace
    _require(workspace.get_device() == index and workspace.is_contiguous(), where)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _transform(q, index, norm, q_weight, k_weight, eps, inv_freq, interleaved, where) -> bytes:
    if q.dim() != 3 or q.dtype not in _DTYPES:
        raise GQEError(GQE_ERR_INVALID_ARG, where)
    d = q.shape[2]
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    return _pack_transform(d, _DTYPES[q.dtype], int(norm), eps,
                           _vector(q_weight, d, torch.float32, index, where),
                           _vector(k_weight, d, torch.float32, index, where), rot,
                           int(interleaved),
                           _vector(inv_freq, rot // 2, torch.float64, index, where))


def gqe_qk_norm_rope(q, k, q_out, k_out, *, positions=None, T=0, norm=True, q_weight=None,
                     k_weight=None, eps=1e-6, inv_freq=None, interleaved=False,
                     stream=None) -> None:
    """RMS norm of every head of q [Hq, M, d_h] and k [Hk, M, d_h] and rotation by position in
    one pass (see include/gqe.h). positions: int32 [M], or None for t % T (T = 0: t)."""
    w = "gqe_qk_norm_rope"
    i = _device(q, w)
    tr = _transform(q, i, norm, q_weight, k_weight, eps, inv_freq, interleaved, w)
    dt, sq = q.dtype, q.shape
    M = sq[1]
    sk = (k.shape[0], M, sq[2])
    _call(lib.gqe_qk_norm_rope, i, stream, w, tr, M, _heads(q, sq, dt, i, w),
          _heads(k, sk, dt, i, w), _vector(positions, M, torch.int32, i, w), T or max(M, 1),
          _heads(q_out, sq, dt, i, w), _heads(k_out, sk, dt, i, w))


def gqe_qk_norm_rope_backward(q, k, dq_out, dk_out, dq, dk, dq_weight=None, dk_weight=None, *,
                              positions=None, T=0, norm=True, q_weight=None, k_weight=None,
                              eps=1e-6, inv_freq=None, interleaved=False, workspace=None,
                              stream=None) -> None:
    """Gradients of gqe_qk_norm_rope given its inputs and the gradients of its outputs (see
    include/gqe.h); dq_weight, dk_weight: float32 [d_h] to fill, or None."""
    w = "gqe_qk_norm_rope_backward"
    i = _device(q, w)
    tr = _transform(q, i, norm, q_weight, k_weight, eps, inv_freq, interleaved, w)
    dt, sq = q.dtype, q.shape
    M, d = sq[1], sq[2]
    sk = (k.shape[0], M, d)
    wq = _vector(dq_weight, d, torch.float32, i, w)
    wk = _vector(dk_weight, d, torch.float32, i, w)
    size = lib.gqe_qk_norm_rope_workspace_bytes(d) if norm and (wq or wk) else 0
    room, size, owner = _room(workspace, size, i, stream, w)
    _call(lib.gqe_qk_norm_rope_backward, i, stream, w, tr, M, _heads(q, sq, dt, i, w),
          _heads(k, sk, dt, i, w), _vector(positions, M, torch.int32, i, w), T or max(M, 1),
          _heads(dq_out, sq, dt, i, w), _heads(dk_out, sk, dt, i, w), _heads(dq, sq, dt, i, w),
          _heads(dk, sk, dt, i, w), wq, wk, room, size)


def gqe_qk_norm_rope_append(q, k, v, lengths, q_out, k_cache, v_cache, *, norm=True,
                            q_weight=None, k_weight=None, eps=1e-6, inv_freq=None,
                            interleaved=False, stream=None) -> None:
    """The serving form: q [Hq, B, d_h], k, v [G, B, d_h] of one new token per sequence at
    positions `lengths` (int32 [B]; -1: idle slot); k and v go to row lengths[b] of the caches
    [G, B, L_max, d_h] (see include/gqe.h)."""
    w = "gqe_qk_norm_rope_append"
    i = _device(q, w)
    tr = _transform(q, i, norm, q_weight, k_weight, eps, inv_freq, interleaved, w)
    sc = k_cache.shape
    if len(sc) != 4:
        raise GQEError(GQE_ERR_INVALID_ARG, w)
    dt, sq = q.dtype, q.shape
    B, d = sq[1], sq[2]
    sk = (k.shape[0], B, d)
    sc = (k.shape[0], B, sc[2], d)
    _call(lib.gqe_qk_norm_rope_append, i, stream, w, tr, B, _heads(q, sq, dt, i, w),
          _heads(k, sk, dt, i, w), _heads(v, sk, dt, i, w),
          _vector(lengths, B, torch.int32, i, w), sc[2], _heads(q_out, sq, dt, i, w),
          _cache(k_cache, sc, dt, i, w), _cache(v_cache, sc, dt, i, w))


def _scores(sq, i, G, B, T, top_k, causal, scale, softcap, slopes, key_begin, key_end, rows,
            where) -> bytes:
    return _pack_scores(B, T, G, top_k, sq[0], sq[2], int(causal), scale, softcap,
                        _vector(slopes, sq[0], torch.float32, i, where),
                        _vector(key_begin, rows, torch.int32, i, where),
                        _vector(key_end, rows, torch.int32, i, where))


def gqe_attention_forward(q, k, v, out, lse, B, T, top_k, *, causal=True, scale=0.0, softcap=0.0,
                          slopes=None, key_begin=None, key_end=None, stream=None) -> None:
    """Attention of the streams q [S, B T, d_h] over k, v [G, B T, d_h] (S = G top_k, or
    G top_k + 1 with the shared stream) with capped, biased and masked scores; lse: float32
    [S, B T] to fill for the backward pass, or None (see include/gqe.h)."""
    w = "gqe_attention_forward"
    i = _device(q, w)
    sq, sk, bf = q.shape, k.shape, torch.bfloat16
    M = B * T
    if len(sq) != 3 or len(sk) != 3 or sq[1] != M:
        raise GQEError(GQE_ERR_INVALID_ARG, w)
    G = sk[0]
    sk = (G, M, sq[2])
    a = _scores(sq, i, G, B, T, top_k, causal, scale, softcap, slopes, key_begin, key_end, M, w)
    _call(lib.gqe_attention_forward, i, stream, w, a, _heads(q, sq, bf, i, w),
          _heads(k, sk, bf, i, w), _heads(v, sk, bf, i, w), _heads(out, sq, bf, i, w),
          _vector(lse, sq[0] * M, torch.float32, i, w))


def gqe_attention_backward(q, k, v, out, lse, dout, dq, dk, dv, B, T, top_k, *, causal=True,
                           scale=0.0, softcap=0.0, slopes=None, key_begin=None, key_end=None,
                           workspace=None, stream=None) -> None:
    """Gradients dq, dk, dv of gqe_attention_forward (same arguments), given its out and lse and
    the upstream gradient dout (see include/gqe.h)."""
    w = "gqe_attention_backward"
    i = _device(q, w)
    sq, sk, bf = q.shape, k.shape, torch.bfloat16
    M = B * T
    if len(sq) != 3 or len(sk) != 3 or sq[1] != M:
        raise GQEError(GQE_ERR_INVALID_ARG, w)
    G = sk[0]
    sk = (G, M, sq[2])
    a = _scores(sq, i, G, B, T, top_k, causal, scale, softcap, slopes, key_begin, key_end, M, w)
    room, size, owner = _room(workspace, lib.gqe_attention_workspace_bytes(a), i, stream, w)
    _call(lib.gqe_attention_backward, i, stream, w, a, _heads(q, sq, bf, i, w),
          _heads(k, sk, bf, i, w), _heads(v, sk, bf, i, w), _heads(out, sq, bf, i, w),
          _vector(lse, sq[0] * M, torch.float32, i, w), _heads(dout, sq, bf, i, w),
          _heads(dq, sq, bf, i, w), _heads(dk, sk, bf, i, w), _heads(dv, sk, bf, i, w), room, size)


def gqe_attention_decode(q, k_cache, v_cache, lengths, out, top_k, *, scale=0.0, softcap=0.0,
                         slopes=None, key_begin=None, workspace=None, stream=None) -> None:
    """The single-token form: q [S, B, d_h] at positions `lengths` (int32 [B]; -1: no key) over
    rows key_begin[b] .. lengths[b] of the caches [G, B, L_max, d_h] (see include/gqe.h)."""
    w = "gqe_attention_decode"
    i = _device(q, w)
    sq, sc, bf = q.shape, k_cache.shape, torch.bfloat16
    if len(sq) != 3 or len(sc) != 4:
        raise GQEError(GQE_ERR_INVALID_ARG, w)
    G, B, L = sc[0], sq[1], sc[2]
    sc = (G, B, L, sq[2])
    a = _scores(sq, i, G, B, 1, top_k, 1, scale, softcap, slopes, key_begin, None, B, w)
    room, size, owner = _room(workspace, lib.gqe_attention_decode_workspace_bytes(a, L), i, stream,
                              w)
    _call(lib.gqe_attention_decode, i, stream, w, a, _heads(q, sq, bf, i, w),
          _cache(k_cache, sc, bf, i, w), _cache(v_cache, sc, bf, i, w), L,
          _vector(lengths, B, torch.int32, i, w), _heads(out, sq, bf, i, w), room, size)


def _on_handle(h, sizes: dict) -> None:
    """Notes the sizes of what has been set on a handle."""
    on = _set_on.get(_address(h))
    if on is not None:
        for name, t in sizes.items():
            if t is None:
                on.pop(name, None)
            else:
                on[name] = t.numel()


def _handle_vector(h, t, n, dtype, where: str) -> int:
    """Address of a dense vector of n values on the handle's device; 0 for None."""
    if t is None:
        return 0
    index = _device(t, where)
    on = _set_on.get(_address(h))
    _require(on is None or on["device"] == index, where)
    return _vector(t, n, dtype, index, where)


def gqe_set_qk_transform(h, d_h=0, dtype=GQE_BF16, *, norm=True, q_weight=None, k_weight=None,
                         eps=1e-6, inv_freq=None, interleaved=False, positions=None,
                         dq_weight=None, dk_weight=None) -> None:
    """Norm and rotation of the handle's queries and keys (see include/gqe.h); d_h = 0 turns
    them off. The tensors must stay alive while calls of the handle read them; a gqe_forward
    whose B T is not the size of `positions` is refused."""
    w = "gqe_set_qk_transform"
    if not d_h:
        _check(lib.gqe_set_qk_transform(h, None, None, None, None), w)
        _on_handle(h, {"positions": None})
        return
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()

    def vec(t, n, dt=torch.float32):
        return _handle_vector(h, t, n, dt, w)

    tr = _pack_transform(d_h, dtype, int(norm), eps, vec(q_weight, d_h), vec(k_weight, d_h), rot,
                         int(interleaved), vec(inv_freq, rot // 2, torch.float64))
    pos = 0 if positions is None else vec(positions, positions.numel(), torch.int32)
    _check(lib.gqe_set_qk_transform(h, tr, pos, vec(dq_weight, d_h), vec(dk_weight, d_h)), w)
    _on_handle(h, {"positions": positions})


def gqe_set_scores(h, *, scale=0.0, softcap=0.0, slopes=None, key_begin=None,
                   key_end=None) -> None:
    """Cap, bias and intervals of the handle's scores (see include/gqe.h); without arguments they
    are off. The tensors must stay alive while calls of the handle read them; a gqe_forward
    (B T) or gqe_decode (B) that would read another number of values than they hold is
    refused."""
    w = "gqe_set_scores"

    def vec(t, dt):
        return 0 if t is None else _handle_vector(h, t, t.numel(), dt, w)

    _check(lib.gqe_set_scores(h, scale, softcap, vec(slopes, torch.float32),
                              vec(key_begin, torch.int32), vec(key_end, torch.int32)), w)
    _on_handle(h, {"slopes": slopes, "key_begin": key_begin, "key_end": key_end})


def gqe_check_op_status(stream=None, device=None) -> int:
    """Synchronises the stream and reads and clears the device's status word of the operators
    above (see include/gqe.h)."""
    index = None if device is None else torch.device(device).index
    if index is None:
        index = torch.cuda.current_device()
    with torch.cuda.device(index):
        raw = stream.cuda_stream if stream is not None else _raw_stream(index)
        return int(lib.gqe_check_op_status(raw))
