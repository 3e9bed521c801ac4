"""Python binding of libqmoe (include/qmoe.h, qmoe_attn.h, qmoe_step.h): the same calls under the same
names, with argument marshalling only -- torch tensors become device
pointers, the current torch stream becomes the hipStream_t, a nonzero status
becomes a QmoeError carrying moe_last_error().  Every computation happens in
the library's kernels or its host quantizer.

Import torch before this module (the library then shares torch's HIP
runtime); a missing libqmoe.so raises at import time, a missing _attn.so when
one of the attention or step calls that need it is made.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

import torch


class _NotBuilt:
    """Stands for a module that is missing or does not load: its calls say so."""

    def __init__(self, name, why):
        self._name, self._why = name, why

    def __getattr__(self, call):
        raise ImportError(f"{self._name} does not load ({self._why}); run `python -m bit_quantized_moe_02_amd.build`")


try:
    from . import _attn
except ImportError as e:                       # (the calls of the expert layer do not need it)
    _attn = _NotBuilt("_attn.so", str(e))

_HERE = os.path.dirname(os.path.abspath(__file__))
# QMOE_LIB names another build of the same library (the host-sanitizer build
# the CPU tests load); by default the one built in this directory.
LIB_PATH = os.environ.get("QMOE_LIB") or os.path.join(_HERE, "libqmoe.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_WORKSPACE = 3
MOE_ERR_HIP = 4

MOE_FMT_BF16 = 0
MOE_FMT_CB2 = 1
MOE_FMT_K2 = 2
MOE_FMT_K4 = 3
MOE_FMT_Q8 = 4
FMT = {"bf16": MOE_FMT_BF16, "cb2": MOE_FMT_CB2, "k2": MOE_FMT_K2, "k4": MOE_FMT_K4, "q8": MOE_FMT_Q8}

EXPORTED = [
    "moe_codebook_generate", "moe_packed_bytes", "moe_quantize_pack",
    "moe_route_workspace_bytes", "moe_route", "moe_group_workspace_bytes",
    "moe_group_tokens", "moe_ffn_workspace_bytes", "moe_expert_ffn_decode",
    "moe_expert_ffn_prefill", "moe_layer_decode_workspace_bytes", "moe_layer_decode",
    "moe_debug_dequant", "moe_profile_next_launch", "moe_last_error", "moe_layer_decode_noalloc",
    "moe_measure_read", "moe_expert_cache_slot_bytes", "moe_expert_cache_create", "moe_expert_cache_destroy",
    "moe_expert_cache_weights", "moe_expert_cache_plan", "moe_expert_cache_fetch", "moe_expert_cache_state",
    "moe_layer_decode_streamed_workspace_bytes", "moe_layer_decode_streamed",
]
# the attention calls (include/qmoe_attn.h)
EXPORTED_ATTN = [
    "moe_kv_code_bytes", "moe_kv_scale_bytes", "moe_rope_freqs", "moe_kv_append", "moe_kv_read",
    "moe_attn_decode_workspace_bytes", "moe_attn_decode", "moe_attn_prefill_workspace_bytes", "moe_attn_prefill",
]
# norm, 4-bit products, pages (include/qmoe_step.h)
EXPORTED_STEP = [
    "moe_rms_norm", "moe_linear_quantize", "moe_linear_packed_bytes", "moe_linear_pack", "moe_linear", "moe_kv_resize",
    "moe_kv_fork_workspace_bytes", "moe_kv_fork", "moe_kv_compact_workspace_bytes", "moe_kv_compact",
]
MOE_NOALLOC_SCRATCH_BYTES = 8 << 20

MOE_DT_BF16 = 0
MOE_DT_F16 = 1
MOE_DT_F32 = 2
MOE_DT_I8 = 3
MOE_ROPE = {"plain": 0, "linear": 1, "base": 2, "parts": 3}

MOE_KERNEL = {"route_logits": 0, "route_topk": 1, "decode_upgate": 2, "decode_down": 3,
              "decode_combine": 4, "group": 5, "prefill_upgate": 6, "prefill_down": 7,
              "prefill_combine": 8, "read": 9}


class QmoeError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"libqmoe error {code}: {msg}")
        self.code = code


class MoeWeights(ctypes.Structure):
    """Mirror of struct moe_weights."""
    _fields_ = [
        ("n_experts", ctypes.c_int32), ("hidden", ctypes.c_int32),
        ("inter", ctypes.c_int32), ("shared_inter", ctypes.c_int32),
        ("fmt_up", ctypes.c_int32), ("fmt_gate", ctypes.c_int32),
        ("fmt_down", ctypes.c_int32), ("fmt_shared", ctypes.c_int32),
        ("up", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("down", ctypes.c_void_p),
        ("codebook", ctypes.c_void_p),
        ("shared_up", ctypes.c_void_p), ("shared_gate", ctypes.c_void_p),
        ("shared_down", ctypes.c_void_p),
    ]


class MoeKvCache(ctypes.Structure):
    """Mirror of struct moe_kv_cache."""
    _fields_ = [("n_pages", ctypes.c_int32), ("page_tokens", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class MoeKvBatch(ctypes.Structure):
    """Mirror of struct moe_kv_batch."""
    _fields_ = [("batch", ctypes.c_int32), ("rows", ctypes.c_int32), ("max_new", ctypes.c_int32),
                ("pages_per_seq", ctypes.c_int32), ("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("kv_lens", ctypes.c_void_p), ("cu_rows", ctypes.c_void_p)]


class MoeRope(ctypes.Structure):
    """Mirror of struct moe_rope."""
    _fields_ = [("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("scale", ctypes.c_float),
                ("freqs", ctypes.c_void_p)]


class MoePacked(ctypes.Structure):
    """Mirror of struct moe_packed."""
    _fields_ = [("batch", ctypes.c_int32), ("rows_q", ctypes.c_int32), ("rows_k", ctypes.c_int32),
                ("max_q", ctypes.c_int32), ("cu_q", ctypes.c_void_p), ("cu_k", ctypes.c_void_p),
                ("q_heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class MoeNorm(ctypes.Structure):
    """Mirror of struct moe_norm."""
    _fields_ = [("rows", ctypes.c_int32), ("heads", ctypes.c_int32), ("cols", ctypes.c_int32), ("x_dtype", ctypes.c_int32),
                ("x", ctypes.c_void_p), ("x_stride", ctypes.c_int64), ("residual_dtype", ctypes.c_int32),
                ("weight_dtype", ctypes.c_int32), ("residual", ctypes.c_void_p), ("residual_stride", ctypes.c_int64),
                ("sum", ctypes.c_void_p), ("sum_stride", ctypes.c_int64), ("weight", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("out_dtype", ctypes.c_int32), ("out", ctypes.c_void_p), ("out_stride", ctypes.c_int64),
                ("codes", ctypes.c_void_p), ("codes_stride", ctypes.c_int64), ("scales", ctypes.c_void_p),
                ("scale_stride", ctypes.c_int64), ("group", ctypes.c_int32)]


class MoeLinearWeights(ctypes.Structure):
    """Mirror of struct moe_linear_weights."""
    _fields_ = [("n", ctypes.c_int32), ("k", ctypes.c_int32), ("group", ctypes.c_int32), ("with_zeros", ctypes.c_int32),
                ("packed", ctypes.c_void_p), ("bias", ctypes.c_void_p)]


class MoeKvPool(ctypes.Structure):
    """Mirror of struct moe_kv_pool."""
    _fields_ = [("n_pages", ctypes.c_int32), ("n_caches", ctypes.c_int32), ("caches", ctypes.POINTER(MoeKvCache)),
                ("refs", ctypes.c_void_p)]


class MoeKvTables(ctypes.Structure):
    """Mirror of struct moe_kv_tables."""
    _fields_ = [("seqs", ctypes.c_int32), ("pages_per_seq", ctypes.c_int32), ("page_tokens", ctypes.c_int32),
                ("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("kv_lens", ctypes.c_void_p)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python -m bit_quantized_moe_02_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    f64 = ctypes.c_double
    sig = {
        "moe_codebook_generate": (ctypes.c_int, [ctypes.c_uint64, vp]),
        "moe_packed_bytes": (sz, [ctypes.c_int, i64, i64]),
        "moe_quantize_pack": (ctypes.c_int, [ctypes.c_int, vp, i64, i64, vp, vp, sz, ctypes.c_int]),
        "moe_route_workspace_bytes": (sz, [i32, i32]),
        "moe_route": (ctypes.c_int, [vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, sz, vp]),
        "moe_group_workspace_bytes": (sz, [i32, i32, i32]),
        "moe_group_tokens": (ctypes.c_int, [vp, i32, i32, i32, vp, vp, vp, vp, sz, vp]),
        "moe_ffn_workspace_bytes": (sz, [ctypes.POINTER(MoeWeights), i32, i32, ctypes.c_int]),
        "moe_expert_ffn_decode": (ctypes.c_int, [ctypes.POINTER(MoeWeights), vp, i32, i32, vp, vp, vp,
                                                 vp, sz, vp]),
        "moe_expert_ffn_prefill": (ctypes.c_int, [ctypes.POINTER(MoeWeights), vp, i32, i32, vp, vp, vp,
                                                  vp, vp, vp, vp, sz, vp]),
        "moe_layer_decode_workspace_bytes": (sz, [ctypes.POINTER(MoeWeights), i32, i32]),
        "moe_layer_decode": (ctypes.c_int, [ctypes.POINTER(MoeWeights), vp, vp, vp, i32, i32, vp, vp, vp,
                                            vp, sz, vp]),
        "moe_layer_decode_noalloc": (ctypes.c_int, [ctypes.POINTER(MoeWeights), vp, vp, vp, i32, i32, vp, vp, vp,
                                                    vp]),
        "moe_debug_dequant": (ctypes.c_int, [ctypes.c_int, vp, i64, i64, vp, vp, vp]),
        "moe_profile_next_launch": (ctypes.c_int, [ctypes.c_int, vp, vp]),
        "moe_measure_read": (ctypes.c_int, [vp, sz, vp, ctypes.c_int, vp]),
        "moe_last_error": (ctypes.c_char_p, []),
        "moe_expert_cache_slot_bytes": (sz, [ctypes.POINTER(MoeWeights), i32]),
        "moe_expert_cache_create": (ctypes.c_int, [ctypes.POINTER(MoeWeights), i32, i32, vp, sz,
                                                   ctypes.POINTER(vp)]),
        "moe_expert_cache_destroy": (ctypes.c_int, [vp]),
        "moe_expert_cache_weights": (ctypes.c_int, [vp, ctypes.POINTER(MoeWeights)]),
        "moe_expert_cache_plan": (ctypes.c_int, [vp, vp, i32, vp, vp, vp, ctypes.POINTER(i32)]),
        "moe_expert_cache_fetch": (ctypes.c_int, [vp, vp, vp, i32, vp]),
        "moe_expert_cache_state": (ctypes.c_int, [vp, vp, ctypes.POINTER(i64), ctypes.POINTER(i64)]),
        "moe_layer_decode_streamed_workspace_bytes": (sz, [vp, i32, i32]),
        "moe_layer_decode_streamed": (ctypes.c_int, [vp, vp, vp, vp, i32, i32, vp, vp, vp, vp, sz, vp, vp]),
        "moe_kv_code_bytes": (sz, [i32, i32, i32, i32]),
        "moe_kv_scale_bytes": (sz, [i32, i32, i32]),
        "moe_rope_freqs": (ctypes.c_int, [i32, f64, ctypes.c_int, f64, f64, f64, f64, vp]),
        "moe_kv_append": (ctypes.c_int, [vp, vp, vp, ctypes.c_int, vp, i64, i32, vp, i64, vp, i64, vp, i64, vp, i64, vp]),
        "moe_kv_read": (ctypes.c_int, [vp, vp, ctypes.c_int, vp, i64, vp, i64, vp]),
        "moe_attn_decode_workspace_bytes": (sz, [vp, vp, i32]),
        "moe_attn_decode": (ctypes.c_int, [vp, vp, ctypes.c_int, vp, i64, i32, ctypes.c_float, vp, i64, vp, vp, sz, vp]),
        "moe_attn_prefill_workspace_bytes": (sz, [vp]),
        "moe_attn_prefill": (ctypes.c_int, [vp, ctypes.c_int, vp, i64, vp, i64, vp, i64, ctypes.c_float, ctypes.c_int, vp, i64,
                                            vp, vp, sz, vp]),
        "moe_rms_norm": (ctypes.c_int, [vp, vp]),
        "moe_linear_quantize": (ctypes.c_int, [vp, i64, i64, i32, vp, vp, vp, ctypes.c_int]),
        "moe_linear_packed_bytes": (sz, [i64, i64, i32, ctypes.c_int]),
        "moe_linear_pack": (ctypes.c_int, [vp, vp, vp, i64, i64, i32, vp, sz, ctypes.c_int]),
        "moe_linear": (ctypes.c_int, [vp, i32, ctypes.c_int, vp, i64, vp, i64, i32, ctypes.c_int, vp, i64, vp]),
        "moe_kv_resize": (ctypes.c_int, [vp, vp, vp, vp, vp]),
        "moe_kv_fork_workspace_bytes": (sz, [vp, vp]),
        "moe_kv_fork": (ctypes.c_int, [vp, vp, vp, vp, vp, sz, vp]),
        "moe_kv_compact_workspace_bytes": (sz, [vp, vp]),
        "moe_kv_compact": (ctypes.c_int, [vp, vp, vp, vp, sz, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


def _check(rc):
    if rc != MOE_OK:
        raise QmoeError(rc, lib.moe_last_error().decode())


def _dev(t, name, dtype, n=0, optional=False):
    """Device address of tensor `t` as a kernel argument, after the checks
    that keep a kernel from touching the wrong memory: a CUDA tensor of
    `dtype`, contiguous, with at least `n` elements.  None passes only where
    the call takes NULL (`optional`)."""
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < n:
        raise ValueError(f"{name} holds {t.numel()} elements; the call needs {n}")
    return t.data_ptr()


def _ws(ws):
    """(address, bytes) of a uint8 device workspace; the library checks the size."""
    return _dev(ws, "ws", torch.uint8), ws.numel()


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream
    return torch.cuda.current_stream().cuda_stream


# ---------------------------------------------------------------------------
# host-only calls


def moe_codebook_generate(seed: int = 0) -> np.ndarray:
    out = np.empty((256, 8), dtype=np.int8)
    _check(lib.moe_codebook_generate(seed, out.ctypes.data))
    return out


def moe_packed_bytes(fmt, rows: int, k: int) -> int:
    return int(lib.moe_packed_bytes(FMT.get(fmt, fmt), rows, k))


def moe_quantize_pack(fmt, w: np.ndarray, codebook: np.ndarray | None = None, n_threads: int = 0,
                      out: np.ndarray | None = None) -> np.ndarray:
    """fp32 host matrix [rows, k] -> packed uint8 bytes (host)."""
    f = FMT.get(fmt, fmt)
    w = np.ascontiguousarray(w, dtype=np.float32)
    rows, k = w.shape
    nbytes = moe_packed_bytes(f, rows, k)
    if out is None:
        out = np.empty(max(nbytes, 1), dtype=np.uint8)
    cb = None if codebook is None else np.ascontiguousarray(codebook, dtype=np.int8)
    _check(lib.moe_quantize_pack(f, w.ctypes.data, rows, k, None if cb is None else cb.ctypes.data,
                                 out.ctypes.data, out.nbytes, n_threads))
    return out[:nbytes]


# ---------------------------------------------------------------------------
# device calls (torch tensors on the current device)


def moe_route_workspace_bytes(T: int, E: int) -> int:
    return int(lib.moe_route_workspace_bytes(T, E))


def moe_route(x_bf16, w_router, logit_bias, T, H, E, k, topk_idx, topk_w, ws, stream=None):
    _check(lib.moe_route(_dev(x_bf16, "x_bf16", torch.bfloat16, T * H), _dev(w_router, "w_router", torch.float32, E * H),
                         _dev(logit_bias, "logit_bias", torch.float32, E, optional=True), T, H, E, k,
                         _dev(topk_idx, "topk_idx", torch.int32, T * k), _dev(topk_w, "topk_w", torch.float32, T * k),
                         *_ws(ws), _stream(stream)))


def moe_group_workspace_bytes(T: int, k: int, E: int) -> int:
    return int(lib.moe_group_workspace_bytes(T, k, E))


def moe_group_tokens(topk_idx, T, k, E, expert_offsets, sorted_slots, slot_pos, ws, stream=None):
    _check(lib.moe_group_tokens(_dev(topk_idx, "topk_idx", torch.int32, T * k), T, k, E,
                                _dev(expert_offsets, "expert_offsets", torch.int32, E + 1),
                                _dev(sorted_slots, "sorted_slots", torch.int32, T * k),
                                _dev(slot_pos, "slot_pos", torch.int32, T * k), *_ws(ws), _stream(stream)))


def moe_ffn_workspace_bytes(w: MoeWeights, T: int, k: int, prefill: bool) -> int:
    return int(lib.moe_ffn_workspace_bytes(ctypes.byref(w), T, k, int(bool(prefill))))


def moe_expert_ffn_decode(w: MoeWeights, x_bf16, T, k, topk_idx, topk_w, y, ws, stream=None):
    H = w.hidden
    _check(lib.moe_expert_ffn_decode(ctypes.byref(w), _dev(x_bf16, "x_bf16", torch.bfloat16, T * H), T, k,
                                     _dev(topk_idx, "topk_idx", torch.int32, T * k),
                                     _dev(topk_w, "topk_w", torch.float32, T * k),
                                     _dev(y, "y", torch.float32, T * H), *_ws(ws), _stream(stream)))


def moe_layer_decode_workspace_bytes(w: MoeWeights, T: int, k: int) -> int:
    return int(lib.moe_layer_decode_workspace_bytes(ctypes.byref(w), T, k))


def moe_layer_decode_noalloc(w: MoeWeights, w_router, logit_bias, x_bf16, T, k, topk_idx, topk_w, y, stream=None):
    """moe_layer_decode with the library's own device scratch (allocates nothing)."""
    E, H = w.n_experts, w.hidden
    _check(lib.moe_layer_decode_noalloc(ctypes.byref(w), _dev(w_router, "w_router", torch.float32, E * H),
                                        _dev(logit_bias, "logit_bias", torch.float32, E, optional=True),
                                        _dev(x_bf16, "x_bf16", torch.bfloat16, T * H), T, k,
                                        _dev(topk_idx, "topk_idx", torch.int32, T * k),
                                        _dev(topk_w, "topk_w", torch.float32, T * k),
                                        _dev(y, "y", torch.float32, T * H), _stream(stream)))


def moe_layer_decode(w: MoeWeights, w_router, logit_bias, x_bf16, T, k, topk_idx, topk_w, y, ws, stream=None):
    E, H = w.n_experts, w.hidden
    _check(lib.moe_layer_decode(ctypes.byref(w), _dev(w_router, "w_router", torch.float32, E * H),
                                _dev(logit_bias, "logit_bias", torch.float32, E, optional=True),
                                _dev(x_bf16, "x_bf16", torch.bfloat16, T * H), T, k,
                                _dev(topk_idx, "topk_idx", torch.int32, T * k),
                                _dev(topk_w, "topk_w", torch.float32, T * k),
                                _dev(y, "y", torch.float32, T * H), *_ws(ws), _stream(stream)))


def moe_expert_ffn_prefill(w: MoeWeights, x_bf16, T, k, topk_idx, topk_w, expert_offsets, sorted_slots,
                           slot_pos, y, ws, stream=None):
    E, H = w.n_experts, w.hidden
    _check(lib.moe_expert_ffn_prefill(ctypes.byref(w), _dev(x_bf16, "x_bf16", torch.bfloat16, T * H), T, k,
                                      _dev(topk_idx, "topk_idx", torch.int32, T * k),
                                      _dev(topk_w, "topk_w", torch.float32, T * k),
                                      _dev(expert_offsets, "expert_offsets", torch.int32, E + 1),
                                      _dev(sorted_slots, "sorted_slots", torch.int32, T * k),
                                      _dev(slot_pos, "slot_pos", torch.int32, T * k),
                                      _dev(y, "y", torch.float32, T * H), *_ws(ws), _stream(stream)))


def moe_debug_dequant(fmt, packed, rows, k, codebook, out, stream=None):
    f = FMT.get(fmt, fmt)
    kp = -(-k // 256) * 256
    _check(lib.moe_debug_dequant(f, _dev(packed, "packed", torch.uint8, moe_packed_bytes(f, rows, k)), rows, k,
                                 _dev(codebook, "codebook", torch.int8, 256 * 8, optional=True),
                                 _dev(out, "out", torch.float32, rows * kp), _stream(stream)))


def moe_profile_next_launch(kernel, start_event, stop_event):
    """Record torch.cuda.Event (or raw hipEvent_t) start/stop around the next
    launch of `kernel` (name or id) by this thread."""
    kid = MOE_KERNEL.get(kernel, kernel)
    ev = lambda e: None if e is None else (e.cuda_event if hasattr(e, "cuda_event") else e)
    _check(lib.moe_profile_next_launch(kid, ev(start_event), ev(stop_event)))


def moe_measure_read(src, out, blocks=0, stream=None):
    """Streaming read of the whole uint8 device tensor `src`; XOR of its words into out (int32 [1])."""
    _check(lib.moe_measure_read(_dev(src, "src", torch.uint8), src.numel(), _dev(out, "out", torch.int32, 1),
                                blocks, _stream(stream)))


def moe_last_error() -> str:
    return lib.moe_last_error().decode()


# ---------------------------------------------------------------------------
# Convenience: a layer's weights resident in device memory.


class DeviceLayer:
    """Device copies of one layer's packed weights plus the MoeWeights view.

    up / gate / down: uint8 device tensors holding E packed matrices back to
    back; shared_*: packed matrices in format `shared_fmt` ("bf16" or "q8")
    or None; codebook: int8 device tensor [256*8] or None; router: fp32
    device tensor [E, H]."""

    def __init__(self, n_experts, hidden, inter, shared_inter, fmts, up, gate, down, codebook=None,
                 shared_up=None, shared_gate=None, shared_down=None, router=None, bias=None,
                 shared_fmt="bf16"):
        self.tensors = dict(up=up, gate=gate, down=down, codebook=codebook, shared_up=shared_up,
                            shared_gate=shared_gate, shared_down=shared_down, router=router, bias=bias)
        self.router = router
        self.bias = bias
        self.n_experts, self.hidden, self.inter, self.shared_inter = n_experts, hidden, inter, shared_inter
        E, H, I, Is = n_experts, hidden, inter, shared_inter
        nb_up, nb_dn = moe_packed_bytes(fmts[0], I, H), moe_packed_bytes(fmts[2], H, I)
        u8 = torch.uint8
        shared = Is > 0
        sf = FMT[shared_fmt]
        self.w = MoeWeights(E, H, I, Is, FMT[fmts[0]], FMT[fmts[1]], FMT[fmts[2]], sf,
                            _dev(up, "up", u8, E * nb_up), _dev(gate, "gate", u8, E * nb_up),
                            _dev(down, "down", u8, E * nb_dn),
                            _dev(codebook, "codebook", torch.int8, 256 * 8, optional=True),
                            _dev(shared_up, "shared_up", u8, moe_packed_bytes(sf, Is, H) if shared else 0,
                                 optional=not shared),
                            _dev(shared_gate, "shared_gate", u8, moe_packed_bytes(sf, Is, H) if shared else 0,
                                 optional=not shared),
                            _dev(shared_down, "shared_down", u8, moe_packed_bytes(sf, H, Is) if shared else 0,
                                 optional=not shared))
        _dev(router, "router", torch.float32, E * H, optional=True)
        _dev(bias, "bias", torch.float32, E, optional=True)


# ---------------------------------------------------------------------------
# Expert streaming: an HBM cache of n_slots experts over a layer whose routed
# experts stay in host memory.


def _host(a, name, nbytes):
    """Address of a host buffer (numpy array or CPU tensor, page-locked for
    asynchronous copies) of at least `nbytes` bytes."""
    if isinstance(a, torch.Tensor):
        if a.is_cuda or not a.is_contiguous():
            raise ValueError(f"{name} must be a contiguous host tensor")
        if a.numel() * a.element_size() < nbytes:
            raise ValueError(f"{name} holds fewer than {nbytes} bytes")
        return a.data_ptr()
    a = np.asarray(a)
    if not a.flags.c_contiguous or a.nbytes < nbytes:
        raise ValueError(f"{name} must be a contiguous host array of at least {nbytes} bytes")
    return a.ctypes.data


class ExpertCache:
    """moe_expert_cache over a layer whose up/gate/down are host buffers
    (`host_up`, `host_gate`, `host_down`: E packed experts each) and whose
    shared expert and codebook come from the device layer `shared_from`
    (a DeviceLayer, or None).  `slot_mem`: uint8 device tensor of at least
    moe_expert_cache_slot_bytes bytes (allocated here when None)."""

    def __init__(self, n_experts, hidden, inter, fmts, host_up, host_gate, host_down, n_slots, keep=0,
                 shared_from=None, slot_mem=None):
        E, H, I = n_experts, hidden, inter
        nb_up, nb_dn = moe_packed_bytes(fmts[0], I, H), moe_packed_bytes(fmts[2], H, I)
        self._keep_alive = [host_up, host_gate, host_down, shared_from]
        sw = shared_from.w if shared_from is not None else None
        self.host_w = MoeWeights(E, H, I, sw.shared_inter if sw else 0, FMT[fmts[0]], FMT[fmts[1]], FMT[fmts[2]],
                                 sw.fmt_shared if sw else 0,
                                 _host(host_up, "host_up", E * nb_up), _host(host_gate, "host_gate", E * nb_up),
                                 _host(host_down, "host_down", E * nb_dn),
                                 sw.codebook if sw else None, sw.shared_up if sw else None,
                                 sw.shared_gate if sw else None, sw.shared_down if sw else None)
        need = int(lib.moe_expert_cache_slot_bytes(ctypes.byref(self.host_w), n_slots))
        if need == 0:
            raise QmoeError(MOE_ERR_INVALID_ARG, "bad layer or n_slots")
        if slot_mem is None:
            slot_mem = torch.empty(need, dtype=torch.uint8, device="cuda")
        self.slot_mem = slot_mem
        self.ptr = ctypes.c_void_p()
        _check(lib.moe_expert_cache_create(ctypes.byref(self.host_w), n_slots, keep,
                                           _dev(slot_mem, "slot_mem", torch.uint8, need), slot_mem.numel(),
                                           ctypes.byref(self.ptr)))
        self.n_slots, self.n_experts, self.hidden = n_slots, E, H
        self.w = MoeWeights()
        _check(lib.moe_expert_cache_weights(self.ptr, ctypes.byref(self.w)))

    def plan(self, ids):
        ids = np.ascontiguousarray(ids, dtype=np.int32).reshape(-1)
        slots = np.empty(ids.size, np.int32)
        me = np.empty(max(ids.size, 1), np.int32)
        ms = np.empty(max(ids.size, 1), np.int32)
        nm = ctypes.c_int32(0)
        _check(lib.moe_expert_cache_plan(self.ptr, ids.ctypes.data, ids.size, slots.ctypes.data, me.ctypes.data,
                                         ms.ctypes.data, ctypes.byref(nm)))
        return slots, me[:nm.value].copy(), ms[:nm.value].copy()

    def fetch(self, miss_experts, miss_slots, stream=None):
        me = np.ascontiguousarray(miss_experts, dtype=np.int32)
        ms = np.ascontiguousarray(miss_slots, dtype=np.int32)
        _check(lib.moe_expert_cache_fetch(self.ptr, me.ctypes.data, ms.ctypes.data, me.size, _stream(stream)))

    def state(self):
        eos = np.empty(self.n_slots, np.int32)
        h, m = ctypes.c_int64(0), ctypes.c_int64(0)
        _check(lib.moe_expert_cache_state(self.ptr, eos.ctypes.data, ctypes.byref(h), ctypes.byref(m)))
        return eos, h.value, m.value

    def decode_workspace_bytes(self, T, k):
        return int(lib.moe_layer_decode_streamed_workspace_bytes(self.ptr, T, k))

    def decode(self, w_router, logit_bias, x_bf16, T, k, topk_idx, topk_w, y, ws, stream=None, copy_stream=None):
        H = self.hidden
        _check(lib.moe_layer_decode_streamed(
            self.ptr, _dev(w_router, "w_router", torch.float32, self.n_experts * H),
            _dev(logit_bias, "logit_bias", torch.float32, self.n_experts, optional=True),
            _dev(x_bf16, "x_bf16", torch.bfloat16, T * H), T, k,
            _dev(topk_idx, "topk_idx", torch.int32, T * k), _dev(topk_w, "topk_w", torch.float32, T * k),
            _dev(y, "y", torch.float32, T * H), *_ws(ws), _stream(stream),
            None if copy_stream is None else _stream(copy_stream)))

    def close(self):
        if self.ptr:
            lib.moe_expert_cache_destroy(self.ptr)
            self.ptr = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---------------------------------------------------------------------------
# Attention (include/qmoe_attn.h).


_DTYPE = {torch.bfloat16: MOE_DT_BF16, torch.float16: MOE_DT_F16}

if not isinstance(_attn, _NotBuilt):
    _attn.use(*(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value
                for f in ("moe_kv_append", "moe_kv_read", "moe_attn_decode", "moe_attn_prefill")))

# index of the current device, where the library launches, and its current
# stream's address: by torch's short ways, where it has them
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _here(t, name, dev):
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on the current device")


def _look_rows(t, name, heads, dim, n, dtype, dev):
    """Raises unless t is a row tensor [>= n, heads, dim] of `dtype` on device `dev`, its heads back to back."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in _DTYPE or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype if dtype in _DTYPE else 'torch.bfloat16 or torch.float16'}, not {t.dtype}")
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dim or t.shape[0] < n:
        raise ValueError(f"{name} has shape {tuple(t.shape)}; the call needs [{n}, {heads}, {dim}]")
    _here(t, name, dev)
    if t.layout != torch.strided or t.stride(2) != 1 or (t.stride(1) != dim and heads != 1):
        raise ValueError(f"{name}'s heads must lie back to back")


def _look_vec(t, name, dtype, n, dev, optional=False):
    """Raises unless t is a contiguous tensor of at least n elements of `dtype` on device `dev`."""
    if _dev(t, name, dtype, n, optional) is not None:
        _here(t, name, dev)


def _refused(rc, rows, vecs=()):
    """Raises what is wrong with a call: the library's error, or the tensor that is not what the call needs."""
    if rc > 0:
        _check(rc)
    for r in rows:
        _look_rows(*r)
    for v in vecs:
        _look_vec(*v)
    raise ValueError("an argument is out of range")


def _heads(t):
    return t.shape[1] if isinstance(t, torch.Tensor) and t.dim() == 3 else 0


def _stream_on(stream, dev):
    return _current_stream(dev) if stream is None else _stream(stream)


def moe_kv_code_bytes(n_pages: int, page_tokens: int, kv_heads: int, head_dim: int) -> int:
    return int(lib.moe_kv_code_bytes(n_pages, page_tokens, kv_heads, head_dim))


def moe_kv_scale_bytes(n_pages: int, page_tokens: int, kv_heads: int) -> int:
    return int(lib.moe_kv_scale_bytes(n_pages, page_tokens, kv_heads))


def moe_rope_freqs(rot_dim, base=10000.0, rule="plain", factor=1.0, trained=0.0, slow=1.0, fast=32.0) -> np.ndarray:
    """Radians a position of each pair, fp64 [rot_dim/2] (host)."""
    out = np.empty(max(int(rot_dim) // 2, 1), np.float64)
    _check(lib.moe_rope_freqs(rot_dim, base, MOE_ROPE.get(rule, rule), factor, trained, slow, fast, out.ctypes.data))
    return out


class KvCache:
    """A paged 8-bit cache (struct moe_kv_cache) over the caller's `codes` and
    `scales` tensors (uint8 and fp32, any shape, contiguous), or over new ones
    where they are None (n_pages is then required)."""

    def __init__(self, codes, scales, page_tokens, kv_heads, head_dim, n_pages=None):
        if n_pages is None:
            per = moe_kv_code_bytes(1, page_tokens, kv_heads, head_dim)
            if codes is None or per == 0:
                raise ValueError("n_pages is required without codes; page_tokens, kv_heads, head_dim must be valid")
            n_pages = codes.numel() // per
        nc, ns = moe_kv_code_bytes(n_pages, page_tokens, kv_heads, head_dim), moe_kv_scale_bytes(n_pages, page_tokens, kv_heads)
        if nc == 0:
            raise ValueError("bad cache geometry")
        if codes is None:
            codes = torch.empty(nc, dtype=torch.uint8, device="cuda")
        if scales is None:
            scales = torch.empty(ns // 4, dtype=torch.float32, device="cuda")
        self.codes, self.scales = codes, scales
        self.n_pages, self.page_tokens, self.kv_heads, self.head_dim = n_pages, page_tokens, kv_heads, head_dim
        self.c = MoeKvCache(n_pages, page_tokens, kv_heads, head_dim, _dev(codes, "codes", torch.uint8, nc),
                            _dev(scales, "scales", torch.float32, ns // 4))
        self.device = codes.get_device()
        _here(scales, "scales", self.device)
        self.ref, self.at = ctypes.byref(self.c), ctypes.addressof(self.c)


class KvBatch:
    """A step's sequences (struct moe_kv_batch): page_table int32 [batch, pages] (rows may be strided), kv_lens
    int32 [batch], `rows` new rows in all, at most `max_new` of one sequence; cu_rows int32 [batch+1] or None (the
    same number each)."""

    def __init__(self, page_table, kv_lens, rows, max_new=None, cu_rows=None):
        if not isinstance(page_table, torch.Tensor) or not page_table.is_cuda or page_table.dim() != 2 or page_table.dtype != torch.int32:
            raise ValueError("page_table must be a 2-dimensional int32 CUDA tensor")
        batch, pages = page_table.shape
        if page_table.stride(1) != 1 and pages > 1:
            raise ValueError("page_table's rows must be contiguous")
        if max_new is None:
            if cu_rows is not None or batch == 0:
                raise ValueError("max_new is required with cu_rows")
            max_new = rows // batch
        self.tensors = (page_table, kv_lens, cu_rows)
        self.batch, self.rows = batch, rows
        self.c = MoeKvBatch(batch, rows, max_new, pages, page_table.data_ptr(),
                            page_table.stride(0) if batch > 1 else max(page_table.stride(0), pages),
                            _dev(kv_lens, "kv_lens", torch.int32, batch),
                            _dev(cu_rows, "cu_rows", torch.int32, batch + 1, optional=True))
        self.device = page_table.get_device()
        for t, name in ((kv_lens, "kv_lens"), (cu_rows, "cu_rows")):
            if t is not None:
                _here(t, name, self.device)
        self.ref, self.at = ctypes.byref(self.c), ctypes.addressof(self.c)


class Rope:
    """Rotary positions (struct moe_rope): freqs fp64 CUDA [rot_dim/2] (moe_rope_freqs)."""

    def __init__(self, freqs, rot_dim, interleaved=False, scale=1.0):
        self.freqs = freqs
        self.c = MoeRope(rot_dim, int(bool(interleaved)), scale,
                         _dev(freqs, "freqs", torch.float64, rot_dim // 2, optional=rot_dim == 0))
        self.device = None if freqs is None else freqs.get_device()
        self.ref, self.at = ctypes.byref(self.c), ctypes.addressof(self.c)


def _step(cache, batch):
    """The current device, which must be the cache's and the batch's."""
    dev = _device()
    if cache.device != dev or batch.device != dev:
        raise ValueError(f"the cache is on device {cache.device}, the batch on {batch.device}, the current one is {dev}")
    return dev


def moe_kv_append(cache, batch, k, v, rope=None, q=None, q_out=None, k_out=None, stream=None):
    """k, v (and q) [rows, heads, head_dim], any row stride; q turned into q_out (may be q), k_out (may be k or None)."""
    H, D, n = cache.kv_heads, cache.head_dim, batch.rows
    dev = _step(cache, batch)
    if rope is not None and rope.device not in (None, dev):
        raise ValueError(f"rope is on device {rope.device}, the current one is {dev}")
    if q is None and q_out is not None:
        raise ValueError("q_out without q")
    rc = _attn.append(cache.at, batch.at, 0 if rope is None else rope.at, H, D, n, dev, _stream_on(stream, dev), k, v, q, q_out,
                      k_out)
    if rc:
        dt, hq = getattr(k, "dtype", None), _heads(q)
        _refused(rc, [(k, "k", H, D, n, dt, dev), (v, "v", H, D, n, dt, dev)] +
                 ([] if q is None else [(q, "q", hq, D, n, dt, dev), (q_out, "q_out", hq, D, n, dt, dev)]) +
                 ([] if k_out is None else [(k_out, "k_out", H, D, n, dt, dev)]))


def moe_kv_read(cache, batch, k_out, v_out, stream=None):
    """Rows of the batch's last positions into k_out, v_out [rows, kv_heads, head_dim]."""
    H, D, n = cache.kv_heads, cache.head_dim, batch.rows
    dev = _step(cache, batch)
    rc = _attn.read(cache.at, batch.at, H, D, n, dev, _stream_on(stream, dev), k_out, v_out)
    if rc:
        dt = getattr(k_out, "dtype", None)
        _refused(rc, [(k_out, "k_out", H, D, n, dt, dev), (v_out, "v_out", H, D, n, dt, dev)])


def moe_attn_decode_workspace_bytes(cache, batch, q_heads: int) -> int:
    return int(lib.moe_attn_decode_workspace_bytes(cache.ref, batch.ref, q_heads))


def moe_attn_decode(cache, batch, q, out, ws, scale, lse=None, stream=None):
    """q, out [rows, q_heads, head_dim]; lse fp32 [rows, q_heads] or None."""
    D, n = cache.head_dim, batch.rows
    dev = _step(cache, batch)
    rc = _attn.decode(cache.at, batch.at, D, n, dev, _stream_on(stream, dev), q, out, ws, scale, lse)
    if rc:
        dt, hq = getattr(q, "dtype", None), _heads(q)
        _refused(rc, [(q, "q", hq, D, n, dt, dev), (out, "out", hq, D, n, dt, dev)],
                 [(ws, "ws", torch.uint8, 0, dev), (lse, "lse", torch.float32, n * hq, dev, True)])


def moe_attn_prefill_workspace_bytes(rows_q: int, batch: int, max_q: int, rows_k: int, q_heads: int, kv_heads: int,
                                     head_dim: int) -> int:
    # (which rows belong to which sequence does not matter here: any offsets stand for them)
    p = MoePacked(batch, rows_q, rows_k, max_q, 16, 16, q_heads, kv_heads, head_dim)
    return int(lib.moe_attn_prefill_workspace_bytes(ctypes.byref(p)))


def moe_attn_prefill(q, k, v, cu_q, cu_k, max_q, out, ws, scale, causal=True, lse=None, stream=None):
    """q, out [rows_q, q_heads, head_dim]; k, v [rows_k, kv_heads, head_dim]; cu_q, cu_k int32 [batch+1]."""
    if not getattr(q, "is_cuda", False):
        raise ValueError("q must be a CUDA tensor")
    dev = _device()
    rc = _attn.prefill(dev, _stream_on(stream, dev), q, k, v, cu_q, cu_k, max_q, out, ws, scale, causal, lse)
    if rc:
        if rc < 0 and any(not isinstance(t, torch.Tensor) or t.dim() != 3 for t in (q, k)):
            raise ValueError("q and k must be CUDA tensors [rows, heads, head_dim]")
        dt, (nq, hq, D), (nk, hk, _) = q.dtype, q.shape, k.shape
        _refused(rc, [(q, "q", hq, D, nq, dt, dev), (k, "k", hk, D, nk, dt, dev), (v, "v", hk, D, nk, dt, dev),
                      (out, "out", hq, D, nq, dt, dev)],
                 [(cu_q, "cu_q", torch.int32, 2, dev), (cu_k, "cu_k", torch.int32, getattr(cu_q, "numel", int)(), dev),
                  (ws, "ws", torch.uint8, 0, dev), (lse, "lse", torch.float32, nq * hq, dev, True)])



# ---------------------------------------------------------------------------
# Norm, 4-bit products, pages of a cache (include/qmoe_step.h).


if not isinstance(_attn, _NotBuilt):
    _attn.step_use(*(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value
                     for f in ("moe_rms_norm", "moe_linear", "moe_kv_resize", "moe_kv_fork", "moe_kv_compact")))

_NORM_TYPES = (torch.bfloat16, torch.float16, torch.float32)


def _look_vectors(t, name, shape, types, dev):
    """Raises unless t is a tensor of vectors of this shape, a row's values back to back, on device `dev`."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in types:
        raise ValueError(f"{name} must be {' or '.join(str(x) for x in types)}, not {t.dtype}")
    if t.dim() not in (2, 3) or (shape is not None and tuple(t.shape) != tuple(shape)):
        raise ValueError(f"{name} has shape {tuple(t.shape)}; the call needs {'[rows, cols] or [rows, heads, cols]' if shape is None else list(shape)}")
    _here(t, name, dev)
    if t.layout != torch.strided or t.stride(-1) != 1 or (t.dim() == 3 and t.shape[1] != 1 and t.stride(1) != t.shape[2]):
        raise ValueError(f"{name}'s rows must be contiguous")


def _look_scales(t, name, groups, rows, dev):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.float32:
        raise ValueError(f"{name} must be a torch.float32 CUDA tensor")
    _here(t, name, dev)
    if t.dim() != 2 or t.shape[0] != groups or t.shape[1] < rows or t.stride(1) != 1:
        raise ValueError(f"{name} has shape {tuple(t.shape)}; the call needs [{groups}, at least {rows}], rows of it contiguous")


def moe_scales_shape(rows: int, cols: int, group: int = 0, heads: int = 1):
    """Shape of the scales of 8-bit rows: [groups of a row, rows (a multiple of 4)]."""
    return heads * (-(-cols // group) if group else 1), max(-(-rows // 4) * 4, 4)


def moe_rms_norm(x, out=None, weight=None, eps=1e-6, residual=None, sum_out=None, codes=None, scales=None, group=0, stream=None):
    """x [rows, cols] or [rows, heads, cols] (+ residual, whose sum with x goes to sum_out), normed into out and/or into
    int8 codes with fp32 scales (moe_scales_shape)."""
    dev = _device()
    rc = _attn.norm(dev, _stream_on(stream, dev), x, out, weight, eps, residual, sum_out, codes, scales, group)
    if rc:
        looks = []
        if rc < 0:
            _look_vectors(x, "x", None, _NORM_TYPES, dev)
            for t, name, types in ((out, "out", _NORM_TYPES), (residual, "residual", _NORM_TYPES),
                                   (sum_out, "sum_out", (getattr(residual, "dtype", None),)), (codes, "codes", (torch.int8,))):
                if t is not None:
                    _look_vectors(t, name, x.shape, types, dev)
            if weight is not None:
                if not isinstance(weight, torch.Tensor) or weight.dtype not in _NORM_TYPES or weight.dim() != 1:
                    raise ValueError("weight must be a 1-dimensional CUDA tensor of 16 or 32 bits")
                looks.append((weight, "weight", weight.dtype, x.shape[-1], dev))
                if weight.numel() != x.shape[-1]:
                    raise ValueError(f"weight holds {weight.numel()} elements; the call needs {x.shape[-1]}")
            if scales is not None and group >= 0:
                _look_scales(scales, "scales", moe_scales_shape(x.shape[0], x.shape[-1], group, x.shape[1] if x.dim() == 3 else 1)[0],
                             x.shape[0], dev)
        _refused(rc, [], looks)


def moe_linear_packed_bytes(n: int, k: int, group: int, with_zeros: bool) -> int:
    return int(lib.moe_linear_packed_bytes(n, k, group, int(bool(with_zeros))))


def moe_linear_quantize(w: np.ndarray, group: int = 128, with_zeros: bool = False, n_threads: int = 0):
    """fp32 host matrix [n, k] -> (codes uint8 [n, k], scales fp16 [n, groups], zero points uint8 [n, groups] or None)."""
    w = np.ascontiguousarray(w, dtype=np.float32)
    n, k = w.shape
    groups = -(-k // group) if group > 0 else 1
    codes, scales = np.empty((n, k), np.uint8), np.empty((n, groups), np.float16)
    zeros = np.empty((n, groups), np.uint8) if with_zeros else None
    _check(lib.moe_linear_quantize(w.ctypes.data, n, k, group, codes.ctypes.data, scales.ctypes.data,
                                   None if zeros is None else zeros.ctypes.data, n_threads))
    return codes, scales, zeros


def _small(a, name):
    """a as contiguous uint8; raises for values that these do not hold (the library refuses the rest of what it must)."""
    a = np.asarray(a)
    b = a if a.dtype == np.uint8 else np.clip(a, 0, 255).astype(np.uint8) if a.dtype.kind in "iuf" and not np.isnan(a).any() else None
    if b is None or (b is not a and not np.array_equal(a, b)):
        raise ValueError(f"{name} must be whole numbers of 0 to 15")
    return np.ascontiguousarray(b)


def moe_linear_pack(codes: np.ndarray, scales: np.ndarray, zeros: np.ndarray | None = None, group: int = 128,
                    n_threads: int = 0) -> np.ndarray:
    """Codes, scales (rounded to fp16) and zero points (host) -> packed uint8 bytes (host)."""
    codes = _small(codes, "codes")
    if codes.ndim != 2:
        raise ValueError("codes must be [n, k]")
    n, k = codes.shape
    groups = (n, -(-k // group) if group > 0 else 1)
    scales = np.ascontiguousarray(scales, dtype=np.float16)
    zeros = None if zeros is None else _small(zeros, "zeros")
    if scales.shape != groups or (zeros is not None and zeros.shape != groups):
        raise ValueError(f"scales and zeros must be {list(groups)}")
    out = np.empty(max(moe_linear_packed_bytes(n, k, group, zeros is not None), 1), np.uint8)
    _check(lib.moe_linear_pack(codes.ctypes.data, scales.ctypes.data, None if zeros is None else zeros.ctypes.data, n, k, group,
                               out.ctypes.data, out.nbytes, n_threads))
    return out


class LinearWeights:
    """A packed 4-bit matrix [n, k] in device memory (struct moe_linear_weights): `packed` uint8 CUDA (moe_linear_pack),
    bias fp32 CUDA [n] or None."""

    def __init__(self, packed, n, k, group=128, with_zeros=False, bias=None):
        need = moe_linear_packed_bytes(n, k, group, with_zeros)
        if need == 0:
            raise ValueError("n must be in [1, 2^24], k a multiple of 8 in [8, 2^20], group 32, 64 or 128")
        self.tensors = (packed, bias)
        self.n, self.k = n, k
        self.c = MoeLinearWeights(n, k, group, int(bool(with_zeros)), _dev(packed, "packed", torch.uint8, need),
                                  _dev(bias, "bias", torch.float32, n, optional=True))
        self.device = packed.get_device()
        if bias is not None:
            _here(bias, "bias", self.device)
        self.at = ctypes.addressof(self.c)


def moe_linear(w, x, y, x_scales=None, x_group=0, stream=None):
    """y [rows, n] = x [rows, k] times the weights' transpose; x 16-bit, or int8 codes with x_scales (moe_scales_shape).
    Rows may also be [rows, heads, dim] with heads * dim columns."""
    dev = _device()
    if w.device != dev:
        raise ValueError(f"the weights are on device {w.device}, the current one is {dev}")
    rc = _attn.linear(w.at, w.n, w.k, dev, _stream_on(stream, dev), x, y, x_scales, x_group)
    if rc:
        if rc < 0:
            _look_vectors(x, "x", None, (torch.bfloat16, torch.float16, torch.int8), dev)
            _look_vectors(y, "y", None, _NORM_TYPES, dev)
            for t, name, cols in ((x, "x", w.k), (y, "y", w.n)):
                if t.shape[1:].numel() != cols or t.shape[0] != x.shape[0]:
                    raise ValueError(f"{name} has shape {tuple(t.shape)}; the call needs [{x.shape[0]}, {cols}]")
            if x_scales is not None and x_group >= 0:
                groups, most = moe_scales_shape(x.shape[0], w.k, x_group)
                _look_scales(x_scales, "x_scales", groups, x.shape[0], dev)
                if x_group and x_scales.storage_offset() + (groups - 1) * x_scales.stride(0) + most > x_scales.untyped_storage().nbytes() // 4:
                    raise ValueError(f"x_scales' last group must have room for {most} rows")
        _refused(rc, [])


class KvPool:
    """The pages of one or more caches of the same n_pages and page_tokens (struct moe_kv_pool): refs int32 CUDA
    [n_pages], how many table entries name each page (zeros: all free)."""

    def __init__(self, refs, caches=()):
        self.caches, self.refs = list(caches), refs
        array = (MoeKvCache * max(len(self.caches), 1))(*(c.c for c in self.caches))
        self.c = MoeKvPool(refs.numel() if isinstance(refs, torch.Tensor) else 0, len(self.caches), array,
                           _dev(refs, "refs", torch.int32, 1))
        self.device = refs.get_device()
        for c in self.caches:
            _here(c.codes, "a cache", self.device)
        self._array = array
        self.ref, self.at = ctypes.byref(self.c), ctypes.addressof(self.c)


class KvTables:
    """Rows of a page table (struct moe_kv_tables): page_table int32 CUDA [seqs, pages] (rows may be strided), kv_lens
    int32 CUDA [seqs]; the tensors of KvBatch."""

    def __init__(self, page_table, kv_lens, page_tokens):
        if not isinstance(page_table, torch.Tensor) or not page_table.is_cuda or page_table.dim() != 2 or page_table.dtype != torch.int32:
            raise ValueError("page_table must be a 2-dimensional int32 CUDA tensor")
        seqs, pages = page_table.shape
        if page_table.stride(1) != 1 and pages > 1:
            raise ValueError("page_table's rows must be contiguous")
        self.tensors = (page_table, kv_lens)
        self.seqs = seqs
        self.c = MoeKvTables(seqs, pages, page_tokens, page_table.data_ptr(),
                             page_table.stride(0) if seqs > 1 else max(page_table.stride(0), pages),
                             _dev(kv_lens, "kv_lens", torch.int32, seqs))
        self.device = page_table.get_device()
        _here(kv_lens, "kv_lens", self.device)
        self.ref, self.at = ctypes.byref(self.c), ctypes.addressof(self.c)


def _pages(pool, tables):
    """The current device, which must be the pool's and the tables'."""
    dev = _device()
    if pool.device != dev or tables.device != dev:
        raise ValueError(f"the pool is on device {pool.device}, the tables on {tables.device}, the current one is {dev}")
    return dev


def moe_kv_resize(pool, tables, new_lens, missing=None, stream=None):
    """new_lens int32 [seqs] (negative: left alone); missing int32 [1] or None."""
    dev = _pages(pool, tables)
    rc = _attn.resize(pool.at, tables.at, tables.seqs, dev, _stream_on(stream, dev), new_lens, missing)
    if rc:
        _refused(rc, [], [(new_lens, "new_lens", torch.int32, tables.seqs, dev), (missing, "missing", torch.int32, 1, dev, True)])


def moe_kv_fork_workspace_bytes(pool, tables) -> int:
    return int(lib.moe_kv_fork_workspace_bytes(pool.ref, tables.ref))


def moe_kv_fork(pool, tables, from_rows, ws, missing=None, stream=None):
    """from_rows int32 [seqs]: the row that each row goes on from (negative: left alone)."""
    dev = _pages(pool, tables)
    rc = _attn.fork(pool.at, tables.at, tables.seqs, dev, _stream_on(stream, dev), from_rows, missing, ws)
    if rc:
        _refused(rc, [], [(from_rows, "from_rows", torch.int32, tables.seqs, dev), (missing, "missing", torch.int32, 1, dev, True),
                          (ws, "ws", torch.uint8, 0, dev)])


def moe_kv_compact_workspace_bytes(pool, tables) -> int:
    return int(lib.moe_kv_compact_workspace_bytes(pool.ref, tables.ref))


def moe_kv_compact(pool, tables, ws, held=None, stream=None):
    """held int32 [1] or None: the number of pages held, which are then the pool's first ones."""
    dev = _pages(pool, tables)
    rc = _attn.compact(pool.at, tables.at, dev, _stream_on(stream, dev), held, ws)
    if rc:
        _refused(rc, [], [(held, "held", torch.int32, 1, dev, True), (ws, "ws", torch.uint8, 0, dev)])
