"""ctypes binding of libpeagle.so (include/peagle*.h): argument marshalling only.

Every step of the drafting path runs in the library's CUDA kernels; PyTorch
is used here for device memory and streams.  Importing this module does not
need a GPU, but calling into the library does; if the library has not been
built the import fails loudly (there is no fallback path).
"""

from __future__ import annotations

import ctypes
import os
import threading
from typing import Dict, List, Optional, Sequence

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libpeagle.so")

PE_OK = 0
PE_ERR_INVALID_ARGUMENT = 1
PE_ERR_UNSUPPORTED = 2
PE_ERR_CUDA = 3
PE_ERR_OUT_OF_MEMORY = 4
PE_ERR_DEVICE = 5
PE_DTYPE_BF16 = 0
PE_DTYPE_F32 = 1

PE_MASK_BOOL_U8 = 0
PE_MASK_ADDITIVE_BF16 = 1

PE_KV_BF16 = 0
PE_KV_F32 = 1
PE_KV_E4M3 = 2

PE_DEV_BAD_BLOCK = 2
PE_DEV_BAD_POSITION = 3
PE_DEV_BAD_TOKEN = 4
PE_DEV_BAD_ROW = 6

# include/peagle.h and include/peagle_train.h (pe_status_string last: it is
# the one that does not return a pe_status)
EXPORTED = ("pe_create", "pe_destroy", "pe_expand_batch", "pe_draft_forward",
            "pe_lmhead_argmax", "pe_get_device_error", "pe_set_trace", "pe_set_phase_events",
            "pe_set_small_batch_stream", "pe_set_stream_prefetch", "pe_set_stream_timeline",
            "pe_set_fusions", "pe_set_split_reduce", "pe_set_tuning", "pe_set_gemm_timeline",
            "pe_linear",
            "pe_get_launch_count", "pe_check_bounded_wait", "pe_linear_static",
            "pe_linear_static_error",
            "pe_set_kv_cache_fp8",
            "pe_train_build_mask",
            "pe_train_mask_view", "pe_train_partition", "pe_status_string")

# include/peagle_cache.h
CACHE_EXPORTED = ("pe_kv_append", "pe_attn_decode_workspace", "pe_attn_decode", "pe_kv_evict",
                  "pe_set_kv_scores")

# include/peagle_w4.h and include/peagle_sample.h
HEAD_EXPORTED = ("pe_w4_bytes", "pe_w4_pack", "pe_w4_quantize", "pe_w4_linear", "pe_sample",
                 "pe_verify")

_vp = ctypes.c_void_p
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64


class pe_model_desc(ctypes.Structure):
    _fields_ = [("d", _i32), ("n_layers", _i32), ("n_heads", _i32), ("n_kv_heads", _i32),
                ("head_dim", _i32), ("ffn", _i32), ("vocab", _i32), ("hidden3", _i32),
                ("page_size", _i32), ("mask_token_id", _i32), ("rope_theta", ctypes.c_float),
                ("rms_eps", ctypes.c_float), ("dtype", _i32)]


class pe_layer_weights(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("qkv", "o", "gate", "up", "down", "norm_e", "norm_h",
                                   "norm_in", "norm_post")]


class pe_weights(ctypes.Structure):
    _fields_ = [("emb", _vp), ("fc", _vp), ("h_shared", _vp), ("norm_final", _vp),
                ("lm_head", _vp), ("layers", ctypes.POINTER(pe_layer_weights))]


class pe_expanded(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("ids", "pos", "slot", "is_rejected", "is_masked",
                                   "new_idx", "hidden_map", "cu_out", "seq_lens", "hidden")] + \
               [("B", _i32), ("K", _i32), ("T", _i32), ("T_out", _i32),
                ("target_hidden", _vp)]


class pe_kv_pool(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("scores", _vp), ("num_blocks", _i32),
                ("n_kv_heads", _i32), ("head_dim", _i32), ("dtype", _i32),
                ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


class pe_dist(ctypes.Structure):
    _fields_ = [("max", ctypes.c_float), ("inv", ctypes.c_float), ("cut", ctypes.c_float),
                ("cut_token", _i32), ("total", _i64), ("token", _i32), ("reserved", _i32)]


class PeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {status_string(status)} ({status})")
        self.status = status


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with "
                          "speculative_drafting_expand_gb300.build.build()")
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER
    lib.pe_create.argtypes = [P(pe_model_desc), P(pe_weights), _i32, _i32, P(_vp)]
    lib.pe_destroy.argtypes = [_vp]
    lib.pe_expand_batch.argtypes = [_vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i32,
                                    _i32, _vp, P(pe_expanded), _vp]
    lib.pe_draft_forward.argtypes = [_vp, P(pe_expanded), _i32, _i32, _vp, _i32, P(_vp), P(_vp),
                                     _i32, _vp, _vp]
    lib.pe_lmhead_argmax.argtypes = [_vp, _vp, _i32, _vp, _vp, _vp]
    lib.pe_get_device_error.argtypes = [_vp, P(_i32), _vp]
    lib.pe_set_trace.argtypes = [_vp, _vp, _vp]
    lib.pe_linear.argtypes = [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp]
    lib.pe_get_launch_count.argtypes = [_vp, P(ctypes.c_int64)]
    lib.pe_linear_static.argtypes = [_vp, _vp, _vp, _i32, _i32, _i32, _vp]
    lib.pe_check_bounded_wait.argtypes = [_vp, _vp, _vp]
    lib.pe_set_phase_events.argtypes = [_vp, P(_vp), _i32]
    lib.pe_set_small_batch_stream.argtypes = [_vp, _i32]
    lib.pe_set_stream_timeline.argtypes = [_vp, _vp]
    lib.pe_set_fusions.argtypes = [_vp, _i32]
    lib.pe_set_split_reduce.argtypes = [_vp, _i32]
    lib.pe_set_tuning.argtypes = [_vp, _i32, _i32]
    lib.pe_set_gemm_timeline.argtypes = [_vp, _vp, _i32]
    lib.pe_set_stream_prefetch.argtypes = [_vp, _i32, _i32]
    lib.pe_linear_static_error.argtypes = [P(_i32), _vp]
    lib.pe_set_kv_cache_fp8.argtypes = [_vp, P(ctypes.c_float), P(ctypes.c_float)]
    lib.pe_train_build_mask.argtypes = [_i32, _i32, _i32, _vp, ctypes.c_int64, _vp]
    lib.pe_train_mask_view.argtypes = [_vp, ctypes.c_int64, _i32, _i32, _i32, P(_vp),
                                       P(ctypes.c_int64), P(ctypes.c_int64)]
    lib.pe_train_partition.argtypes = [_i32, _i32, ctypes.c_float, _vp, _i32, P(_i32), _vp, _vp,
                                       _vp, _vp, _vp, _vp, ctypes.c_int64, _vp]
    lib.pe_status_string.argtypes = [_i32]
    lib.pe_status_string.restype = ctypes.c_char_p
    lib.pe_kv_append.argtypes = [P(pe_kv_pool), _i32, _i32, _i32, ctypes.c_float, _vp, _i64, _vp,
                                 _i64, _vp, _i64, _vp, _vp, _vp, _i32, _vp, _i64, _vp, _vp]
    lib.pe_attn_decode_workspace.argtypes = [_i32, _i32, _i32, _i32, _i32]
    lib.pe_attn_decode.argtypes = [P(pe_kv_pool), _i32, _i32, ctypes.c_float, _vp, _i64, _vp,
                                   _i32, _vp, _i32, _vp, _i64, _vp, _i32, _vp, _i64, _vp, _vp]
    lib.pe_set_kv_scores.argtypes = [_vp, P(_vp)]
    lib.pe_kv_evict.argtypes = [_i32, P(pe_kv_pool), _i32, _vp, _i32, _vp, _i32, _i32, _i32,
                                ctypes.c_float, _vp, _i32, _vp, _vp, _vp, _vp]
    lib.pe_w4_bytes.argtypes = [_i32, _i32, _i32]
    lib.pe_w4_pack.argtypes = [_vp, _vp, _i32, _i32, _i32, _vp, _vp]
    lib.pe_w4_quantize.argtypes = [_vp, _i32, _i64, _i32, _i32, _i32, _vp, _vp]
    lib.pe_w4_linear.argtypes = [_vp, _i32, _i32, _i32, _i32, _i32, _vp, _i64, _i32, _vp, _i64,
                                 _vp]
    lib.pe_sample.argtypes = [_i32, _i32, _i32, _vp, _i64] + [_vp] * 9
    lib.pe_verify.argtypes = ([_i32] * 4 + [_vp, _i64] + [_vp] * 9 + [_i64] + [_vp] * 7)
    for name in EXPORTED[:-1] + CACHE_EXPORTED + HEAD_EXPORTED:
        getattr(lib, name).restype = _i32
    lib.pe_attn_decode_workspace.restype = _i64
    lib.pe_w4_bytes.restype = _i64
    return lib


_LIB: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    global _LIB
    if _LIB is None:
        _LIB = load_library()
    return _LIB


def status_string(s: int) -> str:
    return lib().pe_status_string(s).decode()


def _check(fn: str, s: int):
    if s != PE_OK:
        raise PeError(fn, s)


# ---------------------------------------------------------------------------
# tensors
# ---------------------------------------------------------------------------

def _torch():
    import torch
    return torch


def ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def stream_ptr(stream=None) -> int:
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def to_device(a: np.ndarray, dtype: str, device="cuda"):
    """Host array (bf16 bits as uint16, or float32 / int32 / uint8) -> tensor
    (a tensor is moved as it is)."""
    torch = _torch()
    if isinstance(a, torch.Tensor):
        return a.to(device)
    if dtype == "bf16" and a.dtype == np.uint16:
        t = torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(torch.bfloat16)
    else:
        t = torch.from_numpy(np.ascontiguousarray(a))
    return t.to(device)


def to_host(t) -> np.ndarray:
    """Tensor -> host array (bf16 as uint16 bits)."""
    torch = _torch()
    t = t.detach().cpu().contiguous()
    if t.dtype == torch.bfloat16:
        return t.view(torch.int16).numpy().view(np.uint16)
    return t.numpy()


def model_desc(shape) -> pe_model_desc:
    return pe_model_desc(shape.d, shape.n_layers, shape.n_heads, shape.n_kv_heads,
                         shape.head_dim, shape.ffn, shape.vocab, shape.hidden3,
                         shape.page_size, shape.mask_token_id, shape.rope_theta,
                         shape.rms_eps, PE_DTYPE_BF16 if shape.dtype == "bf16" else PE_DTYPE_F32)


class Drafter:
    """Owns the device copies of the weights and a pe_handle."""

    def __init__(self, shape, host_weights: Dict, max_tokens: int, max_reqs: int,
                 device="cuda"):
        self.shape = shape
        self.device = device
        dt = shape.dtype
        W = host_weights
        self.w = {k: to_device(W[k], dt, device) for k in
                  ("emb", "fc", "h_shared", "norm_final", "lm_head")}
        self.layers = [{k: to_device(v, dt, device) for k, v in lw.items()}
                       for lw in W["layers"]]
        arr = (pe_layer_weights * shape.n_layers)()
        for l, lw in enumerate(self.layers):
            arr[l] = pe_layer_weights(*(ptr(lw.get(f[0])) for f in pe_layer_weights._fields_))
        self._layer_arr = arr
        self._weights = pe_weights(ptr(self.w["emb"]), ptr(self.w["fc"]),
                                   ptr(self.w["h_shared"]), ptr(self.w["norm_final"]),
                                   ptr(self.w["lm_head"]), arr)
        self._desc = model_desc(shape)
        h = _vp()
        _check("pe_create", lib().pe_create(ctypes.byref(self._desc), ctypes.byref(self._weights),
                                            max_tokens, max_reqs, ctypes.byref(h)))
        self.handle = h
        self.max_tokens = max_tokens

    def close(self):
        if getattr(self, "handle", None):
            lib().pe_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---------------------------------------------------------------------------
# the entry points, same names as the C ABI
# ---------------------------------------------------------------------------

class Expanded:
    """Caller-owned device buffers of one expanded batch (pe_expanded)."""

    def __init__(self, T_out: int, T: int, B: int, K: int, hidden3: int, dtype: str,
                 device="cuda"):
        torch = _torch()
        i32 = dict(dtype=torch.int32, device=device)
        self.ids = torch.empty(T_out, **i32)
        self.pos = torch.empty(T_out, **i32)
        self.slot = torch.empty(T_out, **i32)
        self.is_rejected = torch.empty(T_out, dtype=torch.uint8, device=device)
        self.is_masked = torch.empty(T_out, dtype=torch.uint8, device=device)
        self.new_idx = torch.empty(B * K, **i32)
        self.hidden_map = torch.empty(T, **i32)
        self.cu_out = torch.empty(B + 1, **i32)
        self.seq_lens = torch.empty(B, **i32)
        tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.hidden = torch.empty(T_out, hidden3, dtype=tdt, device=device)
        self.struct = pe_expanded(*(ptr(getattr(self, f)) for f in
                                    ("ids", "pos", "slot", "is_rejected", "is_masked",
                                     "new_idx", "hidden_map", "cu_out", "seq_lens", "hidden")),
                                  0, 0, 0, 0, None)


def pe_expand_batch(dr: Drafter, K: int, target_ids, target_pos, cu_in, num_accepted,
                    sampled_ids, block_table, num_blocks: int, target_hidden,
                    out: Expanded, stream=None):
    B = num_accepted.shape[0]
    T = target_ids.shape[0]
    _check("pe_expand_batch", lib().pe_expand_batch(
        dr.handle, B, K, T, ptr(target_ids), ptr(target_pos), ptr(cu_in), ptr(num_accepted),
        ptr(sampled_ids), ptr(block_table), block_table.shape[1], num_blocks,
        ptr(target_hidden), ctypes.byref(out.struct), stream_ptr(stream)))
    return out


def pe_draft_forward(dr: Drafter, ex: Expanded, block_table, k_cache: Sequence,
                     v_cache: Sequence, num_blocks: int, out_hidden, stream=None):
    L = len(k_cache)
    if any(t.shape[0] < num_blocks for t in getattr(dr, "_kv_scores", None) or ()):
        raise ValueError("the scores of pe_set_kv_scores hold fewer blocks than the pools")
    kc = (_vp * L)(*[ptr(t) for t in k_cache])
    vc = (_vp * L)(*[ptr(t) for t in v_cache])
    _check("pe_draft_forward", lib().pe_draft_forward(
        dr.handle, ctypes.byref(ex.struct), ex.struct.B, ex.struct.K, ptr(block_table),
        block_table.shape[1], kc, vc, num_blocks, ptr(out_hidden), stream_ptr(stream)))
    return out_hidden


def pe_lmhead_argmax(dr: Drafter, hidden, out_tokens, out_logits=None, stream=None):
    _check("pe_lmhead_argmax", lib().pe_lmhead_argmax(
        dr.handle, ptr(hidden), hidden.shape[0], ptr(out_tokens), ptr(out_logits),
        stream_ptr(stream)))
    return out_tokens


def pe_get_device_error(dr: Drafter, stream=None) -> int:
    code = _i32(0)
    _check("pe_get_device_error", lib().pe_get_device_error(dr.handle, ctypes.byref(code),
                                                            stream_ptr(stream)))
    return code.value


def pe_check_bounded_wait(dr: Drafter, out, stream=None) -> None:
    """Launch the bounded-wait self-check (out: device int32[2])."""
    _check("pe_check_bounded_wait", lib().pe_check_bounded_wait(dr.handle, ptr(out),
                                                                stream_ptr(stream)))


def pe_set_small_batch_stream(dr: Drafter, enable: bool) -> None:
    _check("pe_set_small_batch_stream", lib().pe_set_small_batch_stream(dr.handle, int(enable)))


PE_FUSE_ROPE_KV = 1
PE_FUSE_NORM = 2
PE_FUSE_ALL = 3


def pe_set_gemm_timeline(dr: Drafter, stamps=None, launches: int = 0) -> None:
    """stamps: int64 device tensor of launches * 512 * 16 entries, or None."""
    _check("pe_set_gemm_timeline",
           lib().pe_set_gemm_timeline(dr.handle, ptr(stamps), int(launches) if stamps is not None else 0))


def pe_set_fusions(dr: Drafter, mask: int) -> None:
    _check("pe_set_fusions", lib().pe_set_fusions(dr.handle, int(mask)))


PE_REDUCE_PULL = 0
PE_REDUCE_PUSH = 1


def pe_set_split_reduce(dr: Drafter, mode: int) -> None:
    _check("pe_set_split_reduce", lib().pe_set_split_reduce(dr.handle, int(mode)))


PE_TUNE_GEMM_PRE_STAGES = 1
PE_TUNE_ATTN_L2_AHEAD = 2
PE_TUNE_GEMM_MAX_SPLIT = 3
PE_TUNE_ATTN_MIN_CHUNKS = 4
PE_TUNE_ATTN_MAX_CHUNKS = 5
PE_TUNE_GEMM_TILE_ORDER = 6


def pe_set_tuning(dr: Drafter, key: int, value: int) -> None:
    _check("pe_set_tuning", lib().pe_set_tuning(dr.handle, int(key), int(value)))


def pe_set_stream_prefetch(dr: Drafter, tiles: int, boundary_tiles: int = -1) -> None:
    _check("pe_set_stream_prefetch",
           lib().pe_set_stream_prefetch(dr.handle, int(tiles), int(boundary_tiles)))


def pe_set_stream_timeline(dr: Drafter, stamps=None) -> None:
    """stamps: int64 device tensor of sm_count * 64 entries, or None."""
    _check("pe_set_stream_timeline", lib().pe_set_stream_timeline(dr.handle, ptr(stamps)))


def pe_set_phase_events(dr: Drafter, events=None) -> None:
    """events: torch.cuda.Event objects (2 + 2 n_layers, timing enabled), or
    None to turn phase timing off."""
    events = list(events or [])
    for e in events:
        if e.cuda_event == 0:      # torch creates the event on first record
            e.record()
    arr = (_vp * max(1, len(events)))(*[e.cuda_event for e in events])
    dr._phase_events = events      # the library keeps the handles
    _check("pe_set_phase_events", lib().pe_set_phase_events(dr.handle, arr, len(events)))


def pe_set_trace(dr: Drafter, residual_trace=None, attn_trace=None) -> None:
    _check("pe_set_trace", lib().pe_set_trace(dr.handle, ptr(residual_trace), ptr(attn_trace)))


def pe_set_kv_cache_fp8(dr: Drafter, k_scales=None, v_scales=None) -> None:
    """Switch the drafter to e4m3 KV pools with per-layer scales (None, None:
    back to pools of the model dtype)."""
    if k_scales is None and v_scales is None:
        _check("pe_set_kv_cache_fp8", lib().pe_set_kv_cache_fp8(dr.handle, None, None))
        return
    ks = (ctypes.c_float * len(k_scales))(*[float(x) for x in k_scales])
    vs = (ctypes.c_float * len(v_scales))(*[float(x) for x in v_scales])
    _check("pe_set_kv_cache_fp8", lib().pe_set_kv_cache_fp8(dr.handle, ks, vs))


def pe_get_launch_count(dr: Drafter) -> int:
    n = ctypes.c_int64(0)
    _check("pe_get_launch_count", lib().pe_get_launch_count(dr.handle, ctypes.byref(n)))
    return n.value


def pe_linear(dr: Drafter, x, w, y, stream=None):
    M, K = x.shape
    N = w.shape[0]
    _check("pe_linear", lib().pe_linear(dr.handle, ptr(x), ptr(w), ptr(y), M, N, K,
                                        stream_ptr(stream)))
    return y


def pe_linear_static(x, w, y, stream=None):
    """y = x w^T (bf16 in, fp32 out) through the entry point that allocates
    nothing: its scratch is a static device array inside the library."""
    M, K = x.shape
    N = w.shape[0]
    _check("pe_linear_static", lib().pe_linear_static(ptr(x), ptr(w), ptr(y), M, N, K,
                                                      stream_ptr(stream)))
    return y


def pe_linear_static_error(stream=None) -> int:
    """Read and clear the device error word of pe_linear_static's static
    array (0: nothing recorded since the last read)."""
    code = _i32(0)
    _check("pe_linear_static_error", lib().pe_linear_static_error(ctypes.byref(code),
                                                                  stream_ptr(stream)))
    return code.value


# ---------------------------------------------------------------------------
# training-side index work (include/peagle_train.h)
# ---------------------------------------------------------------------------

def pe_train_build_mask(out, n_max: int, K: int, mask_type: int, stream=None):
    """Fill out [n_max*K, ld] (uint8 for PE_MASK_BOOL_U8, bfloat16 for
    PE_MASK_ADDITIVE_BF16; ld = out.shape[1]) with the amortized mask."""
    if out.dim() != 2 or out.stride(1) != 1:
        raise ValueError("out must be a row-major 2-D tensor")
    _check("pe_train_build_mask", lib().pe_train_build_mask(
        n_max, K, mask_type, ptr(out), out.stride(0), stream_ptr(stream)))
    return out


def pe_train_mask_view(mask, n_max: int, K: int, n: int):
    """The mask of an n-token sample: a view of the top-left block of the mask
    built for n_max (no copy)."""
    v = _vp()
    rows = ctypes.c_int64(0)
    ld = ctypes.c_int64(0)
    _check("pe_train_mask_view", lib().pe_train_mask_view(
        ptr(mask), mask.stride(0), n_max, K, n, ctypes.byref(v), ctypes.byref(rows),
        ctypes.byref(ld)))
    if v.value != mask.data_ptr() or ld.value != mask.stride(0):
        raise RuntimeError("pe_train_mask_view returned an unexpected view")
    return mask[: rows.value, : rows.value]


def pe_train_partition(n: int, K: int, r: float, u, bounds: Sequence[int], stream=None):
    """COD sampling + sequence partitioning of one n-token sample; u is a
    [n, K] float32 device tensor of draws.  Returns device tensors keep,
    seg, offsets, rows, owned (rows / owned trimmed to offsets[-1] by the
    caller)."""
    torch = _torch()
    S = len(bounds) - 1
    hb = (_i32 * (S + 1))(*[int(b) for b in bounds])
    cap = int(sum(bounds[:-1])) + n * K
    dev = u.device
    out = dict(keep=torch.empty(n, K, dtype=torch.uint8, device=dev),
               seg=torch.empty(n, K, dtype=torch.int32, device=dev),
               counts=torch.empty(max(S, 1), dtype=torch.int32, device=dev),
               offsets=torch.empty(S + 1, dtype=torch.int32, device=dev),
               rows=torch.empty(cap, dtype=torch.int32, device=dev),
               owned=torch.empty(cap, dtype=torch.uint8, device=dev))
    _check("pe_train_partition", lib().pe_train_partition(
        n, K, ctypes.c_float(r), ptr(u), S, hb, ptr(out["keep"]), ptr(out["seg"]),
        ptr(out["counts"]), ptr(out["offsets"]), ptr(out["rows"]), ptr(out["owned"]), cap,
        stream_ptr(stream)))
    return out


# ---------------------------------------------------------------------------
# paged KV cache operators (include/peagle_cache.h)
# ---------------------------------------------------------------------------

class KvPool:
    """One layer's paged pools, borrowed: k, v [num_blocks, n_kv_heads, 16,
    head_dim] (bfloat16, float32, or e4m3 codes as uint8 / float8_e4m3fn) and
    scores, None or float32 [num_blocks, n_kv_heads, 16]."""

    def __init__(self, k, v, scores=None, k_scale: float = 1.0, v_scale: float = 1.0):
        torch = _torch()
        kinds = {torch.bfloat16: PE_KV_BF16, torch.float32: PE_KV_F32, torch.uint8: PE_KV_E4M3,
                 torch.float8_e4m3fn: PE_KV_E4M3}
        if k.dim() != 4 or k.shape[2] != 16 or v.shape != k.shape:
            raise ValueError("k and v must be [num_blocks, n_kv_heads, 16, head_dim]")
        if k.dtype not in kinds or v.dtype != k.dtype:
            raise ValueError("k and v must both be bfloat16, float32 or e4m3 codes")
        if not (k.is_contiguous() and v.is_contiguous()):
            raise ValueError("k and v must be contiguous")
        if scores is not None and (scores.dtype != torch.float32 or not scores.is_contiguous()
                                   or scores.shape != k.shape[:3]):
            raise ValueError("scores must be contiguous float32 [num_blocks, n_kv_heads, 16]")
        if any(t is not None and t.device != k.device for t in (v, scores)):
            raise ValueError("k, v and scores must be on one device")
        self.k, self.v, self.scores, self.device = k, v, scores, k.device
        self.torch, self.i32, self.lib = torch, torch.int32, lib()
        self.index = k.get_device()  # -1: not on a GPU
        self._workspace = {}         # sizes by (requests, query heads, table width)
        self.num_blocks, self.n_kv_heads, _, self.head_dim = k.shape
        self.dtype = kinds[k.dtype]
        self.act_dtype = torch.float32 if self.dtype == PE_KV_F32 else torch.bfloat16
        self.struct = pe_kv_pool(ptr(k), ptr(v), ptr(scores), self.num_blocks, self.n_kv_heads,
                                 self.head_dim, self.dtype, k_scale, v_scale)
        self._ref = ctypes.byref(self.struct)


def _cache_rows(pool: KvPool, name: str, t, rows: int, heads: int) -> int:
    """Row stride (elements) of a [rows, heads, head_dim] tensor whose heads
    are contiguous."""
    dh = pool.head_dim
    if t.dtype is not pool.act_dtype or t.shape != (rows, heads, dh):
        raise ValueError(f"{name} must be {pool.act_dtype} [{rows}, {heads}, {dh}]")
    row, head, one = t.stride()
    if one != 1 or (head != dh and heads > 1):
        raise ValueError(f"{name} must have contiguous heads")
    if t.get_device() != pool.index:
        raise ValueError(f"{name} must be on the pool's device")
    return row if rows > 1 else heads * dh


def _cache_i32(pool: KvPool, name: str, t, shape) -> None:
    if (t.dtype is not pool.i32 or t.shape != shape or not t.is_contiguous()
            or t.get_device() != pool.index):
        raise ValueError(f"{name} must be contiguous int32 {list(shape)} on {pool.device}")


def _cache_table(pool: KvPool, name: str, t, B: int) -> int:
    # contiguous: the library takes a row's length as its stride
    shape = t.shape
    if (t.dtype is not pool.i32 or len(shape) != 2 or shape[0] != B or not t.is_contiguous()
            or t.get_device() != pool.index):
        raise ValueError(f"{name} must be contiguous int32 [{B}, pages] on {pool.device}")
    return shape[1]


def _cache_ints(**values) -> None:
    """ctypes takes an integer modulo 2^32: refuse what that would change."""
    for name, x in values.items():
        if not -2**31 <= x < 2**31:
            raise ValueError(f"{name} must be a 32-bit integer")


def _cache_empty(pool: KvPool, shape, dtype, stream):
    """Memory for a call on `stream`, from that stream's share of the
    allocator: what other streams still do with freed memory cannot meet it."""
    torch = pool.torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=pool.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=pool.device)


# Workspaces of eager calls, one a device and stream: calls on one stream run
# one after another, so they can share it.  Memory of its own goes to a
# captured call (its graph's: a replay may run beside anything), to a call on
# a stream other than the current one or a device other than the current one,
# and to one that wants a lot.
_CACHE_WORKSPACES: Dict = {}
_CACHE_SHARED_MOST = 64 << 20
# held while the launches of a call with a shared workspace are queued: another
# thread's must not come between them
_CACHE_LOCK = threading.Lock()


def _cache_shares(pool: KvPool, nbytes: int, stream) -> bool:
    # the last question is about the current device's stream
    C = pool.torch._C
    return (nbytes <= _CACHE_SHARED_MOST and stream is None and pool.index >= 0
            and C._cuda_getDevice() == pool.index and not C._cuda_isCurrentStreamCapturing())


def _cache_shared_workspace(pool: KvPool, nbytes: int):
    C = pool.torch._C
    key = pool.index, C._cuda_getCurrentRawStream(pool.index)
    ws = _CACHE_WORKSPACES.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = _CACHE_WORKSPACES[key] = _cache_empty(pool, nbytes, pool.torch.uint8, None)
    return ws


def _cache_call(pool: KvPool, stream, name, fn, *args) -> None:
    """Call into the library with the pool's device current; `stream` None is
    that device's current stream."""
    index = pool.index
    if index < 0:
        raise ValueError(f"{name} needs tensors on a GPU")
    # the raw handles behind torch.cuda.current_stream() and current_device()
    C = pool.torch._C
    s = C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if C._cuda_getDevice() == index:
        status = fn(*args, s)
    else:
        with pool.torch.cuda.device(index):
            status = fn(*args, s)
    if status != PE_OK:
        raise PeError(name, status)


def pe_kv_append(pool: KvPool, q, k, v, pos, block_table, rope_theta: float = 0.0, req=None,
                 q_out=None, err=None, stream=None):
    """Rotate the new rows q [T, n_heads, head_dim] (or None) and k [T,
    n_kv_heads, head_dim] to positions pos [T] and write k and v into the
    pages of their requests (req [T]; None: row t is request t's).  Returns
    q_out (made when None)."""
    T, B = k.shape[0], block_table.shape[0]
    ks = _cache_rows(pool, "k", k, T, pool.n_kv_heads)
    vs = _cache_rows(pool, "v", v, T, pool.n_kv_heads)
    _cache_i32(pool, "pos", pos, (T,))
    if req is not None:
        _cache_i32(pool, "req", req, (T,))
    pages = _cache_table(pool, "block_table", block_table, B)
    n_heads = qs = qos = 0
    if q is not None:
        n_heads = q.shape[1]
        qs = _cache_rows(pool, "q", q, T, n_heads)
        if q_out is None:
            q_out = _cache_empty(pool, (T, n_heads, pool.head_dim), q.dtype, stream)
        qos = _cache_rows(pool, "q_out", q_out, T, n_heads)
    elif q_out is not None:
        raise ValueError("q_out without q")
    if err is not None:
        _cache_i32(pool, "err", err, (1,))
    _cache_call(pool, stream, "pe_kv_append", pool.lib.pe_kv_append, pool._ref, T, B, n_heads,
                rope_theta, ptr(q), qs, ptr(k), ks, ptr(v), vs, ptr(pos), ptr(req),
                ptr(block_table), pages, ptr(q_out), qos, ptr(err))
    return q_out


def pe_attn_decode_workspace(B: int, n_heads: int, n_kv_heads: int, head_dim: int,
                             pages: int = 0) -> int:
    """Bytes of workspace of a pe_attn_decode call on the current device; with
    `pages`, the block table's width, room for the logits of a call that
    accumulates (it then works them out once instead of twice; not beyond 16
    query heads a kv head, with float32 pools 8 of head_dim 64 and 4 of 128)."""
    _cache_ints(B=B, n_heads=n_heads, pages=pages)
    n = lib().pe_attn_decode_workspace(B, n_heads, n_kv_heads, head_dim, pages)
    if n <= 0:
        raise ValueError("pe_attn_decode_workspace: bad sizes")
    return n


def _cache_logits_width(pool: KvPool, n_heads: int, pages: int) -> int:
    """Table width to make room for: 0 where a call keeps no logits."""
    most = 16 if pool.dtype != PE_KV_F32 else 8 if pool.head_dim == 64 else 4
    return pages if n_heads <= most * pool.n_kv_heads else 0


def pe_attn_decode(pool: KvPool, q, block_table, seq_lens, scale: Optional[float] = None,
                   window: int = 0, accumulate: bool = False, out=None, lse=None,
                   workspace=None, err=None, stream=None):
    """Attention of one new token per request, q [B, n_heads, head_dim], over
    its seq_lens [B] cached positions (the last `window` of them unless 0).
    scale None: head_dim ** -0.5.  accumulate: each position's weight is added
    to pool.scores.  Returns out and lse [B, n_heads] float32 (made when
    None).  workspace: uint8, pe_attn_decode_workspace bytes; None: the
    stream's own, or memory allocated for the call where it is captured or
    wants more than 64 MiB."""
    torch = pool.torch
    _cache_ints(window=window)
    B, n_heads = q.shape[0], q.shape[1]
    dh = pool.head_dim
    qs = _cache_rows(pool, "q", q, B, n_heads)
    pages = _cache_table(pool, "block_table", block_table, B)
    _cache_i32(pool, "seq_lens", seq_lens, (B,))
    if out is None:
        out = _cache_empty(pool, (B, n_heads, dh), q.dtype, stream)
    if lse is None:
        lse = _cache_empty(pool, (B, n_heads), torch.float32, stream)
    elif (lse.dtype is not torch.float32 or lse.shape != (B, n_heads) or not lse.is_contiguous()
          or lse.get_device() != pool.index):
        raise ValueError(f"lse must be contiguous float32 [{B}, {n_heads}]")
    os_ = _cache_rows(pool, "out", out, B, n_heads)
    if workspace is None:
        room = _cache_logits_width(pool, n_heads, pages) if accumulate else 0
        n = pool._workspace.get((B, n_heads, room))
        if n is None:
            with torch.cuda.device(pool.index):
                n = pe_attn_decode_workspace(B, n_heads, pool.n_kv_heads, dh, room)
            pool._workspace[B, n_heads, room] = n
        if not _cache_shares(pool, n, stream):
            workspace = _cache_empty(pool, n, torch.uint8, stream)
    elif not workspace.is_contiguous() or workspace.get_device() != pool.index:
        raise ValueError("workspace must be contiguous on the pool's device")
    else:
        n = workspace.numel() * workspace.element_size()
    if err is not None:
        _cache_i32(pool, "err", err, (1,))
    args = (pool._ref, B, n_heads, dh ** -0.5 if scale is None else scale, ptr(q), qs,
            ptr(block_table), pages, ptr(seq_lens), window, ptr(out), os_, ptr(lse),
            int(accumulate))
    if workspace is not None:
        _cache_call(pool, stream, "pe_attn_decode", pool.lib.pe_attn_decode, *args,
                    ptr(workspace), n, ptr(err))
    else:
        with _CACHE_LOCK:
            ws = _cache_shared_workspace(pool, n)
            _cache_call(pool, stream, "pe_attn_decode", pool.lib.pe_attn_decode, *args, ptr(ws),
                        n, ptr(err))
    return out, lse


def pe_kv_evict(pools: Sequence[KvPool], block_table, seq_lens, budget: int, sinks: int = 0,
                recent: int = 0, rope_theta: float = 0.0, dst_table=None, kept=None,
                new_lens=None, err=None, stream=None):
    """Trim every request of more than `budget` positions to that many, the
    first `sinks`, the last `recent` and the heaviest of the rest by
    pool.scores, per layer (one pool each) and kv head.  In place, or into
    the pages of dst_table.  Returns kept [layers, B, n_kv_heads, budget] and
    new_lens [B], int32 (made when None)."""
    pools = list(pools)
    if not pools:
        raise ValueError("no pools")
    _cache_ints(budget=budget, sinks=sinks, recent=recent)
    p0, B = pools[0], block_table.shape[0]
    torch = p0.torch
    if any(p.index != p0.index for p in pools):
        raise ValueError("the pools must be on one device")
    pages = _cache_table(p0, "block_table", block_table, B)
    _cache_i32(p0, "seq_lens", seq_lens, (B,))
    dst_pages = _cache_table(p0, "dst_table", dst_table, B) if dst_table is not None else 0
    shape = (len(pools), B, p0.n_kv_heads, budget)
    if budget < 1:
        raise ValueError("budget must be positive")
    if kept is None:
        kept = _cache_empty(p0, shape, torch.int32, stream)
    _cache_i32(p0, "kept", kept, shape)
    if new_lens is None:
        new_lens = _cache_empty(p0, B, torch.int32, stream)
    _cache_i32(p0, "new_lens", new_lens, (B,))
    if err is not None:
        _cache_i32(p0, "err", err, (1,))
    arr = (pe_kv_pool * len(pools))(*[p.struct for p in pools])
    _cache_call(p0, stream, "pe_kv_evict", p0.lib.pe_kv_evict, len(pools), arr, B,
                ptr(block_table), pages, ptr(seq_lens), budget, sinks, recent, rope_theta,
                ptr(dst_table), dst_pages, ptr(kept), ptr(new_lens), ptr(err))
    return kept, new_lens


def pe_set_kv_scores(dr: Drafter, scores: Optional[Sequence] = None) -> None:
    """Let pe_draft_forward add the attention weights of every request's
    next-token row to scores, one float32 tensor [num_blocks, n_kv_heads, 16]
    a layer (None: collect no more)."""
    if scores is None:
        _check("pe_set_kv_scores", lib().pe_set_kv_scores(dr.handle, None))
        dr._kv_scores = None
        return
    scores = list(scores)
    sh, torch = dr.shape, _torch()
    if len(scores) != sh.n_layers:
        raise ValueError(f"one tensor for each of {sh.n_layers} layers")
    for t in scores:
        if (t.dtype != torch.float32 or t.dim() != 3 or not t.is_contiguous() or not t.is_cuda
                or tuple(t.shape[1:]) != (sh.n_kv_heads, 16)):
            raise ValueError(f"scores must be contiguous float32 [num_blocks, {sh.n_kv_heads}, 16]")
    arr = (_vp * len(scores))(*[ptr(t) for t in scores])
    _check("pe_set_kv_scores", lib().pe_set_kv_scores(dr.handle, arr))
    dr._kv_scores = scores         # the library keeps the pointers


# ---------------------------------------------------------------------------
# 4-bit weights, sampling and the verification of drafts (include/peagle_w4.h,
# include/peagle_sample.h)
# ---------------------------------------------------------------------------

def _op_vector(name: str, t, n: int, dtype, index: int) -> int:
    """Address of a contiguous vector of n elements on device `index`."""
    if (t.dtype is not dtype or t.shape != (n,) or not t.is_contiguous()
            or t.get_device() != index):
        raise ValueError(f"{name} must be contiguous {dtype} [{n}] on the same device")
    return t.data_ptr()


def _op_rows(name: str, t, rows: int, width: int, index: int) -> int:
    """Row stride (elements) of a [rows, width] matrix of contiguous rows."""
    if t.shape != (rows, width) or t.get_device() != index:
        raise ValueError(f"{name} must be [{rows}, {width}] on the same device")
    row, one = t.stride()
    if one != 1 and width > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return row if rows > 1 else width


def _op_kind(name: str, t) -> int:
    torch = _torch()
    if t.dtype is torch.bfloat16:
        return PE_DTYPE_BF16
    if t.dtype is torch.float32:
        return PE_DTYPE_F32
    raise ValueError(f"{name} must be bfloat16 or float32")


def _op_empty(shape, dtype, device, stream):
    """Memory for a call on `stream`, from that stream's share of the
    allocator."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _op_stream(index: int, stream) -> int:
    """The stream of a call: `stream`, or device `index`'s current one."""
    if stream is not None:
        return stream.cuda_stream
    return _torch()._C._cuda_getCurrentRawStream(index) if index >= 0 else 0


def _op_call(index: int, stream, name, fn, *args) -> None:
    """Call into the library with device `index` current; `stream` None is
    that device's current stream."""
    if index < 0:
        raise ValueError(f"{name} needs tensors on a GPU")
    torch = _torch()
    C = torch._C
    s = _op_stream(index, stream)
    if C._cuda_getDevice() == index:
        status = fn(*args, s)
    else:
        with torch.cuda.device(index):
            status = fn(*args, s)
    if status != PE_OK:
        raise PeError(name, status)


def _op_used(stream, *tensors) -> None:
    """Memory that is freed after a call on `stream` is not handed out again
    before that stream is done with it."""
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


class W4Weight:
    """A matrix [n, k] of 4-bit codes with a bfloat16 scale for each `group`
    (32, 64 or 128) inputs of a row, laid out for pe_w4_linear.  Entry (i, j)
    is (code - 8) * scale[i, j // group].

    codes uint8 [n, (k + 1) // 2], input 2 j in the low half of byte j; scales
    bfloat16 [n, ceil(k / group)].  The layout is made once, here, on `stream`
    (None: the current one); codes and scales are not kept.  A product on
    another stream has to wait for it; the matrix may be dropped as soon as the
    last product has been called."""

    def __init__(self, codes, scales, k: int, group: int, stream=None):
        torch = _torch()
        n, index = codes.shape[0], codes.get_device()
        self._prepare(n, k, group, codes.device, stream)
        if (codes.dtype is not torch.uint8 or codes.shape != (n, (k + 1) // 2)
                or not codes.is_contiguous()):
            raise ValueError(f"codes must be contiguous uint8 [{n}, {(k + 1) // 2}]")
        if (scales.dtype is not torch.bfloat16 or scales.shape != (n, -(-k // group))
                or not scales.is_contiguous() or scales.get_device() != index):
            raise ValueError(f"scales must be contiguous bfloat16 [{n}, {-(-k // group)}] "
                             "on the codes' device")
        _op_call(index, stream, "pe_w4_pack", lib().pe_w4_pack, ptr(codes), ptr(scales), n, k,
                 group, ptr(self.packed))
        _op_used(stream, codes, scales)

    def _prepare(self, n, k, group, device, stream):
        torch = _torch()
        _cache_ints(n=n, k=k, group=group)
        nbytes = lib().pe_w4_bytes(n, k, group)
        if nbytes <= 0:
            raise ValueError("a 4-bit matrix has n, k >= 1 (k up to 2**17, n up to 2**24) and a "
                             "group of 32, 64 or 128")
        self.n, self.k, self.group, self.device = n, k, group, device
        self.packed = _op_empty(nbytes, torch.uint8, device, stream)
        self.index = self.packed.get_device()
        self._of = _op_stream(self.index, stream)

    @classmethod
    def quantize(cls, weight, group: int = 32, stream=None) -> "W4Weight":
        """Round a bfloat16 or float32 matrix [n, k] to 4 bits: a group's
        scale is its largest absolute value over 7."""
        self = cls.__new__(cls)
        if weight.dim() != 2:
            raise ValueError("weight must be [n, k]")
        n, k = weight.shape
        kind = _op_kind("weight", weight)
        self._prepare(n, k, group, weight.device, stream)
        stride = _op_rows("weight", weight, n, k, self.index)
        _op_call(self.index, stream, "pe_w4_quantize", lib().pe_w4_quantize, ptr(weight), kind,
                 stride, n, k, group, ptr(self.packed))
        _op_used(stream, weight)
        return self


def pe_w4_linear(w: W4Weight, x, out=None, out_dtype=None, stream=None):
    """x [rows, k] (bfloat16 or float32) times the 4-bit matrix w, [rows, n]
    in out_dtype (None: x's type; float32 beside bfloat16 x for logits), in
    `out` where given."""
    if x.dim() != 2:
        raise ValueError("x must be [rows, k]")
    rows = x.shape[0]
    kind = _op_kind("x", x)
    xs = _op_rows("x", x, rows, w.k, w.index)
    if out is None:
        out = _op_empty((rows, w.n), out_dtype or x.dtype, x.device, stream)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise ValueError("out is of another type than out_dtype")
    ok = _op_kind("out", out)
    ys = _op_rows("out", out, rows, w.n, w.index)
    _op_call(w.index, stream, "pe_w4_linear", lib().pe_w4_linear, w.packed.data_ptr(), w.n, w.k,
             w.group, rows, kind, x.data_ptr(), xs, ok, out.data_ptr(), ys)
    _op_used(stream, x, out)
    if _op_stream(w.index, stream) != w._of:      # its memory is of another stream
        _op_used(stream or _torch().cuda.current_stream(w.index), w.packed)
    return out


def _op_filters(n: int, index: int, temperature, top_k, top_p, min_p):
    """Addresses of the filters, None where not set."""
    torch = _torch()
    f32 = torch.float32
    return [None if t is None else _op_vector(name, t, n, dtype, index)
            for name, t, dtype in (("temperature", temperature, f32),
                                   ("top_k", top_k, torch.int32), ("top_p", top_p, f32),
                                   ("min_p", min_p, f32))]


def _op_dist(name: str, t, n: int, index: int) -> int:
    if (t.dtype is not _torch().int32 or t.shape != (n, 8) or not t.is_contiguous()
            or t.get_device() != index):
        raise ValueError(f"{name} must be contiguous int32 [{n}, 8] on the same device")
    return t.data_ptr()


def pe_sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, tokens=None,
              logprobs=None, dist=None, stream=None):
    """A token for each row of logits [rows, vocab] (float32 or bfloat16),
    drawn with u [rows] float32 of [0, 1).  Filters, each None or a vector
    [rows]: temperature (float32; not above 0: greedy), top_k (int32), top_p,
    min_p (float32).  Returns tokens [rows] int32 (-1: a row without any),
    logprobs [rows] float32 and dist [rows, 8] int32, the rows' pe_dist records
    that pe_verify takes of sampled drafts (made when None)."""
    torch = _torch()
    if logits.dim() != 2:
        raise ValueError("logits must be [rows, vocab]")
    rows, vocab = logits.shape
    index, device = logits.get_device(), logits.device
    kind = _op_kind("logits", logits)
    stride = _op_rows("logits", logits, rows, vocab, index)
    pu = _op_vector("u", u, rows, torch.float32, index)
    filters = _op_filters(rows, index, temperature, top_k, top_p, min_p)
    if tokens is None:
        tokens = _op_empty(rows, torch.int32, device, stream)
    if logprobs is None:
        logprobs = _op_empty(rows, torch.float32, device, stream)
    if dist is None:
        dist = _op_empty((rows, 8), torch.int32, device, stream)
    _op_call(index, stream, "pe_sample", lib().pe_sample, rows, vocab, kind, logits.data_ptr(),
             stride, *filters, pu, _op_vector("tokens", tokens, rows, torch.int32, index),
             _op_vector("logprobs", logprobs, rows, torch.float32, index),
             _op_dist("dist", dist, rows, index))
    _op_used(stream, logits, u, temperature, top_k, top_p, min_p, tokens, logprobs, dist)
    return tokens, logprobs, dist


def pe_verify(logits, ids, cu_in, accept_u, u, temperature=None, top_k=None, top_p=None,
              min_p=None, draft_logits=None, draft_dist=None, num_accepted=None,
              sampled_ids=None, logprobs=None, dist=None, err=None, stream=None):
    """Verify drafts by rejection sampling: logits [T, vocab] of the target at
    the rows of the B requests' windows, ids [T] the windows' tokens (a
    window's first token, then its drafts), cu_in [B + 1] where they start, as
    in pe_expand_batch.  accept_u [T] and u [B] float32 of [0, 1); filters as
    in pe_sample, [B].  draft_logits None: the drafts are the drafter's
    largest logits; else [T - B, vocab], the drafter's logits of all drafts in
    order, and draft_dist what pe_sample returned for them.  Returns
    num_accepted [B], sampled_ids [B] (the next pe_expand_batch takes both),
    logprobs [T] and dist [T, 8] (made when None)."""
    torch = _torch()
    if logits.dim() != 2 or cu_in.dim() != 1:
        raise ValueError("logits must be [T, vocab] and cu_in [B + 1]")
    T, vocab = logits.shape
    B = cu_in.shape[0] - 1
    index, device = logits.get_device(), logits.device
    i32, f32 = torch.int32, torch.float32
    kind = _op_kind("logits", logits)
    stride = _op_rows("logits", logits, T, vocab, index)
    pids = _op_vector("ids", ids, T, i32, index)
    pcu = _op_vector("cu_in", cu_in, B + 1, i32, index)
    pau = _op_vector("accept_u", accept_u, T, f32, index)
    pu = _op_vector("u", u, B, f32, index)
    filters = _op_filters(B, index, temperature, top_k, top_p, min_p)
    dl = dd = None
    ds = 0
    if (draft_logits is None) != (draft_dist is None):
        raise ValueError("draft_logits and draft_dist go together")
    if draft_logits is not None:
        if draft_logits.dtype is not logits.dtype:
            raise ValueError("draft_logits must be of the type of logits")
        ds = _op_rows("draft_logits", draft_logits, T - B, vocab, index)
        dd = _op_dist("draft_dist", draft_dist, T - B, index)
        # without any draft there is no row to point to: any address says "sampled"
        dl = draft_logits.data_ptr() or logits.data_ptr()
    if num_accepted is None:
        num_accepted = _op_empty(B, i32, device, stream)
    if sampled_ids is None:
        sampled_ids = _op_empty(B, i32, device, stream)
    if logprobs is None:
        logprobs = _op_empty(T, f32, device, stream)
    if dist is None:
        dist = _op_empty((T, 8), i32, device, stream)
    _op_call(index, stream, "pe_verify", lib().pe_verify, B, T, vocab, kind, logits.data_ptr(),
             stride, pids, pcu, *filters, pau, pu, dl, ds, dd,
             _op_vector("num_accepted", num_accepted, B, i32, index),
             _op_vector("sampled_ids", sampled_ids, B, i32, index),
             _op_vector("logprobs", logprobs, T, f32, index), _op_dist("dist", dist, T, index),
             None if err is None else _op_vector("err", err, 1, i32, index))
    _op_used(stream, logits, ids, cu_in, accept_u, u, temperature, top_k, top_p, min_p,
             draft_logits, draft_dist, num_accepted, sampled_ids, logprobs, dist, err)
    return num_accepted, sampled_ids, logprobs, dist
