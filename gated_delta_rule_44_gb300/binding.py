"""Thin ctypes binding of libgdn (include/gdn.h).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  Functions take torch tensors (device memory and streams come from
PyTorch) and raise ``GdnError`` on a non-zero status.  There is no fallback:
if the library cannot be built or loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import struct
import threading
from typing import Optional

import torch

from . import build as _build

GDN_OK = 0
GDN_ERR_SHAPE = 1
GDN_ERR_INVALID_ARGUMENT = 2
GDN_ERR_DTYPE = 3
GDN_ERR_UNSUPPORTED = 4
GDN_ERR_CUDA = 5
GDN_ERR_TIMEOUT = 6
GDN_ERR_DEVICE_CHECK = 7

GDN_DTYPE_F32 = 0
GDN_DTYPE_BF16 = 1

GDN_PREFILL_AUTO = 0
GDN_PREFILL_CHUNKED = 1
GDN_PREFILL_RECURRENT = 2
GDN_PREFILL_FUSED = 3

_i64 = ctypes.c_int64
_i32 = ctypes.c_int32
_vp = ctypes.c_void_p
_f32 = ctypes.c_float


class gdn_prepare_args(ctypes.Structure):
    _fields_ = [("T", _i64), ("N", _i64), ("Hk", _i64), ("Hv", _i64), ("Dk", _i64), ("Dv", _i64),
                ("K", _i64), ("act_dtype", _i32), ("apply_qk_l2norm", _i32),
                ("mixed_qkv", _vp), ("mixed_qkv_stride", _i64), ("mixed_qkv_len", _i64),
                ("conv_weight", _vp), ("conv_weight_len", _i64),
                ("a_raw", _vp), ("a_raw_stride", _i64), ("a_raw_len", _i64),
                ("b_raw", _vp), ("b_raw_stride", _i64), ("b_raw_len", _i64),
                ("A_log", _vp), ("A_log_len", _i64), ("dt_bias", _vp), ("dt_bias_len", _i64),
                ("cu_seqlens", _vp), ("state_indices", _vp), ("has_initial_state", _vp),
                ("cu_seqlens_host", _vp), ("state_indices_host", _vp),
                ("conv_state", _vp), ("conv_state_slots", _i64), ("conv_state_len", _i64),
                ("q", _vp), ("q_len", _i64), ("k", _vp), ("k_len", _i64), ("v", _vp),
                ("v_len", _i64), ("g", _vp), ("g_len", _i64), ("beta", _vp),
                ("beta_len", _i64)]


class gdn_packed_decode_args(ctypes.Structure):
    _fields_ = [("B", _i64), ("Hk", _i64), ("Hv", _i64), ("Dk", _i64), ("Dv", _i64), ("K", _i64),
                ("act_dtype", _i32), ("apply_qk_l2norm", _i32), ("scale", _f32),
                ("mixed_qkv", _vp), ("mixed_qkv_stride", _i64), ("mixed_qkv_len", _i64),
                ("conv_weight", _vp), ("conv_weight_len", _i64),
                ("a_raw", _vp), ("a_raw_stride", _i64), ("a_raw_len", _i64),
                ("b_raw", _vp), ("b_raw_stride", _i64), ("b_raw_len", _i64),
                ("A_log", _vp), ("A_log_len", _i64), ("dt_bias", _vp), ("dt_bias_len", _i64),
                ("state_indices", _vp), ("state_indices_host", _vp),
                ("conv_state", _vp), ("conv_state_len", _i64),
                ("state", _vp), ("state_slots", _i64), ("state_len", _i64),
                ("out", _vp), ("out_len", _i64)]


class gdn_spec_prepare_args(ctypes.Structure):
    _fields_ = [("base", gdn_prepare_args), ("conv_state_width", _i64), ("num_accepted", _vp),
                ("num_accepted_host", _vp)]


class gdn_out_norm(ctypes.Structure):
    _fields_ = [("z", _vp), ("z_len", _i64), ("z_token_stride", _i64), ("weight", _vp),
                ("weight_len", _i64), ("eps", _f32), ("sigmoid_gate", _i32), ("in_kernel", _i32)]


class gdn_decode_args(ctypes.Structure):
    _fields_ = [("B", _i64), ("Hk", _i64), ("Hv", _i64), ("Dk", _i64), ("Dv", _i64),
                ("act_dtype", _i32), ("use_qk_l2norm", _i32), ("scale", _f32),
                ("q", _vp), ("q_len", _i64), ("k", _vp), ("k_len", _i64), ("v", _vp),
                ("v_len", _i64), ("g", _vp), ("g_len", _i64), ("beta", _vp), ("beta_len", _i64),
                ("state", _vp), ("state_slots", _i64), ("state_len", _i64),
                ("state_indices", _vp), ("state_indices_host", _vp),
                ("out", _vp), ("out_len", _i64), ("out_norm", ctypes.POINTER(gdn_out_norm))]


class gdn_prefill_args(ctypes.Structure):
    _fields_ = [("T", _i64), ("N", _i64), ("Hk", _i64), ("Hv", _i64), ("Dk", _i64), ("Dv", _i64),
                ("act_dtype", _i32), ("use_qk_l2norm", _i32), ("scale", _f32), ("algo", _i32),
                ("q", _vp), ("q_len", _i64), ("k", _vp), ("k_len", _i64), ("v", _vp),
                ("v_len", _i64), ("g", _vp), ("g_len", _i64), ("beta", _vp), ("beta_len", _i64),
                ("state", _vp), ("state_slots", _i64), ("state_len", _i64),
                ("cu_seqlens", _vp), ("state_indices", _vp), ("has_initial_state", _vp),
                ("cu_seqlens_host", _vp), ("state_indices_host", _vp),
                ("out", _vp), ("out_len", _i64), ("workspace", _vp),
                ("workspace_bytes", ctypes.c_size_t),
                ("out_norm", ctypes.POINTER(gdn_out_norm))]


class gdn_kda_args(ctypes.Structure):
    _fields_ = [("T", _i64), ("N", _i64), ("Hk", _i64), ("Hv", _i64), ("Dk", _i64), ("Dv", _i64),
                ("act_dtype", _i32), ("scale", _f32),
                ("q", _vp), ("q_len", _i64), ("k", _vp), ("k_len", _i64), ("v", _vp),
                ("v_len", _i64), ("g", _vp), ("g_len", _i64), ("beta", _vp), ("beta_len", _i64),
                ("state", _vp), ("state_slots", _i64), ("state_len", _i64),
                ("cu_seqlens", _vp), ("state_indices", _vp), ("has_initial_state", _vp),
                ("cu_seqlens_host", _vp), ("state_indices_host", _vp),
                ("out", _vp), ("out_len", _i64), ("algo", _i32), ("workspace", _vp),
                ("workspace_bytes", ctypes.c_size_t)]


class gdn_spec_decode_args(ctypes.Structure):
    _fields_ = [("T", _i64), ("n_reqs", _i64), ("num_cols", _i64), ("Hk", _i64), ("Hv", _i64),
                ("Dk", _i64), ("Dv", _i64), ("act_dtype", _i32), ("scale", _f32),
                ("q", _vp), ("q_len", _i64), ("k", _vp), ("k_len", _i64), ("v", _vp),
                ("v_len", _i64), ("g", _vp), ("g_len", _i64), ("beta", _vp), ("beta_len", _i64),
                ("state", _vp), ("state_slots", _i64), ("state_len", _i64),
                ("cu_seqlens", _vp), ("state_indices", _vp), ("num_accepted", _vp),
                ("cu_seqlens_host", _vp), ("state_indices_host", _vp), ("num_accepted_host", _vp),
                ("out", _vp), ("out_len", _i64)]


class gdn_gated_rmsnorm_args(ctypes.Structure):
    _fields_ = [("tokens", _i64), ("heads", _i64), ("dim", _i64), ("act_dtype", _i32),
                ("sigmoid_gate", _i32), ("eps", _f32), ("core", _vp), ("core_len", _i64),
                ("z", _vp), ("z_len", _i64), ("z_token_stride", _i64), ("weight", _vp),
                ("weight_len", _i64), ("out", _vp), ("out_len", _i64)]


class gdn_mixed_meta(ctypes.Structure):
    _fields_ = [("num_decodes", _i64), ("num_prefills", _i64), ("num_decode_tokens", _i64),
                ("num_prefill_tokens", _i64), ("num_actual_tokens", _i64), ("state_slots", _i64),
                ("allow_inert_padding", _i32), ("cu_seqlens_host", _vp),
                ("state_indices_host", _vp), ("has_initial_state_host", _vp),
                ("cu_seqlens_prefill_host", _vp), ("prefill_state_indices_host", _vp),
                ("prefill_has_initial_state_host", _vp)]


class gdn_attn_rows(ctypes.Structure):
    _fields_ = [("data", _vp), ("len", _i64), ("token_stride", _i64), ("head_stride", _i64)]


class gdn_attn_cache(ctypes.Structure):
    _fields_ = [("k", _vp), ("k_len", _i64), ("k_page_stride", _i64), ("k_head_stride", _i64),
                ("k_token_stride", _i64), ("v", _vp), ("v_len", _i64), ("v_page_stride", _i64),
                ("v_head_stride", _i64), ("v_token_stride", _i64), ("num_pages", _i64),
                ("page_size", _i64), ("block_table", _vp), ("max_pages", _i64),
                ("table_stride", _i64), ("block_table_host", _vp)]


class gdn_attn_prepare_args(ctypes.Structure):
    _fields_ = [("T", _i64), ("N", _i64), ("Hq", _i64), ("Hkv", _i64), ("D", _i64),
                ("rot_dim", _i64), ("act_dtype", _i32), ("norm_eps", _f32),
                ("q", gdn_attn_rows), ("k", gdn_attn_rows), ("v", gdn_attn_rows),
                ("q_norm_weight", _vp), ("q_norm_weight_len", _i64),
                ("k_norm_weight", _vp), ("k_norm_weight_len", _i64),
                ("cos_sin", _vp), ("cos_sin_len", _i64), ("positions", _vp),
                ("cu_seqlens", _vp), ("kv_lens", _vp), ("cu_seqlens_host", _vp),
                ("kv_lens_host", _vp), ("cache", ctypes.POINTER(gdn_attn_cache)),
                ("q_out", _vp), ("q_out_len", _i64), ("k_out", _vp), ("k_out_len", _i64)]


class gdn_attn_varlen_args(ctypes.Structure):
    _fields_ = [("T", _i64), ("N", _i64), ("Hq", _i64), ("Hkv", _i64), ("D", _i64),
                ("act_dtype", _i32), ("scale", _f32), ("q", gdn_attn_rows), ("k", gdn_attn_rows),
                ("v", gdn_attn_rows), ("gate", gdn_attn_rows), ("cu_seqlens", _vp),
                ("cu_seqlens_host", _vp), ("out", _vp), ("out_len", _i64), ("lse", _vp),
                ("lse_len", _i64)]


class gdn_attn_paged_args(ctypes.Structure):
    _fields_ = [("T", _i64), ("N", _i64), ("Hq", _i64), ("Hkv", _i64), ("D", _i64),
                ("max_q_len", _i64), ("act_dtype", _i32), ("scale", _f32), ("q", gdn_attn_rows),
                ("gate", gdn_attn_rows), ("cu_seqlens", _vp), ("kv_lens", _vp),
                ("cu_seqlens_host", _vp), ("kv_lens_host", _vp),
                ("cache", ctypes.POINTER(gdn_attn_cache)), ("out", _vp), ("out_len", _i64),
                ("lse", _vp), ("lse_len", _i64), ("workspace", _vp),
                ("workspace_bytes", ctypes.c_size_t)]


class gdn_attn_cache8(ctypes.Structure):
    _fields_ = [("codes", gdn_attn_cache), ("k_scale", _vp), ("k_scale_len", _i64),
                ("v_scale", _vp), ("v_scale_len", _i64), ("block", _i64)]


class gdn_attn8_prepare_args(ctypes.Structure):
    _fields_ = [("base", gdn_attn_prepare_args), ("cache", ctypes.POINTER(gdn_attn_cache8))]


class gdn_attn8_paged_args(ctypes.Structure):
    _fields_ = [("base", gdn_attn_paged_args), ("cache", ctypes.POINTER(gdn_attn_cache8))]


class gdn_beam_select_args(ctypes.Structure):
    _fields_ = [("B", _i64), ("W", _i64), ("V", _i64), ("K", _i64), ("dtype", _i32),
                ("logits", _vp), ("logits_len", _i64), ("batch_stride", _i64),
                ("beam_stride", _i64), ("scores", _vp), ("scores_len", _i64),
                ("finished", _vp), ("finished_len", _i64), ("pad_token", _i64),
                ("parents", _vp), ("parents_len", _i64), ("tokens", _vp), ("tokens_len", _i64),
                ("out_scores", _vp), ("out_scores_len", _i64), ("workspace", _vp),
                ("workspace_bytes", ctypes.c_size_t)]


class gdn_slot_pool(ctypes.Structure):
    _fields_ = [("data", _vp), ("len", _i64), ("slots", _i64), ("slot_bytes", _i64),
                ("slot_stride", _i64)]


class gdn_copy_slots_args(ctypes.Structure):
    _fields_ = [("pools", ctypes.POINTER(gdn_slot_pool)), ("num_pools", _i64), ("n", _i64),
                ("group", _i64), ("dst", _vp), ("src", _vp), ("dst_host", _vp),
                ("src_host", _vp)]


EXPORTED = ("gdn_prepare", "gdn_decode", "gdn_prefill_varlen", "gdn_kda_varlen",
            "gdn_spec_prepare", "gdn_spec_decode", "gdn_packed_decode", "gdn_gated_rmsnorm",
            "gdn_prefill_workspace_bytes",
            "gdn_prefill_resolve_algo", "gdn_kda_resolve_algo", "gdn_kda_workspace_bytes",
            "gdn_status_string", "gdn_last_error_message",
            "gdn_read_device_status", "gdn_version", "gdn_launch_count", "gdn_validate_mixed",
            "gdn_check_wait_timeout", "gdn_attn_prepare", "gdn_attn_varlen", "gdn_attn_paged",
            "gdn_attn_paged_workspace_bytes", "gdn_attn8_prepare", "gdn_attn8_paged",
            "gdn_attn8_paged_workspace_bytes", "gdn_beam_select",
            "gdn_beam_select_workspace_bytes", "gdn_copy_slots")


class GdnError(RuntimeError):
    def __init__(self, code: int, name: str, msg: str):
        super().__init__(f"{name}: {msg}")
        self.code = code
        self.status = name
        self.msg = msg


_lock = threading.Lock()
_lib = None


def lib() -> ctypes.CDLL:
    """Build (if stale) and load libgdn.so; raises if that is impossible."""
    global _lib
    with _lock:
        if _lib is None:
            L = ctypes.CDLL(_build.build_library())
            for name in ("gdn_prepare", "gdn_decode", "gdn_prefill_varlen", "gdn_kda_varlen",
                         "gdn_spec_prepare", "gdn_spec_decode", "gdn_packed_decode", "gdn_gated_rmsnorm",
                         "gdn_read_device_status", "gdn_version", "gdn_validate_mixed"):
                getattr(L, name).restype = ctypes.c_int
            L.gdn_prepare.argtypes = [ctypes.POINTER(gdn_prepare_args), _vp]
            L.gdn_decode.argtypes = [ctypes.POINTER(gdn_decode_args), _vp]
            L.gdn_prefill_varlen.argtypes = [ctypes.POINTER(gdn_prefill_args), _vp]
            L.gdn_gated_rmsnorm.argtypes = [ctypes.POINTER(gdn_gated_rmsnorm_args), _vp]
            L.gdn_kda_varlen.argtypes = [ctypes.POINTER(gdn_kda_args), _vp]
            L.gdn_spec_decode.argtypes = [ctypes.POINTER(gdn_spec_decode_args), _vp]
            L.gdn_spec_prepare.argtypes = [ctypes.POINTER(gdn_spec_prepare_args), _vp]
            L.gdn_packed_decode.argtypes = [ctypes.POINTER(gdn_packed_decode_args), _vp]
            L.gdn_read_device_status.argtypes = [_vp]
            L.gdn_validate_mixed.argtypes = [ctypes.POINTER(gdn_mixed_meta)]
            L.gdn_check_wait_timeout.restype = ctypes.c_int
            L.gdn_check_wait_timeout.argtypes = [ctypes.c_longlong, _vp]
            L.gdn_prefill_workspace_bytes.restype = ctypes.c_size_t
            L.gdn_prefill_workspace_bytes.argtypes = [_i64, _i64, _i64, _i64, _i64, _i32, _i32]
            L.gdn_prefill_resolve_algo.restype = _i32
            L.gdn_prefill_resolve_algo.argtypes = [_i64, _i64, _i64, _i64, _i32, _i32]
            L.gdn_kda_resolve_algo.restype = _i32
            L.gdn_kda_resolve_algo.argtypes = [_i64, _i64, _i64, _i64, _i32, _i32]
            L.gdn_kda_workspace_bytes.restype = ctypes.c_size_t
            L.gdn_kda_workspace_bytes.argtypes = [_i64, _i64, _i64, _i64, _i64, _i32, _i32]
            for name in ("gdn_attn_prepare", "gdn_attn_varlen", "gdn_attn_paged",
                         "gdn_attn8_prepare", "gdn_attn8_paged", "gdn_beam_select",
                         "gdn_copy_slots"):
                getattr(L, name).restype = ctypes.c_int
                getattr(L, name).argtypes = [_vp, _vp]  # an address of, or a reference to, args
            L.gdn_attn_paged_workspace_bytes.restype = ctypes.c_size_t
            L.gdn_attn_paged_workspace_bytes.argtypes = [_i64] * 6 + [_i32]
            L.gdn_attn8_paged_workspace_bytes.restype = ctypes.c_size_t
            L.gdn_attn8_paged_workspace_bytes.argtypes = [_i64] * 6 + [_i32] + [_i64] * 2
            L.gdn_beam_select_workspace_bytes.restype = ctypes.c_size_t
            L.gdn_beam_select_workspace_bytes.argtypes = [_i64] * 4
            L.gdn_status_string.restype = ctypes.c_char_p
            L.gdn_status_string.argtypes = [ctypes.c_int]
            L.gdn_last_error_message.restype = ctypes.c_char_p
            L.gdn_last_error_message.argtypes = []
            L.gdn_launch_count.restype = ctypes.c_uint64
            L.gdn_launch_count.argtypes = []
            _lib = L
        return _lib


def _check(rc: int) -> None:
    if rc != GDN_OK:
        L = lib()
        raise GdnError(rc, L.gdn_status_string(rc).decode(), L.gdn_last_error_message().decode())


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return GDN_DTYPE_BF16
    if t.dtype == torch.float32:
        return GDN_DTYPE_F32
    raise GdnError(GDN_ERR_DTYPE, "GDN_ERR_DTYPE", f"unsupported activation dtype {t.dtype}")


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _n(t: Optional[torch.Tensor]) -> int:
    """Elements reachable from the tensor's first element (its allocation length)."""
    if t is None:
        return 0
    if t.numel() == 0:
        return 0
    return int(sum((s - 1) * st for s, st in zip(t.shape, t.stride())) + 1)


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _scratch(nbytes, device, stream):
    """A call's own workspace, allocated on the stream that uses it: a block that the
    allocator has for another one may have kernels of that one pending on it."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _host_i32(t: Optional[torch.Tensor]):
    if t is None:
        return None, None
    h = t.detach().to("cpu", torch.int32).contiguous()
    return h, h.data_ptr()


def _prepare_args(mixed_qkv, conv_weight, a_raw, b_raw, A_log, dt_bias, cu_seqlens, conv_state,
                  q, k, v, g, beta, Hk, Hv, Dk, Dv, K, state_indices, has_initial_state,
                  cu_seqlens_host, state_indices_host, apply_qk_l2norm):
    """gdn_prepare_args of the call, and the host mirrors it points to (kept
    alive by the caller)."""
    T = mixed_qkv.shape[0]
    N = cu_seqlens.numel() - 1
    cuh, cuh_p = _host_i32(cu_seqlens_host)
    sih, sih_p = _host_i32(state_indices_host)
    a = gdn_prepare_args(
        T=T, N=N, Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, K=K, act_dtype=_dt(mixed_qkv),
        apply_qk_l2norm=int(apply_qk_l2norm),
        mixed_qkv=_p(mixed_qkv), mixed_qkv_stride=mixed_qkv.stride(0), mixed_qkv_len=_n(mixed_qkv),
        conv_weight=_p(conv_weight), conv_weight_len=_n(conv_weight),
        a_raw=_p(a_raw), a_raw_stride=a_raw.stride(0), a_raw_len=_n(a_raw),
        b_raw=_p(b_raw), b_raw_stride=b_raw.stride(0), b_raw_len=_n(b_raw),
        A_log=_p(A_log), A_log_len=_n(A_log), dt_bias=_p(dt_bias), dt_bias_len=_n(dt_bias),
        cu_seqlens=_p(cu_seqlens), state_indices=_p(state_indices),
        has_initial_state=_p(has_initial_state), cu_seqlens_host=cuh_p,
        state_indices_host=sih_p, conv_state=_p(conv_state),
        conv_state_slots=conv_state.shape[0] if conv_state is not None else 0,
        conv_state_len=_n(conv_state), q=_p(q), q_len=_n(q), k=_p(k), k_len=_n(k), v=_p(v),
        v_len=_n(v), g=_p(g), g_len=_n(g), beta=_p(beta), beta_len=_n(beta))
    return a, (cuh, sih)


def gdn_prepare(mixed_qkv, conv_weight, a_raw, b_raw, A_log, dt_bias, cu_seqlens, conv_state,
                q, k, v, g, beta, *, Hk, Hv, Dk, Dv, K, state_indices=None,
                has_initial_state=None, cu_seqlens_host=None, state_indices_host=None,
                apply_qk_l2norm=True, stream=None) -> None:
    """include/gdn.h gdn_prepare; outputs q, k, v, g, beta are written, the
    conv_state pool is updated in place."""
    a, keep = _prepare_args(mixed_qkv, conv_weight, a_raw, b_raw, A_log, dt_bias, cu_seqlens,
                            conv_state, q, k, v, g, beta, Hk, Hv, Dk, Dv, K, state_indices,
                            has_initial_state, cu_seqlens_host, state_indices_host,
                            apply_qk_l2norm)
    _check(lib().gdn_prepare(ctypes.byref(a), _stream(stream)))


def gdn_spec_prepare(mixed_qkv, conv_weight, a_raw, b_raw, A_log, dt_bias, cu_seqlens,
                     conv_state, conv_indices, num_accepted, q, k, v, g, beta, *, Hk, Hv, Dk, Dv,
                     K, cu_seqlens_host=None, conv_indices_host=None, num_accepted_host=None,
                     apply_qk_l2norm=True, stream=None) -> None:
    """include/gdn.h gdn_spec_prepare; conv_state [slots, C_conv, width] with
    width = (K-1) + (max_q-1), updated in place; conv_indices, num_accepted
    [requests] int32."""
    base, keep = _prepare_args(mixed_qkv, conv_weight, a_raw, b_raw, A_log, dt_bias, cu_seqlens,
                               conv_state, q, k, v, g, beta, Hk, Hv, Dk, Dv, K, conv_indices,
                               None, cu_seqlens_host, conv_indices_host, apply_qk_l2norm)
    nah, nah_p = _host_i32(num_accepted_host)
    a = gdn_spec_prepare_args(base=base, conv_state_width=conv_state.shape[2],
                              num_accepted=_p(num_accepted), num_accepted_host=nah_p)
    _check(lib().gdn_spec_prepare(ctypes.byref(a), _stream(stream)))


def gdn_packed_decode(mixed_qkv, conv_weight, a_raw, b_raw, A_log, dt_bias, state_indices,
                      conv_state, state, out, *, Hk, Hv, Dk, Dv, K, scale=-1.0,
                      apply_qk_l2norm=True, state_indices_host=None, stream=None) -> None:
    """include/gdn.h gdn_packed_decode.  mixed_qkv [B, >= C_conv] raw rows
    (row stride taken from the tensor, so a [B, C_conv + Hv*Dv] qkvz tensor
    works as is); a_raw, b_raw [B, >= Hv] views (see packed_ba_views);
    conv_state and state are updated in place."""
    B_ = mixed_qkv.shape[0]
    sih, sih_p = _host_i32(state_indices_host)
    a = gdn_packed_decode_args(
        B=B_, Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, K=K, act_dtype=_dt(mixed_qkv),
        apply_qk_l2norm=int(apply_qk_l2norm), scale=float(scale),
        mixed_qkv=_p(mixed_qkv), mixed_qkv_stride=mixed_qkv.stride(0), mixed_qkv_len=_n(mixed_qkv),
        conv_weight=_p(conv_weight), conv_weight_len=_n(conv_weight),
        a_raw=_p(a_raw), a_raw_stride=a_raw.stride(0), a_raw_len=_n(a_raw),
        b_raw=_p(b_raw), b_raw_stride=b_raw.stride(0), b_raw_len=_n(b_raw),
        A_log=_p(A_log), A_log_len=_n(A_log), dt_bias=_p(dt_bias), dt_bias_len=_n(dt_bias),
        state_indices=_p(state_indices), state_indices_host=sih_p,
        conv_state=_p(conv_state), conv_state_len=_n(conv_state), state=_p(state),
        state_slots=state.shape[0], state_len=_n(state), out=_p(out), out_len=_n(out))
    _check(lib().gdn_packed_decode(ctypes.byref(a), _stream(stream)))


def packed_ba_views(ba: torch.Tensor, Hv: int):
    """(a_raw, b_raw) views of a merged gate tensor [T, 2*Hv] whose rows hold
    b then a ([cpu.rs] linear_attention_prepare_varlen_packed_qkvz_ba_f32)."""
    return ba[:, Hv:2 * Hv], ba[:, :Hv]


def _out_norm(norm_z, norm_weight, norm_eps, norm_sigmoid, tokens, Hv, Dv, in_kernel=False):
    """The gdn_out_norm option: None, or (struct, pointer) with z's row stride
    taken from the tensor (a [T, Hv, Dv] gate or a [T, >= Hv*Dv] slice)."""
    if norm_weight is None:
        return None, None
    zs = norm_z.stride(0)
    n = gdn_out_norm(z=_p(norm_z), z_len=max(tokens - 1, 0) * zs + Hv * Dv, z_token_stride=zs,
                     weight=_p(norm_weight), weight_len=_n(norm_weight), eps=float(norm_eps),
                     sigmoid_gate=int(bool(norm_sigmoid)), in_kernel=int(bool(in_kernel)))
    return n, ctypes.pointer(n)


def gdn_decode(q, k, v, g, beta, state, out, *, scale=-1.0, state_indices=None,
               state_indices_host=None, use_qk_l2norm=False, norm_z=None, norm_weight=None,
               norm_eps=1e-6, norm_sigmoid=False, norm_in_kernel=False, stream=None) -> None:
    """include/gdn.h gdn_decode; `state` [slots,Hv,Dv,Dk] f32 updated in place.
    With norm_weight (and norm_z) the gated RMSNorm is applied to `out`."""
    B, Hk, Dk = q.shape
    _, Hv, Dv = v.shape
    sih, sih_p = _host_i32(state_indices_host)
    nrm, nrm_p = _out_norm(norm_z, norm_weight, norm_eps, norm_sigmoid, B, Hv, Dv, norm_in_kernel)
    a = gdn_decode_args(
        B=B, Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, act_dtype=_dt(q), use_qk_l2norm=int(use_qk_l2norm),
        scale=float(scale), q=_p(q), q_len=_n(q), k=_p(k), k_len=_n(k), v=_p(v), v_len=_n(v),
        g=_p(g), g_len=_n(g), beta=_p(beta), beta_len=_n(beta), state=_p(state),
        state_slots=state.shape[0], state_len=_n(state), state_indices=_p(state_indices),
        state_indices_host=sih_p, out=_p(out), out_len=_n(out), out_norm=nrm_p)
    _check(lib().gdn_decode(ctypes.byref(a), _stream(stream)))


def gdn_kda_resolve_algo(T, N, Dk, Dv, act_dtype=GDN_DTYPE_BF16, algo=GDN_PREFILL_AUTO) -> int:
    return int(lib().gdn_kda_resolve_algo(T, N, Dk, Dv, act_dtype, algo))


def gdn_kda_workspace_bytes(T, N, Hv, Dk, Dv, act_dtype=GDN_DTYPE_BF16,
                            algo=GDN_PREFILL_AUTO) -> int:
    return int(lib().gdn_kda_workspace_bytes(T, N, Hv, Dk, Dv, act_dtype, algo))


def gdn_kda_varlen(q, k, v, g, beta, state, cu_seqlens, out, *, scale=-1.0, state_indices=None,
                   has_initial_state=None, cu_seqlens_host=None, state_indices_host=None,
                   algo=GDN_PREFILL_AUTO, workspace=None, stream=None) -> None:
    """include/gdn.h gdn_kda_varlen; g [T, Hv, Dk] f32; `state` updated in place.
    `workspace`: a uint8 device tensor of at least gdn_kda_workspace_bytes()
    bytes; when None and the resolved algorithm needs one, one is allocated
    here for the call."""
    T, Hk, Dk = q.shape
    _, Hv, Dv = v.shape
    N = cu_seqlens.numel() - 1
    cuh, cuh_p = _host_i32(cu_seqlens_host)
    sih, sih_p = _host_i32(state_indices_host)
    if workspace is None:
        nbytes = gdn_kda_workspace_bytes(T, N, Hv, Dk, Dv, _dt(q), algo)
        if nbytes:
            workspace = _scratch(nbytes, q.device, stream)
    a = gdn_kda_args(
        T=T, N=N, Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, act_dtype=_dt(q), scale=float(scale),
        q=_p(q), q_len=_n(q), k=_p(k), k_len=_n(k), v=_p(v), v_len=_n(v), g=_p(g), g_len=_n(g),
        beta=_p(beta), beta_len=_n(beta), state=_p(state), state_slots=state.shape[0],
        state_len=_n(state), cu_seqlens=_p(cu_seqlens), state_indices=_p(state_indices),
        has_initial_state=_p(has_initial_state), cu_seqlens_host=cuh_p,
        state_indices_host=sih_p, out=_p(out), out_len=_n(out), algo=int(algo),
        workspace=_p(workspace),
        workspace_bytes=0 if workspace is None else workspace.numel() * workspace.element_size())
    _check(lib().gdn_kda_varlen(ctypes.byref(a), _stream(stream)))


def gdn_spec_decode(q, k, v, g, beta, state, cu_seqlens, state_indices, num_accepted, out, *,
                    scale=-1.0, cu_seqlens_host=None, state_indices_host=None,
                    num_accepted_host=None, stream=None) -> None:
    """include/gdn.h gdn_spec_decode; state_indices [n_reqs, num_cols] int32;
    the snapshots are written into `state` in place."""
    T, Hk, Dk = q.shape
    _, Hv, Dv = v.shape
    n_reqs, num_cols = state_indices.shape
    cuh, cuh_p = _host_i32(cu_seqlens_host)
    sih, sih_p = _host_i32(state_indices_host)
    nah, nah_p = _host_i32(num_accepted_host)
    a = gdn_spec_decode_args(
        T=T, n_reqs=n_reqs, num_cols=num_cols, Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, act_dtype=_dt(q),
        scale=float(scale), q=_p(q), q_len=_n(q), k=_p(k), k_len=_n(k), v=_p(v), v_len=_n(v),
        g=_p(g), g_len=_n(g), beta=_p(beta), beta_len=_n(beta), state=_p(state),
        state_slots=state.shape[0], state_len=_n(state), cu_seqlens=_p(cu_seqlens),
        state_indices=_p(state_indices), num_accepted=_p(num_accepted), cu_seqlens_host=cuh_p,
        state_indices_host=sih_p, num_accepted_host=nah_p, out=_p(out), out_len=_n(out))
    _check(lib().gdn_spec_decode(ctypes.byref(a), _stream(stream)))


def gdn_gated_rmsnorm(core, z, weight, out, *, eps=1e-6, sigmoid_gate=False, stream=None) -> None:
    """include/gdn.h gdn_gated_rmsnorm.  core, out [T, H, D]; weight [D]; z
    [T, H, D] or a [T, >= H*D] tensor whose rows are the gate's token rows
    (e.g. a slice of a merged projection), row stride taken from it."""
    T, H, D = core.shape
    z_stride = z.stride(0)
    a = gdn_gated_rmsnorm_args(
        tokens=T, heads=H, dim=D, act_dtype=_dt(core), sigmoid_gate=int(bool(sigmoid_gate)),
        eps=float(eps), core=_p(core), core_len=_n(core), z=_p(z),
        z_len=(T - 1) * z_stride + H * D, z_token_stride=z_stride, weight=_p(weight),
        weight_len=_n(weight), out=_p(out), out_len=_n(out))
    _check(lib().gdn_gated_rmsnorm(ctypes.byref(a), _stream(stream)))


def gdn_prefill_workspace_bytes(T, N, Hv, Dk, Dv, act_dtype=GDN_DTYPE_BF16,
                                algo=GDN_PREFILL_AUTO) -> int:
    return int(lib().gdn_prefill_workspace_bytes(T, N, Hv, Dk, Dv, act_dtype, algo))


def gdn_prefill_resolve_algo(N, Hv, Dk, Dv, act_dtype=GDN_DTYPE_BF16,
                             algo=GDN_PREFILL_AUTO) -> int:
    return int(lib().gdn_prefill_resolve_algo(N, Hv, Dk, Dv, act_dtype, algo))


def gdn_prefill_varlen(q, k, v, g, beta, state, cu_seqlens, out, *, scale=-1.0,
                       state_indices=None, has_initial_state=None, cu_seqlens_host=None,
                       state_indices_host=None, use_qk_l2norm=False, algo=GDN_PREFILL_AUTO,
                       workspace=None, norm_z=None, norm_weight=None, norm_eps=1e-6,
                       norm_sigmoid=False, stream=None) -> None:
    """include/gdn.h gdn_prefill_varlen; `state` updated in place.  `workspace`
    is a uint8 device tensor of at least gdn_prefill_workspace_bytes() bytes.
    With norm_weight (and norm_z) the gated RMSNorm is applied to `out`."""
    T, Hk, Dk = q.shape
    _, Hv, Dv = v.shape
    N = cu_seqlens.numel() - 1
    cuh, cuh_p = _host_i32(cu_seqlens_host)
    sih, sih_p = _host_i32(state_indices_host)
    nrm, nrm_p = _out_norm(norm_z, norm_weight, norm_eps, norm_sigmoid, T, Hv, Dv)
    a = gdn_prefill_args(
        T=T, N=N, Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, act_dtype=_dt(q), use_qk_l2norm=int(use_qk_l2norm),
        scale=float(scale), algo=int(algo), q=_p(q), q_len=_n(q), k=_p(k), k_len=_n(k),
        v=_p(v), v_len=_n(v), g=_p(g), g_len=_n(g), beta=_p(beta), beta_len=_n(beta),
        state=_p(state), state_slots=state.shape[0], state_len=_n(state),
        cu_seqlens=_p(cu_seqlens), state_indices=_p(state_indices),
        has_initial_state=_p(has_initial_state), cu_seqlens_host=cuh_p,
        state_indices_host=sih_p, out=_p(out), out_len=_n(out), workspace=_p(workspace),
        workspace_bytes=0 if workspace is None else workspace.numel() * workspace.element_size(),
        out_norm=nrm_p)
    _check(lib().gdn_prefill_varlen(ctypes.byref(a), _stream(stream)))


# ---- full attention ----------------------------------------------------------------
#
# A decode step calls these once per layer, so their host side is kept short:
# each tensor is looked at once, and the argument structures are packed into one
# buffer per thread with struct (building them field by field through ctypes
# took 40 us for gdn_attn_prepare).

_MAX_BYTES = 1024


def _packer(cls):
    """struct.Struct of a ctypes structure's fields, nested ones in line."""
    def codes(c):
        out = ""
        for _, t in c._fields_:
            if issubclass(t, ctypes.Structure):
                out += codes(t)
            else:
                out += {_i64: "q", _i32: "i", _f32: "f", ctypes.c_size_t: "N"}.get(t, "P")
        return out
    s = struct.Struct("@" + codes(cls) + "0q")
    assert s.size == ctypes.sizeof(cls) <= _MAX_BYTES
    return s


_PREPARE = _packer(gdn_attn_prepare_args)
_VARLEN = _packer(gdn_attn_varlen_args)
_PAGED = _packer(gdn_attn_paged_args)
_CACHE = _packer(gdn_attn_cache)
_PREPARE8 = _packer(gdn_attn8_prepare_args)
_PAGED8 = _packer(gdn_attn8_paged_args)
_CACHE8 = _packer(gdn_attn_cache8)
_NO_ROWS = (0, 0, 0, 0)
_E4M3 = torch.float8_e4m3fn


class _Args(threading.local):
    """A thread's argument buffer and its address; the same for a cache."""

    def __init__(self):
        self.buf = ctypes.create_string_buffer(_MAX_BYTES)
        self.cache = ctypes.create_string_buffer(_MAX_BYTES)
        self.at, self.cache_at = ctypes.addressof(self.buf), ctypes.addressof(self.cache)


_args = _Args()
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


@functools.lru_cache(maxsize=4096)
def _workspace_need(device, name, *sizes) -> int:
    """Workspace bytes of a call of these sizes on this device (a decode step asks for the
    same ones again and again)."""
    return int(getattr(lib(), name)(*sizes))


def _bad(msg: str):
    return GdnError(GDN_ERR_INVALID_ARGUMENT, "GDN_ERR_INVALID_ARGUMENT", msg)


def _bad_shape(msg: str):
    return GdnError(GDN_ERR_SHAPE, "GDN_ERR_SHAPE", msg)


def _attn_check(name, t, shape, dtype, dev):
    """The C entries see sizes, not tensors: shape, type and device are checked here."""
    if t.shape != shape:
        raise _bad_shape(f"attention {name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if t.dtype is not dtype:
        raise GdnError(GDN_ERR_DTYPE, "GDN_ERR_DTYPE", f"attention {name} is {t.dtype}, not {dtype}")
    if t.device != dev:
        raise _bad(f"attention {name} is on {t.device}, not {dev}")


def _attn_rows(name, t, shape, dtype, dev):
    """The gdn_attn_rows of a [tokens, heads, D] view (any token and head stride)."""
    if t is None:
        return _NO_ROWS
    if t.shape != shape or t.dtype is not dtype or t.device != dev:
        _attn_check(name, t, shape, dtype, dev)
    n, h, d = shape
    ts, hs, ds = t.stride()
    if ds != 1:
        raise _bad(f"attention {name}'s last dimension must be contiguous")
    # A dimension of one entry has no step of its own: its stride is free.
    if n == 1:
        ts = 0
    elif ts == 0:
        raise _bad(f"attention {name} is a broadcast view; pass real rows")
    if h == 1:
        hs = 0
    elif hs == 0:
        raise _bad(f"attention {name} is a broadcast view; pass real rows")
    return t.data_ptr(), (n - 1) * ts + (h - 1) * hs + d, ts, hs


def _attn_flat(name, t, shape, dtype, dev):
    """Address and length of a contiguous tensor (0, 0 for None)."""
    if t is None:
        return 0, 0
    if t.shape != shape or t.dtype is not dtype or t.device != dev:
        _attn_check(name, t, shape, dtype, dev)
    if not t.is_contiguous():
        raise _bad(f"attention {name} must be contiguous")
    return t.data_ptr(), t.numel()


def _attn_i32(name, t, n, dev):
    """Address of a contiguous int32 [n] (0 for None)."""
    if t is None:
        return 0
    if t.shape != (n,) or t.dtype is not torch.int32 or t.device != dev:
        _attn_check(name, t, (n,), torch.int32, dev)
    if not t.is_contiguous():
        raise _bad(f"attention {name} must be contiguous")
    return t.data_ptr()


def _attn_cache(k_cache, v_cache, block_table, N, Hkv, D, dtype, dev, block_table_host, scales=None):
    """Packs the gdn_attn_cache of k_cache, v_cache [pages, Hkv, page_size, D]
    (any strides but the last) and block_table [N, max_pages] int32 into the
    thread's buffer, as a gdn_attn_cache8 with the scales (k_scale, v_scale) of
    one in 8 bits; returns its address and the host mirror to keep."""
    shape = k_cache.shape
    P, _, page, _ = shape if len(shape) == 4 else (0, 0, 0, 0)
    shape = (P, Hkv, page, D)
    parts = []
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if t.shape != shape or t.dtype is not dtype or t.device != dev:
            _attn_check(name, t, shape, dtype, dev)
        ps, hs, ts, ds = t.stride()
        if ds != 1:
            raise _bad(f"attention {name}'s last dimension must be contiguous")
        if (P > 1 and ps == 0) or (Hkv > 1 and hs == 0) or (page > 1 and ts == 0):
            raise _bad(f"attention {name} is a broadcast view; pass a real cache")
        parts += (t.data_ptr(), (P - 1) * ps + (Hkv - 1) * hs + (page - 1) * ts + D,
                  ps if P > 1 else 0, hs if Hkv > 1 else 0, ts if page > 1 else 0)
    rows = block_table.shape
    if len(rows) != 2:
        raise _bad_shape("attention block_table must be [N, max_pages]")
    width = rows[1]
    if rows[0] != N or block_table.dtype is not torch.int32 or block_table.device != dev:
        _attn_check("block_table", block_table, (N, width), torch.int32, dev)
    row, one = block_table.stride()
    if width > 1 and one != 1:
        raise _bad("attention block_table's last dimension must be contiguous")
    if N <= 1:
        row = 0
    host, host_p = None, 0
    if block_table_host is not None:
        host, host_p = _host_i32(block_table_host)
        if host.shape != block_table.shape:
            raise _bad_shape("attention block_table_host must have block_table's shape")
        if N > 1 and row != width:  # the mirror shares the row stride
            wide = torch.zeros((N, row), dtype=torch.int32)
            wide[:, :width] = host
            host, host_p = wide, wide.data_ptr()
    if scales is None:
        _CACHE.pack_into(_args.cache, 0, *parts, P, page, block_table.data_ptr(), width, row,
                         host_p or 0)
        return _args.cache_at, host
    blocks = scales[0].shape[-1] if scales[0].dim() == 3 else 0
    if blocks == 0 or page % blocks != 0:
        raise _bad_shape(f"attention k_scale has shape {tuple(scales[0].shape)}, not [{P}, {Hkv}, "
                         f"blocks of a page of {page} rows]")
    shape = (P, Hkv, blocks)
    _CACHE8.pack_into(_args.cache, 0, *parts, P, page, block_table.data_ptr(), width, row,
                      host_p or 0, *_attn_flat("k_scale", scales[0], shape, torch.float32, dev),
                      *_attn_flat("v_scale", scales[1], shape, torch.float32, dev), page // blocks)
    return _args.cache_at, host


def _attn_mirror(name, t, n):
    if t is None:
        return None, 0
    h, p = _host_i32(t)
    if h.numel() != n:
        raise _bad_shape(f"attention {name} holds {h.numel()} entries, not {n}")
    return h, p


def _attn_dims(q, kv, cu_seqlens):
    shape, heads = q.shape, kv.shape
    if len(shape) != 3 or len(heads) < 2:
        raise _bad_shape("attention query must be [tokens, heads, D]")
    T, Hq, D = shape
    return T, (T if cu_seqlens is None else cu_seqlens.numel() - 1), Hq, heads[1], D


def _attn_call(fn, q, stream) -> None:
    if not q.is_cuda:
        raise _bad(f"attention tensors must be on a CUDA device, got {q.device}")
    if stream is not None:
        s = stream.cuda_stream
    elif _raw_stream is not None:
        s = _raw_stream(q.device.index)
    else:
        s = torch.cuda.current_stream(q.device).cuda_stream
    if q.device.index != _current_device():  # the library launches on the current device
        with torch.cuda.device(q.device):
            _check(fn(_args.at, s))
    else:
        _check(fn(_args.at, s))


def _attn_prepare(packer, fn, q, k, v, cu_seqlens, q_out, kv_lens, block_table, k_cache, v_cache,
                  scales, k_out, q_norm_weight, k_norm_weight, norm_eps, cos_sin, positions,
                  cu_seqlens_host, kv_lens_host, block_table_host, stream):
    """The prepare calls; scales: of a cache in 8 bits, whose address then ends the arguments."""
    T, N, Hq, Hkv, D = _attn_dims(q, k, cu_seqlens)
    dt, dev = q.dtype, q.device
    keep_cu, cu_host = _attn_mirror("cu_seqlens_host", cu_seqlens_host, N + 1)
    keep_kv, kv_host = _attn_mirror("kv_lens_host", kv_lens_host, N)
    keep_table, cache = None, 0
    if k_cache is not None or v_cache is not None or block_table is not None:
        if k_cache is None or v_cache is None or block_table is None:
            raise _bad("attention cache needs k_cache, v_cache and block_table")
        cache, keep_table = _attn_cache(k_cache, v_cache, block_table, N, Hkv, D,
                                        dt if scales is None else _E4M3, dev, block_table_host,
                                        scales)
    rot, cs = 0, (0, 0)
    if cos_sin is not None:
        rot = cos_sin.shape[-1]
        cs = _attn_flat("cos_sin", cos_sin, (cos_sin.shape[0], rot), torch.float32, dev)
    packer.pack_into(
        _args.buf, 0, T, N, Hq, Hkv, D, rot, _dt(q), norm_eps,
        *_attn_rows("query", q, (T, Hq, D), dt, dev), *_attn_rows("key", k, (T, Hkv, D), dt, dev),
        *_attn_rows("value", v, (T, Hkv, D), dt, dev),
        *_attn_flat("q_norm_weight", q_norm_weight, (D,), dt, dev),
        *_attn_flat("k_norm_weight", k_norm_weight, (D,), dt, dev), *cs,
        _attn_i32("positions", positions, T, dev),
        _attn_i32("cu_seqlens", cu_seqlens, N + 1, dev),
        _attn_i32("kv_lens", kv_lens, N, dev), cu_host, kv_host, cache if scales is None else 0,
        *_attn_flat("q_out", q_out, (T, Hq, D), dt, dev),
        *_attn_flat("k_out", k_out, (T, Hkv, D), dt, dev), *(() if scales is None else (cache,)))
    _attn_call(fn, q, stream)


def gdn_attn_prepare(q, k, v, cu_seqlens, q_out, *, kv_lens=None, block_table=None, k_cache=None,
                     v_cache=None, k_out=None, q_norm_weight=None, k_norm_weight=None,
                     norm_eps=1e-6, cos_sin=None, positions=None, cu_seqlens_host=None,
                     kv_lens_host=None, block_table_host=None, stream=None) -> None:
    """include/gdn.h gdn_attn_prepare.  q [T, Hq, D], k, v [T, Hkv, D] views of
    the projection rows; q_out [T, Hq, D] and k_out [T, Hkv, D] are written, and
    the new rows of k_cache, v_cache [pages, Hkv, page_size, D] in place.
    cos_sin [positions, rot_dim] f32; cu_seqlens None: one token per sequence."""
    _attn_prepare(_PREPARE, (_lib or lib()).gdn_attn_prepare, q, k, v, cu_seqlens, q_out, kv_lens,
                  block_table, k_cache, v_cache, None, k_out, q_norm_weight, k_norm_weight, norm_eps,
                  cos_sin, positions, cu_seqlens_host, kv_lens_host, block_table_host, stream)


def gdn_attn8_prepare(q, k, v, cu_seqlens, q_out, *, kv_lens=None, block_table, k_cache, v_cache,
                      k_scale, v_scale, k_out=None, q_norm_weight=None, k_norm_weight=None,
                      norm_eps=1e-6, cos_sin=None, positions=None, cu_seqlens_host=None,
                      kv_lens_host=None, block_table_host=None, stream=None) -> None:
    """include/gdn.h gdn_attn8_prepare: gdn_attn_prepare into a cache in 8 bits.
    k_cache, v_cache [pages, Hkv, page_size, D] float8_e4m3fn; k_scale, v_scale
    [pages, Hkv, page_size / block] f32."""
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache), ("block_table", block_table),
                    ("k_scale", k_scale), ("v_scale", v_scale)):
        if t is None:
            raise _bad(f"{name} is NULL")
    _attn_prepare(_PREPARE8, (_lib or lib()).gdn_attn8_prepare, q, k, v, cu_seqlens, q_out, kv_lens,
                  block_table, k_cache, v_cache, (k_scale, v_scale), k_out, q_norm_weight,
                  k_norm_weight, norm_eps, cos_sin, positions, cu_seqlens_host, kv_lens_host,
                  block_table_host, stream)


def gdn_attn_varlen(q, k, v, cu_seqlens, out, *, scale=-1.0, gate=None, lse=None,
                    cu_seqlens_host=None, stream=None) -> None:
    """include/gdn.h gdn_attn_varlen.  q, gate [T, Hq, D], k, v [T, Hkv, D] (any
    token and head strides); out [T, Hq, D] and lse [T, Hq] f32 are written."""
    T, N, Hq, Hkv, D = _attn_dims(q, k, cu_seqlens)
    dt, dev = q.dtype, q.device
    keep, cu_host = _attn_mirror("cu_seqlens_host", cu_seqlens_host, N + 1)
    _VARLEN.pack_into(
        _args.buf, 0, T, N, Hq, Hkv, D, _dt(q), scale,
        *_attn_rows("query", q, (T, Hq, D), dt, dev), *_attn_rows("key", k, (T, Hkv, D), dt, dev),
        *_attn_rows("value", v, (T, Hkv, D), dt, dev),
        *_attn_rows("gate", gate, (T, Hq, D), dt, dev),
        _attn_i32("cu_seqlens", cu_seqlens, N + 1, dev), cu_host,
        *_attn_flat("out", out, (T, Hq, D), dt, dev),
        *_attn_flat("lse", lse, (T, Hq), torch.float32, dev))
    _attn_call((_lib or lib()).gdn_attn_varlen, q, stream)


def gdn_attn_paged_workspace_bytes(T, N, Hq, Hkv, D, max_q_len=0,
                                   act_dtype=GDN_DTYPE_BF16) -> int:
    return int(lib().gdn_attn_paged_workspace_bytes(T, N, Hq, Hkv, D, max_q_len, act_dtype))


def _attn_paged(packer, fn, q, k_cache, v_cache, scales, block_table, kv_lens, cu_seqlens, out,
                max_q_len, scale, gate, lse, workspace, cu_seqlens_host, kv_lens_host,
                block_table_host, stream):
    """The paged calls; scales: of a cache in 8 bits, whose address then ends the arguments."""
    if k_cache.dim() != 4:
        raise _bad_shape("attention k_cache must be [pages, Hkv, page_size, D]")
    T, N, Hq, Hkv, D = _attn_dims(q, k_cache, cu_seqlens)
    if kv_lens is None:
        raise _bad("kv_lens is NULL")
    dt, dev = q.dtype, q.device
    keep_cu, cu_host = _attn_mirror("cu_seqlens_host", cu_seqlens_host, N + 1)
    keep_kv, kv_host = _attn_mirror("kv_lens_host", kv_lens_host, N)
    cache, keep_table = _attn_cache(k_cache, v_cache, block_table, N, Hkv, D,
                                    dt if scales is None else _E4M3, dev, block_table_host, scales)
    if workspace is None:
        # Without offsets a call has one token per sequence, whatever max_q_len says.
        most = max_q_len if cu_seqlens is not None or scales is None else 1
        nbytes = (gdn_attn_paged_workspace_bytes(T, N, Hq, Hkv, D, most, _dt(q)) if scales is None else
                  _workspace_need(dev.index, "gdn_attn8_paged_workspace_bytes", T, N, Hq, Hkv, D,
                                  most, _dt(q), block_table.shape[1], k_cache.shape[2]))
        if nbytes:
            workspace = _scratch(nbytes, dev, stream)
    elif workspace.device != dev:
        raise _bad(f"attention workspace is on {workspace.device}, not {dev}")
    ws = (0, 0) if workspace is None else (workspace.data_ptr(),
                                           workspace.numel() * workspace.element_size())
    packer.pack_into(
        _args.buf, 0, T, N, Hq, Hkv, D, max_q_len, _dt(q), scale,
        *_attn_rows("query", q, (T, Hq, D), dt, dev), *_attn_rows("gate", gate, (T, Hq, D), dt, dev),
        _attn_i32("cu_seqlens", cu_seqlens, N + 1, dev),
        _attn_i32("kv_lens", kv_lens, N, dev), cu_host, kv_host,
        cache if scales is None else 0,
        *_attn_flat("out", out, (T, Hq, D), dt, dev),
        *_attn_flat("lse", lse, (T, Hq), torch.float32, dev), *ws,
        *(() if scales is None else (cache,)))
    _attn_call(fn, q, stream)


def gdn_attn_paged(q, k_cache, v_cache, block_table, kv_lens, cu_seqlens, out, *, max_q_len=0,
                   scale=-1.0, gate=None, lse=None, workspace=None, cu_seqlens_host=None,
                   kv_lens_host=None, block_table_host=None, stream=None) -> None:
    """include/gdn.h gdn_attn_paged.  q, gate [T, Hq, D]; k_cache, v_cache
    [pages, Hkv, page_size, D]; block_table [N, max_pages], kv_lens [N],
    cu_seqlens [N + 1] (None: one token per sequence) int32; out [T, Hq, D] and
    lse [T, Hq] f32 are written.  `workspace`: a uint8 device tensor of at least
    gdn_attn_paged_workspace_bytes() bytes; when None and one is needed, it is
    allocated here for the call."""
    _attn_paged(_PAGED, (_lib or lib()).gdn_attn_paged, q, k_cache, v_cache, None, block_table,
                kv_lens, cu_seqlens, out, max_q_len, scale, gate, lse, workspace, cu_seqlens_host,
                kv_lens_host, block_table_host, stream)


def gdn_attn8_paged_workspace_bytes(T, N, Hq, Hkv, D, max_q_len=0, act_dtype=GDN_DTYPE_BF16,
                                    max_pages=1, page_size=128) -> int:
    """max_pages, page_size: of the block table and cache that the call will have."""
    return int(lib().gdn_attn8_paged_workspace_bytes(T, N, Hq, Hkv, D, max_q_len, act_dtype,
                                                     max_pages, page_size))


def gdn_attn8_paged(q, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens, out, *,
                    max_q_len=0, scale=-1.0, gate=None, lse=None, workspace=None,
                    cu_seqlens_host=None, kv_lens_host=None, block_table_host=None,
                    stream=None) -> None:
    """include/gdn.h gdn_attn8_paged: gdn_attn_paged over a cache in 8 bits.  k_cache,
    v_cache [pages, Hkv, page_size, D] float8_e4m3fn; k_scale, v_scale [pages, Hkv,
    page_size / block] f32."""
    _attn_paged(_PAGED8, (_lib or lib()).gdn_attn8_paged, q, k_cache, v_cache, (k_scale, v_scale),
                block_table, kv_lens, cu_seqlens, out, max_q_len, scale, gate, lse, workspace,
                cu_seqlens_host, kv_lens_host, block_table_host, stream)


# ---- searches over several continuations ---------------------------------------------

_BEAM = _packer(gdn_beam_select_args)
_SLOTS = _packer(gdn_copy_slots_args)


def _on_device(name, what, t, shape, dtype, dev):
    """A contiguous tensor of this shape, type and device: its address and length."""
    if t.shape != shape:
        raise _bad_shape(f"{what} {name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if t.dtype is not dtype:
        raise GdnError(GDN_ERR_DTYPE, "GDN_ERR_DTYPE", f"{what} {name} is {t.dtype}, not {dtype}")
    if t.device != dev:
        raise _bad(f"{what} {name} is on {t.device}, not {dev}")
    if not t.is_contiguous():
        raise _bad(f"{what} {name} must be contiguous")
    return t.data_ptr(), t.numel()


def gdn_beam_select_workspace_bytes(B, W, V, K) -> int:
    return int(lib().gdn_beam_select_workspace_bytes(B, W, V, K))


def gdn_beam_select(logits, scores, parents, tokens, out_scores, *, finished=None, pad_token=0,
                    workspace=None, stream=None) -> None:
    """include/gdn.h gdn_beam_select.  logits [B, W, V] (bf16 or f32, the vocabulary
    contiguous, any other strides), scores [B, W] f32, finished [B, W] uint8 or bool;
    parents, tokens [B, K] int32 and out_scores [B, K] f32 are written.  `workspace`: a
    uint8 device tensor of at least gdn_beam_select_workspace_bytes() bytes; when None it
    is allocated here for the call."""
    if logits.dim() != 3 or parents.dim() != 2:
        raise _bad_shape("beam_select logits must be [B, W, V] and parents [B, K]")
    (n, W, V), K, dev = logits.shape, parents.shape[1], logits.device
    bs, ws, vs = logits.stride()
    if V > 1 and vs != 1:
        raise _bad("beam_select logits' last dimension must be contiguous")
    if (n > 1 and bs == 0) or (W > 1 and ws == 0):
        raise _bad("beam_select logits is a broadcast view; pass real rows")
    bs, ws = (bs if n > 1 else 0), (ws if W > 1 else 0)
    if bs < 0 or ws < 0:
        raise _bad_shape("beam_select logits strides out of range")
    beams = (n, W)
    fin = (0, 0)
    if finished is not None:
        if finished.dtype is torch.bool:
            finished = finished.view(torch.uint8)
        fin = _on_device("finished", "beam_select", finished, beams, torch.uint8, dev)
    sc = _on_device("scores", "beam_select", scores, beams, torch.float32, dev)
    outs = (n, K)
    par = _on_device("parents", "beam_select", parents, outs, torch.int32, dev)
    tok = _on_device("tokens", "beam_select", tokens, outs, torch.int32, dev)
    best = _on_device("out_scores", "beam_select", out_scores, outs, torch.float32, dev)
    if best[0] == sc[0] and K != W:
        raise _bad("beam_select out_scores may be scores only where K = W")
    dt = _dt(logits)
    if not logits.is_cuda:
        raise _bad(f"beam_select tensors must be on a CUDA device, got {dev}")
    if workspace is None:
        workspace = _scratch(_workspace_need(dev.index, "gdn_beam_select_workspace_bytes", n, W, V, K),
                             dev, stream)
    elif workspace.device != dev:
        raise _bad(f"beam_select workspace is on {workspace.device}, not {dev}")
    length = (n - 1) * bs + (W - 1) * ws + V if n > 0 and W > 0 else 0
    # A group stride of 0 stands for whole groups of beams: one group has no step of its own.
    _BEAM.pack_into(_args.buf, 0, n, W, V, K, dt, logits.data_ptr(), length, bs, ws, *sc, *fin,
                    int(pad_token), *par, *tok, *best, workspace.data_ptr(),
                    workspace.numel() * workspace.element_size())
    _attn_call((_lib or lib()).gdn_beam_select, logits, stream)


def gdn_copy_slots(pools, dst, src, *, groups=False, dst_host=None, src_host=None,
                   stream=None) -> None:
    """include/gdn.h gdn_copy_slots: pool[dst] = pool[src] for every tensor of `pools`
    (slots first, a slot's values contiguous), updated in place.  groups False: dst, src
    [n] int32 slots; True: dst [groups, W] the groups' slots, src [groups, W] places in the
    group (a search's parents)."""
    if not pools:
        raise _bad_shape("copy_slots needs at least one pool")
    dev = pools[0].device
    if dst.dim() != (2 if groups else 1):
        raise _bad_shape(f"copy_slots dst has shape {tuple(dst.shape)}, not "
                         f"{'[groups, W]' if groups else '[n]'}")
    d = _on_device("dst", "copy_slots", dst, dst.shape, torch.int32, dev)
    s = _on_device("src", "copy_slots", src, dst.shape, torch.int32, dev)
    rows = []
    for i, t in enumerate(pools):
        if t.device != dev:
            raise _bad(f"copy_slots pool {i} is on {t.device}, not {dev}")
        n = t.shape[0] if t.dim() else 0
        size = t.nbytes // n if n else 0
        if size == 0:
            raise _bad_shape(f"copy_slots pool {i} has shape {tuple(t.shape)}")
        stride = size
        if not t.is_contiguous():
            if not t[0].is_contiguous():
                raise _bad(f"copy_slots pool {i}: a slot's values must be contiguous")
            if n > 1:
                stride = t.stride(0) * t.element_size()
                if stride == 0:
                    raise _bad(f"copy_slots pool {i} is a broadcast view; pass a real pool")
        rows += (t.data_ptr(), (n - 1) * stride + size, n, size, stride)
    if not pools[0].is_cuda:
        raise _bad(f"copy_slots tensors must be on a CUDA device, got {dev}")
    table = struct.pack(f"@{len(rows)}q", *rows)
    keep = ctypes.create_string_buffer(table, len(table))
    mirrors = []
    for name, t in (("dst_host", dst_host), ("src_host", src_host)):
        h, p = _host_i32(t)
        if h is not None and h.numel() != d[1]:
            raise _bad_shape(f"copy_slots {name} holds {h.numel()} entries, not {d[1]}")
        mirrors.append((h, p or 0))
    _SLOTS.pack_into(_args.buf, 0, ctypes.addressof(keep), len(pools), d[1],
                     dst.shape[1] if groups else 0, d[0], s[0], mirrors[0][1], mirrors[1][1])
    _attn_call((_lib or lib()).gdn_copy_slots, pools[0], stream)


def _host_u8(t: Optional[torch.Tensor]):
    if t is None:
        return None, None
    h = t.detach().to("cpu", torch.uint8).contiguous()
    return h, h.data_ptr()


def gdn_validate_mixed(*, num_decodes, num_prefills, num_actual_tokens, state_slots,
                       cu_seqlens_host, state_indices_host, cu_seqlens_prefill_host,
                       has_initial_state_host=None, prefill_state_indices_host=None,
                       prefill_has_initial_state_host=None, num_decode_tokens=None,
                       num_prefill_tokens=None, allow_inert_padding=True) -> None:
    """include/gdn.h gdn_validate_mixed on host copies of a mixed step's
    metadata (tensors on any device; they are copied to the host).  Raises
    GdnError on the first broken rule; launches nothing."""
    nd_tok = num_decodes if num_decode_tokens is None else num_decode_tokens
    np_tok = (num_actual_tokens - nd_tok) if num_prefill_tokens is None else num_prefill_tokens
    cu, cu_p = _host_i32(cu_seqlens_host)
    si, si_p = _host_i32(state_indices_host)
    hi, hi_p = _host_u8(has_initial_state_host)
    cp, cp_p = _host_i32(cu_seqlens_prefill_host)
    ps, ps_p = _host_i32(prefill_state_indices_host)
    ph, ph_p = _host_u8(prefill_has_initial_state_host)
    nreq = num_decodes + num_prefills
    for name, t, n in (("cu_seqlens", cu, nreq + 1), ("state_indices", si, nreq),
                       ("has_initial_state", hi, nreq), ("cu_seqlens_prefill", cp, num_prefills + 1),
                       ("prefill_state_indices", ps, num_prefills),
                       ("prefill_has_initial_state", ph, num_prefills)):
        if t is not None and t.numel() < n:
            raise GdnError(GDN_ERR_SHAPE, "GDN_ERR_SHAPE",
                           f"{name} holds {t.numel()} entries, the step needs {n}")
    m = gdn_mixed_meta(num_decodes=num_decodes, num_prefills=num_prefills,
                       num_decode_tokens=nd_tok, num_prefill_tokens=np_tok,
                       num_actual_tokens=num_actual_tokens, state_slots=state_slots,
                       allow_inert_padding=int(bool(allow_inert_padding)),
                       cu_seqlens_host=cu_p, state_indices_host=si_p, has_initial_state_host=hi_p,
                       cu_seqlens_prefill_host=cp_p, prefill_state_indices_host=ps_p,
                       prefill_has_initial_state_host=ph_p)
    _check(lib().gdn_validate_mixed(ctypes.byref(m)))


def gdn_read_device_status(stream=None) -> None:
    """Synchronises the stream and raises GdnError if a kernel flagged an error."""
    _check(lib().gdn_read_device_status(_stream(stream)))


def gdn_check_wait_timeout(budget_cycles: int, stream=None) -> None:
    """include/gdn.h gdn_check_wait_timeout: one bounded device wait that runs
    out on purpose; gdn_read_device_status then raises GDN_ERR_TIMEOUT."""
    _check(lib().gdn_check_wait_timeout(int(budget_cycles), _stream(stream)))


def gdn_version() -> int:
    return int(lib().gdn_version())


def gdn_launch_count() -> int:
    """Kernel launches issued through the library by this process so far."""
    return int(lib().gdn_launch_count())
