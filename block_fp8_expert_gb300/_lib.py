"""ctypes binding of libmoe_fp8.so (include/moe_fp8.h).

Argument marshalling only: every function here passes device pointers, sizes
and the current CUDA stream to the C ABI of the same name and turns a non-zero
status into an exception.  Every step of the layer runs in the library's CUDA
kernels; there is no Python or CPU fallback, and a missing library raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_fp8.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_WORKSPACE = 3
MOE_ERR_CUDA = 4
MOE_ERR_DEVICE_STATUS = 5
MOE_ERR_TIMEOUT = 6
MOE_ERR_NOT_IMPLEMENTED = 7
MOE_DEV_BAD_EXPERT_INDEX = 1
MOE_DEV_WAIT_TIMEOUT = 2
MOE_DEV_FP16_RANGE = 4
MOE_DEV_NONFINITE = 8
MOE_DEV_BAD_PAGE = 16
MOE_DEV_BAD_POSITION = 32
MOE_SCORE_SOFTMAX = 0
MOE_SCORE_SIGMOID = 1
MOE_KV_BF16 = 0
MOE_KV_E4M3 = 1


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        super().__init__(f"{where}: status {status}: {message}")
        self.status = status


class Dims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
                ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("I_shared", ctypes.c_int32)]

    def __repr__(self):
        return (f"Dims(T={self.T}, H={self.H}, I={self.I}, E={self.E}, k={self.k}, "
                f"I_shared={self.I_shared})")


class Fp8Mat(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class Fp8Ffn(ctypes.Structure):
    _fields_ = [("gate", Fp8Mat), ("up", Fp8Mat), ("down", Fp8Mat)]


class SelectRule(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("top_groups", ctypes.c_int32), ("group_top", ctypes.c_int32),
                ("renorm", ctypes.c_int32), ("scale", ctypes.c_float)]


class KvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("D", ctypes.c_int32),
                ("format", ctypes.c_int32), ("page_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("scale_page_stride", ctypes.c_int64), ("scale_head_stride", ctypes.c_int64),
                ("scale_token_stride", ctypes.c_int64)]


class QkDims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("Hq", ctypes.c_int32), ("rot", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("n_pos", ctypes.c_int32),
                ("eps", ctypes.c_float), ("qkv_stride", ctypes.c_int64),
                ("q_stride", ctypes.c_int64)]


class AttnDims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("table_width", ctypes.c_int32),
                ("window", ctypes.c_int32), ("scale", ctypes.c_float),
                ("table_stride", ctypes.c_int64), ("q_stride", ctypes.c_int64),
                ("out_stride", ctypes.c_int64)]


class LinearDims(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
                ("x_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64)]


class DraftDims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("n", ctypes.c_int32), ("Hq", ctypes.c_int32),
                ("table_width", ctypes.c_int32), ("window", ctypes.c_int32),
                ("scale", ctypes.c_float), ("table_stride", ctypes.c_int64),
                ("q_stride", ctypes.c_int64), ("q_row_stride", ctypes.c_int64),
                ("out_stride", ctypes.c_int64), ("out_row_stride", ctypes.c_int64),
                ("mask_stride", ctypes.c_int64)]


class LatentPages(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("R", ctypes.c_int32), ("rot", ctypes.c_int32),
                ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64)]


class LatentDims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("n_pos", ctypes.c_int32), ("eps", ctypes.c_float), ("kv_stride", ctypes.c_int64),
                ("q_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
                ("q_out_stride", ctypes.c_int64), ("q_out_head_stride", ctypes.c_int64),
                ("rows_stride", ctypes.c_int64)]


class ExpandedDims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("Tq", ctypes.c_int32), ("Tk", ctypes.c_int32),
                ("H", ctypes.c_int32), ("scale", ctypes.c_float), ("q_stride", ctypes.c_int64),
                ("q_head_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("k_head_stride", ctypes.c_int64), ("rope_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("v_head_stride", ctypes.c_int64),
                ("out_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64)]


_vp = ctypes.c_void_p
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64
_sz = ctypes.c_size_t
_st = ctypes.c_int32

_SIGNATURES = {
    "moe_status_string": (ctypes.c_char_p, [_st]),
    "moe_last_error_message": (ctypes.c_char_p, []),
    "moe_version": (ctypes.c_char_p, []),
    "moe_kernel_launches": (ctypes.c_ulonglong, []),
    "moe_expert_uses_gemm": (ctypes.c_int, [Dims]),
    "moe_workspace_bytes": (_st, [Dims, ctypes.POINTER(_sz)]),
    "moe_route": (_st, [_vp, _vp, _vp, Dims, _vp, _vp, _vp, _sz, _vp]),
    "moe_permute": (_st, [_vp, Dims, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_expert_ffn_fp8": (_st, [_vp, _vp, _vp, Fp8Ffn, Dims, _vp, _vp, _sz, _vp]),
    "moe_combine": (_st, [_vp, _vp, _vp, _vp, Dims, _vp, _vp]),
    "moe_layer_forward": (_st, [_vp, _vp, _vp, Fp8Ffn, ctypes.POINTER(Fp8Ffn), Dims, _vp, _vp,
                                _vp, _vp, _sz, _vp]),
    "moe_layer_forward_gated": (_st, [_vp, _vp, _vp, Fp8Ffn, ctypes.POINTER(Fp8Ffn), _vp, Dims,
                                      _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_layer_forward_act8": (_st, [_vp, _vp, _vp, Fp8Ffn, Dims, _vp, _vp, _vp, _vp, _sz,
                                     _vp]),
    "moe_verify_workspace_bytes": (_st, [Dims, ctypes.c_int, ctypes.POINTER(_sz)]),
    "moe_verify_layer": (_st, [_vp, Fp8Ffn, ctypes.POINTER(Fp8Ffn), _vp, Dims, _vp, _vp, _vp,
                               _vp, ctypes.c_int, _vp, _vp, _sz, _vp]),
    "moe_read_device_status": (_st, [_vp, ctypes.POINTER(ctypes.c_int32), _vp]),
    "moe_permute_static_scratch": (_st, [_vp, Dims, _vp, _vp, _vp, _vp]),
    "moe_select_experts": (_st, [_vp, _i64, _vp, SelectRule, _i32, _i32, _i32, _vp, _vp, _vp]),
    "moe_route_select": (_st, [_vp, _vp, _vp, _vp, SelectRule, Dims, _vp, _vp, _vp, _sz, _vp]),
    "moe_route_select_status": (_st, [_vp, _vp, _vp, _vp, SelectRule, Dims, _vp, _vp, _vp, _sz, _vp,
                                      _vp]),
    "moe_experts_forward": (_st, [_vp, _vp, _vp, Fp8Ffn, ctypes.POINTER(Fp8Ffn), _vp, Dims, _vp,
                                  _vp, _sz, _vp, _vp]),
    "moe_qk_norm_rope": (_st, [_vp, _vp, _vp, _vp, _vp, _vp, QkDims, KvCache, _vp, _vp, _vp]),
    "moe_paged_attention_workspace_bytes": (_st, [AttnDims, _i32, ctypes.POINTER(_sz)]),
    "moe_paged_attention": (_st, [_vp, KvCache, _vp, _vp, AttnDims, _vp, _vp, _sz, _vp, _vp]),
    "moe_tree_attention_workspace_bytes": (_st, [DraftDims, _i32, _i32, ctypes.POINTER(_sz)]),
    "moe_tree_attention": (_st, [_vp, KvCache, _vp, _vp, _vp, _vp, DraftDims, _vp, _vp, _sz, _vp,
                                 _vp]),
    "moe_latent_store": (_st, [_vp, _vp, _vp, _vp, _vp, _vp, LatentDims, LatentPages, _vp, _vp, _vp,
                               _vp]),
    "moe_latent_attention_workspace_bytes": (_st, [DraftDims, _i32, ctypes.POINTER(_sz)]),
    "moe_latent_attention": (_st, [_vp, LatentPages, _vp, _vp, _vp, _vp, DraftDims, _vp, _vp, _sz,
                                   _vp, _vp]),
    "moe_expanded_attention": (_st, [_vp, _vp, _vp, _vp, _vp, _vp, ExpandedDims, _vp, _vp, _vp]),
    "moe_linear_fp8_workspace_bytes": (_st, [LinearDims, ctypes.POINTER(_sz)]),
    "moe_linear_fp8": (_st, [_vp, Fp8Mat, _vp, LinearDims, _vp, _vp, _sz, _vp, _vp]),
}

_lib: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """The loaded library.  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with block_fp8_expert_gb300.build.build(); "
                "this package has no CPU fallback")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _check(status: int, where: str) -> None:
    if status != MOE_OK:
        msg = lib().moe_last_error_message().decode()
        raise MoeError(status, where, msg)


def _ptr(t) -> Optional[int]:
    """Device address of a tensor (or an int address, or None)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    import torch
    return torch.cuda.current_stream().cuda_stream


def dims(T: int, H: int, I: int, E: int, k: int, I_shared: int = 0) -> Dims:
    return Dims(T, H, I, E, k, I_shared)


def ffn(gate_codes, gate_scales, up_codes, up_scales, down_codes, down_scales) -> Fp8Ffn:
    return Fp8Ffn(Fp8Mat(_ptr(gate_codes), _ptr(gate_scales)),
                  Fp8Mat(_ptr(up_codes), _ptr(up_scales)),
                  Fp8Mat(_ptr(down_codes), _ptr(down_scales)))


def version() -> str:
    return lib().moe_version().decode()


def kernel_launches() -> int:
    """Kernel launches this library has issued in this process (diagnostic)."""
    return int(lib().moe_kernel_launches())


def expert_uses_gemm(d) -> bool:
    """True if a layer call with dims d runs its routed experts on the
    tensor-core GEMM (diagnostic; raises on invalid dims)."""
    r = int(lib().moe_expert_uses_gemm(d))
    if r < 0:
        raise ValueError("invalid moe_dims")
    return r == 1


def status_string(status: int) -> str:
    return lib().moe_status_string(status).decode()


def workspace_bytes(d: Dims) -> int:
    n = _sz(0)
    _check(lib().moe_workspace_bytes(d, ctypes.byref(n)), "moe_workspace_bytes")
    return n.value


def _nbytes(ws) -> int:
    return ws.numel() * ws.element_size()


def moe_route(x, Wr, bias, d: Dims, topk_idx, topk_w, ws, stream=None) -> None:
    _check(lib().moe_route(_ptr(x), _ptr(Wr), _ptr(bias), d, _ptr(topk_idx), _ptr(topk_w),
                           _ptr(ws), _nbytes(ws), _stream(stream)), "moe_route")


def moe_permute(topk_idx, d: Dims, expert_off, row_token, tok_slot_row, ws, stream=None) -> None:
    _check(lib().moe_permute(_ptr(topk_idx), d, _ptr(expert_off), _ptr(row_token),
                             _ptr(tok_slot_row), _ptr(ws), _nbytes(ws), _stream(stream)),
           "moe_permute")


def moe_permute_static_scratch(topk_idx, d: Dims, expert_off, row_token, tok_slot_row,
                               stream=None) -> None:
    """moe_permute with its scratch in the library's fixed device array
    (no workspace argument; T*k <= 65536, E <= 512)."""
    _check(lib().moe_permute_static_scratch(_ptr(topk_idx), d, _ptr(expert_off),
                                            _ptr(row_token), _ptr(tok_slot_row),
                                            _stream(stream)), "moe_permute_static_scratch")


def moe_expert_ffn_fp8(x, expert_off, row_token, w: Fp8Ffn, d: Dims, y_perm, ws,
                       stream=None) -> None:
    _check(lib().moe_expert_ffn_fp8(_ptr(x), _ptr(expert_off), _ptr(row_token), w, d,
                                    _ptr(y_perm), _ptr(ws), _nbytes(ws), _stream(stream)),
           "moe_expert_ffn_fp8")


def moe_combine(y_perm, tok_slot_row, topk_w, shared_y, d: Dims, out, stream=None) -> None:
    _check(lib().moe_combine(_ptr(y_perm), _ptr(tok_slot_row), _ptr(topk_w), _ptr(shared_y), d,
                             _ptr(out), _stream(stream)), "moe_combine")


def moe_layer_forward(x, Wr, bias, routed: Fp8Ffn, shared: Optional[Fp8Ffn], d: Dims, out,
                      topk_idx_out, topk_w_out, ws, stream=None) -> None:
    sh = ctypes.byref(shared) if shared is not None else None
    _check(lib().moe_layer_forward(_ptr(x), _ptr(Wr), _ptr(bias), routed, sh, d, _ptr(out),
                                   _ptr(topk_idx_out), _ptr(topk_w_out), _ptr(ws), _nbytes(ws),
                                   _stream(stream)), "moe_layer_forward")


def moe_layer_forward_gated(x, Wr, bias, routed: Fp8Ffn, shared: Fp8Ffn, shared_gate, d: Dims,
                            out, topk_idx_out, topk_w_out, ws, stream=None) -> None:
    _check(lib().moe_layer_forward_gated(_ptr(x), _ptr(Wr), _ptr(bias), routed,
                                         ctypes.byref(shared), _ptr(shared_gate), d, _ptr(out),
                                         _ptr(topk_idx_out), _ptr(topk_w_out), _ptr(ws),
                                         _nbytes(ws), _stream(stream)), "moe_layer_forward_gated")


def moe_layer_forward_act8(x, Wr, bias, routed: Fp8Ffn, d: Dims, out, topk_idx_out, topk_w_out,
                           ws, stream=None) -> None:
    _check(lib().moe_layer_forward_act8(_ptr(x), _ptr(Wr), _ptr(bias), routed, d, _ptr(out),
                                        _ptr(topk_idx_out), _ptr(topk_w_out), _ptr(ws),
                                        _nbytes(ws), _stream(stream)), "moe_layer_forward_act8")


def verify_workspace_bytes(d: Dims, n_tokens: int) -> int:
    n = _sz(0)
    _check(lib().moe_verify_workspace_bytes(d, n_tokens, ctypes.byref(n)),
           "moe_verify_workspace_bytes")
    return n.value


def moe_verify_layer(x, routed: Fp8Ffn, shared: Optional[Fp8Ffn], shared_gate, d: Dims, out,
                     topk_idx, topk_w, tokens, result, ws, stream=None) -> None:
    sh = ctypes.byref(shared) if shared is not None else None
    _check(lib().moe_verify_layer(_ptr(x), routed, sh, _ptr(shared_gate), d, _ptr(out),
                                  _ptr(topk_idx), _ptr(topk_w), _ptr(tokens),
                                  int(tokens.numel()), _ptr(result), _ptr(ws), _nbytes(ws),
                                  _stream(stream)), "moe_verify_layer")


def moe_read_device_status(ws, stream=None) -> int:
    """The workspace's device status bits; raises MoeError when any is set.
    ws=None reads the status word of moe_permute_static_scratch's fixed array."""
    v = ctypes.c_int32(0)
    st = lib().moe_read_device_status(_ptr(ws), ctypes.byref(v), _stream(stream))
    if st not in (MOE_OK, MOE_ERR_DEVICE_STATUS):
        _check(st, "moe_read_device_status")
    if st == MOE_ERR_DEVICE_STATUS:
        raise MoeError(st, "moe_read_device_status", f"device status bits 0x{v.value:x}")
    return v.value


def moe_select_experts(logits, row_stride: int, bias, rule: SelectRule, T: int, E: int, k: int,
                       topk_idx, topk_w, stream=None) -> None:
    _check(lib().moe_select_experts(_ptr(logits), row_stride, _ptr(bias), rule, T, E, k,
                                    _ptr(topk_idx), _ptr(topk_w), _stream(stream)),
           "moe_select_experts")


def moe_route_select(x, Wr, logit_bias, bias, rule: SelectRule, d: Dims, topk_idx, topk_w, ws,
                     status=None, stream=None) -> None:
    _check(lib().moe_route_select_status(_ptr(x), _ptr(Wr), _ptr(logit_bias), _ptr(bias), rule, d,
                                         _ptr(topk_idx), _ptr(topk_w), _ptr(ws), _nbytes(ws),
                                         _ptr(status), _stream(stream)), "moe_route_select")


def moe_experts_forward(x, topk_idx, topk_w, routed: Fp8Ffn, shared: Optional[Fp8Ffn], shared_gate,
                        d: Dims, out, ws, status=None, stream=None) -> None:
    sh = ctypes.byref(shared) if shared is not None else None
    _check(lib().moe_experts_forward(_ptr(x), _ptr(topk_idx), _ptr(topk_w), routed, sh,
                                     _ptr(shared_gate), d, _ptr(out), _ptr(ws), _nbytes(ws),
                                     _ptr(status), _stream(stream)), "moe_experts_forward")


def moe_qk_norm_rope(qkv, q_norm, k_norm, cos_sin, pos, slots, d: QkDims, cache: KvCache, q_out,
                     status=None, stream=None) -> None:
    _check(lib().moe_qk_norm_rope(_ptr(qkv), _ptr(q_norm), _ptr(k_norm), _ptr(cos_sin), _ptr(pos),
                                  _ptr(slots), d, cache, _ptr(q_out), _ptr(status),
                                  _stream(stream)), "moe_qk_norm_rope")


def paged_attention_workspace_bytes(d: AttnDims, D: int) -> int:
    n = _sz(0)
    _check(lib().moe_paged_attention_workspace_bytes(d, D, ctypes.byref(n)),
           "moe_paged_attention_workspace_bytes")
    return n.value


def moe_paged_attention(q, cache: KvCache, block_table, seq_lens, d: AttnDims, out, ws,
                        status=None, stream=None) -> None:
    _check(lib().moe_paged_attention(_ptr(q), cache, _ptr(block_table), _ptr(seq_lens), d,
                                     _ptr(out), _ptr(ws), _nbytes(ws), _ptr(status),
                                     _stream(stream)), "moe_paged_attention")


def tree_attention_workspace_bytes(d: DraftDims, Hkv: int, D: int) -> int:
    n = _sz(0)
    _check(lib().moe_tree_attention_workspace_bytes(d, Hkv, D, ctypes.byref(n)),
           "moe_tree_attention_workspace_bytes")
    return n.value


def moe_tree_attention(q, cache: KvCache, block_table, seq_lens, mask, draft_lens, d: DraftDims, out,
                       ws, status=None, stream=None) -> None:
    _check(lib().moe_tree_attention(_ptr(q), cache, _ptr(block_table), _ptr(seq_lens), _ptr(mask),
                                    _ptr(draft_lens), d, _ptr(out), _ptr(ws), _nbytes(ws),
                                    _ptr(status), _stream(stream)), "moe_tree_attention")


def moe_latent_store(kv, norm, cos_sin, pos, slots, q, d: LatentDims, cache: LatentPages, q_out, rows,
                     status=None, stream=None) -> None:
    _check(lib().moe_latent_store(_ptr(kv), _ptr(norm), _ptr(cos_sin), _ptr(pos), _ptr(slots), _ptr(q),
                                  d, cache, _ptr(q_out), _ptr(rows), _ptr(status), _stream(stream)),
           "moe_latent_store")


def latent_attention_workspace_bytes(d: DraftDims, R: int) -> int:
    n = _sz(0)
    _check(lib().moe_latent_attention_workspace_bytes(d, R, ctypes.byref(n)),
           "moe_latent_attention_workspace_bytes")
    return n.value


def moe_latent_attention(q, cache: LatentPages, block_table, seq_lens, mask, draft_lens, d: DraftDims,
                         out, ws, status=None, stream=None) -> None:
    _check(lib().moe_latent_attention(_ptr(q), cache, _ptr(block_table), _ptr(seq_lens), _ptr(mask),
                                      _ptr(draft_lens), d, _ptr(out), _ptr(ws), _nbytes(ws),
                                      _ptr(status), _stream(stream)), "moe_latent_attention")


def moe_expanded_attention(q, k_nope, k_rope, v, cu_q, cu_k, d: ExpandedDims, out, status=None,
                           stream=None) -> None:
    _check(lib().moe_expanded_attention(_ptr(q), _ptr(k_nope), _ptr(k_rope), _ptr(v), _ptr(cu_q),
                                        _ptr(cu_k), d, _ptr(out), _ptr(status), _stream(stream)),
           "moe_expanded_attention")


def linear_fp8_workspace_bytes(d: LinearDims) -> int:
    n = _sz(0)
    _check(lib().moe_linear_fp8_workspace_bytes(d, ctypes.byref(n)),
           "moe_linear_fp8_workspace_bytes")
    return n.value


def moe_linear_fp8(x, w: Fp8Mat, bias, d: LinearDims, out, ws, status=None, stream=None) -> None:
    _check(lib().moe_linear_fp8(_ptr(x), w, _ptr(bias), d, _ptr(out), _ptr(ws), _nbytes(ws),
                                _ptr(status), _stream(stream)), "moe_linear_fp8")


EXPORTED = tuple(_SIGNATURES)
