"""The operators of a decoder layer around the MoE layer, on PyTorch tensors.

    ExpertSelector   router logits -> chosen experts and weights
    QkNormRope       head norms, rotary positions, store into a paged cache
    PagedCache       the paged key/value cache (bf16 or E4M3)
    PagedAttention   attention of one new token per sequence over it
    Fp8Linear        x W^T with block-FP8 weights and E4M3 activations

Each object holds what a serving program sets up once; ``forward`` takes the
step's tensors, and output buffers and a workspace where the program keeps
them (they are allocated otherwise).  Everything runs in libmoe_fp8.so on the
current stream or the one given; tensors are checked for device, type and
layout here and for their sizes in the library.  What the kernels themselves
find wrong in their data (a page number outside the cache, say) is recorded in
``status``, a device array that ``check()`` reads after synchronising.
"""
from __future__ import annotations

import math
from typing import Optional

import torch

from . import _lib


def _need(t: torch.Tensor, name: str, dtype, ndim: int) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.dim() != ndim:
        raise TypeError(f"{name}: need a {ndim}-d {dtype} tensor, got "
                        f"{getattr(t, 'dtype', type(t))} {tuple(getattr(t, 'shape', ()))}")
    if not t.is_cuda:
        raise ValueError(f"{name} is not on a CUDA device")
    if ndim and t.numel() and t.stride(-1) != 1 and t.shape[-1] != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return t


def _shape(t: torch.Tensor, name: str, *shape) -> torch.Tensor:
    if tuple(t.shape) != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, need {shape}")
    return t


def _dense(t: Optional[torch.Tensor], name: str, dtype, *shape) -> Optional[torch.Tensor]:
    if t is None:
        return None
    _shape(_need(t, name, dtype, len(shape)), name, *shape)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _row_stride(t: torch.Tensor, width: int) -> int:
    """Elements between rows of a tensor whose rows are `width` wide."""
    return t.stride(0) if t.shape[0] > 1 else width


def _new(stream, *shape, dtype, device) -> torch.Tensor:
    """A tensor that a call on `stream` may still be using when the caller has
    dropped it: the allocator is told of a stream other than the current one."""
    t = torch.empty(*shape, dtype=dtype, device=device)
    if stream is not None:
        t.record_stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)
    return t


class _Status:
    """The device status word of one operator object."""

    def __init__(self, device):
        self.status = torch.zeros(16, dtype=torch.int32, device=device)

    def check(self, stream=None) -> None:
        """Synchronise and raise MoeError if a kernel flagged its data."""
        _lib.moe_read_device_status(self.status, stream)


class ExpertSelector:
    """Experts from router logits (moe_select_experts): softmax or sigmoid
    scores, a balance bias [E] that steers the choice only, `top_groups` of
    `groups` expert groups kept by the sum of their `group_top` largest keys,
    the k largest keys, weights renormalised and scaled."""

    def __init__(self, E: int, k: int, score: str = "softmax",
                 bias: Optional[torch.Tensor] = None, groups: int = 1, top_groups: int = 1,
                 group_top: int = 1, renorm: bool = True, scale: float = 1.0):
        if score not in ("softmax", "sigmoid"):
            raise ValueError(f"score {score!r}: need 'softmax' or 'sigmoid'")
        self.E, self.k = E, k
        self.bias = _dense(bias, "bias", torch.float32, E)
        self.rule = _lib.SelectRule(
            _lib.MOE_SCORE_SIGMOID if score == "sigmoid" else _lib.MOE_SCORE_SOFTMAX,
            groups, top_groups, group_top, int(bool(renorm)), scale)

    def forward(self, logits: torch.Tensor, topk_idx: Optional[torch.Tensor] = None,
                topk_w: Optional[torch.Tensor] = None, stream=None):
        """logits float32 [T, E] -> (topk_idx int32 [T, k], topk_w float32 [T, k])."""
        _need(logits, "logits", torch.float32, 2)
        T = logits.shape[0]
        _shape(logits, "logits", T, self.E)
        if topk_idx is None:
            topk_idx = _new(stream, T, self.k, dtype=torch.int32, device=logits.device)
        if topk_w is None:
            topk_w = _new(stream, T, self.k, dtype=torch.float32, device=logits.device)
        _dense(topk_idx, "topk_idx", torch.int32, T, self.k)
        _dense(topk_w, "topk_w", torch.float32, T, self.k)
        _lib.moe_select_experts(logits, _row_stride(logits, self.E), self.bias, self.rule, T,
                                self.E, self.k, topk_idx, topk_w, stream)
        return topk_idx, topk_w


class PagedCache:
    """A paged key/value cache over tensors [pages, Hkv, page_size, D]: bf16,
    or E4M3 codes (uint8 or float8_e4m3fn) with float32 scales [pages, Hkv,
    page_size].  Any strides with D contiguous will do (a cache kept as
    [pages, page_size, Hkv, D] is passed transposed); k and v, and the two
    scales, share theirs."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor,
                 k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None):
        self.e4m3 = k_scale is not None
        if self.e4m3:
            k = k.view(torch.uint8) if k.dtype == torch.float8_e4m3fn else k
            v = v.view(torch.uint8) if v.dtype == torch.float8_e4m3fn else v
        dtype = torch.uint8 if self.e4m3 else torch.bfloat16
        _need(k, "k", dtype, 4)
        _shape(_need(v, "v", dtype, 4), "v", *k.shape)
        if k.stride() != v.stride():
            raise ValueError(f"k and v have different strides: {k.stride()}, {v.stride()}")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.pages, self.Hkv, self.page_size, self.D = k.shape
        ss = (0, 0, 0)
        if (k_scale is None) != (v_scale is None):
            raise ValueError("k_scale and v_scale come together")
        if self.e4m3:
            for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
                if not (t.is_cuda and t.dtype == torch.float32):
                    raise TypeError(f"{name}: need a float32 CUDA tensor")
                _shape(t, name, *k.shape[:3])
            if k_scale.stride() != v_scale.stride():
                raise ValueError("k_scale and v_scale have different strides")
            ss = k_scale.stride()
        self._abi = _lib.KvCache(
            k.data_ptr(), v.data_ptr(), _lib._ptr(k_scale), _lib._ptr(v_scale), self.pages,
            self.page_size, self.Hkv, self.D,
            _lib.MOE_KV_E4M3 if self.e4m3 else _lib.MOE_KV_BF16, *k.stride()[:3], *ss)

    @classmethod
    def empty(cls, pages: int, Hkv: int, page_size: int, D: int, e4m3: bool = False,
              device="cuda") -> "PagedCache":
        shape = (pages, Hkv, page_size, D)
        if not e4m3:
            return cls(torch.zeros(shape, dtype=torch.bfloat16, device=device),
                       torch.zeros(shape, dtype=torch.bfloat16, device=device))
        return cls(torch.zeros(shape, dtype=torch.uint8, device=device),
                   torch.zeros(shape, dtype=torch.uint8, device=device),
                   torch.zeros(shape[:3], dtype=torch.float32, device=device),
                   torch.zeros(shape[:3], dtype=torch.float32, device=device))

    def abi(self) -> _lib.KvCache:
        return self._abi


def rope_cos_sin(n_pos: int, rot: int, base: float = 1e6, factor: float = 1.0,
                 scaling: str = "none", original: int = 0, beta_fast: float = 32.0,
                 beta_slow: float = 1.0, device="cuda") -> torch.Tensor:
    """The rotation table of QkNormRope: float32 [n_pos, rot], the cosines of
    the rot / 2 angles pos * base^(-2i / rot), then their sines, computed in
    float64 and rounded once.

    scaling, for contexts `factor` times longer than the `original` training
    length: "linear" divides every position by `factor`; "yarn" (the "NTK by
    parts" interpolation of the YaRN paper) divides the frequencies that turn
    less than beta_slow times over the original length, keeps those that turn
    more than beta_fast times, blends linearly in between, and multiplies the
    table by the paper's 0.1 ln(factor) + 1."""
    if rot < 2 or rot % 2:
        raise ValueError(f"rot = {rot}: need an even number of dimensions")
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    inv = base ** (-i / rot)
    gain = 1.0
    if scaling == "linear":
        inv = inv / factor
    elif scaling == "yarn":
        if original < 1 or factor < 1:
            raise ValueError("yarn needs the original length and a factor of at least 1")

        def dim_of(turns: float) -> float:  # the pair that turns so often over `original`
            return rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))

        low = max(math.floor(dim_of(beta_fast)), 0)
        high = min(math.ceil(dim_of(beta_slow)), rot - 1)
        ramp = ((i / 2 - low) / max(high - low, 1e-3)).clamp(0, 1)
        inv = inv * (1 - ramp) + inv / factor * ramp
        gain = 0.1 * math.log(factor) + 1.0
    elif scaling != "none":
        raise ValueError(f"scaling {scaling!r}: need 'none', 'linear' or 'yarn'")
    ang = torch.arange(n_pos, dtype=torch.float64)[:, None] * inv
    return (torch.cat([ang.cos(), ang.sin()], 1) * gain).to(torch.float32).to(device)


class QkNormRope(_Status):
    """Query/key head norms and rotary positions, the keys and values stored
    into a paged cache (moe_qk_norm_rope).  q_norm, k_norm: float32 [D] or
    None (no norm); cos_sin: a table of rope_cos_sin or None (no rotation)."""

    def __init__(self, Hq: int, Hkv: int, D: int, q_norm: Optional[torch.Tensor] = None,
                 k_norm: Optional[torch.Tensor] = None, cos_sin: Optional[torch.Tensor] = None,
                 interleaved: bool = False, eps: float = 1e-6, device="cuda"):
        super().__init__(device)
        self.Hq, self.Hkv, self.D, self.eps = Hq, Hkv, D, eps
        self.interleaved = bool(interleaved)
        self.q_norm = _dense(q_norm, "q_norm", torch.float32, D)
        self.k_norm = _dense(k_norm, "k_norm", torch.float32, D)
        self.cos_sin = cos_sin
        self.n_pos, self.rot = (0, 0) if cos_sin is None else cos_sin.shape
        if cos_sin is not None:
            _dense(cos_sin, "cos_sin", torch.float32, self.n_pos, self.rot)

    def forward(self, qkv: torch.Tensor, positions: Optional[torch.Tensor], slots: torch.Tensor,
                cache: PagedCache, q_out: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
        """qkv bf16 [T, (Hq + 2 Hkv) D] (rows may be strided), positions int32
        [T], slots int64 [T] (page * page_size + offset, or < 0 for padding)
        -> q_out bf16 [T, Hq, D]."""
        _need(qkv, "qkv", torch.bfloat16, 2)
        T, width = qkv.shape
        if width != (self.Hq + 2 * self.Hkv) * self.D:
            raise ValueError(f"qkv: rows of {width}, need {(self.Hq + 2 * self.Hkv) * self.D}")
        if cache.Hkv != self.Hkv or cache.D != self.D:
            raise ValueError("the cache has other heads")
        if (positions is None) != (self.cos_sin is None):
            raise ValueError("positions and the rotation table come together")
        _dense(positions, "positions", torch.int32, T)
        _dense(slots, "slots", torch.int64, T)
        if q_out is None:
            q_out = _new(stream, T, self.Hq, self.D, dtype=torch.bfloat16, device=qkv.device)
        _heads(q_out, "q_out", T, self.Hq, self.D)
        d = _lib.QkDims(T, self.Hq, self.rot, int(self.interleaved), self.n_pos, self.eps,
                        _row_stride(qkv, width), _row_stride(q_out, self.Hq * self.D))
        _lib.moe_qk_norm_rope(qkv, self.q_norm, self.k_norm, self.cos_sin, positions, slots, d,
                              cache.abi(), q_out, self.status, stream)
        return q_out


def _heads(t: torch.Tensor, name: str, n: int, H: int, D: int) -> torch.Tensor:
    """A bf16 tensor [n, H, D] whose heads lie one after another."""
    _shape(_need(t, name, torch.bfloat16, 3), name, n, H, D)
    if n and H > 1 and t.stride(1) != D:
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    return t


class PagedAttention(_Status):
    """Attention of one new token per sequence over a paged cache
    (moe_paged_attention); window > 0 keeps the last `window` tokens."""

    def __init__(self, Hq: int, Hkv: int, D: int, scale: Optional[float] = None, window: int = 0,
                 device="cuda"):
        super().__init__(device)
        self.Hq, self.Hkv, self.D, self.window = Hq, Hkv, D, window
        self.scale = 1.0 / math.sqrt(D) if scale is None else scale

    def workspace(self, B: int, stream=None) -> torch.Tensor:
        """A workspace for calls of up to B sequences (of any length)."""
        d = _lib.AttnDims(B, self.Hq, 0, self.window, self.scale, 0, 0, 0)
        return _new(stream, _lib.paged_attention_workspace_bytes(d, self.D), dtype=torch.uint8,
                    device=self.status.device)

    def forward(self, q: torch.Tensor, cache: PagedCache, block_table: torch.Tensor,
                seq_lens: torch.Tensor, out: Optional[torch.Tensor] = None,
                ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """q bf16 [B, Hq, D], block_table int32 [B, pages per sequence],
        seq_lens int32 [B] (the new token included) -> out bf16 [B, Hq, D]."""
        B = q.shape[0]
        _heads(q, "q", B, self.Hq, self.D)
        if cache.Hkv != self.Hkv or cache.D != self.D:
            raise ValueError("the cache has other heads")
        _need(block_table, "block_table", torch.int32, 2)
        width = block_table.shape[1]
        _shape(block_table, "block_table", B, width)
        _dense(seq_lens, "seq_lens", torch.int32, B)
        if out is None:
            out = _new(stream, B, self.Hq, self.D, dtype=torch.bfloat16, device=q.device)
        _heads(out, "out", B, self.Hq, self.D)
        if ws is None:
            ws = self.workspace(B, stream)
        row = self.Hq * self.D
        d = _lib.AttnDims(B, self.Hq, width, self.window, self.scale,
                          _row_stride(block_table, width), _row_stride(q, row),
                          _row_stride(out, row))
        _lib.moe_paged_attention(q, cache.abi(), block_table, seq_lens, d, out, ws, self.status,
                                 stream)
        return out


class Fp8Linear(_Status):
    """x W^T + bias with block-FP8 weights (codes [N, K] uint8 or
    float8_e4m3fn, scales float32 [ceil(N/128), ceil(K/128)]) and E4M3
    activations quantised in the call (moe_linear_fp8)."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor,
                 bias: Optional[torch.Tensor] = None):
        if codes.dtype == torch.float8_e4m3fn:
            codes = codes.view(torch.uint8)
        self.N, self.K = codes.shape
        self.codes = _dense(codes, "codes", torch.uint8, self.N, self.K)
        self.scales = _dense(scales, "scales", torch.float32, -(-self.N // 128),
                             -(-self.K // 128))
        self.bias = _dense(bias, "bias", torch.float32, self.N)
        super().__init__(codes.device)
        self._mat = _lib.Fp8Mat(codes.data_ptr(), scales.data_ptr())

    def workspace(self, M: int, stream=None) -> torch.Tensor:
        """A workspace for calls of up to M rows."""
        n = _lib.linear_fp8_workspace_bytes(_lib.LinearDims(M, self.N, self.K, self.K, self.N))
        return _new(stream, n, dtype=torch.uint8, device=self.codes.device)

    def forward(self, x: torch.Tensor, out: Optional[torch.Tensor] = None,
                ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """x bf16 [M, K] -> out bf16 [M, N]; rows of either may be strided."""
        _need(x, "x", torch.bfloat16, 2)
        M = x.shape[0]
        _shape(x, "x", M, self.K)
        if out is None:
            out = _new(stream, M, self.N, dtype=torch.bfloat16, device=x.device)
        _shape(_need(out, "out", torch.bfloat16, 2), "out", M, self.N)
        if ws is None:
            ws = self.workspace(M, stream)
        d = _lib.LinearDims(M, self.N, self.K, _row_stride(x, self.K), _row_stride(out, self.N))
        _lib.moe_linear_fp8(x, self._mat, self.bias, d, out, ws, self.status, stream)
        return out
