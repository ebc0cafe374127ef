"""The operators of a decoder layer around the MoE layer, on PyTorch tensors.

    ExpertSelector     router logits -> chosen experts and weights
    QkNormRope         head norms, rotary positions, store into a paged cache
    PagedCache         the paged key/value cache (bf16 or E4M3)
    PagedAttention     attention of one new token per sequence over it
    TreeAttention      attention of several, a tree of drafted tokens, over it
    LatentCache        a paged cache of one latent vector per token
    LatentStore        norm, rotary positions, store into it
    LatentAttention    attention over it in the absorbed form (new or drafted tokens)
    ExpandedAttention  the same attention in its expanded form, for prompts
    Fp8Linear          x W^T with block-FP8 weights and E4M3 activations

Each object holds what a serving program sets up once; ``forward`` takes the
step's tensors, and output buffers and a workspace where the program keeps
them (they are allocated otherwise).  Everything runs in libmoe_fp8.so on the
current stream or the one given; tensors are checked for device, type, shape
and layout here and for their sizes in the library.  Their device has to be the
current one.  What the kernels themselves
find wrong in their data (a page number outside the cache, say) is recorded in
``status``, a device array that ``check()`` reads after synchronising; it keeps
what was recorded until ``status.zero_()``.  Host threads may share an object,
each with its own output and workspace.
"""
from __future__ import annotations

import math
from typing import Optional

import torch

from . import _lib
from ._checks import (current_device as _current_device, dense as _dense, refuse as _refuse,
                      refuse_device as _refuse_device)
from .device import new_on

_BF16, _F32, _I32, _I64, _U8 = (torch.bfloat16, torch.float32, torch.int32, torch.int64,
                                torch.uint8)


_raw_stream = torch._C._cuda_getCurrentRawStream


def _handle(stream) -> int:
    return stream if isinstance(stream, int) else stream.cuda_stream


# The checks of a call cost host time on every step, so forward() asks one
# question per tensor, looks for the words only when the answer is no, and takes
# what is fixed at set-up as one tuple (_held).

_ROWS = "the elements of a row must be contiguous"
_HEADS = "the heads of a row must be contiguous"


class _Fixed:
    """What is set up stays: its addresses and sizes are held as the library
    takes them.  Only the attributes in _free may be set again; tensors may be
    written in place."""

    _free = frozenset()

    def __setattr__(self, name, value):
        if name in self.__dict__ and name not in self._free:
            raise AttributeError(f"{type(self).__name__}.{name} is fixed at set-up: "
                                 "make a new object, or write into the tensor")
        object.__setattr__(self, name, value)


class _Status(_Fixed):
    """The device status word of one operator object."""

    def __init__(self, device):
        self.status = torch.zeros(16, dtype=torch.int32, device=device)
        self._status, self._dev = self.status.data_ptr(), self.status.get_device()

    def check(self, stream=None) -> None:
        """Synchronise and raise MoeError if a kernel flagged its data."""
        if self._dev != _current_device():
            _refuse_device(self._dev, _current_device())
        _lib.moe_read_device_status(self.status, stream)


class ExpertSelector(_Fixed):
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
        self._held = (E, k, self.rule, _lib._ptr(bias), None if bias is None else bias.get_device(),
                      _lib.lib().moe_select_experts)

    def forward(self, logits: torch.Tensor, topk_idx: Optional[torch.Tensor] = None,
                topk_w: Optional[torch.Tensor] = None, stream=None):
        """logits float32 [T, E] (rows may be strided) -> (topk_idx int32
        [T, k], topk_w float32 [T, k])."""
        E, k, rule, bias, bias_dev, call = self._held
        dev, shape, ls = logits.get_device(), logits.shape, logits.stride()
        T = shape[0]
        if dev < 0 or logits.dtype != _F32 or shape != (T, E) or (ls[1] != 1 and E > 1):
            _refuse(logits, "logits", _F32, (T, E), layout=_ROWS)
        if dev != _current_device():
            _refuse_device(dev, _current_device())
        if bias is not None and dev != bias_dev:
            _refuse(self.bias, "bias", _F32, (E,), dev)
        if topk_idx is None:
            topk_idx = new_on(stream, T, k, dtype=_I32, device=logits.device)
        if topk_w is None:
            topk_w = new_on(stream, T, k, dtype=_F32, device=logits.device)
        rows = (T, k)
        if (topk_idx.dtype != _I32 or topk_idx.get_device() != dev or topk_idx.shape != rows
                or not topk_idx.is_contiguous()):
            _refuse(topk_idx, "topk_idx", _I32, (T, k), dev)
        if (topk_w.dtype != _F32 or topk_w.get_device() != dev or topk_w.shape != rows
                or not topk_w.is_contiguous()):
            _refuse(topk_w, "topk_w", _F32, (T, k), dev)
        st = call(logits.data_ptr(), ls[0] if T > 1 else E, bias, rule, T, E, k,
                  topk_idx.data_ptr(), topk_w.data_ptr(),
                  _raw_stream(dev) if stream is None else _handle(stream))
        if st:
            _lib._check(st, "moe_select_experts")
        return topk_idx, topk_w

    def route(self, x: torch.Tensor, layer, ws: torch.Tensor,
              topk_idx: Optional[torch.Tensor] = None, topk_w: Optional[torch.Tensor] = None,
              stream=None):
        """The same choice from the tokens x bf16 [T, H] and a DeviceLayer's
        router (moe_route_select_status); ws: the layer's workspace for T
        tokens.  What the router finds wrong is recorded in the layer's
        `status`, which its check() reads."""
        T = x.shape[0]
        if layer.E != self.E or layer.k != self.k:
            raise ValueError(f"the layer routes to {layer.k} of {layer.E} experts, "
                             f"need {self.k} of {self.E}")
        if not x.is_cuda or x.dtype != _BF16 or x.shape != (T, layer.H) or not x.is_contiguous():
            _refuse(x, "x", _BF16, (T, layer.H))
        dev = x.get_device()
        if dev != _current_device():
            _refuse_device(dev, _current_device())
        _dense(self.bias, "bias", _F32, self.E, device=dev)
        _dense(layer.Wr, "the layer's Wr", _F32, self.E, layer.H, device=dev)
        _dense(layer.bias, "the layer's bias", _F32, self.E, device=dev)
        if topk_idx is None:
            topk_idx = new_on(stream, T, self.k, dtype=_I32, device=x.device)
        if topk_w is None:
            topk_w = new_on(stream, T, self.k, dtype=_F32, device=x.device)
        _dense(topk_idx, "topk_idx", _I32, T, self.k, device=dev)
        _dense(topk_w, "topk_w", _F32, T, self.k, device=dev)
        if ws.get_device() != dev or not ws.is_contiguous():
            raise ValueError("ws must be contiguous and on x's device")
        _lib.moe_route_select(x, layer.Wr, layer.bias, self.bias, self.rule, layer.dims(T),
                              topk_idx, topk_w, ws, layer.status, stream)
        return topk_idx, topk_w


class PagedCache(_Fixed):
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
        dtype = _U8 if self.e4m3 else _BF16
        for t, name in ((k, "k"), (v, "v")):
            if not (t.is_cuda and t.dtype == dtype and t.dim() == 4 and t.shape == k.shape
                    and t.stride(3) == 1 and t.get_device() == k.get_device()):
                _refuse(t, name, dtype, k.shape, k.get_device(), _ROWS)
        if k.stride() != v.stride():
            raise ValueError(f"k and v have different strides: {k.stride()}, {v.stride()}")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.pages, self.Hkv, self.page_size, self.D = k.shape
        self.device = k.get_device()
        self._place = (self.Hkv, self.D, self.device)
        ss = (0, 0, 0)
        if (k_scale is None) != (v_scale is None):
            raise ValueError("k_scale and v_scale come together")
        if self.e4m3:
            for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
                if not (t.is_cuda and t.dtype == _F32 and t.shape == k.shape[:3]
                        and t.get_device() == k.get_device()):
                    _refuse(t, name, _F32, k.shape[:3], k.get_device())
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

    def refuse(self, Hkv: int, D: int, device: int) -> None:
        """Raise for a use that needs other heads or another device."""
        raise ValueError(f"the cache has {self.Hkv} heads of {self.D} on device {self.device}, "
                         f"need {Hkv} of {D} on {device}")


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
    None (no norm); cos_sin: a table of rope_cos_sin or None (no rotation).
    eps and interleaved may be set again."""

    _free = frozenset(("_sizes", "eps", "interleaved"))

    def __init__(self, Hq: int, Hkv: int, D: int, q_norm: Optional[torch.Tensor] = None,
                 k_norm: Optional[torch.Tensor] = None, cos_sin: Optional[torch.Tensor] = None,
                 interleaved: bool = False, eps: float = 1e-6, device="cuda"):
        super().__init__(device)
        self.Hq, self.Hkv, self.D, self.eps = Hq, Hkv, D, eps
        self.interleaved = bool(interleaved)
        self.q_norm = _dense(q_norm, "q_norm", torch.float32, D, device=self._dev)
        self.k_norm = _dense(k_norm, "k_norm", torch.float32, D, device=self._dev)
        self.cos_sin = cos_sin
        self.n_pos, self.rot = (0, 0) if cos_sin is None else cos_sin.shape
        if cos_sin is not None:
            _dense(cos_sin, "cos_sin", torch.float32, self.n_pos, self.rot, device=self._dev)
        self.width = (Hq + 2 * Hkv) * D
        self._sizes = None, None  # (read and replaced as one: threads may share the object)
        self._held = (self._dev, Hq, D, self.width, (Hkv, D, self._dev), cos_sin is None,
                      _lib._ptr(q_norm), _lib._ptr(k_norm), _lib._ptr(cos_sin), self._status,
                      _lib.lib().moe_qk_norm_rope)

    def forward(self, qkv: torch.Tensor, positions: Optional[torch.Tensor], slots: torch.Tensor,
                cache: PagedCache, q_out: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
        """qkv bf16 [T, (Hq + 2 Hkv) D] (rows may be strided), positions int32
        [T], slots int64 [T] (page * page_size + offset, or < 0 for padding)
        -> q_out bf16 [T, Hq, D]."""
        here, Hq, D, width, place, bare, q_norm, k_norm, cos_sin, status, call = self._held
        dev, shape, xs = qkv.get_device(), qkv.shape, qkv.stride()
        T = shape[0]
        if dev != here or qkv.dtype != _BF16 or shape != (T, width) or xs[-1] != 1:
            _refuse(qkv, "qkv", _BF16, (T, width), here, _ROWS)
        if dev != _current_device():
            _refuse_device(dev, _current_device())
        if cache._place != place:
            cache.refuse(*place)
        if (positions is None) != bare:
            raise ValueError("positions and the rotation table come together")
        if positions is not None and (positions.dtype != _I32 or positions.get_device() != dev
                                      or positions.shape != (T,) or not positions.is_contiguous()):
            _refuse(positions, "positions", _I32, (T,), dev)
        if (slots.dtype != _I64 or slots.get_device() != dev or slots.shape != (T,)
                or not slots.is_contiguous()):
            _refuse(slots, "slots", _I64, (T,), dev)
        if q_out is None:
            q_out = new_on(stream, T, Hq, D, dtype=_BF16, device=qkv.device)
        qs = q_out.stride()
        if (q_out.dtype != _BF16 or q_out.get_device() != dev or q_out.shape != (T, Hq, D)
                or qs[2] != 1 or (Hq > 1 and qs[1] != D)):
            _refuse(q_out, "q_out", _BF16, (T, Hq, D), dev, _HEADS)
        key = (T, xs[0], qs[0], self.eps, self.interleaved)
        known, dims = self._sizes
        if key != known:
            dims = _lib.QkDims(T, Hq, self.rot, int(bool(key[4])), self.n_pos, key[3],
                               key[1] if T > 1 else width, key[2] if T > 1 else Hq * D)
            self._sizes = key, dims
        st = call(qkv.data_ptr(), q_norm, k_norm, cos_sin,
                  None if bare else positions.data_ptr(), slots.data_ptr(), dims, cache._abi,
                  q_out.data_ptr(), status, _raw_stream(dev) if stream is None else _handle(stream))
        if st:
            _lib._check(st, "moe_qk_norm_rope")
        return q_out


class PagedAttention(_Status):
    """Attention of one new token per sequence over a paged cache
    (moe_paged_attention); window > 0 keeps the last `window` tokens.  scale
    and window may be set again."""

    _free = frozenset(("_sizes", "scale", "window"))

    def __init__(self, Hq: int, Hkv: int, D: int, scale: Optional[float] = None, window: int = 0,
                 device="cuda"):
        super().__init__(device)
        self.Hq, self.Hkv, self.D, self.window = Hq, Hkv, D, window
        self.scale = 1.0 / math.sqrt(D) if scale is None else scale
        self._sizes = None, None  # (read and replaced as one: threads may share the object)
        self._held = (self._dev, Hq, D, (Hkv, D, self._dev), self._status,
                      _lib.lib().moe_paged_attention)

    def workspace(self, B: int, stream=None) -> torch.Tensor:
        """A workspace for calls of up to B sequences (of any length)."""
        if self._dev != _current_device():
            _refuse_device(self._dev, _current_device())
        d = _lib.AttnDims(B, self.Hq, 0, self.window, self.scale, 0, 0, 0)
        return new_on(stream, _lib.paged_attention_workspace_bytes(d, self.D), dtype=torch.uint8,
                    device=self.status.device)

    def forward(self, q: torch.Tensor, cache: PagedCache, block_table: torch.Tensor,
                seq_lens: torch.Tensor, out: Optional[torch.Tensor] = None,
                ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """q bf16 [B, Hq, D], block_table int32 [B, pages per sequence],
        seq_lens int32 [B] (the new token included) -> out bf16 [B, Hq, D]."""
        here, Hq, D, place, status, call = self._held
        dev, shape, qs = q.get_device(), q.shape, q.stride()
        B = shape[0]
        if (dev != here or q.dtype != _BF16 or shape != (B, Hq, D) or qs[2] != 1
                or (Hq > 1 and qs[1] != D)):
            _refuse(q, "q", _BF16, (B, Hq, D), here, _HEADS)
        if dev != _current_device():
            _refuse_device(dev, _current_device())
        if cache._place != place:
            cache.refuse(*place)
        rows, width = block_table.shape
        ts = block_table.stride()
        if (block_table.dtype != _I32 or block_table.get_device() != dev or rows != B
                or (width > 1 and ts[1] != 1)):
            _refuse(block_table, "block_table", _I32, (B, width), dev, _ROWS)
        if (seq_lens.dtype != _I32 or seq_lens.get_device() != dev or seq_lens.shape != (B,)
                or not seq_lens.is_contiguous()):
            _refuse(seq_lens, "seq_lens", _I32, (B,), dev)
        if out is None:
            out = new_on(stream, B, Hq, D, dtype=_BF16, device=q.device)
        os = out.stride()
        if (out.dtype != _BF16 or out.get_device() != dev or out.shape != shape
                or os[2] != 1 or (Hq > 1 and os[1] != D)):
            _refuse(out, "out", _BF16, (B, Hq, D), dev, _HEADS)
        if ws is None:
            ws = self.workspace(B, stream)
        elif ws.get_device() != dev or not ws.is_contiguous():
            raise ValueError("ws must be contiguous and on the tensors' device")
        key = (B, width, ts[0], qs[0], os[0], self.window, self.scale)
        known, dims = self._sizes
        if key != known:
            row = Hq * D
            strides = key[2:5] if B > 1 else (width, row, row)
            dims = _lib.AttnDims(B, Hq, width, key[5], key[6], *strides)
            self._sizes = key, dims
        st = call(q.data_ptr(), cache._abi, block_table.data_ptr(), seq_lens.data_ptr(), dims,
                  out.data_ptr(), ws.data_ptr(), ws.nbytes, status,
                  _raw_stream(dev) if stream is None else _handle(stream))
        if st:
            _lib._check(st, "moe_paged_attention")
        return out


class _DraftAttention(_Status):
    """What attention of several new tokens per sequence has in common."""

    _free = frozenset(("_sizes", "scale", "window"))

    def _set_up(self, H, Dq, Dv, scale, window, place, call, name):
        self.scale, self.window = scale, window
        self._sizes = None, None  # (read and replaced as one: threads may share the object)
        self._held = (self._dev, H, Dq, Dv, place, self._status, call, name)

    def _bytes(self, d) -> int:
        raise NotImplementedError

    def workspace(self, B: int, n: int, stream=None) -> torch.Tensor:
        """A workspace for calls of up to B sequences (of any length) with n
        new tokens each, or fewer."""
        if self._dev != _current_device():
            _refuse_device(self._dev, _current_device())
        d = _lib.DraftDims(B, n, self._held[1], 0, 0, self.scale, 0, 0, 0, 0, 0, 0)
        return new_on(stream, self._bytes(d), dtype=torch.uint8, device=self.status.device)

    def forward(self, q: torch.Tensor, cache, block_table: torch.Tensor, seq_lens: torch.Tensor,
                mask: Optional[torch.Tensor] = None, draft_lens: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
        """q bf16 [B, n, heads, query size], block_table int32 [B, pages per
        sequence], seq_lens int32 [B] (the new tokens included) -> out bf16
        [B, n, heads, value size].  mask int64 [B, n]: bit j of mask[b, i]
        tells whether new token i sees new token j (None: those up to itself;
        mask.expand(B, n) where the sequences share one); draft_lens int32
        [B]: the sequences' new tokens, the last ones of seq_lens (None: n).
        Rows past them are zeros."""
        here, H, Dq, Dv, place, status, call, name = self._held
        dev, shape, qs = q.get_device(), q.shape, q.stride()
        B, n = shape[0], shape[1]
        if (dev != here or q.dtype != _BF16 or shape != (B, n, H, Dq) or qs[3] != 1
                or (H > 1 and qs[2] != Dq)):
            _refuse(q, "q", _BF16, (B, n, H, Dq), here, _HEADS)
        if dev != _current_device():
            _refuse_device(dev, _current_device())
        if cache._place != place:
            cache.refuse(*place)
        rows, width = block_table.shape
        ts = block_table.stride()
        if (block_table.dtype != _I32 or block_table.get_device() != dev or rows != B
                or (width > 1 and ts[1] != 1)):
            _refuse(block_table, "block_table", _I32, (B, width), dev, _ROWS)
        for t, what in ((seq_lens, "seq_lens"), (draft_lens, "draft_lens")):
            if t is not None and (t.dtype != _I32 or t.get_device() != dev or t.shape != (B,)
                                  or not t.is_contiguous()):
                _refuse(t, what, _I32, (B,), dev)
        ms = 0
        if mask is not None:
            ms = mask.stride()
            if (mask.dtype != _I64 or mask.get_device() != dev or mask.shape != (B, n)
                    or (n > 1 and ms[1] != 1)):
                _refuse(mask, "mask", _I64, (B, n), dev, _ROWS)
            ms = ms[0] if B > 1 else 0
        if out is None:
            out = new_on(stream, B, n, H, Dv, dtype=_BF16, device=q.device)
        os = out.stride()
        if (out.dtype != _BF16 or out.get_device() != dev or out.shape != (B, n, H, Dv)
                or os[3] != 1 or (H > 1 and os[2] != Dv)):
            _refuse(out, "out", _BF16, (B, n, H, Dv), dev, _HEADS)
        if ws is None:
            ws = self.workspace(B, n, stream)
        elif ws.get_device() != dev or not ws.is_contiguous():
            raise ValueError("ws must be contiguous and on the tensors' device")
        key = (B, n, width, ts[0], qs[0], qs[1], os[0], os[1], ms, self.window, self.scale)
        known, dims = self._sizes
        if key != known:
            row = (qs[1], os[1]) if n > 1 else (H * Dq, H * Dv)
            seq = (ts[0], qs[0], os[0]) if B > 1 else (width, n * row[0], n * row[1])
            dims = _lib.DraftDims(B, n, H, width, key[9], key[10], seq[0], seq[1], row[0], seq[2],
                                  row[1], ms)
            self._sizes = key, dims
        st = call(q.data_ptr(), cache._abi, block_table.data_ptr(), seq_lens.data_ptr(),
                  None if mask is None else mask.data_ptr(),
                  None if draft_lens is None else draft_lens.data_ptr(), dims, out.data_ptr(),
                  ws.data_ptr(), ws.nbytes, status,
                  _raw_stream(dev) if stream is None else _handle(stream))
        if st:
            _lib._check(st, name)
        return out


class TreeAttention(_DraftAttention):
    """Attention of several new tokens per sequence, which see each other as a
    tree (or a chain), over a PagedCache that holds them already
    (moe_tree_attention); window > 0 leaves out what lies further back.  scale
    and window may be set again."""

    def __init__(self, Hq: int, Hkv: int, D: int, scale: Optional[float] = None, window: int = 0,
                 device="cuda"):
        super().__init__(device)
        self.Hq, self.Hkv, self.D = Hq, Hkv, D
        self._set_up(Hq, D, D, 1.0 / math.sqrt(D) if scale is None else scale, window,
                     (Hkv, D, self._dev), _lib.lib().moe_tree_attention, "moe_tree_attention")

    def _bytes(self, d):
        return _lib.tree_attention_workspace_bytes(d, self.Hkv, self.D)


class LatentCache(_Fixed):
    """A paged cache of latent vectors over a bf16 tensor [pages, page_size,
    R + rot]: R elements of the vector, then rot of the shared key part.  Any
    strides with a token contiguous will do."""

    def __init__(self, data: torch.Tensor, R: int):
        if not (data.is_cuda and data.dtype == _BF16 and data.dim() == 3 and data.shape[2] > R
                and data.stride(2) == 1):
            _refuse(data, "data", _BF16, (*data.shape[:2], R + 64), layout=_ROWS)
        self.data, self.R = data, R
        self.pages, self.page_size = data.shape[:2]
        self.rot = data.shape[2] - R
        self.device = data.get_device()
        self._place = (R, self.rot, self.device)
        self._abi = _lib.LatentPages(data.data_ptr(), self.pages, self.page_size, R, self.rot,
                                     data.stride(0), data.stride(1))

    @classmethod
    def empty(cls, pages: int, page_size: int, R: int, rot: int = 64,
              device="cuda") -> "LatentCache":
        return cls(torch.zeros(pages, page_size, R + rot, dtype=torch.bfloat16, device=device), R)

    def abi(self) -> _lib.LatentPages:
        return self._abi

    def refuse(self, R: int, rot: int, device: int) -> None:
        """Raise for a use that needs another layout or another device."""
        raise ValueError(f"the cache holds vectors of {self.R} + {self.rot} on device "
                         f"{self.device}, need {R} + {rot} on {device}")


class LatentStore(_Status):
    """Latent vectors normed, their shared key part rotated, stored into a
    LatentCache, and the queries' rotated parts on the way (moe_latent_store).
    norm: float32 [R] or None (no norm); cos_sin: a table of rope_cos_sin with
    `rot` columns.  eps and interleaved may be set again."""

    _free = frozenset(("_sizes", "eps", "interleaved"))

    def __init__(self, H: int, R: int, cos_sin: torch.Tensor, norm: Optional[torch.Tensor] = None,
                 rot: int = 64, interleaved: bool = False, eps: float = 1e-6, device="cuda"):
        super().__init__(device)
        self.H, self.R, self.rot, self.eps = H, R, rot, eps
        self.interleaved = bool(interleaved)
        self.norm = _dense(norm, "norm", torch.float32, R, device=self._dev)
        self.n_pos = cos_sin.shape[0]
        self.cos_sin = _dense(cos_sin, "cos_sin", torch.float32, self.n_pos, rot, device=self._dev)
        self._sizes = None, None  # (read and replaced as one: threads may share the object)
        self._held = (self._dev, H, rot, R + rot, (R, rot, self._dev), _lib._ptr(norm),
                      _lib._ptr(cos_sin), self._status, _lib.lib().moe_latent_store)

    def forward(self, kv: torch.Tensor, positions: torch.Tensor, slots: torch.Tensor,
                cache: LatentCache, q: Optional[torch.Tensor] = None,
                q_out: Optional[torch.Tensor] = None, rows: Optional[torch.Tensor] = None,
                stream=None) -> Optional[torch.Tensor]:
        """kv bf16 [T, R + rot] (rows may be strided), positions int32 [T],
        slots int64 [T] (page * page_size + offset, or < 0 for padding), q bf16
        [T, H, rot] (the rotated part of wider heads: any strides between
        tokens and heads) -> q_out, of q's shape, which may be q itself.  rows
        bf16 [T, R + rot]: what was stored, once more by token.  Without q, the
        heads are left alone."""
        here, H, rot, width, place, norm, cos_sin, status, call = self._held
        dev, shape, xs = kv.get_device(), kv.shape, kv.stride()
        T = shape[0]
        if dev != here or kv.dtype != _BF16 or shape != (T, width) or xs[-1] != 1:
            _refuse(kv, "kv", _BF16, (T, width), here, _ROWS)
        if dev != _current_device():
            _refuse_device(dev, _current_device())
        if cache._place != place:
            cache.refuse(*place)
        if (positions.dtype != _I32 or positions.get_device() != dev or positions.shape != (T,)
                or not positions.is_contiguous()):
            _refuse(positions, "positions", _I32, (T,), dev)
        if (slots.dtype != _I64 or slots.get_device() != dev or slots.shape != (T,)
                or not slots.is_contiguous()):
            _refuse(slots, "slots", _I64, (T,), dev)
        qs = ps = (0, 0, 1)
        if q is None:
            if q_out is not None:
                raise ValueError("q_out without q")
            H = 0
        else:
            if q_out is None:
                q_out = new_on(stream, T, H, rot, dtype=_BF16, device=kv.device)
            qs, ps = q.stride(), q_out.stride()
            for t, name, s in ((q, "q", qs), (q_out, "q_out", ps)):
                if (t.dtype != _BF16 or t.get_device() != dev or t.shape != (T, H, rot)
                        or s[2] != 1):
                    _refuse(t, name, _BF16, (T, H, rot), dev, _ROWS)
        rs = (0, 1)
        if rows is not None:
            rs = rows.stride()
            if (rows.dtype != _BF16 or rows.get_device() != dev or rows.shape != (T, width)
                    or rs[1] != 1):
                _refuse(rows, "rows", _BF16, (T, width), dev, _ROWS)
        key = (T, H, xs[0], qs, ps, rs[0], self.eps, self.interleaved)
        known, dims = self._sizes
        if key != known:
            if T > 1:
                kv_s, q_s, p_s, r_s = xs[0], qs[0], ps[0], rs[0]
            else:
                kv_s, q_s, p_s, r_s = width, 0, 0, width
            qh, ph = (qs[1], ps[1]) if H > 1 else (rot, rot)
            dims = _lib.LatentDims(T, H, int(bool(key[7])), self.n_pos, key[6], kv_s, q_s, qh, p_s, ph,
                                   r_s)
            self._sizes = key, dims
        st = call(kv.data_ptr(), norm, cos_sin, positions.data_ptr(), slots.data_ptr(),
                  None if q is None else q.data_ptr(), dims, cache._abi,
                  None if q is None else q_out.data_ptr(),
                  None if rows is None else rows.data_ptr(), status,
                  _raw_stream(dev) if stream is None else _handle(stream))
        if st:
            _lib._check(st, "moe_latent_store")
        return q_out


class LatentAttention(_DraftAttention):
    """Attention of one or several new tokens per sequence over a LatentCache
    in the absorbed form: the latent vector is key and value of every head
    (moe_latent_attention).  q is [B, n, H, R + rot], out [B, n, H, R]; scale
    is that of the expanded heads, 1 / sqrt(their size), and may be set again."""

    def __init__(self, H: int, R: int, scale: float, rot: int = 64, device="cuda"):
        super().__init__(device)
        self.H, self.R, self.rot = H, R, rot
        self._set_up(H, R + rot, R, scale, 0, (R, rot, self._dev),
                     _lib.lib().moe_latent_attention, "moe_latent_attention")

    def _bytes(self, d):
        return _lib.latent_attention_workspace_bytes(d, self.R)


class ExpandedAttention(_Status):
    """Latent attention in its expanded form, for prompts: causal over ragged
    sequences, keys of 128 dimensions per head and 64 that the heads share,
    values of 128 (moe_expanded_attention).  scale may be set again."""

    _free = frozenset(("_sizes", "scale"))

    def __init__(self, H: int, scale: Optional[float] = None, device="cuda"):
        super().__init__(device)
        self.H = H
        self.scale = 1.0 / math.sqrt(192) if scale is None else scale
        self._sizes = None, None  # (read and replaced as one: threads may share the object)
        self._held = (self._dev, H, self._status, _lib.lib().moe_expanded_attention)

    def forward(self, q: torch.Tensor, k_nope: torch.Tensor, k_rope: torch.Tensor, v: torch.Tensor,
                cu_q: torch.Tensor, cu_k: torch.Tensor, out: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
        """q bf16 [Tq, H, 192], k_nope and v bf16 [Tk, H, 128], k_rope bf16
        [Tk, 64], any strides between tokens and heads; cu_q, cu_k int32 [B +
        1]: where each sequence's tokens begin, its queries being its last
        tokens -> out bf16 [Tq, H, 128] (rows of no sequence are left as they
        were)."""
        here, H, status, call = self._held
        dev, qs = q.get_device(), q.stride()
        Tq, Tk, B = q.shape[0], k_rope.shape[0], cu_q.shape[0] - 1
        if dev != here or q.dtype != _BF16 or q.shape != (Tq, H, 192) or qs[-1] != 1:
            _refuse(q, "q", _BF16, (Tq, H, 192), here, _ROWS)
        if dev != _current_device():
            _refuse_device(dev, _current_device())
        ks, rs, vs = k_nope.stride(), k_rope.stride(), v.stride()
        if (k_nope.dtype != _BF16 or k_nope.get_device() != dev or k_nope.shape != (Tk, H, 128)
                or ks[2] != 1):
            _refuse(k_nope, "k_nope", _BF16, (Tk, H, 128), dev, _ROWS)
        if (k_rope.dtype != _BF16 or k_rope.get_device() != dev or k_rope.shape != (Tk, 64)
                or rs[1] != 1):
            _refuse(k_rope, "k_rope", _BF16, (Tk, 64), dev, _ROWS)
        if v.dtype != _BF16 or v.get_device() != dev or v.shape != (Tk, H, 128) or vs[2] != 1:
            _refuse(v, "v", _BF16, (Tk, H, 128), dev, _ROWS)
        for t, name in ((cu_q, "cu_q"), (cu_k, "cu_k")):
            if (t.dtype != _I32 or t.get_device() != dev or t.shape != (B + 1,) or B < 0
                    or not t.is_contiguous()):
                _refuse(t, name, _I32, (max(B, 0) + 1,), dev)
        if out is None:
            out = new_on(stream, Tq, H, 128, dtype=_BF16, device=q.device)
        os = out.stride()
        if (out.dtype != _BF16 or out.get_device() != dev or out.shape != (Tq, H, 128)
                or os[2] != 1):
            _refuse(out, "out", _BF16, (Tq, H, 128), dev, _ROWS)
        key = (B, Tq, Tk, qs, ks, rs[0], vs, os, self.scale)
        known, dims = self._sizes
        if key != known:
            def pair(s, T, width):  # the strides that are used
                return (s[0] if T > 1 else width, s[1] if H > 1 else width)
            dims = _lib.ExpandedDims(B, Tq, Tk, H, key[8], *pair(qs, Tq, 192), *pair(ks, Tk, 128),
                                     rs[0] if Tk > 1 else 64, *pair(vs, Tk, 128), *pair(os, Tq, 128))
            self._sizes = key, dims
        st = call(q.data_ptr(), k_nope.data_ptr(), k_rope.data_ptr(), v.data_ptr(), cu_q.data_ptr(),
                  cu_k.data_ptr(), dims, out.data_ptr(), status,
                  _raw_stream(dev) if stream is None else _handle(stream))
        if st:
            _lib._check(st, "moe_expanded_attention")
        return out


class Fp8Linear(_Status):
    """x W^T + bias with block-FP8 weights (codes [N, K] uint8 or
    float8_e4m3fn, scales float32 [ceil(N/128), ceil(K/128)]) and E4M3
    activations quantised in the call (moe_linear_fp8)."""

    _free = frozenset(("_sizes",))

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor,
                 bias: Optional[torch.Tensor] = None):
        if codes.dtype == torch.float8_e4m3fn:
            codes = codes.view(torch.uint8)
        self.N, self.K = codes.shape
        dev = codes.get_device()
        self.codes = _dense(codes, "codes", torch.uint8, self.N, self.K)
        self.scales = _dense(scales, "scales", torch.float32, -(-self.N // 128),
                             -(-self.K // 128), device=dev)
        self.bias = _dense(bias, "bias", torch.float32, self.N, device=dev)
        super().__init__(codes.device)
        self._sizes = None, None  # (read and replaced as one: threads may share the object)
        self._held = (self._dev, self.N, self.K, _lib.Fp8Mat(codes.data_ptr(), scales.data_ptr()),
                      _lib._ptr(bias), self._status, _lib.lib().moe_linear_fp8)

    def workspace(self, M: int, stream=None) -> torch.Tensor:
        """A workspace for calls of up to M rows."""
        if self._dev != _current_device():
            _refuse_device(self._dev, _current_device())
        n = _lib.linear_fp8_workspace_bytes(_lib.LinearDims(M, self.N, self.K, self.K, self.N))
        return new_on(stream, n, dtype=torch.uint8, device=self.codes.device)

    def forward(self, x: torch.Tensor, out: Optional[torch.Tensor] = None,
                ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """x bf16 [M, K] -> out bf16 [M, N]; rows of either may be strided."""
        here, N, K, mat, bias, status, call = self._held
        dev, shape, xs = x.get_device(), x.shape, x.stride()
        M = shape[0]
        if dev != here or x.dtype != _BF16 or shape != (M, K) or xs[-1] != 1:
            _refuse(x, "x", _BF16, (M, K), here, _ROWS)
        if dev != _current_device():
            _refuse_device(dev, _current_device())
        if out is None:
            out = new_on(stream, M, N, dtype=_BF16, device=x.device)
        os = out.stride()
        if out.dtype != _BF16 or out.get_device() != dev or out.shape != (M, N) or os[1] != 1:
            _refuse(out, "out", _BF16, (M, N), dev, _ROWS)
        if ws is None:
            ws = self.workspace(M, stream)
        elif ws.get_device() != dev or not ws.is_contiguous():
            raise ValueError("ws must be contiguous and on the tensors' device")
        key = (M, xs[0], os[0])
        known, dims = self._sizes
        if key != known:
            dims = _lib.LinearDims(M, N, K, key[1] if M > 1 else K, key[2] if M > 1 else N)
            self._sizes = key, dims
        st = call(x.data_ptr(), mat, bias, dims, out.data_ptr(), ws.data_ptr(), ws.nbytes, status,
                  _raw_stream(dev) if stream is None else _handle(stream))
        if st:
            _lib._check(st, "moe_linear_fp8")
        return out
