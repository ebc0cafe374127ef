"""The decoder operators without a GPU: arguments are refused on the host
before any CUDA call, workspaces are sized, and the rotation tables follow
their formulas."""
import ctypes
import math

import pytest

from block_fp8_expert_gb300 import _lib
from block_fp8_expert_gb300 import build as B

INV, UNS, WS = _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED, _lib.MOE_ERR_WORKSPACE
P = 0x1000  # an aligned address that is never touched


@pytest.fixture(scope="module")
def L():
    B.build()
    return _lib.lib()


def _rule(**kw):
    d = dict(score=1, groups=8, top_groups=4, group_top=2, renorm=1, scale=1.0)
    d.update(kw)
    return _lib.SelectRule(**d)


def _select(L, T=4, E=256, k=8, stride=None, logits=P, bias=None, idx=P, w=P, **rule):
    return L.moe_select_experts(logits, E if stride is None else stride, bias, _rule(**rule), T, E,
                                k, idx, w, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INV), (dict(E=0), UNS), (dict(E=2048), UNS), (dict(score=2), INV),
    (dict(groups=0), UNS), (dict(groups=7), UNS), (dict(groups=64), UNS), (dict(top_groups=0), INV),
    (dict(top_groups=9), INV), (dict(group_top=0), INV), (dict(group_top=3), INV),
    (dict(E=8, k=4, group_top=2), INV),  # one expert per group
    (dict(k=0), UNS), (dict(k=33), UNS), (dict(E=16, k=9, top_groups=4), UNS),
    (dict(stride=255), INV), (dict(logits=None), INV), (dict(logits=P + 4), INV),
    (dict(bias=P + 4), INV), (dict(idx=None), INV), (dict(w=None), INV)])
def test_select_refusals(L, kw, code):
    assert _select(L, **kw) == code
    assert L.moe_last_error_message()


def test_select_no_tokens(L):
    assert _select(L, T=0, logits=None, idx=None, w=None) == _lib.MOE_OK


def _cache(**kw):
    d = dict(k=P, v=P, k_scale=None, v_scale=None, pages=4, page_size=16, Hkv=2, D=128, format=0,
             page_stride=4096, head_stride=2048, token_stride=128, scale_page_stride=0,
             scale_head_stride=0, scale_token_stride=0)
    d.update(kw)
    return _lib.KvCache(**d)


BAD_CACHES = [
    (dict(format=2), INV), (dict(D=96), UNS), (dict(Hkv=0), UNS), (dict(pages=0), INV),
    (dict(page_size=0), INV), (dict(k=None), INV), (dict(v=P + 8), INV), (dict(page_stride=-8), INV),
    (dict(token_stride=132), INV), (dict(head_stride=2052), INV), (dict(k_scale=P), INV),
    (dict(format=1), INV), (dict(format=1, k_scale=P, v_scale=P, token_stride=136), INV)]


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_cache_refusals(L, kw, code):
    d = _lib.AttnDims(2, 8, 4, 0, 0.1, 4, 8 * 128, 8 * 128)
    assert L.moe_paged_attention(P, _cache(**kw), P, P, d, P, P, 1 << 30, None, None) == code
    q = _lib.QkDims(2, 8, 0, 0, 0, 1e-6, 12 * 128, 8 * 128)
    assert L.moe_qk_norm_rope(P, None, None, None, None, P, q, _cache(**kw), P, None, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INV), (dict(Hq=0), UNS), (dict(rot=8), UNS), (dict(rot=144), UNS), (dict(n_pos=0), INV),
    (dict(qkv_stride=12 * 128 - 8), INV), (dict(qkv_stride=12 * 128 + 4), INV), (dict(q_stride=1000), INV),
    (dict(cos_sin=None), INV), (dict(pos=None), INV), (dict(rot=0), INV), (dict(slots=None), INV),
    (dict(qkv=None), INV), (dict(qkv=P + 2), INV), (dict(q_out=None), INV), (dict(status=P + 4), INV),
    (dict(q_norm=P + 4), INV)])
def test_qk_norm_rope_refusals(L, kw, code):
    a = dict(qkv=P, q_norm=P, k_norm=P, cos_sin=P, pos=P, slots=P, q_out=P, status=P, T=2, Hq=8,
             rot=128, n_pos=16, qkv_stride=12 * 128, q_stride=8 * 128)
    a.update(kw)
    d = _lib.QkDims(a["T"], a["Hq"], a["rot"], 0, a["n_pos"], 1e-6, a["qkv_stride"], a["q_stride"])
    assert L.moe_qk_norm_rope(a["qkv"], a["q_norm"], a["k_norm"], a["cos_sin"], a["pos"], a["slots"],
                              d, _cache(), a["q_out"], a["status"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INV), (dict(Hq=0), UNS), (dict(Hq=7), UNS), (dict(window=-1), INV),
    (dict(width=-1), INV), (dict(table_stride=3), INV), (dict(q_stride=1000), INV),
    (dict(out_stride=1028), INV), (dict(q=None), INV), (dict(table=None), INV), (dict(lens=None), INV),
    (dict(out=P + 8), INV), (dict(ws=None), INV), (dict(nws=1000), WS), (dict(status=P + 4), INV),
    (dict(B=1 << 20, width=1 << 14, table_stride=1 << 14), UNS)])
def test_paged_attention_refusals(L, kw, code):
    a = dict(B=2, Hq=8, window=0, width=4, table_stride=4, q_stride=1024, out_stride=1024, q=P, table=P,
             lens=P, out=P, ws=P, nws=1 << 30, status=None)
    a.update(kw)
    d = _lib.AttnDims(a["B"], a["Hq"], a["width"], a["window"], 0.1, a["table_stride"], a["q_stride"],
                      a["out_stride"])
    assert L.moe_paged_attention(a["q"], _cache(), a["table"], a["lens"], d, a["out"], a["ws"],
                                 a["nws"], a["status"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INV), (dict(M=1 << 23), UNS), (dict(N=12), UNS), (dict(N=65544), UNS), (dict(K=8), UNS), (dict(K=136), UNS),
    (dict(xs=120), INV), (dict(xs=132), INV), (dict(os=60), INV), (dict(x=None), INV), (dict(x=P + 2), INV),
    (dict(codes=None), INV), (dict(scales=P + 4), INV), (dict(bias=P + 4), INV), (dict(out=None), INV),
    (dict(ws=None), INV), (dict(nws=0), WS), (dict(status=P + 4), INV)])
def test_linear_refusals(L, kw, code):
    a = dict(M=4, N=64, K=128, xs=128, os=64, x=P, codes=P, scales=P, bias=None, out=P, ws=P,
             nws=1 << 40, status=None)
    a.update(kw)
    d = _lib.LinearDims(a["M"], a["N"], a["K"], a["xs"], a["os"])
    assert L.moe_linear_fp8(a["x"], _lib.Fp8Mat(a["codes"], a["scales"]), a["bias"], d, a["out"],
                            a["ws"], a["nws"], a["status"], None) == code


def test_workspaces(L):
    d = _lib.AttnDims(8, 32, 0, 0, 0.1, 0, 0, 0)
    assert _lib.paged_attention_workspace_bytes(d, 128) >= 16 * 128 * 4
    with pytest.raises(_lib.MoeError):
        _lib.paged_attention_workspace_bytes(d, 96)
    assert _lib.linear_fp8_workspace_bytes(_lib.LinearDims(0, 64, 128, 128, 64)) > 0
    with pytest.raises(_lib.MoeError):
        _lib.linear_fp8_workspace_bytes(_lib.LinearDims(4, 64, 100, 104, 64))


def test_rotation_tables():
    """Each form against its formula, one entry at a time, in Python floats
    (float64); the table is rounded once to fp32 (2^-24 of a value <= 1.5)."""
    pytest.importorskip("torch")
    from block_fp8_expert_gb300.decoder import rope_cos_sin
    rot, base, factor, original = 64, 1e4, 4.0, 4096

    def check(table, inv, gain=1.0):
        for p in (0, 1, 37, 499):
            for i in range(0, rot // 2, 3):
                assert abs(table[p, i].item() - gain * math.cos(p * inv(i))) <= 2 ** -23
                assert abs(table[p, rot // 2 + i].item() - gain * math.sin(p * inv(i))) <= 2 ** -23

    def plain(i):
        return base ** (-2 * i / rot)

    check(rope_cos_sin(500, rot, base, device="cpu"), plain)
    check(rope_cos_sin(500, rot, base, factor, "linear", device="cpu"), lambda i: plain(i) / factor)

    def yarn(i):
        def pair(turns):
            return rot / 2 * math.log(original / (2 * math.pi * turns), base)
        lo, hi = math.floor(pair(32.0)), math.ceil(pair(1.0))
        r = min(max((i - lo) / (hi - lo), 0.0), 1.0)
        return plain(i) * (1 - r) + plain(i) / factor * r

    check(rope_cos_sin(500, rot, base, factor, "yarn", original, device="cpu"), yarn,
          0.1 * math.log(factor) + 1)
    for bad in (dict(scaling="ntk"), dict(scaling="yarn"), dict(scaling="yarn", original=8, factor=0.5)):
        with pytest.raises(ValueError):
            rope_cos_sin(8, rot, base, device="cpu", **bad)
    with pytest.raises(ValueError):
        rope_cos_sin(8, 7, device="cpu")


@pytest.mark.parametrize("kw,code", [
    (dict(H=100), UNS), (dict(k=40), UNS), (dict(x=None), INV), (dict(Wr=P + 4), INV),
    (dict(logit_bias=P + 4), INV), (dict(bias=P + 4), INV), (dict(idx=None), INV), (dict(w=None), INV),
    (dict(ws=None), INV), (dict(nws=100), WS), (dict(groups=5), UNS), (dict(score=3), INV)])
def test_route_select_refusals(L, kw, code):
    a = dict(x=P, Wr=P, logit_bias=None, bias=None, idx=P, w=P, ws=P, nws=1 << 40, H=256, k=2, groups=1, score=0)
    a.update(kw)
    d = _lib.dims(8, a["H"], 128, 16, a["k"])
    r = _rule(groups=a["groups"], top_groups=1, group_top=1, score=a["score"])
    assert L.moe_route_select(a["x"], a["Wr"], a["logit_bias"], a["bias"], r, d, a["idx"], a["w"],
                              a["ws"], a["nws"], None) == code


def test_arrays_of_elements_need_their_alignment_only(L):
    """Half an element off is refused for every array that is read or written
    one element at a time (a whole element off is taken on the GPU)."""
    assert _select(L, idx=P + 2) == INV and _select(L, w=P + 2) == INV
    d = _lib.AttnDims(2, 8, 4, 0, 0.1, 4, 8 * 128, 8 * 128)
    f8 = dict(format=1, k_scale=P, v_scale=P)
    for cache, table, lens in ((_cache(), P + 2, P), (_cache(), P, P + 2),
                               (_cache(**{**f8, "k_scale": P + 2}), P, P),
                               (_cache(**{**f8, "v_scale": P + 1}), P, P)):
        assert L.moe_paged_attention(P, cache, table, lens, d, P, P, 1 << 30, None, None) == INV
    q = _lib.QkDims(2, 8, 16, 0, 4, 1e-6, 12 * 128, 8 * 128)
    for pos, slots in ((P + 2, P), (P, P + 4)):
        assert L.moe_qk_norm_rope(P, None, None, P, pos, slots, q, _cache(), P, None, None) == INV


@pytest.mark.parametrize("kw,code", [
    (dict(H=100), UNS), (dict(k=40), UNS), (dict(x=None), INV), (dict(idx=None), INV), (dict(idx=P + 2), INV),
    (dict(w=None), INV), (dict(w=P + 2), INV), (dict(codes=None), INV), (dict(out=P + 8), INV), (dict(ws=None), INV),
    (dict(nws=100), WS), (dict(status=P + 4), INV), (dict(gate=P), INV), (dict(I_shared=64), INV),
    (dict(shared=True), INV), (dict(I_shared=64, shared=True, gate=P + 4), INV)])
def test_experts_forward_refusals(L, kw, code):
    a = dict(x=P, idx=P, w=P, codes=P, out=P, ws=P, nws=1 << 40, status=None, gate=None, shared=False, H=256, k=2,
             I_shared=0)
    a.update(kw)
    d = _lib.dims(8, a["H"], 128, 16, a["k"], a["I_shared"])
    f = _lib.ffn(*(a["codes"], P) * 3)
    assert L.moe_experts_forward(a["x"], a["idx"], a["w"], f, ctypes.byref(f) if a["shared"] else None, a["gate"],
                                 d, a["out"], a["ws"], a["nws"], a["status"], None) == code
    assert L.moe_last_error_message()


def test_experts_forward_without_tokens(L):
    f = _lib.ffn(*(P, P) * 3)
    assert L.moe_experts_forward(None, None, None, f, None, None, _lib.dims(0, 256, 128, 16, 2), None, None, 0, None,
                                 None) == _lib.MOE_OK
