"""The latent and drafted-token operators without a GPU: arguments are refused
on the host before any CUDA call, workspaces are sized."""
import pytest

from block_fp8_expert_gb300 import _lib
from block_fp8_expert_gb300 import build as B

INV, UNS, WS = _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED, _lib.MOE_ERR_WORKSPACE
P = 0x1000  # an aligned address that is never touched


@pytest.fixture(scope="module")
def L():
    B.build()
    return _lib.lib()


def _cache(**kw):
    d = dict(k=P, v=P, k_scale=None, v_scale=None, pages=4, page_size=16, Hkv=2, D=128, format=0,
             page_stride=4096, head_stride=2048, token_stride=128, scale_page_stride=0,
             scale_head_stride=0, scale_token_stride=0)
    d.update(kw)
    return _lib.KvCache(**d)


def _latent(**kw):
    d = dict(data=P, pages=4, page_size=16, R=512, rot=64, page_stride=16 * 576, token_stride=576)
    d.update(kw)
    return _lib.LatentPages(**d)


def _dims(Dq, Dv, **kw):
    a = dict(B=2, n=4, Hq=8, width=4, window=0, table_stride=4, q_stride=4 * 8 * Dq, q_row_stride=8 * Dq,
             out_stride=4 * 8 * Dv, out_row_stride=8 * Dv, mask_stride=4)
    a.update(kw)
    return _lib.DraftDims(a["B"], a["n"], a["Hq"], a["width"], a["window"], 0.1, a["table_stride"], a["q_stride"],
                          a["q_row_stride"], a["out_stride"], a["out_row_stride"], a["mask_stride"])


SHARED = [
    (dict(B=-1), INV), (dict(n=0), UNS), (dict(n=65), UNS), (dict(Hq=0), UNS), (dict(Hq=2048), UNS), (dict(width=-1), INV),
    (dict(window=-1), INV), (dict(table_stride=3), INV), (dict(q_stride=-8), INV), (dict(q_stride=12), INV),
    (dict(q_row_stride=8), INV), (dict(out_row_stride=8), INV), (dict(out_stride=8), INV), (dict(out_stride=4097), INV),
    (dict(mask_stride=3), INV), (dict(q=None), INV), (dict(q=P + 2), INV), (dict(table=None), INV), (dict(lens=None), INV),
    (dict(lens=P + 2), INV), (dict(mask=P + 4), INV), (dict(drafts=P + 1), INV), (dict(out=None), INV),
    (dict(out=P + 8), INV), (dict(ws=None), INV), (dict(nws=1000), WS), (dict(status=P + 4), INV),
    (dict(B=1 << 22, width=1 << 14, table_stride=1 << 14), UNS)]


def _split(kw, defaults):
    a = dict(q=P, table=P, lens=P, mask=P, drafts=None, out=P, ws=P, nws=1 << 40, status=None)
    a.update({k: v for k, v in kw.items() if k in a})
    return a, {k: v for k, v in kw.items() if k not in a}


def _tree(L, cache=None, **kw):
    a, d = _split(kw, None)
    return L.moe_tree_attention(a["q"], cache or _cache(page_size=64, page_stride=1 << 14, head_stride=1 << 13),
                                a["table"], a["lens"], a["mask"], a["drafts"], _dims(128, 128, **d), a["out"], a["ws"],
                                a["nws"], a["status"], None)


def _absorbed(L, cache=None, **kw):
    a, d = _split(kw, None)
    return L.moe_latent_attention(a["q"], cache or _latent(page_size=256, page_stride=256 * 576), a["table"], a["lens"],
                                  a["mask"], a["drafts"], _dims(576, 512, **d), a["out"], a["ws"], a["nws"], a["status"], None)


@pytest.mark.parametrize("kw,code", SHARED + [(dict(Hq=7), UNS), (dict(window=3), UNS)])
def test_tree_refusals(L, kw, code):
    assert _tree(L, **kw) == code
    assert L.moe_last_error_message()


@pytest.mark.parametrize("kw,code", SHARED + [(dict(window=64), UNS), (dict(Hq=1024, n=9), UNS)])
def test_latent_attention_refusals(L, kw, code):
    assert _absorbed(L, **kw) == code
    assert L.moe_last_error_message()


@pytest.mark.parametrize("kw,code", [
    (dict(format=2), INV), (dict(D=96), UNS), (dict(Hkv=0), UNS), (dict(pages=0), INV), (dict(k=None), INV),
    (dict(token_stride=132), INV), (dict(k_scale=P), INV), (dict(format=1), INV)])
def test_tree_cache_refusals(L, kw, code):
    assert _tree(L, _cache(**kw)) == code


BAD_LATENT = [(dict(R=128), UNS), (dict(rot=32), UNS), (dict(pages=0), INV), (dict(page_size=0), INV), (dict(data=None), INV),
              (dict(data=P + 8), INV), (dict(page_stride=-8), INV), (dict(token_stride=580), INV)]


def _store(L, cache=None, **kw):
    a = dict(T=2, H=4, n_pos=16, kv_stride=576, q_stride=4 * 192, q_head_stride=192, q_out_stride=256, q_out_head_stride=64,
             rows_stride=576, kv=P, norm=P, cos_sin=P, pos=P, slots=P, q=P, q_out=P, rows=P, status=P)
    a.update(kw)
    d = _lib.LatentDims(a["T"], a["H"], 0, a["n_pos"], 1e-6, a["kv_stride"], a["q_stride"], a["q_head_stride"],
                        a["q_out_stride"], a["q_out_head_stride"], a["rows_stride"])
    return L.moe_latent_store(a["kv"], a["norm"], a["cos_sin"], a["pos"], a["slots"], a["q"], d, cache or _latent(),
                              a["q_out"], a["rows"], a["status"], None)


@pytest.mark.parametrize("kw,code", BAD_LATENT)
def test_latent_cache_refusals(L, kw, code):
    assert _absorbed(L, _latent(**kw)) == code
    assert _store(L, _latent(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INV), (dict(H=-1), UNS), (dict(H=2000), UNS), (dict(n_pos=0), INV), (dict(kv_stride=568), INV),
    (dict(kv_stride=580), INV), (dict(rows_stride=64), INV), (dict(q_head_stride=56), INV), (dict(q_out_head_stride=68), INV),
    (dict(q_stride=-8), INV), (dict(q_out_stride=12), INV), (dict(H=0), INV), (dict(kv=None), INV), (dict(kv=P + 2), INV),
    (dict(norm=P + 4), INV), (dict(cos_sin=None), INV), (dict(pos=None), INV), (dict(pos=P + 2), INV),
    (dict(slots=None), INV), (dict(slots=P + 4), INV), (dict(q=None), INV), (dict(q_out=None), INV), (dict(rows=P + 8), INV),
    (dict(status=P + 4), INV)])
def test_latent_store_refusals(L, kw, code):
    assert _store(L, **kw) == code
    assert L.moe_last_error_message()


def _expanded(L, **kw):
    a = dict(B=2, Tq=8, Tk=9, H=4, scale=0.1, q_stride=768, q_head_stride=192, k_stride=1024, k_head_stride=256,
             rope_stride=64, v_stride=1024, v_head_stride=256, out_stride=512, out_head_stride=128, q=P, k=P, rope=P, v=P,
             cu_q=P, cu_k=P, out=P, status=None)
    a.update(kw)
    d = _lib.ExpandedDims(a["B"], a["Tq"], a["Tk"], a["H"], a["scale"], a["q_stride"], a["q_head_stride"], a["k_stride"],
                          a["k_head_stride"], a["rope_stride"], a["v_stride"], a["v_head_stride"], a["out_stride"],
                          a["out_head_stride"])
    return L.moe_expanded_attention(a["q"], a["k"], a["rope"], a["v"], a["cu_q"], a["cu_k"], d, a["out"], a["status"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INV), (dict(Tq=-1), INV), (dict(Tk=-1), INV), (dict(H=0), UNS), (dict(H=1025), UNS), (dict(scale=0.0), INV),
    (dict(scale=-1.0), INV), (dict(scale=float("nan")), INV), (dict(Tq=2 ** 31 - 1), UNS), (dict(Tk=2 ** 31 - 1), UNS),
    (dict(q_stride=184), INV), (dict(q_head_stride=196), INV), (dict(k_stride=120), INV), (dict(k_head_stride=64), INV),
    (dict(rope_stride=56), INV), (dict(v_stride=132), INV), (dict(v_head_stride=120), INV), (dict(out_stride=64), INV),
    (dict(out_head_stride=132), INV), (dict(k_stride=1 << 39), UNS), (dict(B=1 << 22, H=1024), UNS), (dict(q=None), INV),
    (dict(k=None), INV), (dict(rope=P + 8), INV), (dict(v=P + 2), INV), (dict(cu_q=None), INV), (dict(cu_k=P + 2), INV),
    (dict(out=None), INV), (dict(status=P + 4), INV)])
def test_expanded_refusals(L, kw, code):
    assert _expanded(L, **kw) == code
    assert L.moe_last_error_message()


def test_nothing_to_do(L):
    assert _tree(L, B=0, q=None, table=None, lens=None, out=None, ws=None, nws=0) == _lib.MOE_OK
    assert _absorbed(L, B=0, q=None, table=None, lens=None, out=None, ws=None, nws=0) == _lib.MOE_OK
    assert _store(L, T=0, kv=None, pos=None, slots=None, q=None, q_out=None) == _lib.MOE_OK
    assert _expanded(L, Tq=0, q=None, out=None) == _lib.MOE_OK
    assert _expanded(L, B=0, cu_q=None, cu_k=None) == _lib.MOE_OK


def test_workspaces(L):
    d = _dims(128, 128, B=300)
    assert _lib.tree_attention_workspace_bytes(d, 2, 128) >= 300 * 2 * 8 + 64 * 130 * 4
    assert _lib.latent_attention_workspace_bytes(_dims(576, 512), 512) >= 64 * 514 * 4
    for bad in (lambda: _lib.tree_attention_workspace_bytes(d, 2, 96), lambda: _lib.tree_attention_workspace_bytes(d, 3, 128),
                lambda: _lib.latent_attention_workspace_bytes(_dims(576, 512), 300)):
        with pytest.raises(_lib.MoeError):
            bad()
    # fewer sequences or new tokens never need more
    for B, n in ((1, 4), (2, 1), (2, 3)):
        assert _lib.tree_attention_workspace_bytes(_dims(128, 128, B=B, n=n), 2, 128) <= \
            _lib.tree_attention_workspace_bytes(_dims(128, 128, B=2, n=4), 2, 128)
