"""The decoder operators against plain float64 statements of their formulas.

Tolerances, each derived from the roundings the operator makes:

* U16 = 2^-8, the largest relative error of one rounding to bf16; U11 = 2^-11
  of one to fp16; E4M3 rounds within 2^-4 of a value, or 2^-10 of the scale
  among its subnormals.
* fp32 work before a rounding adds a few 2^-24 of the largest terms involved
  (F32 below: 64 of them).
* attention: with weights p rounded by at most u and normalised by the sum of
  the rounded weights, the output moves by at most u (A + |out|), A = sum p |v|
  / sum p; the scores' own fp32 error e moves it by 2 e A.
* tensor-core sums of 128 products may truncate each addition: 128 x 2^-23 of
  the sum of magnitudes.
"""
import math

import numpy as np
import pytest

from gpu_common import require_gpu

pytestmark = pytest.mark.gpu

U16, U11 = 2.0 ** -8, 2.0 ** -11
F32 = 64 * 2.0 ** -24


@pytest.fixture(scope="module")
def torch():
    return require_gpu()


def _dec():
    from block_fp8_expert_gb300 import decoder
    return decoder


def _lib():
    from block_fp8_expert_gb300 import _lib
    return _lib


def _gen(torch, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _check(got, ref, tol, what):
    got, ref, tol = (np.asarray(t, dtype=np.float64) for t in (got, ref, tol))
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what
    err = np.abs(got - ref)
    bad = ~(err <= tol) & ~np.isnan(ref)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst err/tol " \
                          f"{np.nanmax(err / np.maximum(tol, 1e-300)):.3g}"


def _np(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------ expert selection

def _ref_select(l, bias, k, sigmoid, groups, top_groups, group_top, renorm, scale):
    """Keys, indices and weights row by row in float64, by sorting."""
    l = l.astype(np.float64)
    T, E = l.shape
    idx, w = np.zeros((T, k), np.int32), np.zeros((T, k))
    for t in range(T):
        if sigmoid:
            s = 1.0 / (1.0 + np.exp(-l[t]))
        else:
            top = l[t].max()
            e = np.exp(l[t] - (top if np.isfinite(top) else 0.0))
            s = e / e.sum() if e.sum() > 0 else e
        key = s + (0.0 if bias is None else bias.astype(np.float64))
        cand = list(range(E))
        if groups > 1:
            n = E // groups
            gs = [sum(sorted(key[g * n:(g + 1) * n], reverse=True)[:group_top]) for g in range(groups)]
            best = sorted(range(groups), key=lambda g: (-gs[g], g))[:top_groups]
            cand = [e for e in cand if e // n in best]
        cand.sort(key=lambda e: (-key[e], e))
        idx[t] = cand[:k]
        w[t] = s[idx[t]]
        if renorm:
            w[t] = w[t] / w[t].sum() if w[t].sum() > 0 else 0.0
    return idx, scale * w


def _clear_rows(l, bias, c):
    """Rows whose choice does not hang on a difference under 1e-5."""
    T, E = l.shape
    rng = np.random.default_rng(5)
    keep = np.ones(T, bool)
    base = _ref_select(l, bias, **c)[0]
    for _ in range(3):  # the choice withstands disturbances of the logits of that size
        keep &= (_ref_select(l + 1e-5 * rng.uniform(-1, 1, l.shape), bias, **c)[0] == base).all(1)
    return l[keep]


SELECT = [  # T, E, k, sigmoid, bias, groups, top_groups, group_top, renorm, scale
    (1, 8, 2, False, False, 1, 1, 1, True, 1.0), (7, 1, 1, True, False, 1, 1, 1, True, 1.0),
    (33, 60, 4, False, True, 1, 1, 1, False, 1.0), (65, 128, 8, False, False, 1, 1, 1, True, 1.0),
    (40, 160, 6, False, False, 8, 3, 1, False, 16.0), (50, 256, 8, True, True, 8, 4, 2, True, 2.5),
    (9, 512, 10, True, True, 16, 3, 2, True, 1.0), (5, 1024, 32, False, True, 32, 5, 2, True, 1.0),
    (12, 96, 3, True, False, 32, 1, 2, False, 0.5)]


@pytest.mark.parametrize("case", SELECT)
def test_select(torch, case):
    T, E, k, sigmoid, has_bias, groups, top_groups, group_top, renorm, scale = case
    rng = np.random.default_rng(E)
    bias = (0.2 * rng.standard_normal(E)).astype(np.float32) if has_bias else None
    c = dict(k=k, sigmoid=sigmoid, groups=groups, top_groups=top_groups, group_top=group_top,
             renorm=renorm, scale=scale)
    l = _clear_rows((1.5 * rng.standard_normal((T + 8, E))).astype(np.float32), bias, c)[:T]
    assert len(l)
    ref_i, ref_w = _ref_select(l, bias, **c)
    wide = torch.full((len(l), E + 5), math.nan, device="cuda")  # strided rows
    wide[:, :E] = torch.from_numpy(l).cuda()
    op = _dec().ExpertSelector(E, k, "sigmoid" if sigmoid else "softmax",
                               None if bias is None else torch.from_numpy(bias).cuda(), groups,
                               top_groups, group_top, renorm, scale)
    idx, w = op.forward(wide[:, :E])
    assert np.array_equal(idx.cpu().numpy(), ref_i)
    # exp of a rounded difference (|l| < 16: 2^-20), its own 2 ulp, a sum of E / 32 + 5 rounded terms
    _check(_np(w), ref_w, np.abs(ref_w) * (2.0 ** -20 + (E / 32 + 16) * 2.0 ** -24), "weights")


def test_select_ties_and_switched_off_experts(torch):
    E, k = 64, 4
    l = torch.zeros(6, E, device="cuda")           # all equal: the lowest experts
    l[1, :] = -math.inf                            # nothing left: valid indices, zero weights
    l[2, :] = -math.inf
    l[2, 40] = 3.0                                 # one left
    l[3, 5] = l[3, 9] = 2.0                        # a tie at the top
    l[4] = math.nan
    l[5, 17] = -math.nan
    for score in ("softmax", "sigmoid"):
        for groups, top in ((1, 1), (8, 2)):
            op = _dec().ExpertSelector(E, k, score, None, groups, top, 2 if groups > 1 else 1)
            idx, w = (t.cpu().numpy() for t in op.forward(l))
            assert idx.min() >= 0 and idx.max() < E
            assert all(len(set(r)) == k for r in idx)
            assert idx[0].tolist() == [0, 1, 2, 3] and np.allclose(w[0], 0.25)
            assert (w[1] == 0).all() and idx[1].tolist() == [0, 1, 2, 3]
            assert idx[2, 0] == 40 and w[2, 0] == 1 and (w[2, 1:] == 0).all()
            assert idx[3, :2].tolist() == [5, 9] and w[3, 0] == w[3, 1]
            assert np.isnan(w[4]).all()
    off = torch.zeros(E, device="cuda")
    off[:60] = -math.inf                           # a bias of -inf keeps an expert out
    idx, w = _dec().ExpertSelector(E, k, "softmax", off).forward(l[:1])
    assert idx.tolist() == [[60, 61, 62, 63]] and torch.allclose(w, torch.full_like(w, 0.25))


def test_select_feeds_the_experts(torch):
    """The chosen experts and weights run through permute, experts and combine
    like moe_route's: same routing, same layer output."""
    import moe_inputs as mi
    from block_fp8_expert_gb300.device import DeviceLayer, x_to_device
    lib = _lib()
    layer = mi.make_layer("tiny", seed=3)
    D = DeviceLayer.from_host(layer)
    xb, _ = mi.make_tokens(layer, 24, seed=3)
    x = x_to_device(xb)
    d = D.dims(24)
    idx0 = torch.empty(24, layer.k, dtype=torch.int32, device="cuda")
    w0 = torch.empty(24, layer.k, device="cuda")
    out0 = D.forward(x, topk_idx=idx0, topk_w=w0)
    idx, w = _dec().ExpertSelector(layer.E, layer.k).forward(x.float() @ D.Wr.t())
    assert torch.equal(idx, idx0)
    ws = D.workspace(24)
    P = 24 * layer.k
    off = torch.empty(layer.E + 1, dtype=torch.int32, device="cuda")
    rt, tsr = (torch.empty(P, dtype=torch.int32, device="cuda") for _ in range(2))
    y = torch.empty(P, layer.H, device="cuda")
    out = torch.empty_like(out0)
    lib.moe_permute(idx, d, off, rt, tsr, ws)
    lib.moe_expert_ffn_fp8(x, off, rt, D.routed.abi(), d, y, ws)
    lib.moe_combine(y, tsr, w, None, d, out)
    a, b = _np(out), _np(out0)
    assert np.all(np.abs(a - b) <= 2e-2 * (np.abs(b) + np.sqrt(np.mean(b * b))))


# ------------------------------------------------------------------ norms, positions, cache store

def _ref_norm_rope(x, weight, eps, cos, sin, interleaved):
    """x [heads, D] float64, one token."""
    D = x.shape[1]
    y = x.copy() if weight is None else x / np.sqrt((x * x).sum(1, keepdims=True) / D + eps) * weight
    out = y.copy()
    n = len(cos)
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        out[:, a] = y[:, a] * cos[i] - y[:, b] * sin[i]
        out[:, b] = y[:, b] * cos[i] + y[:, a] * sin[i]
    return out


QK = [  # T, Hq, Hkv, D, rot, interleaved, e4m3, page_size, normed
    (1, 4, 1, 64, 64, False, False, 16, True), (3, 7, 1, 128, 128, False, False, 1, True),
    (17, 32, 4, 128, 128, False, True, 16, True), (5, 6, 2, 128, 32, True, False, 7, True),
    (33, 3, 3, 64, 16, True, True, 5, False), (8, 8, 2, 256, 64, False, True, 32, True),
    (2, 1, 1, 256, 256, True, False, 64, True), (70, 5, 2, 64, 0, False, False, 16, True),
    (40, 16, 8, 128, 96, False, False, 16, False), (600, 32, 4, 128, 128, False, False, 16, True)]


@pytest.mark.parametrize("case", QK)
def test_qk_norm_rope(torch, case):
    T, Hq, Hkv, D, rot, inter, e4m3, ps, normed = case
    dec, g = _dec(), _gen(torch, T * D)
    heads = Hq + 2 * Hkv
    wide = torch.randn(T, heads * D + 8, generator=g, device="cuda").mul(3).to(torch.bfloat16)
    qkv = wide[:, :heads * D]                       # strided rows
    if T > 4:
        qkv[2] = 0                                  # rows of zeros: eps and a = 0
        qkv[3] *= 1e-20                             # all but eps
    n_pos = 50
    cs = dec.rope_cos_sin(n_pos, rot, 1e4) if rot else None
    pos = torch.randint(0, n_pos, (T,), generator=g, device="cuda").to(torch.int32) if rot else None
    qn, kn = ((1 + 0.2 * torch.randn(D, generator=g, device="cuda")) for _ in range(2))
    pages = -(-T // ps) + 3
    if T % 2:
        cache = dec.PagedCache.empty(pages, Hkv, ps, D, e4m3)
    else:  # tokens outside, heads inside, keys and values in one tensor
        c = torch.zeros(pages, 2, ps, Hkv, D, device="cuda",
                        dtype=torch.uint8 if e4m3 else torch.bfloat16)
        sc = torch.zeros(pages, 2, ps, Hkv, device="cuda") if e4m3 else None
        cache = dec.PagedCache(c[:, 0].transpose(1, 2), c[:, 1].transpose(1, 2),
                               *([s.transpose(1, 2) for s in (sc[:, 0], sc[:, 1])] if e4m3 else []))
    slots = torch.randperm(pages * ps, generator=g, device="cuda")[:T]
    if T > 2:
        slots[1] = -1
    op = dec.QkNormRope(Hq, Hkv, D, qn if normed else None, kn if normed else None, cs, inter, 1e-6)
    buf = torch.full((T, Hq + 1, D), math.nan, dtype=torch.bfloat16, device="cuda")
    q = op.forward(qkv, pos, slots, cache, buf[:, :Hq])
    op.check()
    assert torch.isnan(buf[:, Hq]).all()            # nothing beyond the rows' heads
    x = _np(qkv).reshape(T, heads, D)
    written = set()
    K = cache.k.view(torch.float8_e4m3fn) if e4m3 else cache.k
    V = cache.v.view(torch.float8_e4m3fn) if e4m3 else cache.v
    K, V = _np(K), _np(V)
    ks, vs = (_np(cache.k_scale), _np(cache.v_scale)) if e4m3 else (None, None)
    csn = _np(cs) if rot else None
    for t in range(T):
        cos, sin = (csn[pos[t]][:rot // 2], csn[pos[t]][rot // 2:]) if rot else ((), ())
        rq = _ref_norm_rope(x[t, :Hq], _np(qn) if normed else None, 1e-6, cos, sin, inter)
        top = np.abs(rq).max(1, keepdims=True)
        _check(_np(q[t]), rq, U16 * np.abs(rq) + F32 * top + 1e-40, f"q {t}")
        s = int(slots[t])
        if s < 0:
            continue
        written.add(s)
        rk = _ref_norm_rope(x[t, Hq:Hq + Hkv], _np(kn) if normed else None, 1e-6, cos, sin, inter)
        for got, sc, ref in ((K, ks, rk), (V, vs, x[t, Hq + Hkv:])):
            got = got[s // ps, :, s % ps]
            top = np.abs(ref).max(1, keepdims=True)
            if not e4m3:
                _check(got, ref, U16 * np.abs(ref) + F32 * top + 1e-40, f"cache {t}")
                continue
            scale = sc[s // ps, :, s % ps][:, None]
            real = top >= 2.0 ** -117
            _check(scale, np.where(real, top / 448, 0), F32 * top / 448, f"scale {t}")
            _check(got * scale, np.where(real, ref, 0),
                   np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * scale) + F32 * top, f"code {t}")
    for s in range(pages * ps):                     # nothing else was touched
        if s not in written:
            assert (K[s // ps, :, s % ps] == 0).all() and (V[s // ps, :, s % ps] == 0).all()


def test_qk_norm_rope_flags_what_it_cannot_place(torch):
    dec, lib = _dec(), _lib()
    cache = dec.PagedCache.empty(2, 1, 16, 64)
    op = dec.QkNormRope(2, 1, 64, cos_sin=dec.rope_cos_sin(10, 64))
    qkv = torch.ones(3, 4 * 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.tensor([3, 10, -1], dtype=torch.int32, device="cuda")
    slots = torch.tensor([32, 1, 2], device="cuda")
    q = op.forward(qkv, pos, slots, cache)
    with pytest.raises(lib.MoeError, match="0x30"):
        op.check()
    assert not torch.isnan(q[0]).any() and torch.isnan(q[1:]).all()
    assert (cache.k == 0).all() and (cache.v == 0).all()
    assert op.forward(qkv[:0], pos[:0], slots[:0], cache).shape == (0, 2, 64)


# ------------------------------------------------------------------ paged attention

def _paged(torch, g, lens, Hkv, D, ps, e4m3, garbage=True):
    """A cache with scattered pages whose elements outside the sequences are NaN."""
    dec = _dec()
    need = [-(-n // ps) for n in lens]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=g, device="cuda").tolist()
    width = max(need + [1]) + 1
    table = torch.full((len(lens), width), -7, dtype=torch.int32)   # unused entries are no pages
    k = torch.randn(pages, Hkv, ps, D, generator=g, device="cuda")
    v = torch.randn(pages, Hkv, ps, D, generator=g, device="cuda") + 0.5
    live = torch.zeros(pages, ps, dtype=torch.bool)
    for b, n in enumerate(lens):
        for i in range(need[b]):
            p = order.pop()
            table[b, i] = p
            live[p, :min(ps, n - i * ps)] = True
    dead = (~live).cuda()[:, None, :].expand(pages, Hkv, ps)
    if e4m3:
        def quant(x):
            s = x.abs().amax(-1) / 448
            return (x / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), s.contiguous()
        (kc, ks), (vc, vs) = quant(k), quant(v)
        for t in (kc, vc):
            t[dead] = 0x7F
        for t in (ks, vs):
            t[dead] = math.nan
        cache = dec.PagedCache(kc, vc, ks, vs)
        kd = kc.view(torch.float8_e4m3fn).double() * ks[..., None].double()
        vd = vc.view(torch.float8_e4m3fn).double() * vs[..., None].double()
    else:
        k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
        k[dead], v[dead] = math.nan, math.inf
        cache = dec.PagedCache(k, v)
        kd, vd = k.double(), v.double()
    return cache, table.cuda(), kd, vd


def _ref_attention(torch, q, kd, vd, table, lens, ps, scale, window):
    """(out, A) in float64, sequence by sequence."""
    B, Hq, D = q.shape
    Hkv = kd.shape[1]
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
    A = torch.zeros_like(out)
    for b, n in enumerate(lens):
        lo = max(0, n - window) if window else 0
        if n <= lo:
            continue
        t = torch.arange(lo, n, device="cuda")
        page, off = table[b].long()[t // ps], t % ps
        k, v = kd[page, :, off], vd[page, :, off]           # [t, Hkv, D]
        for h in range(Hq):
            s = (k[:, h // (Hq // Hkv)] @ q[b, h].double()) * scale
            p = torch.exp(s - s.max())
            p = p / p.sum()
            out[b, h] = p @ v[:, h // (Hq // Hkv)]
            A[b, h] = p @ v[:, h // (Hq // Hkv)].abs()
    return out, A


def _attn_tol(ref, A, e4m3):
    u = U11 if e4m3 else U16
    # scores: |s| < 64, D products and the scales in fp32, and 2^-21 of ex2 and log2
    e = 64 * F32 + 2.0 ** -20
    return 1.01 * ((u + 2 * e) * (A + np.abs(ref)) + U16 * np.abs(ref))


ATTN = [  # lens, Hq, Hkv, D, page_size, e4m3, window
    ([1], 1, 1, 64, 16, False, 0), ([1], 8, 1, 128, 16, True, 0), ([15, 16, 17, 0, 31, 33], 4, 2, 64, 16, False, 0),
    ([0, 0], 4, 2, 128, 16, False, 0), ([129, 0, 1, 640, 37], 32, 4, 128, 16, False, 0),
    ([129, 0, 1, 640, 37], 32, 4, 128, 16, True, 0), ([77, 500], 14, 2, 128, 7, False, 0),
    ([77, 500], 12, 4, 64, 5, True, 0), ([300, 45], 16, 1, 256, 32, False, 0),
    ([300, 45], 8, 2, 256, 64, True, 0), ([513], 17, 1, 128, 16, False, 0), ([513, 2], 40, 1, 64, 16, True, 0),
    ([900, 33, 100], 8, 2, 128, 16, False, 100), ([900, 33, 100], 8, 2, 128, 3, True, 33),
    ([64] * 70, 6, 2, 64, 1, False, 0), ([20000], 8, 2, 128, 16, False, 0), ([20000], 8, 2, 128, 64, True, 0),
    ([70000, 3], 4, 1, 64, 64, False, 0), ([9000, 8999], 2, 2, 256, 16, False, 0),
    ([30, 7] * 300, 2, 1, 64, 16, False, 0), ([0, 5, 0] * 250, 2, 1, 64, 16, True, 0)]


@pytest.mark.parametrize("case", ATTN)
def test_paged_attention(torch, case):
    lens, Hq, Hkv, D, ps, e4m3, window = case
    g = _gen(torch, sum(lens) + D + e4m3)
    cache, table, kd, vd = _paged(torch, g, lens, Hkv, D, ps, e4m3)
    wide = torch.randn(len(lens), Hq + 2, D, generator=g, device="cuda").mul(1.5).to(torch.bfloat16)
    q = wide[:, 1:Hq + 1]                           # strided rows
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    scale = 1.0 / math.sqrt(D)
    op = _dec().PagedAttention(Hq, Hkv, D, scale, window)
    out = torch.full((len(lens), Hq, D), math.nan, dtype=torch.bfloat16, device="cuda")
    op.forward(q, cache, table, sl, out)
    op.check()
    ref, A = _ref_attention(torch, q, kd, vd, table, lens, ps, scale, window)
    ref, A = _np(ref), _np(A)
    _check(_np(out), ref, _attn_tol(ref, A, e4m3), "attention")
    again = op.forward(q, cache, table, sl)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("e4m3", [False, True])
def test_paged_attention_extreme_values(torch, e4m3):
    """Scores far apart, a dominating token, tokens whose values are tiny or
    zero next to others: the running maximum and the weights' range hold."""
    g = _gen(torch, 11)
    lens, Hq, Hkv, D, ps = [700, 90], 4, 1, 128, 16
    cache, table, kd, vd = _paged(torch, g, lens, Hkv, D, ps, e4m3)
    if e4m3:
        cache.v_scale[table[0, 3].item()] *= 1e-12
        cache.v_scale[table[0, 5].item()] = 0
        cache.v_scale[table[0, 7].item()] *= 1e12
        cache.k_scale[table[1, 2].item()] *= 30
        kd = cache.k.view(torch.float8_e4m3fn).double() * cache.k_scale[..., None].double()
        vd = cache.v.view(torch.float8_e4m3fn).double() * cache.v_scale[..., None].double()
    else:
        cache.v[table[0, 3].item()] *= 1e-12
        cache.v[table[0, 7].item()] *= 1e12
        cache.k[table[1, 2].item()] *= 8
        kd, vd = cache.k.double(), cache.v.double()
    q = torch.randn(2, Hq, D, generator=g, device="cuda").to(torch.bfloat16)
    q[1] *= 4
    q[1, 3] = 0                                     # equal scores
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = _dec().PagedAttention(Hq, Hkv, D).forward(q, cache, table, sl)
    ref, A = (_np(t) for t in _ref_attention(torch, q, kd, vd, table, lens, ps, 1 / math.sqrt(D), 0))
    s = 30 * 8 * 4 * 16                              # the largest |score| here is far below this
    tol = _attn_tol(ref, A, e4m3) + 2 * s * 2.0 ** -22 * (A + np.abs(ref))
    _check(_np(out), ref, tol, "extreme values")


def test_paged_attention_nan_and_flags(torch):
    dec, lib = _dec(), _lib()
    g = _gen(torch, 4)
    lens, ps = [40, 40, 40], 16
    cache, table, kd, vd = _paged(torch, g, lens, 1, 64, ps, False)
    q = torch.randn(3, 2, 64, generator=g, device="cuda").to(torch.bfloat16)
    op = dec.PagedAttention(2, 1, 64)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    clean = op.forward(q, cache, table, sl)
    op.check()
    # a NaN inside a sequence reaches that sequence and no other
    cache.v[table[1, 1].item(), 0, 3, 5] = math.nan
    out = op.forward(q, cache, table, sl)
    assert torch.isnan(out[1, :, 5]).all()
    assert torch.equal(out[0], clean[0]) and torch.equal(out[2], clean[2])
    # a page outside the cache: flagged, its tokens left out
    bad = table.clone()
    bad[0, 1], bad[2, 0] = cache.pages, -1
    out = op.forward(q, cache, bad, sl)
    with pytest.raises(lib.MoeError, match="0x10"):
        op.check()
    for b, toks in ((0, list(range(16)) + list(range(32, 40))), (2, list(range(16, 40)))):
        t = torch.tensor(toks, device="cuda")
        k, v = kd[table[b].long()[t // ps], 0, t % ps], vd[table[b].long()[t // ps], 0, t % ps]
        p = torch.softmax(k @ q[b].double().t() / 8, 0)
        ref, A = _np(p.t() @ v), _np(p.t() @ v.abs())
        _check(_np(out[b]), ref, _attn_tol(ref, A, False), f"sequence {b}")
    # lengths outside the table: flagged and clamped
    op = dec.PagedAttention(2, 1, 64)
    out = op.forward(q, cache, table[:, :3].contiguous(), torch.tensor([40, -5, 4000], dtype=torch.int32, device="cuda"))
    with pytest.raises(lib.MoeError, match="0x10"):
        op.check()
    assert torch.equal(out[0], clean[0]) and (out[1] == 0).all()
    assert op.forward(q[:0], cache, table[:0], sl[:0]).shape == (0, 2, 64)


def test_paged_attention_long_offsets(torch):
    """Element offsets past 2^31: the pages of a 9 GB cache's end."""
    g = _gen(torch, 9)
    pages, Hkv, ps, D = 70000, 4, 64, 128
    k = torch.empty(pages, Hkv, ps, D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    use = torch.tensor([69999, 0, 69998, 40000, 5], device="cuda")
    for t in (k, v):
        t[use] = torch.randn(5, Hkv, ps, D, generator=g, device="cuda").to(torch.bfloat16)
    cache = _dec().PagedCache(k, v)
    lens = [300]
    table = use.to(torch.int32)[None].contiguous()
    q = torch.randn(1, 8, D, generator=g, device="cuda").to(torch.bfloat16)
    out = _dec().PagedAttention(8, Hkv, D).forward(q, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    small = torch.arange(5, device="cuda")[None]
    ref, A = (_np(t) for t in _ref_attention(torch, q, k[use].double(), v[use].double(), small, lens, ps,
                                             1 / math.sqrt(D), 0))
    _check(_np(out), ref, _attn_tol(ref, A, False), "long offsets")


# ------------------------------------------------------------------ linear

def _linear_case(torch, M, N, K, seed=0):
    g = _gen(torch, seed + M + N + K)
    x = torch.randn(M, K, generator=g, device="cuda") * torch.exp(torch.randn(K, generator=g, device="cuda"))
    codes = torch.randn(N, K, generator=g, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    scales = 0.005 + 0.015 * torch.rand(-(-N // 128), -(-K // 128), generator=g, device="cuda")
    return x.to(torch.bfloat16), codes, scales


def _ref_linear(torch, x, codes, scales, bias=None):
    """(out, S) in float64 from the codes the definition gives, S = the sum of
    the products' magnitudes."""
    M, K = x.shape
    N = codes.shape[0]
    out = np.zeros((M, N))
    S = np.zeros((M, N))
    w = codes.view(torch.float8_e4m3fn).double()
    for b in range(-(-K // 128)):
        xb = x[:, 128 * b:128 * b + 128].float().cpu().numpy()
        a = np.abs(xb).max(1, keepdims=True)
        real = a >= np.float32(2.0 ** -117)
        with np.errstate(divide="ignore", over="ignore"):
            f = np.where(real, np.float32(448) * (np.float32(1) / a), np.float32(0)).astype(np.float32)
            s = np.where(real, a / np.float32(448), np.float32(0)).astype(np.float32)
        c = torch.from_numpy((xb * f).clip(-448, 448)).to(torch.float8_e4m3fn).double().cuda()
        wb = w[:, 128 * b:128 * b + 128] * scales[:, b].double().repeat_interleave(128)[:N, None]
        sx = torch.from_numpy(s).cuda().double()
        out += ((c @ wb.t()) * sx).cpu().numpy()
        S += ((c.abs() @ wb.abs().t()) * sx).cpu().numpy()
    if bias is not None:
        out += _np(bias)[None]
        S += np.abs(_np(bias))[None]
    return out, S


def _linear_tol(ref, S):
    return 1.001 * U16 * np.abs(ref) + (128 * 2.0 ** -23 + F32) * S


LINEAR = [(1, 64, 128), (1, 8, 16), (3, 136, 80), (8, 512, 2048), (9, 128, 256), (16, 264, 400),
          (17, 128, 128), (31, 1000, 1040), (33, 256, 512), (64, 2048, 4096), (65, 384, 896), (127, 136, 272),
          (128, 640, 1024), (200, 1288, 528), (257, 512, 16), (300, 264, 2048), (513, 1024, 1152),
          (1030, 2056, 336), (2600, 2056, 272), (1300, 4104, 1040), (4097, 1288, 640)]


@pytest.mark.parametrize("M,N,K", LINEAR)
def test_linear(torch, M, N, K):
    x, codes, scales = _linear_case(torch, M, N, K)
    g = _gen(torch, 1)
    bias = torch.randn(N, generator=g, device="cuda") if M % 2 else None
    wide = torch.full((M, K + 8), math.nan, dtype=torch.bfloat16, device="cuda")
    wide[:, :K] = x
    if M > 4:
        wide[2, :K] = 0                             # empty groups
        wide[3, :min(K, 128)] = 1e-38
    x = wide[:, :K]                                 # strided rows, NaN between them
    buf = torch.full((M, N + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    op = _dec().Fp8Linear(codes, scales, bias)
    op.forward(x, buf[:, :N])
    op.check()
    assert (buf[:, N:] == 7).all()
    ref, S = _ref_linear(torch, x, codes, scales, bias)
    _check(_np(buf[:, :N]), ref, _linear_tol(ref, S), "linear")
    ws = op.workspace(M)
    ws.fill_(0xA5)                                  # whatever the workspace held
    again = op.forward(x, ws=ws)
    assert torch.equal(again.view(torch.int16), buf[:, :N].contiguous().view(torch.int16))


@pytest.mark.parametrize("M", [5, 300])
def test_linear_flags_what_is_not_finite(torch, M):
    lib = _lib()
    x, codes, scales = _linear_case(torch, M, 256, 512)
    op = _dec().Fp8Linear(codes, scales)
    clean = op.forward(x)
    op.check()
    x[1, 300] = math.inf
    x[4, 7] = math.nan
    out = op.forward(x)
    with pytest.raises(lib.MoeError, match="0x8"):
        op.check()
    keep = [i for i in range(M) if i not in (1, 4)]
    assert torch.equal(out[keep], clean[keep])
    assert not torch.isfinite(out[[1, 4]]).any()
    assert op.forward(x[:0]).shape == (0, 256)


def test_linear_scales_of_any_magnitude(torch):
    for gain in (1e-30, 1e25):
        x, codes, scales = _linear_case(torch, 40, 128, 512)
        x = (x.float() * 1e8).to(torch.bfloat16)
        scales = scales * gain
        out = _dec().Fp8Linear(codes, scales).forward(x)
        ref, S = _ref_linear(torch, x, codes, scales)
        _check(_np(out), ref, _linear_tol(ref, S), f"scales times {gain}")


# ------------------------------------------------------------------ streams, captures, Python-side checks

def test_other_streams_and_graphs(torch):
    """The operators on a side stream and replayed from a captured graph give
    the bits of a plain call."""
    dec, g = _dec(), _gen(torch, 21)
    x, codes, scales = _linear_case(torch, 6, 12 * 64, 256)
    lin = dec.Fp8Linear(codes, scales)
    lens = [60, 5, 200, 0, 31, 16]
    cache, table, _, _ = _paged(torch, g, lens, 2, 64, 16, False)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    rope = dec.QkNormRope(8, 2, 64, cos_sin=dec.rope_cos_sin(300, 64))
    spare = dec.PagedCache.empty(4, 2, 16, 64)
    attn = dec.PagedAttention(8, 2, 64)
    pos = torch.arange(6, dtype=torch.int32, device="cuda")
    slots = torch.arange(6, device="cuda")

    def step(stream=None):
        q = rope.forward(lin.forward(x, stream=stream), pos, slots, spare, stream=stream)
        return attn.forward(q, cache, table, sl, stream=stream)

    plain = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    other = step(side)
    side.synchronize()
    assert torch.equal(other, plain)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    held.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held, plain)
    for op in (lin, rope, attn):
        op.check()


def test_python_side_checks(torch):
    dec = _dec()
    x, codes, scales = _linear_case(torch, 4, 64, 128)
    lin = dec.Fp8Linear(codes, scales)
    for bad in (x.float(), x[:, :64], x.t().contiguous().t(), x.cpu()):
        with pytest.raises((TypeError, ValueError)):
            lin.forward(bad)
    with pytest.raises(ValueError):
        dec.Fp8Linear(codes, scales[:, :0])
    with pytest.raises(ValueError):
        dec.ExpertSelector(8, 2, "relu")
    with pytest.raises(TypeError):
        dec.ExpertSelector(8, 2).forward(torch.zeros(4, 8, device="cuda", dtype=torch.float64))
    with pytest.raises(ValueError):
        lin.forward(x, ws=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(_lib().MoeError):
        lin.forward(x, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    c = dec.PagedCache.empty(2, 2, 16, 64)
    with pytest.raises(ValueError):
        dec.PagedCache(c.k, c.v.transpose(0, 1).contiguous().transpose(0, 1))
    with pytest.raises(ValueError):
        dec.PagedAttention(4, 1, 64).forward(torch.zeros(1, 4, 64, device="cuda", dtype=torch.bfloat16), c,
                                             torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                                             torch.ones(1, dtype=torch.int32, device="cuda"))


def test_index_arrays_out_of_longer_ones(torch):
    """Routings, positions, slots, lengths, a table's columns and a cache's
    scales that begin anywhere in a longer array give the bits of a plain call."""
    dec, g = _dec(), _gen(torch, 23)

    def inside(t, room=3):  # a copy that begins 1 element into its buffer
        buf = torch.empty(t.numel() + room, dtype=t.dtype, device="cuda")
        part = buf[1:1 + t.numel()].view(t.shape)
        part.copy_(t)
        assert part.data_ptr() % 16
        return part

    lens = [40, 1, 0, 97]
    B, Hkv, D, page = len(lens), 2, 64, 16
    _, table, _, _ = _paged(torch, g, lens, Hkv, D, page, True)
    qkv = torch.randn(B, 8 * D, generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.tensor(lens, dtype=torch.int32, device="cuda")
    slots = torch.arange(B, device="cuda") * page
    logits = torch.randn(B, 64, generator=g, device="cuda")
    rope = dec.QkNormRope(4, Hkv, D, cos_sin=dec.rope_cos_sin(100, D))
    attn = dec.PagedAttention(4, Hkv, D)
    pick = dec.ExpertSelector(64, 3)
    codes = torch.randint(0, 120, (2, 64, Hkv, page, D), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.rand(2, 64, Hkv, page, generator=g, device="cuda")
    res = []
    for f in (lambda t: t, inside):
        cache = dec.PagedCache(codes[0].clone(), codes[1].clone(), f(scales[0]), f(scales[1]))
        q = rope.forward(qkv, f(pos), f(slots), cache)
        wide = torch.cat([table[:, :1], table], 1)
        o = attn.forward(q, cache, table if f is not inside else wide[:, 1:], f(pos))
        idx, w = pick.forward(logits, f(torch.zeros(B, 3, dtype=torch.int32, device="cuda")),
                              f(torch.zeros(B, 3, device="cuda")))
        res.append([q, o, idx, w, cache.k, cache.v, cache.k_scale, cache.v_scale])
    for a, b in zip(*res):
        assert torch.equal(a, b)
    rope.check()
    attn.check()


def test_memory_of_a_call_on_another_stream(torch):
    """What a call on another stream allocates does not come from memory that
    the current stream has just let go of, which its work may still be using."""
    dec = _dec()
    x, codes, scales = _linear_case(torch, 300, 512, 256)
    lin = dec.Fp8Linear(codes, scales)
    plain = lin.forward(x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        held = [torch.empty_like(plain), lin.workspace(300)]
        gone = {t.data_ptr() for t in held}
        del held
        ws = lin.workspace(300, stream)
        out = lin.forward(x, ws=ws, stream=stream)
        side.synchronize()
        assert not gone & {out.data_ptr(), ws.data_ptr()}
        assert torch.equal(out, plain)
    with torch.cuda.stream(side):  # and the default stream from another one
        side.wait_stream(torch.cuda.default_stream())
        held = torch.empty_like(plain)
        gone = held.data_ptr()
        del held
        out = lin.forward(x, stream=0)
        assert out.data_ptr() != gone
    torch.cuda.synchronize()
    assert torch.equal(out, plain)
    lin.check()


@pytest.mark.parametrize("lens", [[777], [700, 90, 0, 333], [9000, 40], [40000], [130] * 60])
def test_paged_attention_workspaces_of_any_content(torch, lens):
    """Whatever the workspace holds, and however often a captured call is
    replayed over it, the bits are those of the first call, which is checked."""
    dec, g = _dec(), _gen(torch, 31)
    Hq, Hkv, D, page = 8, 2, 64, 16
    cache, table, kd, vd = _paged(torch, g, lens, Hkv, D, page, False)
    B = len(lens)
    q = torch.randn(B, Hq, D, generator=g, device="cuda").to(torch.bfloat16)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    attn = dec.PagedAttention(Hq, Hkv, D)
    ws = attn.workspace(B)
    first = attn.forward(q, cache, table, sl, ws=ws)
    ref, A = _ref_attention(torch, q, kd, vd, table, lens, page, attn.scale, 0)
    _check(_np(first), _np(ref), _attn_tol(_np(ref), _np(A), False), str(lens))
    graph, held = torch.cuda.CUDAGraph(), torch.empty_like(first)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        attn.forward(q, cache, table, sl, out=held, ws=ws)
    for fill in (0, 0xFF, 0x7F, None, None, "own"):
        if fill is None:
            ws.random_(256)
        elif fill != "own":  # (own: as the last call left it)
            ws.fill_(fill)
        assert torch.equal(attn.forward(q, cache, table, sl, ws=ws), first)
        for _ in range(20):
            held.zero_()
            graph.replay()
            assert torch.equal(held, first)
    attn.check()


@pytest.mark.parametrize("E,groups,top_groups,group_top,k", [
    (1020, 17, 9, 2, 8), (1020, 15, 4, 1, 32), (1023, 3, 2, 2, 10), (1023, 31, 7, 2, 5), (45, 9, 4, 2, 3),
    (105, 7, 3, 1, 6), (160, 5, 2, 2, 8), (20, 20, 6, 1, 4), (992, 31, 31, 2, 30), (64, 2, 1, 2, 16)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_select_groups_of_any_size(torch, E, groups, top_groups, group_top, k, sigmoid):
    rng = np.random.default_rng(E + groups)
    c = dict(k=k, sigmoid=sigmoid, groups=groups, top_groups=top_groups, group_top=group_top, renorm=True,
             scale=2.0)
    bias = (0.05 * rng.standard_normal(E)).astype(np.float32)
    l = _clear_rows((1.5 * rng.standard_normal((24, E))).astype(np.float32), bias, c)
    assert len(l) > 4
    idx, w = _ref_select(l, bias, **c)
    sel = _dec().ExpertSelector(E, k, "sigmoid" if sigmoid else "softmax", torch.from_numpy(bias).cuda(),
                                groups, top_groups, group_top, True, 2.0)
    for pad in (0, 4, 5):  # rows on 16-byte boundaries or not
        wide = torch.full((len(l), E + pad), math.nan, device="cuda")
        wide[:, :E] = torch.from_numpy(l).cuda()
        gi, gw = sel.forward(wide[:, :E])
        assert np.array_equal(gi.cpu().numpy(), idx)
        # exponentials and sums of fp32: some tens of roundings of each weight
        _check(_np(gw), w, 2.0 ** -18 * np.abs(w), f"E {E}, {groups} groups")


@pytest.mark.parametrize("M,N,K", [(9, 8200, 2048), (16, 8192, 2048), (16, 8192, 2064), (12, 4112, 4112)])
def test_linear_where_sixteen_rows_change_kernels(torch, M, N, K):
    """Either side of 2^24 weights with 9 to 16 rows."""
    x, codes, scales = _linear_case(torch, M, N, K)
    lin = _dec().Fp8Linear(codes, scales)
    out = lin.forward(x)
    lin.check()
    ref, S = _ref_linear(torch, x, codes, scales)
    _check(_np(out), ref, _linear_tol(ref, S), f"{M} x {N} x {K}")


@pytest.mark.parametrize("M,N", [(40, 4864), (150, 2432), (64, 4352), (33, 9728)])
def test_linear_around_a_wave_of_clusters(torch, M, N):
    """Tile counts near those at which K is divided over fewer CTAs."""
    x, codes, scales = _linear_case(torch, M, N, 2048, seed=3)
    lin = _dec().Fp8Linear(codes, scales)
    out = lin.forward(x)
    lin.check()
    ref, S = _ref_linear(torch, x, codes, scales)
    _check(_np(out), ref, _linear_tol(ref, S), f"{M} x {N}")
