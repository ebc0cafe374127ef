"""Attention of drafted tokens and latent attention on the edges: queries and keys
that are NaN, scores of -infinity, E4M3 value scales at the ends of fp32, the
smallest pages and pages that are no power of two, negative scales, and every
sequence of the divisions.

Tolerances as in test_gpu_draft_attention.py.
"""
import math

import pytest

from gpu_common import require_gpu
from test_gpu_draft_attention import Batch, _close, _dec
from test_gpu_latent import _expanded, _expanded_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return require_gpu()


def _batch(torch, kind, lens, n, Hq, Hkv, D, ps=16, **kw):
    Dk = D + 64 if kind == "latent" else D
    return Batch(torch, lens, [min(n, x) for x in lens], n, Hq, Hkv, Dk, D, ps, kind, **kw)


# 64 or 128 rows of a CTA, one or two row tiles
SHAPES = [("bf16", 3, 8, 2, 64), ("bf16", 20, 4, 1, 128), ("bf16", 2, 4, 1, 256), ("e4m3", 3, 8, 2, 64),
          ("e4m3", 20, 4, 1, 128), ("e4m3", 2, 4, 1, 256), ("latent", 3, 8, 1, 256), ("latent", 1, 20, 1, 512)]
# segments of one part each; of many parts; of shares that end inside them
LENS = {"whole": [120, 90, 6], "parts": [9000], "shares": [2000] * 100}


# ------------------------------------------------------------------ NaN

@pytest.mark.parametrize("lens", LENS.values(), ids=LENS.keys())
@pytest.mark.parametrize("kind,n,Hq,Hkv,D", SHAPES)
def test_a_nan_query_answers_nan(torch, kind, n, Hq, Hkv, D, lens):
    """However the cache is divided; the other rows do not notice."""
    b = _batch(torch, kind, lens, n, Hq, Hkv, D)
    ref, tol = b.reference()
    hit = torch.zeros(len(lens), n, Hq, dtype=torch.bool, device="cuda")
    for s, i, h in ((0, 0, 2), (len(lens) - 1, n // 2, Hq - 1)):
        b.q[s, i, h, 5] = math.nan
        hit[s, i, h] = i < b.drafts[s]
    got = b.run()
    assert torch.isnan(got[hit]).all()
    _close(torch, got[~hit], ref[~hit], tol[~hit])


@pytest.mark.parametrize("lens", LENS.values(), ids=LENS.keys())
@pytest.mark.parametrize("kind,n,Hq,Hkv,D", SHAPES)
def test_nan_keys_of_whole_tiles_answer_nan(torch, kind, n, Hq, Hkv, D, lens):
    """A context with tiles, and so parts, of nothing but NaN scores."""
    b = _batch(torch, kind, lens, n, Hq, Hkv, D)
    ref, tol = b.reference()
    t = torch.arange(640, 1024) if lens[0] > 1100 else torch.arange(0, 64)
    page, off = b.table[0].long()[t.cuda() // b.ps], t.cuda() % b.ps
    if kind == "latent":
        b.data[page, off, D + 3] = math.nan  # of the shared key part: the values stay
    elif kind == "bf16":
        b.k[page, :, off] = math.nan
    else:
        b.k.view(torch.uint8)[page, :, off] = 0x7F
    got = b.run()
    assert torch.isnan(got[0, :b.drafts[0]]).all()
    _close(torch, got[1:], ref[1:], tol[1:])
    if kind != "latent" and lens[0] > 1100:  # a window that they lie behind
        _close(torch, b.run(window=300), *b.reference(window=300))


def test_a_nan_query_of_a_prompt_answers_nan(torch):
    q, kv, rope, cu_q, cu_k = _expanded(torch, [300, 90], [0, 700], 3)
    op = _dec().ExpandedAttention(3)
    ref, tol = _expanded_ref(torch, q, kv, rope, cu_q, cu_k, op.scale)
    hit = torch.zeros(390, 3, dtype=torch.bool, device="cuda")
    for i, h in ((0, 1), (299, 0), (320, 2)):
        q[i, h, 100] = math.nan
        hit[i, h] = True
    got = op.forward(q, kv[..., :128], rope, kv[..., 128:], cu_q, cu_k)
    assert torch.isnan(got[hit]).all()
    _close(torch, got[~hit], ref[~hit], tol[~hit])


# ------------------------------------------------------------------ scores of -infinity

@pytest.mark.parametrize("lens", LENS.values(), ids=LENS.keys())
@pytest.mark.parametrize("kind,n,Hq,Hkv,D", [c for c in SHAPES if c[0] != "e4m3"])
def test_scores_of_minus_infinity_are_not_seen(torch, kind, n, Hq, Hkv, D, lens):
    """Tokens with such scores have no weight; rows with nothing else answer zeros."""
    b = _batch(torch, kind, lens, n, Hq, Hkv, D)
    b.q[..., -2] = 1.0
    keys = b.data if kind == "latent" else b.k
    clean = keys.clone()

    def spoil(s, lo, hi):
        t = torch.arange(lo, hi, device="cuda")
        page, off = b.table[s].long()[t // b.ps], t % b.ps
        if kind == "latent":
            keys[page, off, -2] = -math.inf
        else:
            keys[page, :, off, -2] = -math.inf
    gone = min(70, lens[0] - n) if lens[0] < 1100 else 1000
    spoil(0, 0, gone)
    if len(lens) > 1:
        spoil(1, 0, lens[1])
    got = b.run()
    keys.copy_(clean)
    b.seen = lambda s, i, *a: [t for t in Batch.seen(b, s, i, *a) if s > 1 or (s == 0 and t >= gone)]
    _close(torch, got, *b.reference())


def test_scores_of_minus_infinity_in_a_prompt(torch):
    q, kv, rope, cu_q, cu_k = _expanded(torch, [500], [0], 2)
    q[..., 190] = 1.0
    later = torch.tensor([0, 400], dtype=torch.int32, device="cuda")
    op = _dec().ExpandedAttention(2)
    ref, tol = _expanded_ref(torch, q[100:], kv[100:], rope[100:], later, later, op.scale)
    rope[:100, 62] = -math.inf
    got = op.forward(q, kv[..., :128], rope, kv[..., 128:], cu_q, cu_k)
    assert (got[:100] == 0).all()
    _close(torch, got[100:], ref, tol)


# ------------------------------------------------------------------ E4M3 scales

def _scaled(torch, lens, n, Hq, Hkv, D, ps, e):
    """A batch whose value scales lie in [2^e, 2^(e + 1)), its values' codes within
    1/2, with reference and tolerance: that of the formula, and half a step of bf16's
    subnormals (2^-134) where the outputs are."""
    b = _batch(torch, "e4m3", lens, n, Hq, Hkv, D, ps)
    g = torch.Generator(device="cuda")
    g.manual_seed(e + 1000)
    f = 1 + 0.99 * torch.rand(b.vs.shape, generator=g, device="cuda", dtype=torch.float64)
    b.vs.copy_((f * 2.0 ** e).float())
    b.v.copy_((0.25 * torch.randn(b.v.shape, generator=g, device="cuda")).clamp(-0.5, 0.5).to(torch.float8_e4m3fn))
    ref, tol = b.reference()
    return b, ref, (tol - 1e-30).clamp(min=0) + 2.0 ** -133


@pytest.mark.parametrize("e", [-140, -126, -121, -60, 60, 119, 120, 121, 122, 125, 126, 127])
@pytest.mark.parametrize("n,Hq,Hkv,D,ps", [(3, 8, 2, 64, 16), (16, 8, 1, 128, 16), (2, 4, 1, 256, 64), (3, 8, 2, 128, 24)])
def test_value_scales_of_any_size(torch, n, Hq, Hkv, D, ps, e):
    """Outputs are finite in bf16, and so are the weights."""
    b, ref, tol = _scaled(torch, [120, 90, 6], n, Hq, Hkv, D, ps, e)
    _close(torch, b.run(), ref, tol)


@pytest.mark.parametrize("e", [-140, -126, -110, -90, 90, 105, 115, 121, 127])
@pytest.mark.parametrize("n,Hq,Hkv,D,ps", [(3, 8, 2, 64, 16), (16, 8, 1, 128, 16), (2, 4, 1, 256, 64), (3, 8, 2, 128, 24)])
@pytest.mark.parametrize("lens", [[9000], [1500] * 100], ids=["parts", "shares"])
def test_value_scales_of_any_size_over_parts(torch, lens, n, Hq, Hkv, D, ps, e):
    """What a part of a long sequence sums up is beyond fp32 where the outputs are
    not."""
    b, ref, tol = _scaled(torch, lens, n, Hq, Hkv, D, ps, e)
    _close(torch, b.run(), ref, tol)


# ------------------------------------------------------------------ pages

@pytest.mark.parametrize("ps", [8, 192, 320])
@pytest.mark.parametrize("kind,n,Hq,Hkv,D", SHAPES + [("bf16", 6, 8, 2, 128), ("e4m3", 16, 8, 1, 64), ("latent", 6, 4, 1, 512)])
def test_pages_of_one_core_row_and_of_several_tiles(torch, kind, n, Hq, Hkv, D, ps):
    """Pages of 8 tokens, eight boxes to a tile, and of several tiles whose number
    is no power of two."""
    b = _batch(torch, kind, [700, 64, 193, 5, 0, 383], n, Hq, Hkv, D, ps)
    _close(torch, b.run(), *b.reference())


@pytest.mark.parametrize("ps", [8, 64, 192])
@pytest.mark.parametrize("window", [20, 101, 200])
@pytest.mark.parametrize("kind,n,Hq,Hkv,D", [c for c in SHAPES if c[0] != "latent"])
def test_windows_that_begin_inside_a_page(torch, kind, n, Hq, Hkv, D, window, ps):
    """Pages before every row's window have been given away."""
    b = _batch(torch, kind, [700, 64, 193, 5, 0, 383], n, Hq, Hkv, D, ps)
    keep = b.table.clone()
    for s, (length, d) in enumerate(zip(b.lens, b.drafts)):
        b.table[s, :max(0, length - d + 1 - window) // ps] = -7
    got = b.run(window=window)
    b.table.copy_(keep)
    _close(torch, got, *b.reference(window=window))


# ------------------------------------------------------------------ scores

@pytest.mark.parametrize("scale", [-2.0, -0.3, 3.0])
@pytest.mark.parametrize("kind,n,Hq,Hkv,D", SHAPES)
def test_scales_of_either_sign(torch, kind, n, Hq, Hkv, D, scale):
    """Scores that grow along the keys, within the formula's tolerance (of the
    same scores from queries of the other sign where the scale is negative)."""
    b = _batch(torch, kind, [900, 300], n, Hq, Hkv, D, spread=0.25)
    t = torch.arange(900, device="cuda")
    page, off = b.table[0].long()[t // 16], t % 16
    if kind == "latent":
        b.data[page, off] = (b.data[page, off].float() * (0.2 + t / 900.0).view(-1, 1)).to(torch.bfloat16)
    elif kind == "bf16":
        b.k[page, :, off] = (b.k[page, :, off].float() * (0.2 + t / 900.0).view(-1, 1, 1)).to(torch.bfloat16)
    else:
        b.ks[page, :, off] *= (0.2 + t / 900.0).view(-1, 1)
    b.op.scale = scale
    got = b.run()
    b.scale = abs(scale)
    b.q = b.q if scale > 0 else -b.q
    _close(torch, got, *b.reference())


# ------------------------------------------------------------------ division

@pytest.mark.parametrize("lens", [[6000] * 3 + [130] * 150, [40] * 400, [3000, 2999, 64, 1, 700], [2] * 1000,
                                  [100 + 37 * (i * 5 % 23) for i in range(160)], [1000] * 90])
@pytest.mark.parametrize("kind,n,Hq,Hkv,D", [("bf16", 2, 8, 2, 64), ("e4m3", 2, 8, 2, 64), ("latent", 2, 8, 1, 256),
                                             ("bf16", 9, 16, 2, 128), ("e4m3", 9, 8, 1, 128)])
def test_every_sequence_of_a_division(torch, kind, n, Hq, Hkv, D, lens):
    """Wherever columns begin and end in them."""
    b = _batch(torch, kind, lens, n, Hq, Hkv, D)
    _close(torch, b.run(), *b.reference())
