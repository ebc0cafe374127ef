"""The decoder operators where their answers are easily a little wrong: bounds
tighter than the plain parity tests', plans, rings and kernels that only some
sizes reach, values at the ends of their ranges."""
import math

import numpy as np
import pytest

from gpu_common import require_gpu
from test_gpu_decoder import F32, U16, _check, _dec, _gen, _np, _paged, _ref_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return require_gpu()


# ------------------------------------------------------------------ attention: the weights' precision

@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 128), (12, 1, 64), (4, 2, 256)])
def test_attention_weights_next_to_bf16_values(torch, Hq, Hkv, D):
    """Values that cancel show the softmax weights' own rounding, which next to
    bf16 values is far below that of the output.

    With |s| < 1 (the queries are small) the scores' error is F32 + 2^-20.  The
    weights enter the second product as two parts: the larger one drops less
    than 2^-7 of them, the smaller one rounds that by 2^-9.  A warp's sums take
    at most 10 steps of two products, each within 2^-22 of sum p |v|, in four
    warps, and the joins as many again."""
    g = _gen(torch, 5 + D)
    lens, ps = [2, 7, 33, 150, 600], 16
    cache, table, kd, vd = _paged(torch, g, lens, Hkv, D, ps, False)
    sign = 1.0 - 2.0 * (torch.rand(vd.shape, generator=g, device="cuda") < 0.5)
    cache.v.mul_(sign.to(torch.bfloat16))
    vd = cache.v.double()
    q = (0.02 * torch.randn(len(lens), Hq, D, generator=g, device="cuda")).to(torch.bfloat16)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    scale = 1.0 / math.sqrt(D)
    op = _dec().PagedAttention(Hq, Hkv, D, scale)
    out = op.forward(q, cache, table, sl)
    op.check()
    ref, A = (_np(t) for t in _ref_attention(torch, q, kd, vd, table, lens, ps, scale, 0))
    e = F32 + 2.0 ** -20
    tol = 1.01 * (U16 * np.abs(ref) + (2.0 ** -16 + 2 * e + 160 * 2.0 ** -22) * (A + np.abs(ref)))
    _check(_np(out), ref, tol, "attention")


def test_attention_infinite_value(torch):
    """An infinite value of a token that is attended to gives infinity, in its
    dimension alone, whatever the weights' own bits."""
    g = _gen(torch, 6)
    lens, ps, D = [40, 300], 16, 64
    cache, table, kd, vd = _paged(torch, g, lens, 1, D, ps, False)
    cache.v[table[0, 1].item(), 0, 3, 5] = math.inf
    cache.v[table[1, 2].item(), 0, 7, 9] = -math.inf
    q = torch.randn(2, 4, D, generator=g, device="cuda").to(torch.bfloat16)
    q[:, 0] = 0                                     # equal weights, which are exact
    out = _dec().PagedAttention(4, 1, D).forward(q, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    assert (out[0, :, 5] == math.inf).all() and (out[1, :, 9] == -math.inf).all()
    out[0, :, 5] = out[1, :, 9] = 0
    assert torch.isfinite(out).all()


def test_attention_value_without_weight(torch):
    """A token whose weight is below fp32's range adds nothing, however large
    its values."""
    g = _gen(torch, 8)
    lens, ps, D = [33], 16, 64
    cache, table, _, _ = _paged(torch, g, lens, 1, D, ps, False)
    cache.k[table[0].long().clamp(min=0)] = 0
    cache.k[table[0, 1].item(), 0, 3] = -40.0       # score -320 next to zeros
    cache.v[table[0, 1].item(), 0, 3] = 3e38
    q = torch.ones(1, 4, D, dtype=torch.bfloat16, device="cuda")
    out = _dec().PagedAttention(4, 1, D).forward(q, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    t = torch.tensor([i for i in range(33) if i != 19], device="cuda")
    ref = cache.v.double()[table[0].long()[t // ps], 0, t % ps].mean(0)
    A = cache.v.double()[table[0].long()[t // ps], 0, t % ps].abs().mean(0)
    tol = U16 * ref.abs() + 2.0 ** -15 * A          # equal weights: exact; a few sums in fp32
    assert ((out.double() - ref).abs() <= tol).all()


# ------------------------------------------------------------------ selection

@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("groups,top_groups", [(1, 1), (8, 2)])
@pytest.mark.parametrize("renorm", [True, False])
def test_softmax_of_a_row_with_a_nan(torch, value, groups, top_groups, renorm):
    """One NaN (or infinite) logit makes every softmax score of the row NaN, so
    the weights are, whichever experts are chosen; other rows are as ever."""
    E, k = 64, 4
    l = torch.randn(3, E, generator=_gen(torch, 3), device="cuda")
    clean = l.clone()
    l[1, 40] = value
    op = _dec().ExpertSelector(E, k, "softmax", None, groups, top_groups, 1, renorm)
    idx, w = op.forward(l)
    assert torch.isnan(w[1]).all()
    assert idx.min() >= 0 and idx.max() < E and len(set(idx[1].tolist())) == k
    i2, w2 = op.forward(clean)
    for t in (0, 2):
        assert torch.equal(idx[t], i2[t]) and torch.equal(w[t], w2[t])


@pytest.mark.parametrize("groups,top_groups", [(1, 1), (4, 2)])
def test_sigmoid_scores_near_the_end_of_fp32(torch, groups, top_groups):
    """Logits about -88, whose scores are subnormal (4e-39 to 1e-38): they order
    the experts and make the weights.  exp is within 2^-21 of its argument's
    rounding (88 x 2^-24), the reciprocal within 2^-23, a subnormal score of
    4e-39 is rounded by 2^-22, twice."""
    E, k = 64, 6
    rng = np.random.default_rng(2)
    l = np.stack([rng.permutation(np.linspace(-88.4, -87.0, E)) for _ in range(5)]).astype(np.float32)
    s = 1 / (1 + np.exp(-l.astype(np.float64)))
    n = E // groups
    for renorm in (False, True):
        op = _dec().ExpertSelector(E, k, "sigmoid", None, groups, top_groups, 1, renorm)
        idx, w = op.forward(torch.from_numpy(l).cuda())
        for t in range(5):
            best = sorted(range(groups), key=lambda g: -s[t, g * n:(g + 1) * n].max())[:top_groups]
            cand = sorted((e for e in range(E) if e // n in best), key=lambda e: -s[t, e])[:k]
            assert idx[t].tolist() == cand
            ref = s[t, cand] / (s[t, cand].sum() if renorm else 1)
            _check(_np(w[t]), ref, 2.0 ** -17 * ref, "weights")
    idx, w = _dec().ExpertSelector(E, k, "sigmoid", renorm=False).forward(torch.full((1, E), -200.0, device="cuda"))
    assert (w == 0).all() and idx[0].tolist() == list(range(k))
    idx, w = _dec().ExpertSelector(E, k, "sigmoid", renorm=False).forward(torch.full((1, E), 200.0, device="cuda"))
    assert (w == 1).all()
