"""The decoder operators where their answers are easily a little wrong: bounds
tighter than the plain parity tests', plans, rings and kernels that only some
sizes reach, values at the ends of their ranges."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest

from gpu_common import require_gpu
from test_gpu_decoder import F32, U16, _attn_tol, _check, _dec, _gen, _np, _paged, _ref_attention

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


# ------------------------------------------------------------------ attention: how the work is divided

def _division(torch, lens, Hq, Hkv, D, ps, e4m3, window, width):
    """How the tiles of these sequences are divided, by the kernel's rules:
    'short' (each segment its own parts of at most 8 tiles), 'even' (its own
    parts of an even share and a little more) or 'row' (equal shares of all)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    G = Hq // Hkv
    nh = 1 if G <= 8 else 2
    tile = 16 * (1 if (D if e4m3 else 2 * D) >= 256 else 2)
    per_sm = (2 if e4m3 else 1) if D == 256 else (3 if nh == 1 else 2)
    HG = Hkv * -(-G // (8 * nh))
    spans = []
    for n in lens:
        lo = max(0, n - window) if window else 0
        spans.append(-(-n // tile) - lo // tile if n > 0 else 0)
    most = len(lens) * HG * (-(-width * ps // tile) + 9) // 8 + len(lens) * HG
    grid = max(1, min(per_sm * sms, most))

    def parts(most):
        return HG * sum(-(-t // most) for t in spans)

    if parts(8) <= grid:
        return "short"
    share = max(8, -(-HG * sum(t + 8 for t in spans if t) // grid))
    if len(lens) * HG * 16 >= grid and parts(share + max(8, share // 6)) <= grid:
        return "even"
    return "row"


def _ragged(n, top, seed):
    """n lengths up to top, one of them 0 and one 1."""
    rng = np.random.default_rng(seed)
    return [0, 1, top] + [int(v) for v in rng.integers(1, top + 1, n - 3)]


DIVIDED = [  # lens, Hq, Hkv, D, page_size, e4m3, window, how
    (_ragged(48, 4096, 1), 32, 4, 128, 16, True, 0, "even"), (_ragged(64, 3000, 2), 16, 2, 128, 32, False, 0, "even"),
    (_ragged(40, 2500, 3), 24, 4, 64, 16, False, 0, "even"), (_ragged(33, 2000, 4), 8, 4, 256, 16, True, 0, "even"),
    (_ragged(30, 1500, 5), 4, 2, 256, 16, False, 0, "even"), (_ragged(40, 3000, 6), 24, 2, 128, 7, True, 0, "even"),
    (_ragged(64, 4000, 7), 32, 2, 128, 16, False, 900, "even"), ([2000] * 64, 8, 2, 128, 16, False, 0, "even"),
    ([2000] * 32, 8, 2, 128, 16, False, 0, "even"), ([30000] * 9, 8, 1, 128, 64, False, 0, "row"),
    (_ragged(300, 900, 8), 8, 2, 128, 16, True, 0, "row"), (_ragged(5, 40000, 9), 12, 2, 128, 16, True, 0, "row"),
    ([30000, 1, 0, 9000, 29999], 8, 2, 64, 16, False, 25000, "row"), (_ragged(20, 250, 10), 8, 2, 128, 16, False, 0, "short")]


@pytest.mark.parametrize("case", DIVIDED, ids=[f"{len(c[0])}x{max(c[0])}-{c[3]}-{c[-1]}" for c in DIVIDED])
def test_attention_divided_each_way(torch, case):
    """Ragged batches over every division of the work, each against float64 and
    repeated on a workspace of any content."""
    lens, Hq, Hkv, D, ps, e4m3, window, how = case
    g = _gen(torch, len(lens) + D)
    cache, table, kd, vd = _paged(torch, g, lens, Hkv, D, ps, e4m3)
    assert _division(torch, lens, Hq, Hkv, D, ps, e4m3, window, table.shape[1]) == how
    q = torch.randn(len(lens), Hq, D, generator=g, device="cuda").mul(1.5).to(torch.bfloat16)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    op = _dec().PagedAttention(Hq, Hkv, D, None, window)
    ws = op.workspace(len(lens))
    ws.random_(256, generator=g)
    out = op.forward(q, cache, table, sl, ws=ws)
    op.check()
    ref, A = (_np(t) for t in _ref_attention(torch, q, kd, vd, table, lens, ps, op.scale, window))
    _check(_np(out), ref, _attn_tol(ref, A, e4m3), how)
    for _ in range(3):
        assert torch.equal(op.forward(q, cache, table, sl, ws=ws), out)


@pytest.mark.parametrize("lens,Hq,Hkv,D,ps,e4m3,window", [
    ([700, 0, 45], 16, 1, 128, 16, True, 0), ([700, 0, 45], 12, 1, 256, 16, True, 0), ([700, 0, 45], 16, 1, 64, 16, False, 0),
    ([5000, 333], 16, 1, 256, 64, True, 1000), ([12000], 24, 2, 128, 5, True, 0), ([9000, 40], 32, 2, 64, 16, False, 2500),
    ([6000], 16, 1, 256, 16, False, 0), ([20000], 14, 1, 64, 16, True, 0)])
def test_attention_of_more_than_eight_heads(torch, lens, Hq, Hkv, D, ps, e4m3, window):
    """More than eight query heads on a key/value head, in every type and head
    size: short, joined from many parts, windowed."""
    g = _gen(torch, sum(lens) + Hq)
    cache, table, kd, vd = _paged(torch, g, lens, Hkv, D, ps, e4m3)
    q = torch.randn(len(lens), Hq, D, generator=g, device="cuda").mul(1.5).to(torch.bfloat16)
    op = _dec().PagedAttention(Hq, Hkv, D, None, window)
    out = op.forward(q, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    op.check()
    ref, A = (_np(t) for t in _ref_attention(torch, q, kd, vd, table, lens, ps, op.scale, window))
    _check(_np(out), ref, _attn_tol(ref, A, e4m3), "attention")


# ------------------------------------------------------------------ head norms: many steps per warp

def _steps_per_warp(torch, T, Hq, Hkv, D):
    """How many steps of 512 / D heads a warp takes, by the launch's rules."""
    warps = torch.cuda.get_device_properties(0).multi_processor_count * 6 * 4
    heads = 512 // D
    steps = -(-Hq // heads) + 2 * -(-Hkv // heads)
    chunks = min(steps, max(-(-steps // 16), warps // T))
    return -(-steps // chunks)


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter,e4m3,ps", [
    (3700, 32, 4, 128, 128, False, False, 64), (3700, 30, 5, 128, 64, True, True, 16), (3650, 17, 3, 64, 64, False, True, 64),
    (2600, 16, 2, 256, 128, True, False, 7), (4001, 32, 8, 256, 256, False, True, 32), (3800, 64, 8, 128, 32, True, False, 1)])
def test_head_norms_of_long_prompts(torch, T, Hq, Hkv, D, rot, inter, e4m3, ps):
    """Prompts so long that a warp takes more steps than its ring of loads
    holds (four), every element against float64."""
    assert _steps_per_warp(torch, T, Hq, Hkv, D) >= 5
    dec, g = _dec(), _gen(torch, T + D)
    heads = Hq + 2 * Hkv
    qkv = torch.randn(T, heads * D, generator=g, device="cuda").mul(2).to(torch.bfloat16)
    qn, kn = ((1 + 0.2 * torch.randn(D, generator=g, device="cuda")) for _ in range(2))
    cs = dec.rope_cos_sin(5000, rot, 1e4)
    pos = torch.randint(0, 5000, (T,), generator=g, device="cuda").to(torch.int32)
    pages = -(-T // ps) + 2
    cache = dec.PagedCache.empty(pages, Hkv, ps, D, e4m3)
    slots = torch.randperm(pages * ps, generator=g, device="cuda")[:T]
    slots[::97] = -1
    op = dec.QkNormRope(Hq, Hkv, D, qn, kn, cs, inter, 1e-6)
    q = op.forward(qkv, pos, slots, cache)
    op.check()

    x = qkv.double().view(T, heads, D)
    cos, sin = (c[:, None] for c in cs.double()[pos.long()].split(rot // 2, 1))

    def norm_rope(x, w):
        y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.double()
        out = y.clone()
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
        out[..., a] = y[..., a] * cos - y[..., b] * sin
        out[..., b] = y[..., b] * cos + y[..., a] * sin
        return out

    def close(got, ref, tol, what):
        bad = ~((got - ref).abs() <= tol)
        assert not bad.any(), (what, int(bad.sum()), float(((got - ref).abs() / tol).max()))

    def top(t):
        return t.abs().amax(-1, keepdim=True)

    rq = norm_rope(x[:, :Hq], qn)
    close(q.double(), rq, U16 * rq.abs() + F32 * top(rq), "queries")
    kept = slots >= 0
    at = slots[kept]
    for codes, scales, ref, what in ((cache.k, cache.k_scale, norm_rope(x[:, Hq:Hq + Hkv], kn), "keys"),
                                     (cache.v, cache.v_scale, x[:, Hq + Hkv:], "values")):
        got, ref = codes[at // ps, :, at % ps], ref[kept]
        if not e4m3:
            close(got.double(), ref, U16 * ref.abs() + F32 * top(ref), what)
            continue
        s = scales[at // ps, :, at % ps].double()[..., None]
        close(s, top(ref) / 448, F32 * top(ref) / 448, what)
        close(got.view(torch.float8_e4m3fn).double() * s, ref,
              torch.maximum(2.0 ** -4 * ref.abs(), 2.0 ** -10 * s) + F32 * top(ref), what)
    # nothing else was touched
    free = torch.ones(pages * ps, dtype=torch.bool, device="cuda")
    free[at] = False
    left = free.nonzero().flatten()
    assert (cache.k[left // ps, :, left % ps] == 0).all() and (cache.v[left // ps, :, left % ps] == 0).all()


# ------------------------------------------------------------------ captures, the functions on addresses, the example's routing

@pytest.mark.parametrize("M,N,K", [(200, 1024, 2048), (300, 2048, 1024), (1100, 2048, 512), (24, 5120, 2048), (64, 640, 512)])
def test_linear_in_a_graph(torch, M, N, K):
    """Every kernel of the linear layer captured and replayed on new inputs:
    quantisation and tcgen05 with K over a cluster or not, and the streamed one."""
    dec, g = _dec(), _gen(torch, M)
    codes = torch.randn(N, K, generator=g, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    scales = 0.005 + 0.015 * torch.rand(-(-N // 128), -(-K // 128), generator=g, device="cuda")
    lin = dec.Fp8Linear(codes, scales)
    xs = [torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3)]
    plain = [lin.forward(x) for x in xs]
    x, held, ws = xs[0].clone(), torch.empty_like(plain[0]), lin.workspace(M)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        lin.forward(x, held, ws)
    for i in (1, 2, 0, 1):
        x.copy_(xs[i])
        ws.fill_(0xA5)
        graph.replay()
        assert torch.equal(held, plain[i])
    lin.check()


FIRST_CALL = """
import sys, torch
from block_fp8_expert_gb300 import decoder
g = torch.Generator(device="cuda"); g.manual_seed(0)
M, N, K = {M}, 2048, 2048
codes = torch.randn(N, K, generator=g, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
lin = decoder.Fp8Linear(codes, torch.rand(16, 16, generator=g, device="cuda"))
x = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
out, ws = torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), lin.workspace(M)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    lin.forward(x, out, ws)
graph.replay()
torch.cuda.synchronize()
held = out.clone()
assert torch.equal(lin.forward(x), held) and torch.isfinite(held).all()
lin.check()
print("same")
"""


@pytest.mark.parametrize("M", [200, 1300])
def test_first_call_of_a_process_in_a_capture(torch, M):
    """What a first call sets up (shared-memory limits, the clusters that fit,
    the tensor maps' encoder) can be set up while a stream is captured."""
    r = subprocess.run([sys.executable, "-c", FIRST_CALL.format(M=M)], capture_output=True, text=True, timeout=280,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]


def test_functions_on_addresses_are_the_objects_calls(torch):
    """The functions of the binding that take plain addresses and structures
    give the bits of the objects, which call the library themselves."""
    from block_fp8_expert_gb300 import _lib as lib
    import block_fp8_expert_gb300 as package
    dec, g = _dec(), _gen(torch, 12)
    T, E, k, Hq, Hkv, D, ps = 5, 64, 4, 8, 2, 64, 16
    logits = torch.randn(T, E, generator=g, device="cuda")
    bias = 0.1 * torch.randn(E, generator=g, device="cuda")
    sel = dec.ExpertSelector(E, k, "sigmoid", bias, 8, 4, 2)
    idx, w = sel.forward(logits)
    i2, w2 = torch.empty_like(idx), torch.empty_like(w)
    package.moe_select_experts(logits, E, bias, sel.rule, T, E, k, i2, w2)
    assert torch.equal(idx, i2) and torch.equal(w, w2)

    qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g, device="cuda").to(torch.bfloat16)
    table = dec.rope_cos_sin(50, D)
    pos = torch.tensor([3, 0, 49, 7, 8], dtype=torch.int32, device="cuda")
    slots = torch.tensor([17, 2, 40, 0, 33], device="cuda")
    a, b = (dec.PagedCache.empty(4, Hkv, ps, D) for _ in range(2))
    rope = dec.QkNormRope(Hq, Hkv, D, cos_sin=table)
    q = rope.forward(qkv, pos, slots, a)
    q2 = torch.empty_like(q)
    d = lib.QkDims(T, Hq, D, 0, 50, 1e-6, qkv.stride(0), Hq * D)
    package.moe_qk_norm_rope(qkv, None, None, table, pos, slots, d, b.abi(), q2, rope.status)
    assert torch.equal(q, q2) and torch.equal(a.k, b.k) and torch.equal(a.v, b.v)

    pages = torch.tensor([[1, 0], [0, 2], [2, 1], [3, 3], [2, 0]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([20, 1, 32, 0, 17], dtype=torch.int32, device="cuda")
    attn = dec.PagedAttention(Hq, Hkv, D)
    o = attn.forward(q, a, pages, lens)
    o2 = torch.empty_like(o)
    d = lib.AttnDims(T, Hq, 2, 0, D ** -0.5, 2, Hq * D, Hq * D)
    ws = torch.empty(lib.paged_attention_workspace_bytes(d, D), dtype=torch.uint8, device="cuda")
    package.moe_paged_attention(q, b.abi(), pages, lens, d, o2, ws, attn.status)
    assert torch.equal(o, o2)

    codes = torch.randn(128, Hq * D, generator=g, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    scales = torch.rand(1, Hq * D // 128, generator=g, device="cuda")
    lin = dec.Fp8Linear(codes, scales)
    x = o.view(T, Hq * D)
    y = lin.forward(x)
    y2 = torch.empty_like(y)
    d = lib.LinearDims(T, 128, Hq * D, Hq * D, 128)
    ws = torch.empty(lib.linear_fp8_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    package.moe_linear_fp8(x, lib.Fp8Mat(codes.data_ptr(), scales.data_ptr()), None, d, y2, ws, lin.status)
    assert torch.equal(y, y2)
    for op in (rope, attn, lin):
        op.check()


def test_example_layers_routing(torch):
    """The example's router and selection against float64 on tokens whose choice
    hangs on no small difference, which most have to be."""
    from examples.decoder_layer import DecoderLayer
    E, k, groups, top = 16, 2, 4, 2
    L = DecoderLayer(64, 16, H=256, Hq=4, Hkv=2, D=64, I=128, E=E, k=k, groups=groups, top_groups=top, page=4, seed=7)
    h = torch.randn(64, 256, generator=_gen(torch, 2), device="cuda").to(torch.bfloat16)
    idx, w = L.select.route(h, L.moe, L.moe_ws)
    L.check()
    score = torch.sigmoid(h.double() @ L.moe.Wr.double().t())
    key = (score + L.select.bias.double()).view(64, groups, -1)
    gs = key.topk(2, -1).values.sum(-1).sort(1, descending=True)
    keep = torch.zeros(64, groups, device="cuda").scatter(1, gs.indices[:, :top], 1.0).unsqueeze(-1) > 0
    flat = key.masked_fill(~keep, -math.inf).flatten(1).sort(1, descending=True)
    clear = (gs.values[:, top - 1] - gs.values[:, top] > 1e-4) & (
        flat.values[:, :k] - flat.values[:, 1:k + 1] > 1e-4).all(1)
    assert clear.sum() > 48
    assert torch.equal(idx[clear].long(), flat.indices[clear, :k])
    s = score.gather(1, idx.long())
    ref = s / s.sum(1, keepdim=True)
    assert ((w.double() - ref).abs() <= 1e-4 * ref).all()
