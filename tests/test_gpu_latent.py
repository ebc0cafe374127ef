"""The latent store and the expanded attention against their formulas in
float64, and a prompt with decoding through both forms of latent attention.

Tolerances as in test_gpu_draft_attention.py: U16 = 2^-8 for one rounding to
bf16, F32 = 64 x 2^-24 of the largest terms for fp32 work before it.
"""
import math

import pytest

from gpu_common import require_gpu

pytestmark = pytest.mark.gpu

U16 = 2.0 ** -8
F32 = 64 * 2.0 ** -24


@pytest.fixture(scope="module")
def torch():
    return require_gpu()


def _dec():
    from block_fp8_expert_gb300 import decoder
    return decoder


def _gen(torch, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _bf16(torch, g, *shape, spread=1.0):
    return (spread * torch.randn(*shape, generator=g, device="cuda")).to(torch.bfloat16)


def _close(got, ref, tol):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst err/tol {(err / tol.clamp(min=1e-30)).max().item():.3g}"


# ------------------------------------------------------------------ store

def _rotated(torch, x, cs, inter):
    """x float64 [..., 64], cs [..., 64]: cosines, then sines."""
    c, s = cs[..., :32], cs[..., 32:]
    a, b = (x[..., 0::2], x[..., 1::2]) if inter else (x[..., :32], x[..., 32:])
    ra, rb = a * c - b * s, b * c + a * s
    size = a.abs() + b.abs()
    if inter:
        return torch.stack([ra, rb], -1).flatten(-2), torch.stack([size, size], -1).flatten(-2)
    return torch.cat([ra, rb], -1), torch.cat([size, size], -1)


def _normed(torch, x, norm, eps=1e-6):
    if norm is None:
        return x
    return x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * norm.double()


STORE = [  # T, H, R, interleaved, page size, norm, rows
    (1, 1, 512, False, 16, True, False), (1, 128, 256, True, 64, True, True), (5, 32, 512, True, 64, True, True),
    (37, 20, 256, False, 1, True, True), (300, 7, 512, False, 24, False, True), (1000, 64, 512, True, 16, True, False),
    (3000, 8, 256, True, 64, True, True), (63, 0, 512, False, 16, True, True)]


@pytest.mark.parametrize("case", STORE, ids=str)
def test_store(torch, case):
    T, H, R, inter, ps, normed, want_rows = case
    dec, g = _dec(), _gen(torch, T)
    pages = -(-T // ps) + 2
    norm = 1 + 0.1 * torch.randn(R, generator=g, device="cuda") if normed else None
    table = dec.rope_cos_sin(500, 64, 1e4)
    cache = dec.LatentCache.empty(pages, ps, R)
    op = dec.LatentStore(H, R, table, norm, interleaved=inter)
    kv = _bf16(torch, g, T, R + 72, spread=2.0)[:, :R + 64]   # strided rows
    pos = torch.randint(0, 500, (T,), generator=g, device="cuda").to(torch.int32)
    slots = torch.randperm(pages * ps, generator=g, device="cuda")[:T]
    if T > 4:
        slots[3] = -1
    q = _bf16(torch, g, T, H, 192)[..., 128:] if H else None
    rows = torch.full((T, R + 64), 5.0, dtype=torch.bfloat16, device="cuda") if want_rows else None
    wide = torch.full((T, H, 192), 5.0, dtype=torch.bfloat16, device="cuda")
    got = op.forward(kv, pos, slots, cache, q=q, q_out=wide[..., 128:] if H else None, rows=rows)
    op.check()
    cs = table.double()[pos.long()]
    lat = _normed(torch, kv[:, :R].double(), norm)
    key, size = _rotated(torch, kv[:, R:].double(), cs, inter)
    ref = torch.cat([lat, key], 1)
    tol = U16 * ref.abs() + F32 * torch.cat([lat.abs(), size], 1) + 1e-30
    flat = cache.data.view(-1, R + 64)
    keep = slots >= 0
    _close(flat[slots[keep]], ref[keep], tol[keep])
    rest = torch.ones(pages * ps, dtype=torch.bool, device="cuda")
    rest[slots[keep]] = False
    assert (flat[rest] == 0).all()
    if want_rows:
        _close(rows, ref, tol)
        assert torch.equal(rows[keep], flat[slots[keep]])
    if H:
        qr, size = _rotated(torch, q.double(), cs.unsqueeze(1), inter)
        _close(got, qr, U16 * qr.abs() + F32 * size + 1e-30)
        assert (wide[..., :128] == 5.0).all()
        # in place, and into a new tensor
        new = op.forward(kv, pos, slots, cache, q=q)
        assert torch.equal(new, got)
        op.forward(kv, pos, slots, cache, q=q, q_out=q)
        assert torch.equal(q, got)
    else:
        assert got is None


def test_store_bad_positions_and_slots(torch):
    from block_fp8_expert_gb300 import MoeError
    dec, g = _dec(), _gen(torch, 1)
    cache = dec.LatentCache.empty(2, 16, 256)
    op = dec.LatentStore(3, 256, dec.rope_cos_sin(50, 64))
    kv, q = _bf16(torch, g, 6, 320), _bf16(torch, g, 6, 3, 64)
    rows = torch.zeros(6, 320, dtype=torch.bfloat16, device="cuda")
    pos = torch.tensor([0, 50, -1, 3, 4, 5], dtype=torch.int32, device="cuda")
    slots = torch.tensor([0, 1, 2, 32, 2 ** 40, -9], dtype=torch.int64, device="cuda")
    out = op.forward(kv, pos, slots, cache, q=q, rows=rows)
    with pytest.raises(MoeError, match="0x30"):
        op.check()
    assert torch.isnan(out[1:3]).all() and torch.isnan(rows[1:3]).all()
    assert torch.isfinite(out[[0, 3, 4, 5]]).all() and torch.isfinite(rows[[0, 3, 4, 5]]).all()
    flat = cache.data.view(-1, 320)
    assert torch.equal(flat[0], rows[0]) and (flat[1:] == 0).all()


# ------------------------------------------------------------------ expanded attention

def _expanded(torch, lens, ctx, H, seed=0, spread=1.0):
    g = _gen(torch, seed)
    Tq, Tk = sum(lens), sum(lens) + sum(ctx)
    q = _bf16(torch, g, Tq, H, 192, spread=spread)
    kv = _bf16(torch, g, Tk, H, 256)
    rope = _bf16(torch, g, Tk, 64)
    cu = lambda n: torch.tensor([0] + n, device="cuda").cumsum(0).to(torch.int32)  # noqa: E731
    return q, kv, rope, cu(lens), cu([a + b for a, b in zip(lens, ctx)])


def _expanded_ref(torch, q, kv, rope, cu_q, cu_k, scale):
    out = torch.zeros(*q.shape[:2], 128, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    cu_q, cu_k = cu_q.tolist(), cu_k.tolist()
    for b in range(len(cu_q) - 1):
        lq, lk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        for h in range(q.shape[1]):
            k = torch.cat([kv[cu_k[b]:cu_k[b + 1], h, :128], rope[cu_k[b]:cu_k[b + 1]]], 1).double()
            v = kv[cu_k[b]:cu_k[b + 1], h, 128:].double()
            x = q[cu_q[b]:cu_q[b + 1], h].double()
            i, t = torch.arange(lq, device="cuda"), torch.arange(lk, device="cuda")
            live = i + (lk - lq) >= 0
            if not live.any():
                continue
            hidden = t > (i + (lk - lq))[:, None]
            s = (x @ k.t() * scale).masked_fill(hidden, -math.inf)[live]
            p = torch.softmax(s, -1)
            o, A = p @ v, p @ v.abs()
            e = scale * (x[live].abs() @ k.abs().t()).amax(-1, keepdim=True) * 192 * 2.0 ** -23 + 2.0 ** -20
            rows = torch.arange(cu_q[b], cu_q[b + 1], device="cuda")[live]
            out[rows, h] = o
            tol[rows, h] = (U16 * o.abs() + U16 * (A + o.abs()) + (2 * e + lk * 2.0 ** -23) * A) * 1.01 + 1e-30
    return out, tol


EXPANDED = [  # lens, context lengths, heads
    ([1], [0], 1), ([1], [300], 5), ([2, 1, 3], [0, 0, 0], 20), ([127], [0], 3), ([128], [0], 3), ([129], [0], 3),
    ([255], [1], 2), ([256], [128], 2), ([257], [127], 2), ([600, 1, 300], [0, 700, 5], 4), ([9, 4, 1], [700, 130, 129], 7),
    ([0, 40, 0, 7], [0, 3, 9, 0], 5), ([1500], [0], 2), ([10, 20], [-4, -20], 3), ([300], [-200], 2), ([400], [-399], 2)]


@pytest.mark.parametrize("case", EXPANDED, ids=str)
def test_expanded(torch, case):
    """Rows of every kind: first and last of tiles, with and without a context,
    sequences without tokens, and (negative contexts) rows that see no key."""
    lens, ctx, H = case
    q, kv, rope, cu_q, cu_k = _expanded(torch, lens, ctx, H)
    op = _dec().ExpandedAttention(H)
    out = torch.full((sum(lens), H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    got = op.forward(q, kv[..., :128], rope, kv[..., 128:], cu_q, cu_k, out=out)
    op.check()
    _close(got, *_expanded_ref(torch, q, kv, rope, cu_q, cu_k, op.scale))


def test_expanded_layouts(torch):
    """Heads before tokens, odd strides, outputs in a wider tensor, keys of the
    next sequences and past the last: none of it shows."""
    lens, ctx, H = [70, 200], [10, 0], 3
    q, kv, rope, cu_q, cu_k = _expanded(torch, lens, ctx, H)
    op = _dec().ExpandedAttention(H)
    base = op.forward(q, kv[..., :128], rope, kv[..., 128:], cu_q, cu_k)
    q2 = torch.zeros(H, 275, 192, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    k2 = torch.full((300, H, 136), math.nan, dtype=torch.bfloat16, device="cuda")[..., :128]
    v2 = torch.full((H, 300, 128), math.inf, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    r2 = torch.full((300, 576), math.nan, dtype=torch.bfloat16, device="cuda")[:, 512:]
    q2[:270], k2[:280], v2[:280], r2[:280] = q, kv[..., :128], kv[..., 128:], rope
    big = torch.full((275, H + 1, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    op.forward(q2, k2, r2, v2, cu_q, cu_k, out=big[:, :H])
    op.check()
    assert torch.equal(big[:270, :H], base)
    assert (big[270:] == 3.0).all() and (big[:, H] == 3.0).all()  # rows of no sequence stay


def test_expanded_what_is_not_seen_may_be_anything(torch):
    """NaN and infinities in a later token's key and value, and in another
    sequence's: rows that do not see them keep their outputs, those that see an
    infinite value hold it."""
    q, kv, rope, cu_q, cu_k = _expanded(torch, [200, 100], [0, 20], 2)
    op = _dec().ExpandedAttention(2)
    ref, tol = _expanded_ref(torch, q, kv, rope, cu_q, cu_k, op.scale)
    kv[150, 0, :128] = math.nan
    kv[150, 0, 130], kv[150, 0, 131] = math.inf, math.nan
    kv[140, 1, 128 + 70] = -math.inf
    kv[201, 1, 128 + 9] = math.inf       # the other sequence's context
    got = op.forward(q, kv[..., :128], rope, kv[..., 128:], cu_q, cu_k)
    op.check()
    _close(got[:150, 0], ref[:150, 0], tol[:150, 0])
    assert torch.isnan(got[150:200, 0]).all()
    _close(got[:140, 1], ref[:140, 1], tol[:140, 1])
    assert (got[140:200, 1, 70] == -math.inf).all()
    keep = torch.arange(128, device="cuda") != 70
    _close(got[140:200, 1][:, keep], ref[140:200, 1][:, keep], tol[140:200, 1][:, keep])
    _close(got[200:, 0], ref[200:, 0], tol[200:, 0])
    assert (got[200:, 1, 9] == math.inf).all()


def test_expanded_bad_offsets(torch):
    from block_fp8_expert_gb300 import MoeError
    q, kv, rope, cu_q, cu_k = _expanded(torch, [50, 60], [0, 0], 2)
    op = _dec().ExpandedAttention(2)
    ref, tol = _expanded_ref(torch, q, kv, rope, cu_q, cu_k, op.scale)
    for t, i, v in ((cu_q, 2, 200), (cu_k, 2, 2 ** 31 - 1), (cu_q, 0, -3), (cu_k, 0, -2 ** 31), (cu_q, 1, -1), (cu_k, 1, 500)):
        keep = t.clone()
        t[i] = v
        op.forward(q, kv[..., :128], rope, kv[..., 128:], cu_q, cu_k)
        with pytest.raises(MoeError, match="0x20"):
            op.check()
        t.copy_(keep)
        op.status.zero_()
    _close(op.forward(q, kv[..., :128], rope, kv[..., 128:], cu_q, cu_k), ref, tol)
    op.check()


@pytest.mark.parametrize("B,H", [(1, 33), (3, 70), (31, 3), (32, 3), (33, 3), (70, 3), (128, 2), (129, 2), (300, 1)])
def test_expanded_many_sequences(torch, B, H):
    """Every block of every sequence and head is found, and the last sequence's offsets are
    checked as the first one's."""
    from block_fp8_expert_gb300 import MoeError
    lens = [(b * 7 % 5) * (b * 37 % 211) for b in range(B)]
    lens[B // 2] = 700
    q, kv, rope, cu_q, cu_k = _expanded(torch, lens, [b % 3 for b in range(B)], H)
    op = _dec().ExpandedAttention(H)
    ref, tol = _expanded_ref(torch, q, kv, rope, cu_q, cu_k, op.scale)
    _close(op.forward(q, kv[..., :128], rope, kv[..., 128:], cu_q, cu_k), ref, tol)
    op.check()
    cu_k[B] += 1
    op.forward(q, kv[..., :128], rope, kv[..., 128:], cu_q, cu_k)
    with pytest.raises(MoeError, match="0x20"):
        op.check()


def test_expanded_large_scores(torch):
    """Scores whose maximum moves along the keys, and a graph's replay."""
    q, kv, rope, cu_q, cu_k = _expanded(torch, [500], [100], 2, spread=4.0)
    kv[..., :128] *= (1 + torch.arange(600, device="cuda") / 200).view(-1, 1, 1).to(torch.bfloat16)
    op = _dec().ExpandedAttention(2, scale=0.5)
    ref, tol = _expanded_ref(torch, q, kv, rope, cu_q, cu_k, 0.5)
    got = op.forward(q, kv[..., :128], rope, kv[..., 128:], cu_q, cu_k)
    _close(got, ref, tol)
    out, graph = torch.empty_like(got), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.forward(q, kv[..., :128], rope, kv[..., 128:], cu_q, cu_k, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, got)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = op.forward(q, kv[..., :128], rope, kv[..., 128:], cu_q, cu_k, stream=side)
    side.synchronize()
    assert torch.equal(other, got)


def test_expanded_without_tokens(torch):
    dec = _dec()
    op = dec.ExpandedAttention(3)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    none = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert op.forward(torch.zeros(0, 3, 192, **bf), torch.zeros(0, 3, 128, **bf), torch.zeros(0, 64, **bf),
                      torch.zeros(0, 3, 128, **bf), none, none).shape == (0, 3, 128)
    five = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    out = op.forward(torch.ones(5, 3, 192, **bf), torch.zeros(0, 3, 128, **bf), torch.zeros(0, 64, **bf),
                     torch.zeros(0, 3, 128, **bf), five, none)
    op.check()
    assert (out == 0).all()


# ------------------------------------------------------------------ together

def test_prompt_and_drafted_tokens_of_a_layer(torch):
    """A latent attention layer as a server runs it: a prompt through the store
    and the expanded form, then drafted tokens through the store and the absorbed
    form over what both have stored.  The absorbed rows are those that the
    expanded form gives for the same tokens."""
    dec, g = _dec(), _gen(torch, 11)
    H, R, ps, n_prompt, n_draft = 20, 512, 16, 75, 4
    T = n_prompt + n_draft
    scale = 1 / math.sqrt(192)
    c = _bf16(torch, g, T, R + 64)                       # what the down-projection gives
    q = _bf16(torch, g, T, H, 192)
    w_k = torch.randn(H, 128, R, generator=g, device="cuda") / math.sqrt(R)
    w_v = torch.randn(H, 128, R, generator=g, device="cuda") / math.sqrt(R)
    w_k, w_v = w_k.to(torch.bfloat16), w_v.to(torch.bfloat16)
    norm = 1 + 0.1 * torch.randn(R, generator=g, device="cuda")
    store = dec.LatentStore(H, R, dec.rope_cos_sin(200, 64), norm, interleaved=True)
    cache = dec.LatentCache.empty(9, ps, R)
    table = torch.randperm(9, generator=g, device="cuda").to(torch.int32)[None, :7].contiguous()
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    slots = table[0].long()[pos.long() // ps] * ps + pos.long() % ps
    rows = torch.empty(T, R + 64, dtype=torch.bfloat16, device="cuda")
    first, last = slice(0, n_prompt), slice(n_prompt, T)
    for part in (first, last):
        store.forward(c[part], pos[part].contiguous(), slots[part].contiguous(), cache, q=q[part][..., 128:],
                      q_out=q[part][..., 128:], rows=rows[part])
    store.check()
    # expanded, prompt and drafted tokens as one sequence (a chain)
    kv = torch.empty(T, H, 256, dtype=torch.bfloat16, device="cuda")
    kv[..., :128] = torch.einsum("tr,hdr->thd", rows[:, :R].float(), w_k.float())
    kv[..., 128:] = torch.einsum("tr,hdr->thd", rows[:, :R].float(), w_v.float())
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    exp = dec.ExpandedAttention(H, scale)
    full = exp.forward(q, kv[..., :128], rows[:, R:], kv[..., 128:], cu, cu)
    exp.check()
    # a chunk on its own, with the prompt's keys as context
    part = exp.forward(q[last], kv[..., :128], rows[:, R:], kv[..., 128:],
                       torch.tensor([0, n_draft], dtype=torch.int32, device="cuda"), cu)
    ref, tol = _expanded_ref(torch, q, kv, rows[:, R:], cu, cu, scale)
    _close(full, ref, tol)
    _close(part, ref[last], tol[last])
    # absorbed
    qa = torch.empty(1, n_draft, H, R + 64, dtype=torch.bfloat16, device="cuda")
    qa[0, ..., :R] = torch.einsum("thd,hdr->thr", q[last][..., :128].float(), w_k.float())
    qa[0, ..., R:] = q[last][..., 128:]
    att = dec.LatentAttention(H, R, scale)
    got = att.forward(qa, cache, table, torch.tensor([T], dtype=torch.int32, device="cuda"))
    att.check()
    x, t = qa[0].double(), rows.double()
    s = torch.einsum("ihr,tr->iht", x, t) * scale
    s = s.masked_fill(torch.arange(T, device="cuda") > (n_prompt + torch.arange(n_draft, device="cuda"))[:, None, None],
                      -math.inf)
    p = torch.softmax(s, -1)
    o, A = p @ t[:, :R], p @ t[:, :R].abs()
    e = scale * (x.abs() @ t.abs().t()).amax(-1, keepdim=True) * 576 * 2.0 ** -23 + 2.0 ** -20
    _close(got[0], o, (U16 * o.abs() + U16 * (A + o.abs()) + 2 * e * A) * 1.01)
    # and through the value projections it is the expanded form, up to the
    # roundings of keys, values and queries on either way (U16 each of terms
    # whose size the products' magnitudes bound)
    out = torch.einsum("ihr,hdr->ihd", got[0].double(), w_v.double())
    size = torch.einsum("iht,thd->ihd", p, torch.einsum("tr,hdr->thd", t[:, :R].abs(), w_v.double().abs()))
    ds = 2 * U16 * scale * torch.einsum("ihd,thd->iht", q[last].double().abs()[..., :128],
                                        torch.einsum("tr,hdr->thd", t[:, :R].abs(), w_k.double().abs())).amax(-1, keepdim=True)
    _close(out, ref[last], (4 * U16 + 2 * ds) * size)
