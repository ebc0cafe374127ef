"""Attention of drafted tokens over a paged cache (TreeAttention, and
LatentAttention over latent vectors) against their formula in float64.

Tolerances count the roundings: U16 = 2^-8 is the largest relative error of one
rounding to bf16.  The softmax weights p, rounded by at most u (two bf16 parts:
2^-15; one fp16 part, next to E4M3 values: 2^-11; one bf16 part, summed as
rounded, next to latent vectors: U16), move a normalised output by at most u (A +
|out|), A = sum p |v| / sum p.  A score's fp32 error e (a sum of `size` products
that may truncate each addition, 2^-23 of the sum of magnitudes each, and 2^-20
for the exponent's own) moves it by 2 e A, the sum over t tokens by t 2^-23 A.
An fp16 weight below 2^-14 is rounded by 2^-25: they are held times 2^9 of the
row's largest weight (which is at least 1 there, and their sum with it), over the
largest scale's exponent, so t of them move an output by t 2^-34 of the largest
scale times the largest code.
"""
import math

import pytest

from gpu_common import require_gpu

pytestmark = pytest.mark.gpu

U16 = 2.0 ** -8


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


def _signed(m):
    return m - (1 << 64) if m >> 63 else m


def _trees(rng, B, n):
    """Ancestors and self of each token of a random tree, as int64 bits."""
    rows = []
    for _ in range(B):
        seen = []
        for i in range(n):
            up = rng.randint(-1, i - 1) if i else -1
            seen.append((seen[up] if up >= 0 else 0) | 1 << i)
        rows.append([_signed(s) for s in seen])
    return rows


class Batch:
    """A batch over a paged cache in float64 and as the operators take it."""

    def __init__(self, torch, lens, drafts, n, Hq, Hkv, Dk, Dv, ps, kind, seed=0, spread=1.0):
        import random
        self.torch, self.kind, self.ps = torch, kind, ps
        self.lens, self.drafts, self.n, self.Hq, self.Hkv, self.Dk, self.Dv = lens, drafts, n, Hq, Hkv, Dk, Dv
        B = len(lens)
        g = _gen(torch, seed)
        need = [-(-x // ps) for x in lens]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        width = max(1, max(need))
        self.table = torch.zeros(B, width, dtype=torch.int32, device="cuda")
        at = 0
        for b in range(B):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
        self.q = (spread * torch.randn(B, n, Hq, Dk, generator=g, device="cuda")).to(torch.bfloat16)
        self.mask = torch.tensor(_trees(random.Random(seed), B, n), dtype=torch.int64, device="cuda")
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.draft_lens = torch.tensor(drafts, dtype=torch.int32, device="cuda")
        dec = _dec()
        if kind == "latent":
            self.data = torch.randn(pages, ps, Dk, generator=g, device="cuda").to(torch.bfloat16)
            self.cache = dec.LatentCache(self.data, R=Dv)
            self.scale = 0.07
            self.op = dec.LatentAttention(H=Hq, R=Dv, scale=self.scale)
            return
        shape = (pages, Hkv, ps, Dk)
        self.k, self.v = (torch.randn(shape, generator=g, device="cuda") for _ in range(2))
        self.scale = 1 / math.sqrt(Dk)
        if kind == "e4m3":
            self.ks, self.vs = (0.5 + torch.rand(shape[:3], generator=g, device="cuda") for _ in range(2))
            self.k, self.v = (x.to(torch.float8_e4m3fn) for x in (self.k, self.v))
            self.cache = dec.PagedCache(self.k, self.v, self.ks, self.vs)
        else:
            self.k, self.v = self.k.to(torch.bfloat16), self.v.to(torch.bfloat16)
            self.cache = dec.PagedCache(self.k, self.v)
        self.op = dec.TreeAttention(Hq, Hkv, Dk)

    def tokens(self, b, h):
        """Keys and values of sequence b, head h, in float64."""
        t = self.torch.arange(self.lens[b], device="cuda")
        page, off = self.table[b].long()[t // self.ps], t % self.ps
        if self.kind == "latent":
            k = self.data[page, off].double()
            return k, k[:, :self.Dv]
        k, v = self.k[page, h, off].double(), self.v[page, h, off].double()
        if self.kind == "e4m3":
            k = k * self.ks[page, h, off].double().unsqueeze(1)
            v = v * self.vs[page, h, off].double().unsqueeze(1)
        return k, v

    def seen(self, b, i, mask="own", window=0):
        """Tokens that row i of sequence b sees, as a list."""
        d = self.drafts[b]
        if i >= d:
            return []
        ctx = self.lens[b] - d
        bits = (2 << i) - 1 if mask is None else int(self.mask[b, i])
        mine = [j for j in range(d) if bits >> j & 1]
        low = max(0, ctx + max(1, len(mine)) - window) if window else 0
        return list(range(low, ctx)) + [ctx + j for j in mine]

    def reference(self, mask="own", window=0):
        """Outputs and tolerances in float64 (values that no weight reaches are
        left out of the sums, so that they may be anything)."""
        torch = self.torch
        B, G = len(self.lens), self.Hq // self.Hkv
        out = torch.zeros(B, self.n, self.Hq, self.Dv, dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(out)
        u = {"latent": U16, "e4m3": 2.0 ** -11, "bf16": 2.0 ** -15}[self.kind]
        for b in range(B):
            if not self.lens[b]:
                continue
            for h in range(self.Hkv):
                k, v = self.tokens(b, h)
                for i in range(self.n):
                    t = self.seen(b, i, mask, window)
                    if not t:
                        continue
                    t = torch.tensor(t, device="cuda")
                    q = self.q[b, i, h * G:(h + 1) * G].double()
                    p = torch.softmax(q @ k[t].t() * self.scale, -1)
                    o = p @ v[t]
                    A = p @ v[t].abs()
                    e = self.scale * (q.abs() @ k[t].abs().t()).amax(-1, keepdim=True) * self.Dk * 2.0 ** -23 + 2.0 ** -20
                    out[b, i, h * G:(h + 1) * G] = o
                    tol[b, i, h * G:(h + 1) * G] = (U16 * o.abs() + u * (A + o.abs())
                                                   + (2 * e + len(t) * 2.0 ** -23) * A) * 1.01 + 1e-30
                    if self.kind == "e4m3":
                        page, off = self.table[b].long()[t // self.ps], t % self.ps
                        top = self.vs[page, h, off].double().max() * self.v[page, h, off].double().abs().max()
                        tol[b, i, h * G:(h + 1) * G] += len(t) * 2.0 ** -34 * top
        return out, tol

    def run(self, mask="own", window=0, **kw):
        if self.kind != "latent":
            self.op.window = window
        m = self.mask if isinstance(mask, str) else mask
        out = self.op.forward(self.q, self.cache, self.table, self.seq_lens, m, self.draft_lens, **kw)
        self.op.check()
        return out


def _close(torch, got, ref, tol):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst err/tol {(err / tol.clamp(min=1e-30)).max().item():.3g}"


# lens, drafts, n, Hq, Hkv, D, page size, kind
TREES = [
    ([5], [5], 5, 4, 4, 64, 16, "bf16"), ([1], [1], 1, 1, 1, 128, 16, "bf16"),
    ([64, 65, 63, 128], [1, 1, 1, 1], 1, 8, 2, 64, 64, "bf16"),
    ([300, 0, 7, 40], [7, 0, 7, 3], 7, 8, 1, 128, 32, "bf16"),
    ([1000, 129, 700], [8, 8, 2], 8, 20, 4, 128, 64, "bf16"),
    ([200, 77], [64, 64], 64, 4, 2, 128, 16, "bf16"), ([130, 66], [64, 2], 64, 5, 1, 256, 16, "bf16"),
    ([2500, 64, 63, 1], [33, 33, 5, 1], 33, 16, 2, 64, 128, "bf16"),
    ([400, 300], [6, 6], 6, 6, 6, 256, 32, "bf16"),
    ([90, 257], [4, 4], 4, 8, 2, 128, 24, "bf16"), ([70, 130], [9, 3], 9, 4, 1, 64, 1, "bf16"),
    ([150], [5], 5, 6, 2, 256, 5, "bf16"),
    ([300, 0, 17], [7, 0, 7], 7, 8, 1, 128, 32, "e4m3"), ([1300, 129], [16, 9], 16, 16, 2, 128, 16, "e4m3"),
    ([640, 33], [3, 3], 3, 8, 4, 64, 64, "e4m3"), ([257, 64], [12, 12], 12, 4, 1, 256, 16, "e4m3"),
    ([100, 41], [5, 5], 5, 8, 2, 128, 24, "e4m3"), ([77], [2], 2, 4, 4, 64, 7, "e4m3"), ([200], [4], 4, 4, 2, 256, 1, "e4m3"),
]
LATENT = [
    ([3], [3], 3, 8, 256, 16), ([1, 64, 65], [1, 1, 1], 1, 20, 512, 16), ([777], [1], 1, 32, 512, 64),
    ([900, 0, 5, 130], [5, 0, 5, 2], 5, 20, 512, 32), ([300, 200], [2, 2], 2, 128, 512, 64),
    ([129, 400], [7, 3], 7, 5, 256, 16), ([1500], [1], 1, 128, 256, 128), ([70, 500], [64, 10], 64, 2, 256, 64),
    ([90, 33], [4, 4], 4, 8, 512, 24), ([130], [1], 1, 64, 256, 1),
]
EACH = [(c[0], c[1], c[2], c[3], c[4], c[5], c[5], c[6], c[7]) for c in TREES] + \
       [(c[0], c[1], c[2], c[3], 1, c[4] + 64, c[4], c[5], "latent") for c in LATENT]


def _id(c):
    return f"{c[8]}-{max(c[0])}-n{c[2]}-{c[3]}x{c[4]}x{c[5]}-p{c[7]}"


@pytest.mark.parametrize("case", EACH, ids=_id)
def test_trees(torch, case):
    b = Batch(torch, *case)
    _close(torch, b.run(), *b.reference())


@pytest.mark.parametrize("case", [EACH[3], EACH[9], EACH[12], EACH[22], EACH[27]], ids=_id)
def test_chain(torch, case):
    """Without a mask each new token sees those up to itself."""
    b = Batch(torch, *case)
    _close(torch, b.run(mask=None), *b.reference(mask=None))


@pytest.mark.parametrize("window", [8, 64, 100, 5000])
@pytest.mark.parametrize("case", [EACH[4], EACH[3], EACH[9], EACH[12]], ids=_id)
def test_window(torch, case, window):
    b = Batch(torch, *case)
    # pages that lie behind every row's window may have been given away
    for s, (n, d) in enumerate(zip(b.lens, b.drafts)):
        gone = max(0, n - d + 1 - window) // b.ps
        b.table[s, :gone] = -7
    if b.n > window:
        with pytest.raises(Exception, match="window"):
            b.run(window=window)
        return
    keep = b.table.clone()
    got = b.run(window=window)
    b.table.copy_(keep.clamp(min=0))
    _close(torch, got, *b.reference(window=window))


def test_one_new_token_is_paged_attention(torch):
    """Both operators within their tolerances of the same formula."""
    b = Batch(torch, [500, 0, 33], [1, 0, 1], 1, 8, 2, 128, 128, 16, "bf16")
    ref, tol = b.reference()
    _close(torch, b.run(), ref, tol)
    one = _dec().PagedAttention(8, 2, 128).forward(b.q[:, 0], b.cache, b.table, b.seq_lens)
    _close(torch, one.unsqueeze(1), ref, tol)


@pytest.mark.parametrize("lens", [[6000] * 3 + [130] * 150, [40] * 400, [9000], [3000, 2999, 64, 1, 700], [2] * 1000])
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "latent"])
def test_division(torch, lens, kind):
    """Single parts, shares with several segments, many sequences per thread: the
    rows of a few sequences, against the formula."""
    n = 2
    Dk, Dv, Hq, Hkv = (320, 256, 8, 1) if kind == "latent" else (64, 64, 8, 2)
    b = Batch(torch, lens, [min(n, x) for x in lens], n, Hq, Hkv, Dk, Dv, 16, kind)
    got = b.run()
    pick = sorted({0, len(lens) // 2, len(lens) - 1})
    b.lens, b.drafts = [lens[i] for i in pick], [min(n, lens[i]) for i in pick]
    b.table, b.q, b.mask = b.table[pick], b.q[pick], b.mask[pick]
    _close(torch, got[pick], *b.reference())


@pytest.mark.parametrize("n,Hq,Hkv,D,tiles", [(1, 3, 3, 256, 101), (1, 5, 5, 256, 301), (2, 5, 5, 64, 121),
                                              (1, 7, 7, 128, 131), (32, 64, 8, 128, 19), (2, 11, 11, 256, 29)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_one_sequence_whose_heads_do_not_divide_the_columns(torch, n, Hq, Hkv, D, tiles, kind):
    """All of its parts have a column: the last head's last tokens are there, and
    a call of other lengths before it leaves nothing behind."""
    for t in (tiles, tiles + 1, tiles - 2):
        b = Batch(torch, [64 * t - 3], [n], n, Hq, Hkv, D, D, 64, kind, seed=t)
        ws = b.op.workspace(1, n)
        ws.fill_(0x7f)
        _close(torch, b.run(ws=ws), *b.reference())


@pytest.mark.parametrize("Hq,Hkv,D,lens", [(1024, 8, 64, [200]), (128, 1, 128, [700, 64, 0, 90]), (256, 2, 256, [130])])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_as_many_rows_as_there_may_be(torch, Hq, Hkv, D, lens, kind):
    """64 new tokens of 128 heads per key/value head: more row tiles than there
    are columns for every head."""
    b = Batch(torch, lens, [min(64, x) for x in lens], 64, Hq, Hkv, D, D, 64, kind)
    _close(torch, b.run(), *b.reference())


@pytest.mark.parametrize("n,Hq,Hkv,D,window", [(6, 4, 2, 128, 0), (6, 32, 2, 128, 0), (6, 4, 1, 64, 70), (5, 4, 4, 256, 0)])
@pytest.mark.parametrize("ps", [16, 24])
def test_a_huge_scale_stays_with_those_who_see_it(torch, n, Hq, Hkv, D, window, ps):
    """A new token whose E4M3 scales are finite and huge: rows that do not see it
    answer as if it were an ordinary one (alone, behind a context, across parts)."""
    b = Batch(torch, [7, 150, 1500, 64 + n], [n] * 4, n, Hq, Hkv, D, D, ps, "e4m3")
    b.mask[:] = torch.tensor([(1 << i) | 1 for i in range(n)], device="cuda")
    ref, tol = b.reference(window=window)
    for s, x in enumerate(b.lens):
        t = x - n + 2  # new token 2, which none but itself sees
        page, off = int(b.table[s, t // ps]), t % ps
        b.ks[page, :, off], b.vs[page, :, off] = 1e20, 1e30
    after = b.run(window=window)
    others = [i for i in range(n) if i != 2]
    _close(torch, after[:, others], ref[:, others], tol[:, others])


@pytest.mark.parametrize("kind,n,Hq,Hkv,D", [("bf16", 16, 8, 1, 128), ("e4m3", 16, 8, 1, 128), ("e4m3", 4, 8, 1, 128),
                                             ("bf16", 3, 8, 2, 64), ("e4m3", 16, 16, 2, 64), ("e4m3", 5, 4, 1, 256),
                                             ("latent", 2, 20, 1, 512), ("latent", 1, 64, 1, 256)])
def test_maxima_that_move_in_every_tile(torch, kind, n, Hq, Hkv, D):
    """Keys that grow along long ragged sequences: every tile moves the maxima and
    rescales what is there, the last tile of each part of a sequence among them."""
    lens = [700 + 331 * (i * 7 % 11) for i in range(40)]
    Dk, Dv = (D + 64, D) if kind == "latent" else (D, D)
    b = Batch(torch, lens, [n] * 40, n, Hq, Hkv, Dk, Dv, 16, kind, spread=2.0)
    for s, length in enumerate(lens):
        t = torch.arange(length, device="cuda")
        page, off = b.table[s].long()[t // 16], t % 16
        grow = 0.05 + t / 1500.0
        if kind == "latent":
            b.data[page, off] = (b.data[page, off].float() * grow.unsqueeze(1)).to(torch.bfloat16)
        elif kind == "bf16":
            b.k[page, :, off] = (b.k[page, :, off].float() * grow.view(-1, 1, 1)).to(torch.bfloat16)
        else:
            b.ks[page, :, off] *= grow.unsqueeze(1)
            b.vs[page, :, off] *= grow.unsqueeze(1)
    if kind != "latent":
        b.scale = b.op.scale = 3.0 / math.sqrt(D)
    got = [b.run() for _ in range(3)]
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
    _close(torch, got[0], *b.reference())


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "latent"])
def test_what_is_not_seen_may_be_anything(torch, kind):
    """Tokens past the end of a page that is used, pages that are not, and new
    tokens that a row does not see hold NaN and infinities: the row's outputs are
    those without them; rows that do see a NaN value are NaN in its dimension."""
    Dk, Dv, Hq, Hkv = (576, 512, 8, 1) if kind == "latent" else (128, 128, 4, 2)
    b = Batch(torch, [100, 64 + 5, 6], [6, 6, 6], 6, Hq, Hkv, Dk, Dv, 16, kind)
    chain = [_signed((2 << i) - 1) for i in range(6)]
    chain[3] = 0b001011  # does not see token 2
    chain[5] = 0b101011
    b.mask[:] = torch.tensor(chain, device="cuda")
    ref, tol = b.reference()
    used = torch.zeros(b.cache.pages, b.ps, dtype=torch.bool, device="cuda")
    third = []  # where new token 2 of each sequence lies
    for s, n in enumerate(b.lens):
        t = torch.arange(n, device="cuda")
        used[b.table[s].long()[t // b.ps], t % b.ps] = True
        third.append((int(b.table[s, (n - 4) // b.ps]), (n - 4) % b.ps))
    if kind == "latent":
        b.data[~used] = math.nan
        for p, o in third:
            b.data[p, o, 7], b.data[p, o, 300] = math.nan, -math.inf
    elif kind == "bf16":
        for x in (b.k, b.v):
            x.permute(0, 2, 1, 3)[~used] = math.inf
        for p, o in third:
            b.k[p, :, o] = math.nan
            b.v[p, :, o, 7], b.v[p, :, o, 100] = math.nan, -math.inf
    else:
        for x in (b.ks, b.vs):
            x.permute(0, 2, 1)[~used] = math.nan
        b.k.view(torch.uint8).permute(0, 2, 1, 3)[~used] = 0x7F
        b.v.view(torch.uint8).permute(0, 2, 1, 3)[~used] = 0xFF
        for p, o in third:
            b.vs[p, :, o] = math.nan
            b.v.view(torch.uint8)[p, :, o, 7] = 0x7F
    got = b.run()
    for i in (0, 1, 3, 5):
        _close(torch, got[:, i], ref[:, i], tol[:, i])
    for i in (2, 4):
        assert torch.isnan(got[:, i, :, 7]).all()


def test_infinite_value_reaches_those_who_see_it(torch):
    """An infinite value of a new token, seen by some rows: infinite there."""
    b = Batch(torch, [70], [3], 3, 4, 1, 64, 64, 16, "bf16")
    b.mask[:] = torch.tensor([1, 2, 7], device="cuda")
    ref, tol = b.reference()
    t = 68  # new token 1
    b.v[b.table[0, t // 16].long(), 0, t % 16, 9] = math.inf
    got = b.run()
    assert (got[0, 1:, :, 9] == math.inf).all()
    _close(torch, got[:, 0], ref[:, 0], tol[:, 0])
    keep = torch.arange(64, device="cuda") != 9
    _close(torch, got[..., keep], ref[..., keep], tol[..., keep])


@pytest.mark.parametrize("kind", ["bf16", "latent"])
def test_rows_that_see_nothing(torch, kind):
    Dk, Dv = (320, 256) if kind == "latent" else (128, 128)
    b = Batch(torch, [4, 0, 3], [4, 0, 1], 4, 4, 1, Dk, Dv, 16, kind)
    b.mask[0, 2] = 0
    b.mask[2] = 0  # context alone
    out = torch.full((3, 4, 4, Dv), 7.0, dtype=torch.bfloat16, device="cuda")
    got = b.run(out=out)
    ref, tol = b.reference()
    _close(torch, got, ref, tol)
    assert (got[0, 2] == 0).all() and (got[1] == 0).all() and (got[2, 1:] == 0).all()
    assert (got[2, 0] != 0).any()


def test_values_that_cancel(torch):
    """Weights next to values +v and -v in pairs: what is left of them is small
    beside their own size, and still within the weights' rounding."""
    b = Batch(torch, [600], [4], 4, 8, 1, 128, 128, 16, "bf16", spread=0.05)
    t = torch.arange(600, device="cuda")
    page, off = b.table[0].long()[t // 16], t % 16
    sign = torch.where(t % 2 == 0, 1.0, -1.0).unsqueeze(1)
    b.v[page, 0, off] = (sign * 100.0 * torch.ones(600, 128, device="cuda")).to(torch.bfloat16)
    _close(torch, b.run(), *b.reference())


@pytest.mark.parametrize("kind", ["bf16", "latent"])
def test_layouts(torch, kind):
    """Strided sequences, tokens, tables and masks; a mask that sequences share;
    caches kept as [pages, tokens, heads, size]; what lies around the outputs
    stays."""
    Dk, Dv, Hq, Hkv = (576, 512, 4, 1) if kind == "latent" else (128, 128, 4, 2)
    b = Batch(torch, [100, 70, 33], [5, 5, 5], 5, Hq, Hkv, Dk, Dv, 16, kind)
    base = b.run()
    q = torch.zeros(5, 3, Hq + 1, Dk, dtype=torch.bfloat16, device="cuda")[:, :, :Hq].permute(1, 0, 2, 3)
    q.copy_(b.q)
    big = torch.full((3, 7, Hq + 2, Dv), 3.0, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(3, 50, dtype=torch.int32, device="cuda")[:, 7:7 + b.table.shape[1]]
    table.copy_(b.table)
    mask = torch.zeros(3, 11, dtype=torch.int64, device="cuda")[:, 1:6]
    mask.copy_(b.mask)
    b.q, b.table, b.mask = q, table, mask
    b.run(out=big[:, 1:6, :Hq])
    assert torch.equal(big[:, 1:6, :Hq], base)
    big[:, 1:6, :Hq] = 3.0
    assert (big == 3.0).all()
    if kind == "bf16":
        k, v = (x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for x in (b.k, b.v))
        b.cache = _dec().PagedCache(k, v)
        assert torch.equal(b.run(), base)
    shared = b.mask[:1].expand(3, 5)
    b.mask = b.mask[:1].repeat(3, 1)
    _close(torch, b.run(mask=shared), *b.reference())


def test_streams_graphs_and_equal_bits(torch):
    b = Batch(torch, [5000, 64, 900], [4, 4, 4], 4, 16, 2, 128, 128, 16, "bf16")
    lat = Batch(torch, [5000, 64, 900], [4, 4, 4], 4, 32, 1, 576, 512, 64, "latent")
    for x in (b, lat):
        base = x.run()
        assert torch.equal(x.run(), base)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        other = x.op.forward(x.q, x.cache, x.table, x.seq_lens, x.mask, x.draft_lens, stream=side)
        side.synchronize()
        assert torch.equal(other, base)
        # two graphs that share a workspace, one after the other
        ws, outs, graphs = x.op.workspace(3, 4), [torch.empty_like(base) for _ in range(2)], []
        for o in outs:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                x.op.forward(x.q, x.cache, x.table, x.seq_lens, x.mask, x.draft_lens, out=o, ws=ws)
            graphs.append(g)
        for _ in range(3):
            ws.fill_(255)
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], base) and torch.equal(outs[1], base)
        # lengths that change under a captured graph
        x.seq_lens.copy_(torch.tensor([70, 5000, 4], dtype=torch.int32))
        x.table.copy_(x.table.roll(1, 0))
        x.lens = [70, 5000, 4]
        graphs[0].replay()
        _close(torch, outs[0], *x.reference())


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "latent"])
@pytest.mark.parametrize("ps", [16, 5])
def test_bad_pages_and_lengths(torch, kind, ps):
    """Out-of-range page numbers and lengths are flagged and left out."""
    from block_fp8_expert_gb300 import MoeError
    Dk, Dv, Hq, Hkv = (320, 256, 4, 1) if kind == "latent" else (64, 64, 4, 2)
    b = Batch(torch, [100, 80, 90], [3, 3, 3], 3, Hq, Hkv, Dk, Dv, ps, kind)
    ref, tol = b.reference()
    good = b.table.clone()
    for page in (-1, b.cache.pages, 2 ** 31 - 1, -2 ** 31):
        b.table[1, 1] = page
        with pytest.raises(MoeError, match="0x10"):
            b.run()
        got = b.op.forward(b.q, b.cache, b.table, b.seq_lens, b.mask, b.draft_lens)
        b.op.status.zero_()
        # the tokens of the page are left out
        hole = Batch.seen
        b.seen = lambda s, i, *a: [t for t in hole(b, s, i, *a) if s != 1 or t // ps != 1]
        b.table.copy_(good)
        _close(torch, got, *b.reference())
        del b.seen
    for name, value in (("seq_lens", -5), ("seq_lens", 2 ** 31 - 1), ("draft_lens", 4), ("draft_lens", -1)):
        t = getattr(b, name)
        keep = t.clone()
        t[1] = value
        if value == 2 ** 31 - 1:
            b.table[1] = b.table[1].clamp(min=0)
        with pytest.raises(MoeError, match="0x10"):
            b.run()
        got = b.op.forward(b.q, b.cache, b.table, b.seq_lens, b.mask, b.draft_lens)
        for s in (0, 2):
            _close(torch, got[s], ref[s], tol[s])
        t.copy_(keep)
        b.op.status.zero_()
    _close(torch, b.run(), ref, tol)


@pytest.mark.parametrize("kind", ["bf16", "latent"])
def test_offsets_past_32_bits(torch, kind):
    """The last pages of a cache of more than 2^32 bytes and 2^31 elements."""
    dec = _dec()
    g = _gen(torch, 3)
    if kind == "latent":
        pages = 2 ** 31 // (64 * 320) + 10
        data = torch.empty(pages, 64, 320, dtype=torch.bfloat16, device="cuda")
        b = Batch(torch, [130], [2], 2, 8, 1, 320, 256, 64, kind)
        data[-5:] = torch.randn(5, 64, 320, generator=g, device="cuda").to(torch.bfloat16)
        b.data, b.cache = data, dec.LatentCache(data, R=256)
    else:
        pages = 2 ** 31 // (4 * 64 * 128) + 10
        k, v = (torch.empty(pages, 4, 64, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        b = Batch(torch, [130], [2], 2, 8, 4, 128, 128, 64, kind)
        for x in (k, v):
            x[-5:] = torch.randn(5, 4, 64, 128, generator=g, device="cuda").to(torch.bfloat16)
        b.k, b.v, b.cache = k, v, dec.PagedCache(k, v)
    b.table[0] = torch.tensor([pages - 1, pages - 4, pages - 3], dtype=torch.int32)
    _close(torch, b.run(), *b.reference())


def test_empty_batch(torch):
    b = Batch(torch, [5], [2], 2, 4, 1, 64, 64, 16, "bf16")
    out = b.op.forward(b.q[:0], b.cache, b.table[:0], b.seq_lens[:0], b.mask[:0], b.draft_lens[:0])
    assert out.shape == (0, 2, 4, 64)
    b.op.check()


def test_large_scores_and_negative_scale(torch):
    """Scores of hundreds, whose maximum moves again and again along the cache."""
    for scale in (3.0, -2.0):
        b = Batch(torch, [900, 300], [4, 4], 4, 8, 2, 64, 64, 16, "bf16", spread=0.5)
        t = torch.arange(900, device="cuda")
        page, off = b.table[0].long()[t // 16], t % 16
        b.k[page, :, off] = (b.k[page, :, off].float() * (1 + t / 200.0).view(-1, 1, 1)).to(torch.bfloat16)
        b.scale = b.op.scale = scale
        ref, _ = b.reference()
        got = b.run()
        # the winner takes nearly all: compare with the weights' own sensitivity
        e = 64 * 2.0 ** -23 * abs(scale) * 64 * 4 * 3 + 2.0 ** -12
        assert (got.double() - ref).abs().max() <= (U16 + 2 * e) * 6
