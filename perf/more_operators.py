"""Latent attention and attention of drafted tokens, as cases to time and compare.

Four operators of decoder layers, each with a plain form (elementary torch
operations in fp32, rounded once at the end) and the call a user makes of this
package:

* store: the latent vector of every token, normed, with its shared key part
  rotated, stored into a paged cache; the queries' rotated parts on the way;
* latent: attention over that cache in the absorbed form (the latent vector is
  key and value of every head), one or several new tokens per sequence, which
  see each other as a tree;
* expanded: the prompt form of the same attention: keys and values of every
  head, the rotated key part shared, causal over ragged sequences;
* tree: attention of a tree of drafted tokens over a paged cache of grouped
  key/value heads (bf16, or E4M3 with one scale per token and head).

Head layouts and sizes are generic.
"""
import math
import random

import numpy as np
import torch

own = False

ROT, NOPE, VD = 64, 128, 128
E4M3_MAX = 448.0


def listed():
    return [
        # a decode step of a few users: latency is all
        dict(name="store_T5_H32", op="store", T=5, H=32, R=512, interleaved=True, page=64, rows=False),
        # a ragged chunk of a prompt of a smaller model
        dict(name="store_T517_H20_R256", op="store", T=517, H=20, R=256, interleaved=False, page=16,
             rows=True),
        # a long prompt with many heads, the normed rows kept for the up-projection
        dict(name="store_T8192_H128", op="store", T=8192, H=128, R=512, interleaved=True, page=64,
             rows=True),
        # one user with a short history
        dict(name="latent_B1_L777_H32", op="latent", B=1, L=777, n=1, ragged=False, H=32, R=512,
             page=64),
        # a serving batch of mixed histories (one slot empty), all heads of a large model
        dict(name="latent_B40_ragged_L6000_H128", op="latent", B=40, L=6000, n=1, ragged=True, H=128,
             R=512, page=64),
        # two users with very long documents, a share of the heads
        dict(name="latent_B2_L131072_H64", op="latent", B=2, L=131072, n=1, ragged=False, H=64, R=512,
             page=64),
        # a batch that verifies small trees of drafted tokens, small pages
        dict(name="latent_B16_ragged_L3000_n5_H20", op="latent", B=16, L=3000, n=5, ragged=True, H=20,
             R=512, page=16),
        # the last tokens of a few chunked prompts: mostly history
        dict(name="expanded_B3_L9_ctx700_H32", op="expanded", B=3, L=9, ctx=700, H=32),
        # a batch of ragged prompts
        dict(name="expanded_B7_L1900_H20", op="expanded", B=7, L=1900, ctx=0, H=20),
        # one long prompt
        dict(name="expanded_B1_L8192_H32", op="expanded", B=1, L=8192, ctx=0, H=32),
        # one user's small tree of drafted tokens
        dict(name="tree_B1_L900_n8", op="tree", B=1, L=900, n=8, ragged=False, Hq=32, Hkv=4, D=128,
             e4m3=False, page=64, window=0),
        # a serving batch that verifies drafts over mixed histories, E4M3 cache
        dict(name="tree_B32_ragged_L4096_n16_e4m3", op="tree", B=32, L=4096, n=16, ragged=True, Hq=32,
             Hkv=4, D=128, e4m3=True, page=16, window=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(("store", "latent", "expanded", "tree"))
    if op == "store":
        H, R = rng.choice((8, 20, 32, 64, 128)), rng.choice((256, 512))
        return dict(op=op, T=_log_int(rng, 1, 8192), H=H, R=R, interleaved=rng.random() < 0.5,
                    page=rng.choice((1, 16, 32, 64)), rows=rng.random() < 0.5)
    if op == "latent":
        H, R = rng.choice((8, 20, 32, 64, 128)), rng.choice((256, 512))
        n = rng.choice((1, 1, 1, 2, 4, 7))
        B = _log_int(rng, 1, 64)
        L = _log_int(rng, n, max(n, min(131072, 2 * 131072 * 64 // (B * max(H * n, 64)))))
        return dict(op=op, B=B, L=L, n=n, ragged=rng.random() < 0.7, H=H, R=R,
                    page=rng.choice((16, 32, 64)))
    if op == "expanded":
        H, B = rng.choice((5, 8, 20, 32, 64)), _log_int(rng, 1, 16)
        ctx = rng.choice((0, 0, _log_int(rng, 1, 2000)))
        L = _log_int(rng, 1, min(8192, int(math.sqrt(8192 * 8192 * 32 / (B * H))) - ctx))
        return dict(op=op, B=B, L=L, ctx=ctx, H=H)
    D = rng.choice((64, 128, 256))
    Hkv, G = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 4, 5, 8, 16))
    n, B = rng.choice((1, 2, 5, 8, 16, 33, 64)), _log_int(rng, 1, 64)
    # no more than the largest listed case's work, in the plain form's terms
    top = 32 * 4096 * 4 * 128 // (B * Hkv * D)
    L = _log_int(rng, n, max(n, min(65536, top, top * 16 * 8 // (n * G))))
    return dict(op=op, B=B, L=L, n=n, ragged=rng.random() < 0.7, Hq=Hkv * G, Hkv=Hkv, D=D,
                e4m3=rng.random() < 0.5, page=rng.choice((16, 32, 64)),
                window=rng.choice((0, 0, 0, 512)))


# ------------------------------------------------------------------ inputs

def _gen(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + sum(ord(c) for c in case["op"]))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _e4m3(v):
    """fp32 [..., n] -> (E4M3 tensor, fp32 scale [...]): one scale per last-axis group."""
    a = v.abs().amax(-1)
    codes = (v * (E4M3_MAX / a).unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes, a / E4M3_MAX


def _prompt_lens(c):
    """The lengths of an expanded case's sequences: uneven, of one to L tokens."""
    return [max(1, c["L"] * (b + 1) ** 2 // c["B"] ** 2) for b in range(c["B"])]


def _trees(rng, B, n):
    """The tokens that each drafted token sees of its own tree (its ancestors
    and itself), as bits: a branching chain per sequence, int64 [B, n]."""
    rows = []
    for _ in range(B):
        seen = []
        for i in range(n):
            up = rng.randint(max(0, i - 4), i - 1) if i else -1
            seen.append((seen[up] if i else 0) | 1 << i)
        rows.append([s - (1 << 64) if s >> 63 else s for s in seen])
    return torch.tensor(rows, dtype=torch.int64, device="cuda")


def _paged(g, c, seed):
    """Lengths, page tables and trees of a batch whose slots are mixed: an
    empty one, one that holds its drafted tokens alone, one with fewer of them."""
    B, L, n, ps = c["B"], c["L"], c["n"], c["page"]
    lens = torch.full((B,), L, dtype=torch.int64, device="cuda")
    draft = torch.full((B,), n, dtype=torch.int32, device="cuda")
    if c["ragged"]:
        u = torch.rand(B, generator=g, device="cuda", dtype=torch.float32)
        lens = (L * u ** 1.5).long().clamp(n, L)
        if B >= 4:
            lens[1], lens[2], lens[3] = 0, n, L
            draft[1], draft[3] = 0, (n + 1) // 2
    need = (lens + ps - 1) // ps
    pages = max(1, int(need.sum()))
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(-(-L // ps), device="cuda")
    first = need.cumsum(0) - need
    table = torch.where(col < need[:, None], order[(first[:, None] + col).clamp(max=pages - 1)],
                        torch.zeros((), dtype=torch.int32, device="cuda")).contiguous()
    return dict(lens=lens.to(torch.int32), draft=draft, table=table,
                mask=_trees(random.Random(seed), B, n)), pages


def prepare(case, seed):
    c = case
    g = _gen(c, seed)
    st = {"case": c}
    if c["op"] == "store":
        T, H, R, ps, n_pos = c["T"], c["H"], c["R"], c["page"], 40960
        inv = 1e4 ** (-torch.arange(0, ROT, 2, dtype=torch.float64, device="cuda") / ROT)
        ang = torch.arange(n_pos, dtype=torch.float64, device="cuda")[:, None] * inv
        pages = -(-T // ps) + 2
        slots = torch.randperm(pages * ps, generator=g, device="cuda")[:T]
        slots[torch.rand(T, generator=g, device="cuda") < 0.02] = -1  # padding tokens store nothing
        st.update(
            kv=(2.0 * _randn(g, T, R + ROT)).to(torch.bfloat16),
            q=(2.0 * _randn(g, T, H, NOPE + ROT)).to(torch.bfloat16),
            norm=1 + 0.1 * _randn(g, R), slots=slots, eps=1e-6,
            cos_sin=torch.cat([ang.cos(), ang.sin()], 1).float().contiguous(),
            positions=torch.randint(0, n_pos, (T,), generator=g, device="cuda").to(torch.int32),
            cache=torch.zeros(pages, ps, R + ROT, dtype=torch.bfloat16, device="cuda"))
    elif c["op"] == "latent":
        more, pages = _paged(g, c, seed)
        st.update(more)
        st["q"] = _randn(g, c["B"], c["n"], c["H"], c["R"] + ROT).to(torch.bfloat16)
        st["cache"] = torch.empty(pages, c["page"], c["R"] + ROT, device="cuda", dtype=torch.bfloat16)
        for i in range(0, pages, 4096):
            st["cache"][i:i + 4096] = _randn(g, min(4096, pages - i), c["page"], c["R"] + ROT)
        st["scale"] = 1.0 / math.sqrt(NOPE + ROT)
    elif c["op"] == "expanded":
        lens = _prompt_lens(c)
        cu = torch.tensor([0] + lens, device="cuda").cumsum(0)
        st["cu_q"] = cu.to(torch.int32)
        st["cu_k"] = (cu + c["ctx"] * torch.arange(c["B"] + 1, device="cuda")).to(torch.int32)
        Tq = sum(lens)
        Tk = Tq + c["B"] * c["ctx"]
        st["q"] = (1.5 * _randn(g, Tq, c["H"], NOPE + ROT)).to(torch.bfloat16)
        # as the up-projection leaves them: per head the key part, then the value
        st["kv"] = _randn(g, Tk, c["H"], NOPE + VD).to(torch.bfloat16)
        st["k_rope"] = _randn(g, Tk, ROT).to(torch.bfloat16)
        st["scale"] = 1.0 / math.sqrt(NOPE + ROT)
    else:
        more, pages = _paged(g, c, seed)
        st.update(more)
        st["q"] = (1.5 * _randn(g, c["B"], c["n"], c["Hq"], c["D"])).to(torch.bfloat16)
        shape = (c["Hkv"], c["page"], c["D"])
        for name in ("k", "v"):
            t = torch.empty(pages, *shape, device="cuda",
                            dtype=torch.uint8 if c["e4m3"] else torch.bfloat16)
            s = torch.empty(pages, *shape[:2], device="cuda") if c["e4m3"] else None
            for i in range(0, pages, 4096):
                f = _randn(g, min(4096, pages - i), *shape)
                if c["e4m3"]:
                    codes, s[i:i + 4096] = _e4m3(f)
                    t[i:i + 4096] = codes.view(torch.uint8)
                else:
                    t[i:i + 4096] = f.to(torch.bfloat16)
            st[name], st[name + "s"] = t, s
        st["scale"] = 1.0 / math.sqrt(c["D"])
    if own:
        _plan(st)
    return st


def _plan(st):
    """What a serving program sets up once: the operator's handle, its output
    buffers and its workspace."""
    from block_fp8_expert_gb300 import decoder
    c = st["case"]
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    if c["op"] == "store":
        st["op"] = decoder.LatentStore(H=c["H"], R=c["R"], rot=ROT, norm=st["norm"],
                                       cos_sin=st["cos_sin"], interleaved=c["interleaved"],
                                       eps=st["eps"])
        st["paged"] = decoder.LatentCache(st["cache"], R=c["R"])
        # the rotated parts go where the attention reads them
        st["q_out"] = torch.empty(c["T"], c["H"], NOPE + ROT, **bf16)[..., NOPE:]
        st["rows"] = torch.empty(c["T"], c["R"] + ROT, **bf16) if c["rows"] else None
    elif c["op"] == "latent":
        st["op"] = decoder.LatentAttention(H=c["H"], R=c["R"], rot=ROT, scale=st["scale"])
        st["paged"] = decoder.LatentCache(st["cache"], R=c["R"])
        st["ws"] = st["op"].workspace(c["B"], c["n"])
        st["out"] = torch.empty(c["B"], c["n"], c["H"], c["R"], **bf16)
    elif c["op"] == "expanded":
        st["op"] = decoder.ExpandedAttention(H=c["H"], scale=st["scale"])
        st["out"] = torch.empty(st["q"].shape[0], c["H"], VD, **bf16)
    else:
        st["op"] = decoder.TreeAttention(Hq=c["Hq"], Hkv=c["Hkv"], D=c["D"], scale=st["scale"],
                                         window=c["window"])
        st["paged"] = decoder.PagedCache(st["k"], st["v"], st["ks"], st["vs"])
        st["ws"] = st["op"].workspace(c["B"], c["n"])
        st["out"] = torch.empty(c["B"], c["n"], c["Hq"], c["D"], **bf16)


# ------------------------------------------------------------------ one pass

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    op = st["case"]["op"]
    if op == "store":
        st["op"].forward(st["kv"], st["positions"], st["slots"], st["paged"],
                         q=st["q"][..., NOPE:], q_out=st["q_out"], rows=st["rows"])
        out = {"q": st["q_out"], "cache": st["cache"]}
        return {**out, "rows": st["rows"]} if st["case"]["rows"] else out
    if op == "expanded":
        st["op"].forward(st["q"], st["kv"][..., :NOPE], st["k_rope"], st["kv"][..., NOPE:], st["cu_q"],
                         st["cu_k"], out=st["out"])
    else:
        st["op"].forward(st["q"], st["paged"], st["table"], st["lens"], st["mask"], st["draft"],
                         out=st["out"], ws=st["ws"])
    return {"out": st["out"]}


def _run_plain(st):
    return {"store": _plain_store, "latent": _plain_paged, "expanded": _plain_expanded,
            "tree": _plain_paged}[st["case"]["op"]](st)


def _plain_rotate(x, cs, interleaved):
    """x fp32 [..., ROT], cs [..., ROT]: the cosines, then the sines."""
    cos, sin = cs[..., :ROT // 2], cs[..., ROT // 2:]
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :ROT // 2], x[..., ROT // 2:])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    return torch.stack([ra, rb], -1).flatten(-2) if interleaved else torch.cat([ra, rb], -1)


def _plain_store(st):
    c = st["case"]
    R, ps = c["R"], c["page"]
    cs = st["cos_sin"][st["positions"].long()]
    q = _plain_rotate(st["q"][..., NOPE:].float(), cs.unsqueeze(1), c["interleaved"])
    x = st["kv"].float()
    lat = x[:, :R]
    lat = lat * torch.rsqrt((lat * lat).mean(-1, keepdim=True) + st["eps"]) * st["norm"]
    rows = torch.cat([lat, _plain_rotate(x[:, R:], cs, c["interleaved"])], -1).to(torch.bfloat16)
    tok = (st["slots"] >= 0).nonzero().squeeze(1)
    st["cache"][st["slots"][tok] // ps, st["slots"][tok] % ps] = rows[tok]
    out = {"q": q.to(torch.bfloat16), "cache": st["cache"]}
    return {**out, "rows": rows} if c["rows"] else out


def _plain_paged(st):
    """Both forms over a paged cache: the latent one has one key/value head,
    whose values are the leading dimensions of its keys."""
    c = st["case"]
    t = st["table"].long()
    if c["op"] == "latent":
        Hkv, Dv = 1, c["R"]
        k = st["cache"][t].flatten(1, 2).float().unsqueeze(1)
        v = k[..., :Dv]
    else:
        Hkv, Dv = c["Hkv"], c["D"]
        kv = []
        for name in ("k", "v"):
            x = st[name][t]
            x = (x.view(torch.float8_e4m3fn).float() * st[name + "s"][t].unsqueeze(-1) if c["e4m3"]
                 else x.float())
            kv.append(x.transpose(1, 2).flatten(2, 3))
        k, v = kv
    B, n, H, Dk = st["q"].shape
    q = st["q"].float().view(B, n, Hkv, H // Hkv, Dk).permute(0, 2, 1, 3, 4).flatten(2, 3)
    s = (q @ k.transpose(2, 3)).view(B, Hkv, n, H // Hkv, -1) * st["scale"]
    pos = torch.arange(s.shape[-1], device=s.device)
    ctx = (st["lens"] - st["draft"]).long()[:, None]
    at = pos - ctx                                               # [B, tokens]: place in the tree
    real = (at < st["draft"][:, None]).unsqueeze(1)
    bits = (st["mask"].unsqueeze(-1) >> at.clamp(0, 63).unsqueeze(1)) & 1   # [B, n, tokens]
    seen = (at < 0).unsqueeze(1) | (real & (bits == 1) & (at >= 0).unsqueeze(1))
    if c.get("window"):
        depth = ((st["mask"].unsqueeze(-1) >> torch.arange(64, device=s.device)) & 1
                 & (torch.arange(64, device=s.device) < st["draft"][:, None, None])).sum(-1)
        low = ctx + depth - c["window"]                          # [B, n]
        seen = seen & ((pos >= low.unsqueeze(-1)) | (at >= 0).unsqueeze(1))
    row = torch.arange(n, device=s.device) < st["draft"][:, None]  # [B, n]: rows that exist
    seen = (seen & row.unsqueeze(-1))[:, None, :, None]
    s = torch.where(seen, s, torch.full_like(s, -torch.inf))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -torch.inf, torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).view(B, Hkv, n, H // Hkv, Dv) / torch.where(l == 0, torch.ones_like(l), l)
    return {"out": o.permute(0, 2, 1, 3, 4).reshape(B, n, H, Dv).to(torch.bfloat16)}


def _plain_expanded(st):
    c = st["case"]
    out = torch.empty(st["q"].shape[0], c["H"], VD, dtype=torch.bfloat16, device="cuda")
    q0 = k0 = 0
    for n in _prompt_lens(c):
        m = n + c["ctx"]
        later = torch.arange(m, device="cuda") > torch.arange(n, device="cuda")[:, None] + (m - n)
        for h in range(0, c["H"], 8):  # (a few heads at a time: the scores are large)
            q = st["q"][q0:q0 + n, h:h + 8].float().transpose(0, 1)
            kv = st["kv"][k0:k0 + m, h:h + 8].float().transpose(0, 1)
            s = q[..., :NOPE] @ kv[..., :NOPE].transpose(1, 2)
            s = (s + q[..., NOPE:] @ st["k_rope"][k0:k0 + m].float().t()) * st["scale"]
            s = s.masked_fill(later, -torch.inf)
            p = torch.exp(s - s.amax(-1, keepdim=True))
            o = (p @ kv[..., NOPE:]) / p.sum(-1, keepdim=True)
            out[q0:q0 + n, h:h + 8] = o.transpose(0, 1).to(torch.bfloat16)
        q0, k0 = q0 + n, k0 + m
    return {"out": out}


# ------------------------------------------------------------------ what a pass cannot do without

def _tokens(c):
    # a ragged batch's lengths are L u^1.5: 0.4 L on average
    return c["B"] * (0.4 * c["L"] if c["ragged"] else c["L"])


def work(case):
    c = case
    if c["op"] == "store":
        T, H, R = c["T"], c["H"], c["R"]
        return {"bytes": T * (2 * (R + ROT) * (3 if c["rows"] else 2) + 4 * H * ROT + 4 * ROT + 12) + 4 * R,
                "flops": T * (4 * R + 3 * ROT * (H + 1))}
    if c["op"] == "latent":
        rows, tokens = c["n"] * c["H"], _tokens(c)
        return {"bytes": 2 * tokens * (c["R"] + ROT) + 2 * c["B"] * rows * (2 * c["R"] + ROT)
                + 4 * tokens / c["page"] + c["B"] * (8 + 8 * c["n"]),
                "flops": 2 * tokens * rows * (2 * c["R"] + ROT)}
    if c["op"] == "expanded":
        lens = _prompt_lens(c)
        pairs = sum(n * c["ctx"] + n * (n + 1) // 2 for n in lens)
        Tq, Tk = sum(lens), sum(lens) + c["B"] * c["ctx"]
        return {"bytes": 2 * c["H"] * (Tq * (NOPE + ROT + VD) + Tk * (NOPE + VD)) + 2 * Tk * ROT,
                "flops": 2 * c["H"] * pairs * (NOPE + ROT + VD)}
    tokens = _tokens(c)
    if c["window"]:
        tokens = min(tokens, c["B"] * (c["window"] + c["n"]))
    per = 2 * c["Hkv"] * ((c["D"] + 4) if c["e4m3"] else 2 * c["D"])
    return {"bytes": tokens * per + 4 * c["B"] * c["n"] * c["Hq"] * c["D"] + 4 * tokens / c["page"]
            + c["B"] * (8 + 8 * c["n"]),
            "flops": 4 * tokens * c["n"] * c["Hq"] * c["D"]}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """The operators' definitions in 64 bits, on the inputs of prepare()."""
    st = prepare(case, seed)
    return {"store": _exact_store, "latent": _exact_paged, "expanded": _exact_expanded,
            "tree": _exact_paged}[case["op"]](st)


def _exact_turn(x, turn, interleaved):
    """The rotation as a product of complex numbers, x float64 [..., ROT]."""
    pair = torch.arange(ROT // 2, device=x.device)
    ia = 2 * pair if interleaved else pair
    ib = ia + (1 if interleaved else ROT // 2)
    y = torch.complex(x[..., ia].contiguous(), x[..., ib].contiguous()) * turn
    out = torch.empty_like(x)
    out[..., ia], out[..., ib] = y.real, y.imag
    return out


def _exact_store(st):
    c = st["case"]
    R = c["R"]
    cs = st["cos_sin"].double()[st["positions"].long()]
    turn = torch.complex(cs[:, :ROT // 2].contiguous(), cs[:, ROT // 2:].contiguous())
    q = torch.cat([_exact_turn(x.double(), w.unsqueeze(1), c["interleaved"])
                   for x, w in zip(st["q"][..., NOPE:].split(1024), turn.split(1024))])
    x = st["kv"].double()
    size = torch.sqrt(x[:, :R].square().sum(-1, keepdim=True) / R + st["eps"])
    rows = torch.cat([x[:, :R] / size * st["norm"].double(), _exact_turn(x[:, R:], turn, c["interleaved"])], 1)
    cache = torch.zeros_like(st["cache"], dtype=torch.float64)
    flat = cache.view(-1, R + ROT)
    for t in range(c["T"]):
        slot = int(st["slots"][t]) if c["T"] <= 64 else None
        if slot is None:
            keep = st["slots"] >= 0
            flat[st["slots"][keep]] = rows[keep]
            break
        if slot >= 0:
            flat[slot] = rows[t]
    out = {"q": q, "cache": cache}
    return {**out, "rows": rows} if c["rows"] else out


def _exact_paged(st):
    c = st["case"]
    latent = c["op"] == "latent"
    B, n, H, Dk = st["q"].shape
    Hkv, Dv, ps = (1, c["R"], c["page"]) if latent else (c["Hkv"], c["D"], c["page"])
    out = torch.zeros(B, n, H, Dv, dtype=torch.float64, device="cuda")
    lens, drafts, masks = st["lens"].tolist(), st["draft"].tolist(), st["mask"].tolist()
    for b in range(B):
        ctx = lens[b] - drafts[b]
        t = torch.arange(lens[b], device="cuda")
        page, off = st["table"][b].long()[t // ps], t % ps
        seen = torch.zeros(n, lens[b], dtype=torch.bool)
        for i in range(drafts[b]):
            mine = [j for j in range(drafts[b]) if masks[b][i] >> j & 1]
            low = max(0, ctx + len(mine) - c["window"]) if c.get("window") else 0
            seen[i, low:ctx] = True
            seen[i, [ctx + j for j in mine]] = True
        seen = seen[:drafts[b]].cuda()
        if not drafts[b]:
            continue
        for h in range(Hkv):
            if latent:
                k = st["cache"][page, off].double()
                v = k[:, :Dv]
            else:
                k, v = (st[x][page, h, off] for x in "kv")
                if c["e4m3"]:
                    k, v = (x.view(torch.float8_e4m3fn).double() * st[s][page, h, off].double().unsqueeze(1)
                            for x, s in ((k, "ks"), (v, "vs")))
                k, v = k.double(), v.double()
            G = H // Hkv
            q = st["q"][b, :drafts[b], h * G:(h + 1) * G].double()
            s = torch.einsum("igd,td->igt", q, k) * st["scale"]
            s = s.masked_fill(~seen.unsqueeze(1), -torch.inf)
            out[b, :drafts[b], h * G:(h + 1) * G] = torch.einsum("igt,td->igd", torch.softmax(s, -1), v)
    return {"out": out}


def _exact_expanded(st):
    c = st["case"]
    out = torch.empty(st["q"].shape[0], c["H"], VD, dtype=torch.float64, device="cuda")
    cu_q, cu_k = st["cu_q"].tolist(), st["cu_k"].tolist()
    for b in range(c["B"]):
        for h in range(c["H"]):
            k = torch.cat([st["kv"][cu_k[b]:cu_k[b + 1], h, :NOPE], st["k_rope"][cu_k[b]:cu_k[b + 1]]], 1).double()
            v = st["kv"][cu_k[b]:cu_k[b + 1], h, NOPE:].double()
            for i in range(cu_q[b], cu_q[b + 1], 1024):
                e = min(i + 1024, cu_q[b + 1])
                last = k.shape[0] - (cu_q[b + 1] - e)     # keys that the block's last row sees
                s = (st["q"][i:e, h].double() @ k[:last].t()) * st["scale"]
                s += torch.full_like(s, -torch.inf).triu(last - (e - i) + 1)
                out[i:e, h] = torch.softmax(s, -1) @ v[:last]
    return {"out": out}
