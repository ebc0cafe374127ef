"""The decoder operators next to the MoE layer, as cases to time and compare.

Four operators of a block-FP8 mixture-of-experts decoder layer, each with a
plain form (elementary torch operations in fp32, rounded once at the end) and
the call a user makes of this package:

* select: experts chosen from the router's logits: softmax or sigmoid scores,
  a balance bias that only steers the choice, expert groups, top-k and the
  selected experts' weights;
* qknorm: RMS norm of every query and key head and the rotary position
  embedding, the keys and values stored into a paged cache (bf16, or E4M3
  with one scale per token and head);
* attention: one new token per sequence over that paged cache;
* linear: x W^T with E4M3 activations (one scale per row and 128 input
  features, quantised in the call) and block-FP8 weights (one scale per 128 x
  128 block).

Sizes: hidden size 2048 and the 128 x 128 scale blocks are those of the
layers this package is benchmarked on; the head layouts are generic.
"""
import math

import numpy as np
import torch

own = False

HEAD_DIMS = (64, 128, 256)
E4M3_MAX = 448.0


def listed():
    return [
        # a decode step of a few sequences through a 512-expert layer, softmax scores
        dict(name="select_T5_E512_softmax", op="select", T=5, E=512, k=10, sigmoid=False,
             bias=False, groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0),
        # a long prompt through a layer with sigmoid scores, balance bias and groups
        dict(name="select_T8192_E256_groups", op="select", T=8192, E=256, k=8, sigmoid=True,
             bias=True, groups=8, top_groups=4, group_top=2, renorm=True, scale=2.5),
        # the decode step of a small batch: 32 query heads on 4 key/value heads
        dict(name="qknorm_T8_D128", op="qknorm", T=8, Hq=32, Hkv=4, D=128, rot=128,
             interleaved=False, e4m3=False, page=64),
        # a ragged chunk of a prompt, part of the head rotated in pairs, E4M3 cache
        dict(name="qknorm_T517_D256_e4m3", op="qknorm", T=517, Hq=16, Hkv=2, D=256, rot=64,
             interleaved=True, e4m3=True, page=16),
        # a long prompt into a bf16 cache
        dict(name="qknorm_T8192_D128", op="qknorm", T=8192, Hq=32, Hkv=4, D=128, rot=128,
             interleaved=False, e4m3=False, page=64),
        # one user with a short history: latency is all
        dict(name="attention_B1_L777", op="attention", B=1, L=777, ragged=False, Hq=32, Hkv=4,
             D=128, e4m3=False, page=64, window=0),
        # a serving batch of mixed histories (one slot empty, one with a single token), E4M3 cache
        dict(name="attention_B48_ragged_e4m3", op="attention", B=48, L=4096, ragged=True, Hq=32,
             Hkv=4, D=128, e4m3=True, page=16, window=0),
        # two users with very long documents
        dict(name="attention_B2_L131072", op="attention", B=2, L=131072, ragged=False, Hq=32,
             Hkv=4, D=128, e4m3=False, page=64, window=0),
        # a full serving batch with long histories
        dict(name="attention_B64_ragged_L12000", op="attention", B=64, L=12000, ragged=True,
             Hq=16, Hkv=2, D=128, e4m3=False, page=32, window=0),
        # the query/key/value projection of a single decoding user
        dict(name="linear_M1_N5120_K2048", op="linear", M=1, N=5120, K=2048),
        # the output projection of a ragged mid-size batch
        dict(name="linear_M203_N2048_K4096", op="linear", M=203, N=2048, K=4096),
        # the query/key/value projection of a long prompt
        dict(name="linear_M4096_N5120_K2048", op="linear", M=4096, N=5120, K=2048),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("select", "qknorm", "attention", "linear"))
    if op == "select":
        E = rng.choice((64, 128, 160, 256, 512))
        groups = rng.choice((1, 1, 4, 8))
        top_groups = groups if groups == 1 else rng.choice((groups // 2, groups // 2 + 1))
        k = rng.randint(1, 10)
        return dict(op=op, T=_log_int(rng, 1, 8192 * 256 // E if E > 256 else 8192), E=E, k=k,
                    sigmoid=rng.random() < 0.6, bias=rng.random() < 0.6, groups=groups,
                    top_groups=top_groups, group_top=rng.choice((1, 2)),
                    renorm=rng.random() < 0.7, scale=rng.choice((1.0, 2.5)))
    if op == "qknorm":
        D = rng.choice(HEAD_DIMS)
        Hkv = rng.choice((1, 2, 4, 8))
        Hq = Hkv * rng.choice((1, 2, 3, 4, 7, 8))
        top = max(1, 8192 * 40 * 128 // ((Hq + 2 * Hkv) * D))
        return dict(op=op, T=_log_int(rng, 1, min(8192, top)), Hq=Hq, Hkv=Hkv, D=D,
                    rot=rng.choice((D, D // 2, D // 4)), interleaved=rng.random() < 0.5,
                    e4m3=rng.random() < 0.5, page=rng.choice((16, 32, 64)))
    if op == "attention":
        D = rng.choice(HEAD_DIMS)
        Hkv = rng.choice((1, 2, 4, 8))
        G = rng.choice((1, 2, 3, 4, 7, 8, 16))
        B = _log_int(rng, 1, 64)
        # the plain form's cost goes with B L D times the heads: no more than the largest listed case
        L = _log_int(rng, 1, max(1, min(131072, 64 * 12000 * 2 * 128 // (B * Hkv * D),
                                        64 * 12000 * 16 * 128 // (B * Hkv * G * D))))
        return dict(op=op, B=B, L=L, ragged=rng.random() < 0.7, Hq=Hkv * G, Hkv=Hkv, D=D,
                    e4m3=rng.random() < 0.5, page=rng.choice((16, 32, 64)),
                    window=rng.choice((0, 0, 0, 512, 4096)))
    N = 8 * _log_int(rng, 16, 640)
    K = 64 * _log_int(rng, 4, 64)
    M = _log_int(rng, 1, min(4096, 4096 * 5120 * 2048 // (N * K)))
    return dict(op="linear", M=M, N=N, K=K)


# ------------------------------------------------------------------ inputs

def _gen(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + sum(ord(c) for c in case["op"]))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda", dtype=torch.float32)


def _e4m3(v):
    """fp32 [..., n] -> (E4M3 tensor, fp32 scale [...]): one scale per last-axis group."""
    a = v.abs().amax(-1)
    zero = a == 0
    inv = torch.where(zero, torch.zeros_like(a), E4M3_MAX / a)
    scale = torch.where(zero, torch.zeros_like(a), a / E4M3_MAX)
    codes = (v * inv.unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes, scale


def _gaps_ok(c, logits, bias):
    """Tokens whose choice is clear: every comparison that decides it has a
    gap of 1e-5 of the keys' size (both forms then choose alike)."""
    l = logits.double()
    s = torch.sigmoid(l) if c["sigmoid"] else torch.softmax(l, -1)
    key = s + bias.double() if bias is not None else s
    top = key.abs().amax(-1)
    ok = torch.ones(l.shape[0], dtype=torch.bool, device=l.device)
    if c["groups"] > 1:
        per = key.view(l.shape[0], c["groups"], -1)
        gs = per.sort(-1, descending=True).values[..., :c["group_top"]].sum(-1)
        srt = gs.sort(-1, descending=True)
        n = c["top_groups"]
        ok &= (srt.values[:, n - 1] - srt.values[:, n]) > 2e-5 * top
        keep = torch.zeros_like(gs).scatter(1, srt.indices[:, :n], 1.0)
        key = torch.where(keep.unsqueeze(-1) > 0, per, torch.full_like(per, -torch.inf)).flatten(1)
    v = key.sort(-1, descending=True).values[:, :c["k"] + 1]
    return ok & ((v[:, :-1] - v[:, 1:]) > 1e-5 * top.unsqueeze(-1)).all(-1)


def prepare(case, seed):
    c = case
    g = _gen(c, seed)
    st = {"case": c}
    if c["op"] == "select":
        T, E = c["T"], c["E"]
        bias = 0.1 * _randn(g, E) if c["bias"] else None
        logits = torch.empty(0, E, device="cuda")
        while logits.shape[0] < T:
            more = 1.2 * _randn(g, T + T // 8 + 16, E)
            logits = torch.cat([logits, more[_gaps_ok(c, more, bias)]])[:T]
        st.update(logits=logits.contiguous(), bias=bias)
    elif c["op"] == "qknorm":
        T, Hq, Hkv, D, ps = c["T"], c["Hq"], c["Hkv"], c["D"], c["page"]
        n_pos = 40960
        inv = 1e6 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda") / c["rot"])
        ang = torch.arange(n_pos, dtype=torch.float64, device="cuda")[:, None] * inv
        pages = -(-T // ps) + 2
        slots = torch.randperm(pages * ps, generator=g, device="cuda")[:T]
        slots[_rand(g, T) < 0.02] = -1  # padding tokens store nothing
        dt = torch.uint8 if c["e4m3"] else torch.bfloat16
        st.update(
            qkv=(2.0 * _randn(g, T, (Hq + 2 * Hkv) * D)).to(torch.bfloat16),
            q_norm=1 + 0.1 * _randn(g, D), k_norm=1 + 0.1 * _randn(g, D),
            cos_sin=torch.cat([ang.cos(), ang.sin()], 1).float().contiguous(),
            positions=torch.randint(0, n_pos, (T,), generator=g, device="cuda").to(torch.int32),
            slots=slots, eps=1e-6,
            k=torch.zeros(pages, Hkv, ps, D, dtype=dt, device="cuda"),
            v=torch.zeros(pages, Hkv, ps, D, dtype=dt, device="cuda"))
        if c["e4m3"]:
            st.update(ks=torch.zeros(pages, Hkv, ps, device="cuda"),
                      vs=torch.zeros(pages, Hkv, ps, device="cuda"))
    elif c["op"] == "attention":
        B, L, Hq, Hkv, D, ps = c["B"], c["L"], c["Hq"], c["Hkv"], c["D"], c["page"]
        lens = torch.full((B,), L, dtype=torch.int64, device="cuda")
        if c["ragged"]:
            lens = (L * _rand(g, B) ** 1.5).long().clamp(1, L)
            if B >= 4:
                lens[1], lens[2], lens[3] = 0, 1, L
        width = -(-L // ps)
        need = (lens + ps - 1) // ps
        pages = max(1, int(need.sum()))
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        first = need.cumsum(0) - need
        col = torch.arange(width, device="cuda")
        table = torch.where(col < need[:, None], order[(first[:, None] + col).clamp(max=pages - 1)],
                            torch.zeros((), dtype=torch.int32, device="cuda")).contiguous()
        st.update(q=(1.5 * _randn(g, B, Hq, D)).to(torch.bfloat16), table=table,
                  lens=lens.to(torch.int32))
        for n in ("k", "v"):
            # in pieces: a long cache takes several times its size in fp32
            parts = torch.empty(pages, Hkv, ps, D, device="cuda",
                                dtype=torch.uint8 if c["e4m3"] else torch.bfloat16)
            scales = torch.empty(pages, Hkv, ps, device="cuda") if c["e4m3"] else None
            for i in range(0, pages, 4096):
                f = _randn(g, min(4096, pages - i), Hkv, ps, D)
                if c["e4m3"]:
                    q, s = _e4m3(f)
                    parts[i:i + 4096], scales[i:i + 4096] = q.view(torch.uint8), s
                else:
                    parts[i:i + 4096] = f.to(torch.bfloat16)
            st[n] = parts
            if c["e4m3"]:
                st[n + "s"] = scales
        st["scale"] = 1.0 / math.sqrt(D)
    else:
        M, N, K = c["M"], c["N"], c["K"]
        x = _randn(g, M, K) * torch.exp(0.5 * _randn(g, K))  # a few strong features, as layers have
        codes = (1.0 * _randn(g, N, K)).to(torch.float8_e4m3fn).view(torch.uint8)
        scales = 0.005 + 0.015 * _rand(g, -(-N // 128), -(-K // 128))
        st.update(x=x.to(torch.bfloat16), codes=codes, scales=scales)
    if own:
        _plan(st)
    return st


def _plan(st):
    """What a serving program sets up once: the operator's handle, its output
    buffers and its workspace."""
    from block_fp8_expert_gb300 import decoder
    c = st["case"]
    if c["op"] == "select":
        st["op"] = decoder.ExpertSelector(
            E=c["E"], k=c["k"], score="sigmoid" if c["sigmoid"] else "softmax", bias=st["bias"],
            groups=c["groups"], top_groups=c["top_groups"], group_top=c["group_top"],
            renorm=c["renorm"], scale=c["scale"])
        st["idx"] = torch.empty(c["T"], c["k"], dtype=torch.int32, device="cuda")
        st["w"] = torch.empty(c["T"], c["k"], dtype=torch.float32, device="cuda")
    elif c["op"] == "qknorm":
        st["cache"] = decoder.PagedCache(st["k"], st["v"], st.get("ks"), st.get("vs"))
        st["op"] = decoder.QkNormRope(
            Hq=c["Hq"], Hkv=c["Hkv"], D=c["D"], q_norm=st["q_norm"], k_norm=st["k_norm"],
            cos_sin=st["cos_sin"], interleaved=c["interleaved"], eps=st["eps"])
        st["q_out"] = torch.empty(c["T"], c["Hq"], c["D"], dtype=torch.bfloat16, device="cuda")
    elif c["op"] == "attention":
        st["cache"] = decoder.PagedCache(st["k"], st["v"], st.get("ks"), st.get("vs"))
        st["op"] = decoder.PagedAttention(Hq=c["Hq"], Hkv=c["Hkv"], D=c["D"], scale=st["scale"],
                                          window=c["window"])
        st["ws"] = st["op"].workspace(c["B"])
        st["out"] = torch.empty(c["B"], c["Hq"], c["D"], dtype=torch.bfloat16, device="cuda")
    else:
        st["op"] = decoder.Fp8Linear(st["codes"], st["scales"])
        st["ws"] = st["op"].workspace(c["M"])
        st["out"] = torch.empty(c["M"], c["N"], dtype=torch.bfloat16, device="cuda")


# ------------------------------------------------------------------ one pass

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _cache_outputs(st):
    if not st["case"]["e4m3"]:
        return {"k": st["k"], "v": st["v"]}
    return {"k": st["k"].view(torch.float8_e4m3fn), "v": st["v"].view(torch.float8_e4m3fn),
            "k_scale": st["ks"], "v_scale": st["vs"]}


def _run_own(st):
    op = st["case"]["op"]
    if op == "select":
        st["op"].forward(st["logits"], st["idx"], st["w"])
        return {"idx": st["idx"], "w": st["w"]}
    if op == "qknorm":
        st["op"].forward(st["qkv"], st["positions"], st["slots"], st["cache"], st["q_out"])
        return {"q": st["q_out"], **_cache_outputs(st)}
    if op == "attention":
        st["op"].forward(st["q"], st["cache"], st["table"], st["lens"], st["out"], st["ws"])
        return {"out": st["out"]}
    st["op"].forward(st["x"], st["out"], st["ws"])
    return {"out": st["out"]}


def _run_plain(st):
    return {"select": _plain_select, "qknorm": _plain_qknorm, "attention": _plain_attention,
            "linear": _plain_linear}[st["case"]["op"]](st)


def _plain_select(st):
    c, l = st["case"], st["logits"]
    T, E, k = c["T"], c["E"], c["k"]
    if c["sigmoid"]:
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        e = torch.exp(l - l.amax(-1, keepdim=True))
        s = e / e.sum(-1, keepdim=True)
    key = s + st["bias"] if st["bias"] is not None else s
    if c["groups"] > 1:
        per = key.view(T, c["groups"], E // c["groups"])
        gs = per.sort(-1, descending=True).values[..., :c["group_top"]].sum(-1)
        best = gs.sort(dim=-1, descending=True, stable=True).indices[:, :c["top_groups"]]
        kept = torch.zeros_like(gs).scatter(1, best, 1.0)
        key = torch.where(kept.unsqueeze(-1) > 0, per, torch.full_like(per, -torch.inf)).view(T, E)
    idx = key.sort(dim=-1, descending=True, stable=True).indices[:, :k]
    w = s.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return {"idx": idx.to(torch.int32), "w": w * c["scale"]}


def _plain_norm_rope(st, x, weight):
    """x [T, heads, D] fp32 -> normed and rotated, fp32."""
    c = st["case"]
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + st["eps"]) * weight
    r = c["rot"]
    cs = st["cos_sin"][st["positions"].long()].unsqueeze(1)
    cos, sin = cs[..., :r // 2], cs[..., r // 2:]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if c["interleaved"] else (x[..., :r // 2], x[..., r // 2:r])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    rot = torch.stack([ra, rb], -1).flatten(-2) if c["interleaved"] else torch.cat([ra, rb], -1)
    return torch.cat([rot, x[..., r:]], -1)


def _plain_qknorm(st):
    c = st["case"]
    T, Hq, Hkv, D, ps = c["T"], c["Hq"], c["Hkv"], c["D"], c["page"]
    x = st["qkv"].float().view(T, Hq + 2 * Hkv, D)
    q = _plain_norm_rope(st, x[:, :Hq], st["q_norm"]).to(torch.bfloat16)
    k = _plain_norm_rope(st, x[:, Hq:Hq + Hkv], st["k_norm"])
    v = x[:, Hq + Hkv:]
    tok = (st["slots"] >= 0).nonzero().squeeze(1)
    page, off = st["slots"][tok] // ps, st["slots"][tok] % ps
    if c["e4m3"]:
        kc, ks = _e4m3(k)
        vc, vs = _e4m3(v)
        st["k"][page, :, off] = kc.view(torch.uint8)[tok]
        st["v"][page, :, off] = vc.view(torch.uint8)[tok]
        st["ks"][page, :, off] = ks[tok]
        st["vs"][page, :, off] = vs[tok]
    else:
        st["k"][page, :, off] = k.to(torch.bfloat16)[tok]
        st["v"][page, :, off] = v.to(torch.bfloat16)[tok]
    return {"q": q, **_cache_outputs(st)}


def _plain_pages(st, n):
    """The sequences' keys or values [B, Hkv, width * page, D], fp32."""
    c = st["case"]
    t = st["table"].long()
    x = st[n][t]
    x = x.view(torch.float8_e4m3fn).float() * st[n + "s"][t].unsqueeze(-1) if c["e4m3"] else x.float()
    return x.transpose(1, 2).reshape(c["B"], c["Hkv"], -1, c["D"])


def _plain_attention(st):
    c = st["case"]
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    q = st["q"].float().view(B, Hkv, Hq // Hkv, D)
    s = (q @ _plain_pages(st, "k").transpose(2, 3)) * st["scale"]
    pos = torch.arange(s.shape[-1], device=s.device)
    lens = st["lens"].long()[:, None, None, None]
    seen = pos < lens
    if c["window"]:
        seen = seen & (pos >= lens - c["window"])
    s = torch.where(seen, s, torch.full_like(s, -torch.inf))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -torch.inf, torch.zeros_like(m), m))
    o = (p @ _plain_pages(st, "v")) / p.sum(-1, keepdim=True)
    o = torch.where(lens > 0, o, torch.zeros_like(o))  # an empty sequence answers zeros
    return {"out": o.reshape(B, Hq, D).to(torch.bfloat16)}


def _plain_linear(st):
    c = st["case"]
    M, N, K = c["M"], c["N"], c["K"]
    Kp = -(-K // 128) * 128
    x = torch.nn.functional.pad(st["x"].float(), (0, Kp - K)).view(M, -1, 128)
    codes, sx = _e4m3(x)
    xq = (codes.float() * sx.unsqueeze(-1)).view(M, Kp)[:, :K]
    sw = st["scales"].repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return {"out": (xq @ (st["codes"].view(torch.float8_e4m3fn).float() * sw).t()).to(torch.bfloat16)}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "select":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": 4 * T * E + (4 * E if c["bias"] else 0) + 8 * T * k, "flops": 4 * T * E}
    if c["op"] == "qknorm":
        T, Hq, Hkv, D, r = c["T"], c["Hq"], c["Hkv"], c["D"], c["rot"]
        kv = 2 * T * Hkv * ((D + 4) if c["e4m3"] else 2 * D)
        return {"bytes": 2 * T * (Hq + 2 * Hkv) * D + 2 * T * Hq * D + kv + T * (4 * r + 12) + 8 * D,
                "flops": T * (Hq + Hkv) * (4 * D + 3 * r) + (4 * T * Hkv * D if c["e4m3"] else 0)}
    if c["op"] == "attention":
        B, L, Hq, Hkv, D = c["B"], c["L"], c["Hq"], c["Hkv"], c["D"]
        # a ragged batch's lengths are L u^1.5: 0.4 L on average (a window cuts them, too)
        w = c["window"] or L
        mean = 0.4 * L if c["ragged"] else L
        if c["ragged"] and w < L:
            f = (w / L) ** (2 / 3)
            mean = 0.4 * L * f ** 2.5 + w * (1 - f)
        tokens = B * min(mean, w)
        per = 2 * Hkv * ((D + 4) if c["e4m3"] else 2 * D)
        return {"bytes": tokens * per + 4 * B * Hq * D + 4 * tokens / c["page"] + 4 * B,
                "flops": 4 * tokens * Hq * D}
    M, N, K = c["M"], c["N"], c["K"]
    return {"bytes": 2 * M * K + N * K + 4 * -(-N // 128) * -(-K // 128) + 2 * M * N,
            "flops": 2 * M * N * K}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """The operators' definitions in 64 bits, on the inputs of prepare()."""
    st = prepare(case, seed)
    c = case
    if c["op"] == "select":
        return _exact_select(st)
    if c["op"] == "qknorm":
        return _exact_qknorm(st)
    if c["op"] == "attention":
        return _exact_attention(st)
    return _exact_linear(st)


def _exact_select(st):
    c = st["case"]
    l = st["logits"].double().cpu().numpy()
    if c["sigmoid"]:
        s = 1.0 / (1.0 + np.exp(-l))
    else:
        s = np.exp(l - l.max(1, keepdims=True))
        s /= s.sum(1, keepdims=True)
    key = s.copy()
    if st["bias"] is not None:
        key += st["bias"].double().cpu().numpy()
    T, E = key.shape
    if c["groups"] > 1:
        n = E // c["groups"]
        score = np.sort(key.reshape(T, c["groups"], n), -1)[:, :, n - c["group_top"]:].sum(-1)
        out = np.argsort(-score, 1, kind="stable")[:, c["top_groups"]:]
        dead = np.zeros((T, c["groups"]), bool)
        np.put_along_axis(dead, out, True, 1)
        key[np.repeat(dead, n, 1)] = -np.inf
    idx = np.argsort(-key, 1, kind="stable")[:, :c["k"]]
    w = np.take_along_axis(s, idx, 1)
    if c["renorm"]:
        w = w / w.sum(1, keepdims=True)
    return {"idx": idx.astype(np.int32), "w": c["scale"] * w}


def _exact_qknorm(st):
    c = st["case"]
    T, Hq, Hkv, D, r, ps = c["T"], c["Hq"], c["Hkv"], c["D"], c["rot"], c["page"]
    x = st["qkv"].double().view(T, Hq + 2 * Hkv, D)
    z = x[:, :Hq + Hkv]
    wt = torch.cat([st["q_norm"].double().expand(Hq, D), st["k_norm"].double().expand(Hkv, D)])
    z = z / torch.sqrt(z.square().sum(-1, keepdim=True) / D + st["eps"]) * wt
    # the rotation as a complex product
    pair = torch.arange(r // 2, device=z.device)
    ia = 2 * pair if c["interleaved"] else pair
    ib = 2 * pair + 1 if c["interleaved"] else pair + r // 2
    cs = st["cos_sin"].double()[st["positions"].long()]
    turn = torch.complex(cs[:, :r // 2], cs[:, r // 2:]).unsqueeze(1)
    y = torch.complex(z[..., ia], z[..., ib]) * turn
    z = z.clone()
    z[..., ia], z[..., ib] = y.real, y.imag
    k, v = torch.zeros_like(st["k"], dtype=torch.float64), torch.zeros_like(st["v"], dtype=torch.float64)
    scales = {}
    for n, dst, src in (("k", k, z[:, Hq:]), ("v", v, x[:, Hq + Hkv:])):
        if c["e4m3"]:
            a = src.abs().amax(-1)
            scales[n + "_scale"] = torch.zeros_like(st["ks"], dtype=torch.float64)
            src = src * (E4M3_MAX / a).unsqueeze(-1)  # before its rounding to E4M3
        for t in (st["slots"] >= 0).nonzero().flatten().split(1024):
            page, off = st["slots"][t] // ps, st["slots"][t] % ps
            dst[page, :, off] = src[t]
            if c["e4m3"]:
                scales[n + "_scale"][page, :, off] = a[t] / E4M3_MAX
    return {"q": z[:, :Hq], "k": k, "v": v, **scales}


def _exact_attention(st):
    c = st["case"]
    B, Hq, Hkv, D, ps = c["B"], c["Hq"], c["Hkv"], c["D"], c["page"]
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
    lens = st["lens"].cpu().tolist()
    for b in range(B):
        n = lens[b]
        lo = max(0, n - c["window"]) if c["window"] else 0
        if n <= lo:
            continue
        t = torch.arange(lo, n, device="cuda")
        page, off = st["table"][b].long()[t // ps], t % ps
        kv = []
        for name in ("k", "v"):
            x = st[name][page, :, off]
            if c["e4m3"]:
                x = x.view(torch.float8_e4m3fn).double() * st[name + "s"][page, :, off].double().unsqueeze(-1)
            kv.append(x.double())
        q = st["q"][b].double().view(Hkv, Hq // Hkv, D)
        s = torch.einsum("hgd,thd->hgt", q, kv[0]) * st["scale"]
        out[b] = torch.einsum("hgt,thd->hgd", torch.softmax(s, -1), kv[1]).reshape(Hq, D)
    return {"out": out}


def _round_e4m3(y):
    """float64 -> the nearest E4M3 value, ties to even, |y| <= 448."""
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(y / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_linear(st):
    c = st["case"]
    M, N, K = c["M"], c["N"], c["K"]
    x = st["x"].float()
    w = st["codes"].view(torch.float8_e4m3fn).double()
    out = torch.zeros(M, N, dtype=torch.float64, device="cuda")
    for b in range(-(-K // 128)):
        g = x[:, 128 * b:128 * (b + 1)]
        a = g.abs().max(1, keepdim=True).values
        # the operator's definition rounds 448 / a, v (448 / a) and a / 448 to fp32
        f = torch.where(a > 0, E4M3_MAX / a, a)
        part = _round_e4m3((g * f).double()) @ w[:, 128 * b:128 * (b + 1)].t()
        rows = st["scales"][:, b].double().repeat_interleave(128)[:N]
        out += part * (a / E4M3_MAX).double() * rows
    return {"out": out}
