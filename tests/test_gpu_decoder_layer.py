"""The decoder operators together: the example's layer decodes several tokens
of several sequences from an empty cache, and every step agrees with a float64
layer that keeps its own contiguous history.

Both sides take the same hidden states at every step, and each operator's
float64 form takes the GPU's values of the operator before it: a projection's
input rounds to E4M3, where a difference of one bf16 rounding can move a value
by a sixteenth.  The operators are held to the layer tolerance of 1e-2 (|ref| +
rms) that the MoE layer has; the step itself gives the bits of the operators
called one by one."""
import math
import subprocess
import sys
import os

import pytest

from gpu_common import require_gpu

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _dense_weight(torch, codes, scales):
    w = codes.view(torch.float8_e4m3fn).double()
    s = scales.double().repeat_interleave(128, -2).repeat_interleave(128, -1)
    return w * s[..., :w.shape[-2], :w.shape[-1]]


def _quantised(torch, x):
    """The values that E4M3 quantisation per row and 128 columns gives x."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for b in range(0, x.shape[1], 128):
        g = x[:, b:b + 128].float()
        a = g.abs().amax(1, keepdim=True)
        f = torch.where(a > 0, 448 * a.reciprocal(), a)
        out[:, b:b + 128] = (g * f).to(torch.float8_e4m3fn).double() * (a.double() / 448)
    return out


@pytest.mark.parametrize("e4m3", [False, True])
def test_decoding_layer_matches_float64(e4m3):
    torch = require_gpu()
    from examples.decoder_layer import DecoderLayer
    B, H, Hq, Hkv, D, E, k, groups, top = 3, 256, 4, 2, 64, 16, 2, 4, 2
    L = DecoderLayer(B, 40, H, Hq, Hkv, D, 128, E, k, groups, top, page=4, e4m3=e4m3, seed=7)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    Wqkv, Wo = (_dense_weight(torch, w.codes, w.scales) for w in (L.qkv, L.o))
    f = L.moe.routed
    Wg, Wu, Wd = (_dense_weight(torch, c, s) for c, s in (
        (f.gate_codes, f.gate_scales), (f.up_codes, f.up_scales), (f.down_codes, f.down_scales)))
    keys = torch.zeros(B, 0, Hkv, D, dtype=torch.float64, device="cuda")
    vals = torch.zeros_like(keys)

    def norm(x, w):
        return x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.double()

    def rotate(x, p):
        cos, sin = L.rope.cos_sin[p].double().split(D // 2)
        a, b = x[..., :D // 2], x[..., D // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    def kept(c, scales, slots):  # the rows that the cache holds for these slots
        r = c[slots // 4, :, slots % 4]
        if not e4m3:
            return r.double()
        return r.view(torch.float8_e4m3fn).double() * scales[slots // 4, :, slots % 4].double().unsqueeze(-1)

    def close_kept(got, ref, what):
        """bf16: half of a 2^-7 step; E4M3: half of a 2^-3 step, or of the
        subnormals' 2^-9 of the scale; and fp32 noise of the row's largest."""
        top = ref.abs().amax(-1, keepdim=True)
        bound = torch.maximum(2.0 ** -4 * ref.abs(), 2.0 ** -10 * top / 448) if e4m3 else 2.0 ** -8 * ref.abs()
        assert ((got - ref).abs() <= bound + 1e-5 * top).all(), what

    def close(got, ref, what):
        got, ref = got.double(), ref.double()
        bound = 1e-2 * (ref.abs() + ref.square().mean().sqrt())
        assert ((got - ref).abs() <= bound).all(), (what, ((got - ref).abs() / bound).max().item())

    for step in range(9):
        x = torch.randn(B, H, generator=g, device="cuda").to(torch.bfloat16)
        out = L.step(x)
        # the same, operator by operator
        L.lens -= 1
        pos = L.lens.clone()
        L.lens += 1
        slots = L.table[:, step // 4].long() * 4 + step % 4
        h = L.rms_norm(x, L.norm1)
        qkv = L.qkv.forward(h)
        q = L.rope.forward(qkv, pos, slots, L.cache)
        a = L.attention.forward(q, L.cache, L.table, L.lens)
        y = x + L.o.forward(a.view(B, Hq * D))
        h2 = L.rms_norm(y, L.norm2)
        idx, w = L.select.route(h2, L.moe, L.moe_ws)
        assert torch.equal(out, y + L.moe.experts(h2, idx, w))
        L.check()
        # against float64
        close(qkv, _quantised(torch, h) @ Wqkv.t(), "qkv")
        heads = qkv.double().view(B, Hq + 2 * Hkv, D)
        close(q, rotate(norm(heads[:, :Hq], L.rope.q_norm), step), "q")
        kn = rotate(norm(heads[:, Hq:Hq + Hkv], L.rope.k_norm), step)
        kc, vc = kept(L.cache.k, L.cache.k_scale, slots), kept(L.cache.v, L.cache.v_scale, slots)
        close_kept(kc, kn, "cached keys")
        close_kept(vc, heads[:, Hq + Hkv:], "cached values")
        keys = torch.cat([keys, kc.unsqueeze(1)], 1)
        vals = torch.cat([vals, vc.unsqueeze(1)], 1)
        s = torch.einsum("bhgd,bthd->bhgt", q.double().view(B, Hkv, Hq // Hkv, D), keys) / math.sqrt(D)
        close(a, torch.einsum("bhgt,bthd->bhgd", torch.softmax(s, -1), vals).reshape(B, Hq, D), "attention")
        close(y, x.double() + _quantised(torch, a.view(B, Hq * D)) @ Wo.t(), "o")
        score = torch.sigmoid(h2.double() @ L.moe.Wr.double().t())
        key = (score + L.select.bias.double()).view(B, groups, -1)
        gs = key.topk(2, -1).values.sum(-1)
        srt = gs.sort(1, descending=True)
        keep = torch.zeros_like(gs).scatter(1, srt.indices[:, :top], 1.0).unsqueeze(-1) > 0
        flat = key.masked_fill(~keep, -math.inf).flatten(1).sort(1, descending=True)
        clear = (srt.values[:, top - 1] - srt.values[:, top] > 1e-4) & (
            flat.values[:, :k] - flat.values[:, 1:k + 1] > 1e-4).all(1)
        assert (idx[clear] == flat.indices[clear, :k]).all()
        ws = score.gather(1, idx.long())
        close(w, ws / ws.sum(1, keepdim=True), "weights")
        ref = y.double().clone()
        for b in range(B):
            for j in range(k):
                e = idx[b, j]
                hid = torch.nn.functional.silu(Wg[e] @ h2[b].double()) * (Wu[e] @ h2[b].double())
                ref[b] += w[b, j].double() * (Wd[e] @ hid)
        close(out, ref, "layer")
    assert (L.lens == 9).all()


def test_route_select_matches_route_and_its_own_logits():
    """moe_route_select over all experts is moe_route; with a rule it is
    moe_select_experts on the same logits (both sizes of router)."""
    torch = require_gpu()
    import moe_inputs as mi
    from block_fp8_expert_gb300 import _lib, decoder
    from block_fp8_expert_gb300.device import DeviceLayer, x_to_device
    layer = mi.make_layer("tiny", seed=2)
    D = DeviceLayer.from_host(layer)
    for T in (1, 7, 200):
        xb, _ = mi.make_tokens(layer, T, seed=T)
        x = x_to_device(xb)
        ws = D.workspace(T)
        idx0 = torch.empty(T, layer.k, dtype=torch.int32, device="cuda")
        w0 = torch.empty(T, layer.k, device="cuda")
        _lib.moe_route(x, D.Wr, D.bias, D.dims(T), idx0, w0, ws)
        idx, w = decoder.ExpertSelector(layer.E, layer.k).route(x, D, ws)
        assert torch.equal(idx, idx0)
        assert torch.allclose(w, w0, rtol=1e-5)
        # (the inputs keep the logits' gaps above 1e-4, so the scores' order is
        # that of the logits on either side)
        logits = (x.double() @ D.Wr.double().t()).float()
        sel = decoder.ExpertSelector(layer.E, layer.k, "sigmoid", None, 1, 1, 1, False, 2.5)
        idx, w = sel.route(x, D, ws)
        idx1, w1 = sel.forward(logits)
        assert torch.equal(idx, idx1) and torch.allclose(w, w1, rtol=1e-4)
    with pytest.raises(ValueError):
        decoder.ExpertSelector(8, 2).route(x, D, ws)
    with pytest.raises(_lib.MoeError):
        sel.route(x, D, ws[:100])


@pytest.mark.parametrize("extra", [[], ["--e4m3-cache"]])
def test_example_runs(extra):
    require_gpu()
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "decoder_layer.py"),
                        "--batch", "4", "--context", "512", "--steps", "5", *extra],
                       capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "us per step" in r.stdout
