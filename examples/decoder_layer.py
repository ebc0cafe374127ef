"""One decoder layer of a block-FP8 mixture-of-experts model, decoding.

    python examples/decoder_layer.py [--batch 16] [--context 4096] [--steps 50]

A step takes the hidden states of one new token per sequence through

    x' = x + Wo attention(norms and positions(Wqkv norm(x)), cache)
    x'' = x' + experts(norm(x'))

with the projections in block FP8 (Fp8Linear), the head norms, rotary
positions and cache store in one pass (QkNormRope), attention over the paged
cache (PagedAttention), experts chosen by sigmoid scores with a balance bias
in groups (ExpertSelector) and the block-FP8 experts (DeviceLayer).  The two
norms over the hidden size and the residual sums are left to PyTorch.  Weights
are random; the step is captured in a CUDA graph and replayed.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from block_fp8_expert_gb300 import decoder  # noqa: E402
from block_fp8_expert_gb300.device import DeviceFfn, DeviceLayer  # noqa: E402


def fp8_weight(g, n, rows, cols):
    """Random block-FP8 matrices [n, rows, cols]: E4M3 codes and block scales
    that give the weights a standard deviation of about cols^-1/2."""
    codes = torch.randn(n, rows, cols, generator=g, device="cuda").to(torch.float8_e4m3fn)
    scales = (0.75 + 0.5 * torch.rand(n, -(-rows // 128), -(-cols // 128), generator=g,
                                      device="cuda")) * cols ** -0.5
    return codes.view(torch.uint8), scales


class DecoderLayer:
    """The layer's weights and what its decode step needs, set up once."""

    def __init__(self, batch, context, H=2048, Hq=32, Hkv=4, D=128, I=768, E=128, k=8, groups=8,
                 top_groups=4, page=64, e4m3=False, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.B, self.H, self.Hq, self.D, self.page = batch, H, Hq, D, page
        self.norm1, self.norm2 = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")
                                  for _ in range(2))
        codes, scales = fp8_weight(g, 1, (Hq + 2 * Hkv) * D, H)
        self.qkv = decoder.Fp8Linear(codes[0], scales[0])
        codes, scales = fp8_weight(g, 1, H, Hq * D)
        self.o = decoder.Fp8Linear(codes[0], scales[0])
        q_norm, k_norm = (1 + 0.1 * torch.randn(D, generator=g, device="cuda") for _ in range(2))
        per_seq = -(-context // page)
        self.rope = decoder.QkNormRope(Hq, Hkv, D, q_norm, k_norm,
                                       decoder.rope_cos_sin(per_seq * page, D))
        self.cache = decoder.PagedCache.empty(batch * per_seq, Hkv, page, D, e4m3)
        self.attention = decoder.PagedAttention(Hq, Hkv, D)
        Wr = 0.02 * torch.randn(E, H, generator=g, device="cuda")
        bias = 0.02 * torch.randn(E, generator=g, device="cuda")
        self.select = decoder.ExpertSelector(E, k, "sigmoid", bias, groups, top_groups, 2,
                                             renorm=True, scale=1.0)
        (gc, gs), (uc, us), (dc, ds) = (fp8_weight(g, E, *s) for s in ((I, H), (I, H), (H, I)))
        self.moe = DeviceLayer(H, I, E, k, 0, Wr, None, DeviceFfn(gc, gs, uc, us, dc, ds), None)
        # the sequences' pages, scattered over the cache
        order = torch.randperm(batch * per_seq, generator=g, device="cuda").to(torch.int32)
        self.table = order.view(batch, per_seq).contiguous()
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.attn_ws = self.attention.workspace(batch)
        self.qkv_ws, self.o_ws = self.qkv.workspace(batch), self.o.workspace(batch)
        self.moe_ws = self.moe.workspace(batch)

    @staticmethod
    def rms_norm(x, weight):
        f = x.float()
        return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6) * weight).to(x.dtype)

    def step(self, x):
        """x bf16 [B, H], the new tokens' hidden states -> the layer's output;
        the tokens join the cache and self.lens grows by one."""
        pos = self.lens.clone()  # (at most context - 1: the cache has room)
        self.lens += 1
        page = self.table.gather(1, (pos // self.page).long().unsqueeze(1)).squeeze(1)
        slots = page.long() * self.page + pos % self.page
        qkv = self.qkv.forward(self.rms_norm(x, self.norm1), ws=self.qkv_ws)
        q = self.rope.forward(qkv, pos, slots, self.cache)
        a = self.attention.forward(q, self.cache, self.table, self.lens, ws=self.attn_ws)
        x = x + self.o.forward(a.view(self.B, self.Hq * self.D), ws=self.o_ws)
        h = self.rms_norm(x, self.norm2)
        idx, w = self.select.route(h, self.moe, self.moe_ws)
        return x + self.moe.experts(h, idx, w, ws=self.moe_ws)

    def check(self):
        """Raise if a kernel flagged its data."""
        for op in (self.qkv, self.rope, self.attention, self.o, self.moe):
            op.check()


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--batch", type=int, default=16)
    p.add_argument("--context", type=int, default=4096)
    p.add_argument("--steps", type=int, default=50)
    p.add_argument("--e4m3-cache", action="store_true")
    a = p.parse_args()
    layer = DecoderLayer(a.batch, a.context, e4m3=a.e4m3_cache)
    start = a.context - a.steps - 4
    if start < 0:
        p.error("the context has no room for the steps")
    x = torch.randn(a.batch, layer.H, device="cuda").to(torch.bfloat16)
    # a history: random keys and values up to where decoding starts
    shape = layer.cache.k.shape
    if a.e4m3_cache:
        for t in (layer.cache.k, layer.cache.v):
            t.copy_(torch.randn(shape, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8))
        layer.cache.k_scale.fill_(1.0)
        layer.cache.v_scale.fill_(1.0)
    else:
        layer.cache.k.normal_()
        layer.cache.v.normal_()
    layer.lens.fill_(start)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step(x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.step(x)
    graph.replay()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(a.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    layer.check()
    ms = begin.elapsed_time(end) / a.steps
    print(f"batch {a.batch}, about {start} tokens of history each, "
          f"{'E4M3' if a.e4m3_cache else 'bf16'} cache: {ms * 1e3:.1f} us per step, "
          f"{a.batch / ms * 1e3:.0f} tokens/s through this layer; output rms "
          f"{out.float().square().mean().sqrt().item():.3f}")


if __name__ == "__main__":
    main()
