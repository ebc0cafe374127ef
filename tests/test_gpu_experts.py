"""The experts on a routing made elsewhere (moe_experts_forward,
DeviceLayer.experts): the layer call's result, the flags that stay, routings
with invalid experts."""
import numpy as np
import pytest

import moe_inputs as mi
from gpu_common import host_layer, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return require_gpu()


def _lib():
    from block_fp8_expert_gb300 import _lib
    return _lib


def _routed(torch, name, T, seed=0):
    """(layer, x, topk_idx, topk_w, the layer call's output)."""
    from block_fp8_expert_gb300.device import DeviceLayer, x_to_device
    host = host_layer(name)
    D = DeviceLayer.from_host(host)
    x = x_to_device(mi.make_tokens(host, T, seed=seed)[0])
    idx = torch.empty(T, D.k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, D.k, device="cuda")
    out = D.forward(x, topk_idx=idx, topk_w=w)
    return D, x, idx, w, out


# streamed experts (fused combine or not, over 4096 pairs), tensor-core GEMM
# (one launch and two, row gather and, in the layer call, token gather)
@pytest.mark.parametrize("name,T", [("tiny", 1), ("tiny", 8), ("tiny", 200), ("tiny", 300), ("tiny", 2100),
                                    ("qwen3moe_decode", 1), ("qwen3moe_decode", 8),
                                    ("qwen3moe_decode", 64), ("qwen3moe_decode", 1100)])
def test_experts_on_the_routers_choice_are_the_layer_call(torch, name, T):
    D, x, idx, w, out = _routed(torch, name, T)
    got = D.experts(x, idx, w)
    D.check()
    assert torch.equal(got, out)


def test_routing_arrays_need_their_elements_alignment_only(torch):
    D, x, idx, w, out = _routed(torch, "tiny", 8)
    i2, w2 = torch.zeros(8 * 2 + 3, dtype=torch.int32, device="cuda"), torch.zeros(8 * 2 + 3, device="cuda")
    i2[1:17].copy_(idx.flatten())
    w2[3:19].copy_(w.flatten())
    assert torch.equal(D.experts(x, i2[1:17].view(8, 2), w2[3:19].view(8, 2)), out)


@pytest.mark.parametrize("name,T", [("tiny", 8), ("tiny", 600), ("qwen3moe_decode", 64)])
def test_flags_of_every_stage_stay(torch, name, T):
    """An expert outside the layer is flagged after the whole chain, and adds
    nothing; so are infinite tokens; neither a clean call nor the workspace's
    own word changes with it."""
    lib = _lib()
    D, x, idx, w, _ = _routed(torch, name, T)
    ws = D.workspace(T)
    ws[:4].view(torch.int32).fill_(lib.MOE_DEV_WAIT_TIMEOUT)  # as a router call on it might have left it
    bad, w0, ok = idx.clone(), w.clone(), idx.clone()
    bad[T // 2, 1], bad[0, 0] = D.E, -1
    w0[T // 2, 1] = w0[0, 0] = 0
    out = D.experts(x, bad, w, ws=ws)
    with pytest.raises(lib.MoeError, match="0x1"):
        D.check()
    assert torch.equal(D.experts(x, ok, w0, ws=ws), out)
    with pytest.raises(lib.MoeError, match="0x1"):
        D.check()
    D.status.zero_()
    D.experts(x, ok, w, ws=ws)
    D.check()
    y = x.clone()
    y[T - 1, 5] = float("inf")
    D.experts(y, ok, w, ws=ws)
    D.experts(x, ok, w, ws=ws)
    with pytest.raises(lib.MoeError, match="device status bits"):
        D.check()
    assert D.status[0].item() & lib.MOE_DEV_NONFINITE
    assert ws[:4].view(torch.int32).item() == lib.MOE_DEV_WAIT_TIMEOUT


@pytest.mark.parametrize("name,T", [("tiny", 1), ("tiny", 40), ("tiny", 1100), ("qwen3moe_decode", 20)])
def test_no_valid_expert_at_all(torch, name, T):
    lib = _lib()
    D, x, idx, w, out = _routed(torch, name, T)
    ws = D.workspace(T)
    ws.fill_(0xFF)
    got = D.experts(x, torch.full_like(idx, D.E + 3), w, torch.full_like(out, 7.0), ws)
    assert (got == 0).all()
    with pytest.raises(lib.MoeError, match="0x1"):
        D.check()
    assert torch.equal(D.experts(x, idx, w, ws=ws), out)
    assert D.experts(x[:0], idx[:0], w[:0]).shape == (0, D.H)


def test_one_expert_chosen_twice(torch):
    """A routing may name an expert twice: its output counts with both weights."""
    D, x, idx, w, _ = _routed(torch, "tiny", 24)
    one = D.experts(x, idx[:, :1].expand(-1, 2).contiguous(), torch.tensor([[0.5, 0.5]], device="cuda").expand(24, 2).contiguous())
    two = D.experts(x, idx, torch.tensor([[1.0, 0.0]], device="cuda").expand(24, 2).contiguous())
    D.check()
    assert torch.equal(one, two)                    # (halves are exact)


def test_experts_in_a_graph_and_on_a_stream(torch):
    D, x, idx, w, out = _routed(torch, "tiny", 24)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = D.experts(x, idx, w, stream=side)
    side.synchronize()
    assert torch.equal(got, out)
    ws, held = D.workspace(24), torch.empty_like(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        D.experts(x, idx, w, held, ws)
    for _ in range(3):
        held.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, out)
    D.check()


def test_example_layer_reports_its_experts(torch):
    """The example's check() reads what the experts' kernels recorded."""
    from examples.decoder_layer import DecoderLayer
    L = DecoderLayer(2, 16, H=256, Hq=4, Hkv=2, D=64, I=128, E=16, k=2, groups=4, top_groups=2, page=4)
    x = torch.randn(2, 256, device="cuda").to(torch.bfloat16)
    L.step(x)
    L.check()
    h = x.clone()
    h[0, 0] = float("nan")
    idx = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    L.moe.experts(h, idx, torch.ones(2, 2, device="cuda"), ws=L.moe_ws)
    L.step(x)
    with pytest.raises(_lib().MoeError, match="0x8"):
        L.check()


# the shared expert streamed with the routed ones or by itself, or on the GEMM
@pytest.mark.parametrize("name,T", [("large_sparse", 1), ("large_sparse", 16), ("large_sparse", 60), ("large_sparse", 256),
                                    ("large_sparse", 1100)])
@pytest.mark.parametrize("gated", [False, True])
def test_layers_with_a_shared_expert(torch, name, T, gated):
    from block_fp8_expert_gb300.device import DeviceLayer, x_to_device
    host = host_layer(name)
    D = DeviceLayer.from_host(host)
    if gated:
        g = torch.Generator(device="cuda")
        g.manual_seed(T)
        D.shared_gate_w = 0.02 * torch.randn(D.H, generator=g, device="cuda")
    x = x_to_device(mi.make_tokens(host, T, seed=1)[0])
    idx = torch.empty(T, D.k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, D.k, device="cuda")
    out = D.forward(x, topk_idx=idx, topk_w=w)
    assert torch.equal(D.experts(x, idx, w), out)
    D.check()
    # the selector's choice on the same layer
    from block_fp8_expert_gb300.decoder import ExpertSelector
    i2, w2 = ExpertSelector(D.E, D.k).route(x, D, D.workspace(T))
    assert torch.equal(i2, idx)
    # (weights within 2^-17 of the router's, through one bf16 rounding)
    got, ref = D.experts(x, i2, w2).double(), out.double()
    assert ((got - ref).abs() <= 2.0 ** -7 * ref.abs() + 2.0 ** -10 * ref.square().mean().sqrt()).all()
    # no valid routed expert: the shared one's output alone, flagged
    alone = D.experts(x, torch.full_like(idx, -1), w)
    same = D.experts(x, idx, torch.zeros_like(w))
    assert torch.equal(alone, same) and (alone != 0).any()
    with pytest.raises(_lib().MoeError, match="0x1"):
        D.check()


@pytest.mark.parametrize("name,T", [("tiny", 8), ("tiny", 300), ("qwen3moe_decode", 200)])
def test_route_keeps_what_the_layer_recorded(torch, name, T):
    """A clean router call neither clears nor adds to the layer's flags, and is
    the call without them (both routers; many warps of tokens)."""
    from block_fp8_expert_gb300 import decoder
    lib = _lib()
    D, x, idx, w, _ = _routed(torch, name, T)
    ws = D.workspace(T)
    ws.fill_(0xFF)
    sel = decoder.ExpertSelector(D.E, D.k)
    i2, w2 = sel.route(x, D, ws)
    D.check()
    D.status[0] = lib.MOE_DEV_NONFINITE
    i3, w3 = sel.route(x, D, ws)
    assert D.status.tolist() == [lib.MOE_DEV_NONFINITE] + [0] * 15
    assert torch.equal(i2, idx) and torch.equal(i3, idx) and torch.equal(w2, w3)
    i4, w4 = torch.empty_like(i2), torch.empty_like(w2)
    lib.moe_route_select(x, D.Wr, D.bias, None, sel.rule, D.dims(T), i4, w4, ws)
    assert torch.equal(i4, idx) and torch.equal(w4, w2)
    assert lib.moe_read_device_status(ws) == 0
