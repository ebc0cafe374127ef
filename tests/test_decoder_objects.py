"""The decoder objects' host side without a GPU: tensors on the host that say
they are on the device, and a library that notes what it is given."""
import sys
import threading
import types

import pytest

torch = pytest.importorskip("torch")

from block_fp8_expert_gb300 import _lib, decoder, device  # noqa: E402

BF16, I32 = torch.bfloat16, torch.int32


class Fake(torch.Tensor):
    """A host tensor that the objects take for a CUDA tensor (its device's
    number is the host's, -1)."""
    is_cuda = property(lambda self: True)


def fake(*shape, dtype):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Fake)


class Elsewhere(Fake):
    """The same on another device than the other tensors."""

    def get_device(self):
        return 3


def elsewhere(*shape, dtype):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Elsewhere)


class Library:
    """In place of the library: notes each call's arguments."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    L = Library()
    monkeypatch.setattr(_lib, "lib", lambda: L)
    monkeypatch.setattr(decoder, "_current_device", lambda: -1, raising=False)
    monkeypatch.setattr(device, "_current_device", lambda: -1, raising=False)
    return L


def linear():
    op = decoder.Fp8Linear(fake(64, 128, dtype=torch.uint8), fake(1, 1, dtype=torch.float32))

    def call(M):
        op.forward(call.x(M), fake(M, 64, dtype=BF16), fake(256, dtype=torch.uint8), stream=0)
    call.x = lambda M: fake(M, 128, dtype=BF16)
    return op, call, lambda dims: dims.M


def attention():
    op = decoder.PagedAttention(4, 2, 64, device="cpu")
    cache = decoder.PagedCache(fake(3, 2, 16, 64, dtype=BF16), fake(3, 2, 16, 64, dtype=BF16))

    def call(B):
        op.forward(call.x(B), cache, fake(B, 2, dtype=I32), fake(B, dtype=I32), fake(B, 4, 64, dtype=BF16),
                   fake(256, dtype=torch.uint8), stream=0)
    call.x = lambda B: fake(B, 4, 64, dtype=BF16)
    return op, call, lambda dims: dims.B


def norm():
    op = decoder.QkNormRope(4, 2, 64, device="cpu")
    cache = decoder.PagedCache(fake(3, 2, 16, 64, dtype=BF16), fake(3, 2, 16, 64, dtype=BF16))

    def call(T):
        op.forward(call.x(T), None, fake(T, dtype=torch.int64), cache, fake(T, 4, 64, dtype=BF16), stream=0)
    call.x = lambda T: fake(T, 512, dtype=BF16)
    return op, call, lambda dims: dims.T


def sizes(library, of):
    """The number of rows that each call was given."""
    kinds = (_lib.LinearDims, _lib.AttnDims, _lib.QkDims)
    return [of(next(a for a in args if isinstance(a, kinds))) for _, args in library.calls]


@pytest.mark.parametrize("make", [linear, attention, norm])
def test_a_call_between_another_calls_lines(library, make):
    """A call of another size, as from another thread, while a call gathers its
    arguments: each reaches the library with its own size, then and later."""
    op, call, of = make()

    class Interrupting(Fake):
        def data_ptr(self):
            if not seen:
                seen.append(1)
                inner(7)
            return super().data_ptr()

    seen, plain = [], call.x

    def inner(n):
        call.x = plain
        call(n)

    call.x = lambda n: plain(n).as_subclass(Interrupting)
    call(3)
    assert sizes(library, of) == [7, 3]
    call.x = plain
    for n in (3, 7, 3):
        call(n)
    assert sizes(library, of) == [7, 3, 3, 7, 3]


@pytest.mark.parametrize("make", [linear, attention, norm])
def test_threads_share_an_object(make, monkeypatch):
    """Two threads, two sizes, one object: every call is given the size of the
    tensor that it is given."""
    wrong, mine = [], threading.local()
    kinds = (_lib.LinearDims, _lib.AttnDims, _lib.QkDims)

    def check(*args):
        if of(next(a for a in args if isinstance(a, kinds))) != mine.n:
            wrong.append(mine.n)
        return 0

    monkeypatch.setattr(_lib, "lib", lambda: types.SimpleNamespace(
        moe_linear_fp8=check, moe_paged_attention=check, moe_qk_norm_rope=check))
    monkeypatch.setattr(decoder, "_current_device", lambda: -1, raising=False)
    op, call, of = make()

    def work(n):
        mine.n = n
        for _ in range(300):
            call(n)

    before = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        threads = [threading.Thread(target=work, args=(n,)) for n in (2, 5)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(before)
    assert not wrong


def test_settings_take_effect_at_the_next_call(library):
    """scale, window, eps and interleaved, set again between calls of one size."""
    op, call, _ = attention()
    call(2)
    op.window, op.scale = 5, 0.25
    call(2)
    a, b = (args[4] for _, args in library.calls)
    assert (a.window, a.scale) == (0, 0.125) and (b.window, b.scale) == (5, 0.25)
    library.calls.clear()
    op, call, _ = norm()
    call(2)
    op.eps, op.interleaved = 0.5, True
    call(2)
    a, b = (args[6] for _, args in library.calls)
    assert a.interleaved == 0 and (b.eps, b.interleaved) == (0.5, 1)


def test_what_is_held_as_addresses_and_sizes_is_fixed(library):
    """Another tensor or size in place of one whose address or value the object
    holds is refused, not ignored (the old tensor's memory may be gone)."""
    f32 = torch.float32
    lin, attn, rope = linear()[0], attention()[0], norm()[0]
    sel = decoder.ExpertSelector(8, 2, bias=fake(8, dtype=f32))
    cache = decoder.PagedCache(fake(3, 2, 16, 64, dtype=BF16), fake(3, 2, 16, 64, dtype=BF16))
    for op, names in ((lin, ("codes", "scales", "bias", "N", "K", "status")), (attn, ("Hq", "Hkv", "D", "status")),
                      (rope, ("q_norm", "k_norm", "cos_sin", "rot", "n_pos", "width")),
                      (sel, ("bias", "E", "k", "rule")), (cache, ("k", "v", "k_scale", "pages", "page_size"))):
        for name in names:
            was = getattr(op, name)
            with pytest.raises(AttributeError, match=name):
                setattr(op, name, fake(8, dtype=f32))
            assert getattr(op, name) is was
    sel.bias.fill_(1.0)  # in place, as a balance bias is kept
    sel.rule.scale = 2.0


def selector():
    op = decoder.ExpertSelector(8, 2)

    def call(T):
        op.forward(call.x(T), fake(T, 2, dtype=I32), fake(T, 2, dtype=torch.float32), stream=0)
    call.x = lambda T: OnDevice0.zeros(T, 8)
    return op, call


class OnDevice0(Fake):
    def get_device(self):
        return 0

    @staticmethod
    def zeros(*shape):
        return torch.zeros(*shape, dtype=torch.float32).as_subclass(OnDevice0)


@pytest.mark.parametrize("make", [linear, attention, norm])
def test_another_current_device_is_refused(library, monkeypatch, make):
    """The library launches on the current device: tensors of another one never
    reach it."""
    op, call, _ = make()
    call(2)
    monkeypatch.setattr(decoder, "_current_device", lambda: 1)
    library.calls.clear()
    for refused in (lambda: call(2), op.check, *([lambda: op.workspace(2)] if hasattr(op, "workspace") else [])):
        with pytest.raises(ValueError, match="current device"):
            refused()
    assert not library.calls


def test_selector_on_another_current_device_is_refused(library, monkeypatch):
    monkeypatch.setattr(decoder, "_current_device", lambda: 1)
    op, call = selector()
    with pytest.raises(ValueError, match="current device"):
        call(2)
    assert not library.calls


def _layer(**kw):
    at = dict(E=8, k=2, H=64, Wr=fake(8, 64, dtype=torch.float32), bias=None, dims=lambda T: _lib.dims(T, 64, 64, 8, 2),
              status=fake(16, dtype=I32))
    at.update(kw)
    return types.SimpleNamespace(**at)


def test_tensors_of_several_devices_are_refused(library):
    """At set-up and in a call; nothing reaches the library."""
    f32, u8 = torch.float32, torch.uint8
    codes, table = fake(64, 128, dtype=u8), fake(9, 32, dtype=f32)
    for scales, bias in ((elsewhere(1, 1, dtype=f32), None), (fake(1, 1, dtype=f32), elsewhere(64, dtype=f32))):
        with pytest.raises(ValueError, match="device 3"):
            decoder.Fp8Linear(codes, scales, bias)
    for bad in (dict(q_norm=elsewhere(64, dtype=f32)), dict(k_norm=elsewhere(64, dtype=f32)),
                dict(cos_sin=table.as_subclass(Elsewhere))):
        with pytest.raises(ValueError, match="device 3"):
            decoder.QkNormRope(4, 2, 64, device="cpu", **bad)
    x, ws = fake(3, 64, dtype=BF16), fake(1 << 16, dtype=u8)
    idx, w, bias = fake(3, 2, dtype=I32), fake(3, 2, dtype=f32), fake(8, dtype=f32)
    plain, biased = decoder.ExpertSelector(8, 2, bias=bias), decoder.ExpertSelector(8, 2, bias=elsewhere(8, dtype=f32))
    plain.route(x, _layer(), ws, idx, w, stream=0)
    for op, layer, ws_, idx_, w_ in (
            (biased, _layer(), ws, idx, w), (plain, _layer(Wr=elsewhere(8, 64, dtype=f32)), ws, idx, w),
            (plain, _layer(bias=elsewhere(8, dtype=f32)), ws, idx, w),
            (plain, _layer(), elsewhere(1 << 16, dtype=u8), idx, w),
            (plain, _layer(), ws, elsewhere(3, 2, dtype=I32), w), (plain, _layer(), ws, idx, elsewhere(3, 2, dtype=f32))):
        with pytest.raises(ValueError, match="device"):
            op.route(x, layer, ws_, idx_, w_, stream=0)
    assert len(library.calls) == 1


def test_selector_bias_of_another_device_is_refused(library, monkeypatch):
    monkeypatch.setattr(decoder, "_current_device", lambda: 0)
    op = decoder.ExpertSelector(8, 2, bias=elsewhere(8, dtype=torch.float32))
    with pytest.raises(ValueError, match="bias is on device 3"):
        op.forward(OnDevice0.zeros(2, 8), stream=0)
    assert not library.calls


def _moe_layer():
    f32, u8 = torch.float32, torch.uint8
    I, E, H = 64, 8, 64
    routed = device.DeviceFfn(*(fake(E, *s, dtype=t) for m in ((I, H), (I, H), (H, I))
                                for s, t in ((m, u8), ((1, 1), f32))))
    return device.DeviceLayer(H, I, E, 2, 0, fake(E, H, dtype=f32), None, routed, None)


def test_experts_refuse_what_they_would_misread(library, monkeypatch):
    """A routing made elsewhere in another type (torch.topk's indices are int64),
    shape, layout or place, and tokens or results likewise: refused, and nothing
    reaches the library."""
    f32, u8 = torch.float32, torch.uint8
    L = _moe_layer()
    good = dict(x=fake(4, 64, dtype=BF16), topk_idx=fake(4, 2, dtype=I32), topk_w=fake(4, 2, dtype=f32),
                out=fake(4, 64, dtype=BF16), ws=fake(1 << 16, dtype=u8), stream=0)
    # (the scratch comes from the CUDA allocator)
    monkeypatch.setattr(device, "new_on", lambda stream, *shape, dtype, device: fake(*shape, dtype=dtype))
    L.experts(**good)
    assert library.calls
    library.calls.clear()
    bad = dict(
        x=[fake(4, 64, dtype=f32), fake(4, 32, dtype=BF16), fake(4, 128, dtype=BF16)[:, ::2], fake(64, 4, dtype=BF16).t(),
           torch.zeros(4, 64, dtype=BF16)],
        topk_idx=[fake(4, 2, dtype=torch.int64), fake(4, 3, dtype=I32), fake(3, 2, dtype=I32), fake(2, 4, dtype=I32).t(),
                  torch.zeros(4, 2, dtype=I32), elsewhere(4, 2, dtype=I32), None],
        topk_w=[fake(4, 2, dtype=BF16), fake(4, 1, dtype=f32), fake(4, 4, dtype=f32)[:, :2], elsewhere(4, 2, dtype=f32), None],
        out=[fake(4, 64, dtype=f32), fake(3, 64, dtype=BF16), fake(4, 65, dtype=BF16)[:, :64], elsewhere(4, 64, dtype=BF16)],
        ws=[fake(256, 256, dtype=u8).t()[:, ::2], elsewhere(1 << 16, dtype=u8)])
    for name, values in bad.items():
        for v in values:
            with pytest.raises((TypeError, ValueError), match=name):
                L.experts(**{**good, name: v})
    monkeypatch.setattr(device, "_current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        L.experts(**good)
    assert not library.calls


def test_route_records_in_the_layers_status(library):
    """What a router call finds goes to the layer's own array, which no later
    call on the workspace clears."""
    L = _moe_layer()
    decoder.ExpertSelector(8, 2).route(fake(3, 64, dtype=BF16), L, fake(1 << 16, dtype=torch.uint8),
                                       fake(3, 2, dtype=I32), fake(3, 2, dtype=torch.float32), stream=0)
    (name, args), = library.calls
    assert L.status.data_ptr() in args
