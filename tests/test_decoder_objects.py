"""The decoder objects' host side without a GPU: tensors on the host that say
they are on the device, and a library that notes what it is given."""
import sys
import threading
import types

import pytest

torch = pytest.importorskip("torch")

from block_fp8_expert_gb300 import _lib, decoder  # noqa: E402

BF16, I32 = torch.bfloat16, torch.int32


class Fake(torch.Tensor):
    """A host tensor that the objects take for a CUDA tensor (its device's
    number is the host's, -1)."""
    is_cuda = property(lambda self: True)


def fake(*shape, dtype):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Fake)


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
