"""The latent and drafted-token objects' host side without a GPU: tensors on the
host that say they are on the device, and a library that notes what it is given."""
import pytest

torch = pytest.importorskip("torch")

from block_fp8_expert_gb300 import _lib, decoder  # noqa: E402
from test_decoder_objects import Fake, Library, elsewhere, fake  # noqa: E402

BF16, I32, I64, U8 = torch.bfloat16, torch.int32, torch.int64, torch.uint8
F32 = torch.float32


@pytest.fixture
def library(monkeypatch):
    L = Library()
    monkeypatch.setattr(_lib, "lib", lambda: L)
    monkeypatch.setattr(decoder, "_current_device", lambda: -1, raising=False)
    monkeypatch.setattr(decoder, "new_on", lambda stream, *shape, dtype, device: fake(*shape, dtype=dtype))
    return L


def tree():
    op = decoder.TreeAttention(4, 2, 64, device="cpu")
    cache = decoder.PagedCache(fake(3, 2, 16, 64, dtype=BF16), fake(3, 2, 16, 64, dtype=BF16))
    return op, dict(q=fake(2, 3, 4, 64, dtype=BF16), cache=cache, block_table=fake(2, 5, dtype=I32),
                    seq_lens=fake(2, dtype=I32), mask=fake(2, 3, dtype=I64), draft_lens=fake(2, dtype=I32),
                    out=fake(2, 3, 4, 64, dtype=BF16), ws=fake(64, dtype=U8), stream=0)


def latent():
    op = decoder.LatentAttention(4, 256, 0.1, device="cpu")
    cache = decoder.LatentCache(fake(3, 16, 320, dtype=BF16), 256)
    return op, dict(q=fake(2, 3, 4, 320, dtype=BF16), cache=cache, block_table=fake(2, 5, dtype=I32),
                    seq_lens=fake(2, dtype=I32), mask=fake(2, 3, dtype=I64), draft_lens=fake(2, dtype=I32),
                    out=fake(2, 3, 4, 256, dtype=BF16), ws=fake(64, dtype=U8), stream=0)


def store():
    op = decoder.LatentStore(4, 256, fake(9, 64, dtype=F32), fake(256, dtype=F32), device="cpu")
    return op, dict(kv=fake(3, 320, dtype=BF16), positions=fake(3, dtype=I32), slots=fake(3, dtype=I64),
                    cache=decoder.LatentCache(fake(3, 16, 320, dtype=BF16), 256), q=fake(3, 4, 64, dtype=BF16),
                    q_out=fake(3, 4, 64, dtype=BF16), rows=fake(3, 320, dtype=BF16), stream=0)


def expanded():
    op = decoder.ExpandedAttention(4, device="cpu")
    return op, dict(q=fake(6, 4, 192, dtype=BF16), k_nope=fake(7, 4, 128, dtype=BF16), k_rope=fake(7, 64, dtype=BF16),
                    v=fake(7, 4, 128, dtype=BF16), cu_q=fake(3, dtype=I32), cu_k=fake(3, dtype=I32),
                    out=fake(6, 4, 128, dtype=BF16), stream=0)


def _bad(t):
    """Tensors in place of t that would be misread."""
    other = F32 if t.dtype in (BF16, I32) else I32
    found = [fake(*t.shape, dtype=other), fake(*t.shape[:-1], t.shape[-1] + 1, dtype=t.dtype),
             elsewhere(*t.shape, dtype=t.dtype), fake(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype)[..., ::2]]
    return found


SKIP = {"cache", "stream", "ws", "block_table"}


@pytest.mark.parametrize("make", [tree, latent, store, expanded])
def test_what_would_be_misread_is_refused(library, make):
    op, good = make()
    op.forward(**good)
    assert len(library.calls) == 1
    for name, t in good.items():
        if name in SKIP or t is None:
            continue
        for bad in _bad(t):
            if name in ("cu_q", "cu_k") and bad.dtype == I32 and bad.is_contiguous() and type(bad) is Fake:
                continue  # (another number of sequences, refused with its partner)
            with pytest.raises((TypeError, ValueError)):
                op.forward(**{**good, name: bad})
    for name in {"block_table", "ws"} & set(good):
        with pytest.raises((TypeError, ValueError)):
            op.forward(**{**good, name: elsewhere(*good[name].shape, dtype=good[name].dtype)})
    assert len(library.calls) == 1
    for bad in (fake(2, dtype=I32), fake(4, dtype=I32)):
        if "cu_k" in good:
            with pytest.raises(ValueError):
                op.forward(**{**good, "cu_k": bad})


@pytest.mark.parametrize("make", [tree, latent, store, expanded])
def test_another_current_device_is_refused(library, monkeypatch, make):
    op, good = make()
    monkeypatch.setattr(decoder, "_current_device", lambda: 1)
    for refused in (lambda: op.forward(**good), op.check, *([lambda: op.workspace(2, 3)] if hasattr(op, "workspace") else [])):
        with pytest.raises(ValueError, match="current device"):
            refused()
    assert not library.calls


def test_caches_of_another_layout_are_refused(library):
    op, good = tree()
    other = decoder.PagedCache(fake(3, 4, 16, 64, dtype=BF16), fake(3, 4, 16, 64, dtype=BF16))
    with pytest.raises(ValueError, match="heads"):
        op.forward(**{**good, "cache": other})
    for make in (latent, store):
        op, good = make()
        with pytest.raises(ValueError, match="256"):
            op.forward(**{**good, "cache": decoder.LatentCache(fake(3, 16, 576, dtype=BF16), 512)})
    for bad in (fake(3, 16, 320, dtype=F32), fake(48, 320, dtype=BF16), fake(3, 16, 640, dtype=BF16)[..., ::2]):
        with pytest.raises((TypeError, ValueError)):
            decoder.LatentCache(bad, 256)
    assert not library.calls


def test_sizes_and_settings_of_each_call(library):
    """The strides that are used, a shared mask, and settings between calls."""
    op, good = tree()
    op.forward(**good)
    op.scale, op.window = 0.5, 9
    op.forward(**{**good, "mask": fake(1, 3, dtype=I64).expand(2, 3), "draft_lens": None})
    (_, a), (_, b) = library.calls
    assert (a[6].B, a[6].n, a[6].mask_stride, a[6].window) == (2, 3, 3, 0)
    assert (b[6].mask_stride, b[6].window, b[6].scale) == (0, 9, 0.5) and b[5] is None
    op, good = store()
    library.calls.clear()
    op.forward(**good)
    op.eps, op.interleaved = 0.5, True
    op.forward(**{**good, "q": None, "q_out": None, "rows": None})
    (_, a), (_, b) = library.calls
    assert (a[6].H, a[6].interleaved) == (4, 0) and (b[6].H, b[6].interleaved, b[6].eps) == (0, 1, 0.5)
    assert b[5] is None and b[8] is None and b[9] is None
    with pytest.raises(ValueError, match="q_out"):
        op.forward(**{**good, "q": None})


def test_what_is_held_is_fixed(library):
    for make, names in ((tree, ("Hq", "Hkv", "D", "status")), (latent, ("H", "R", "status")),
                        (store, ("norm", "cos_sin", "H", "R")), (expanded, ("H", "status"))):
        op, good = make()
        for name in names:
            with pytest.raises(AttributeError, match=name):
                setattr(op, name, fake(8, dtype=F32))
        if "cache" in good:
            with pytest.raises(AttributeError):
                good["cache"].pages = 3
