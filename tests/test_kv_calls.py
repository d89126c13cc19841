"""What the PyTorch side of cached decoding refuses, and what it hands to the C ABI, on the
host: CPU tensors that say they are on device 0, and a library that takes notes."""

import pytest

torch = pytest.importorskip("torch")

from dense_decoder_layer_gb300 import kv, pds


class Cuda(torch.Tensor):
    def get_device(self):
        return 0


def cuda(t):
    return t.as_subclass(Cuda)


class Notes:
    """Stands for libpds.so: every entry point succeeds and its arguments are kept."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append((name, args)) or 0


@pytest.fixture
def lib(monkeypatch):
    notes = Notes()
    monkeypatch.setattr(pds, "load", lambda: notes)
    monkeypatch.setattr(kv, "_current_device", lambda: 0)
    monkeypatch.setattr(kv, "_raw_stream", lambda device: 0)
    return notes


def make_cache(fmt="bf16", n=2, cap=16, hkv=2, hd=64):
    k = torch.zeros(n, cap, hkv, hd, dtype=torch.bfloat16)
    cache = kv.KvCache(fmt, n, cap, hkv, hd, k=k, v=k.clone(),
                       lens=torch.zeros(n, dtype=torch.int32))
    cache.index = 0
    return cache


def rows(*shape):
    return cuda(torch.zeros(*shape, dtype=torch.bfloat16))


def test_a_workspace_has_to_be_memory_of_the_device(lib):
    cache, q = make_cache(), rows(2, 1, 4, 64)
    good = cuda(torch.empty(64, dtype=torch.int32))
    cache.attend(q, out=rows(2, 1, 4, 64), workspace=good)
    assert lib.calls[-1][1][-3:-1] == (good.data_ptr(), 256)  # bytes
    for bad in (torch.empty(256, dtype=torch.uint8),                       # of the host
                cuda(torch.empty(1, dtype=torch.uint8)).expand(1 << 20),   # one byte
                cuda(torch.empty(512, dtype=torch.uint8))[::2]):
        with pytest.raises(ValueError, match="workspace"):
            cache.attend(q, out=rows(2, 1, 4, 64), workspace=bad)
    assert len(lib.calls) == 1


@pytest.mark.parametrize("far", [2 ** 32, 2 ** 31, 2 ** 32 + 3, -2 ** 31 - 1])
def test_numbers_past_32_bits_are_refused(lib, far):
    """ctypes would keep the low 32 bits: a window of 2^32 would be none."""
    cache, spec = make_cache(), kv.RopeSpec(1.0e4, 64)
    q = rows(2, 1, 4, 64)
    ws = cuda(torch.empty(64, dtype=torch.uint8))
    calls = [lambda: cache.attend(q, out=rows(2, 1, 4, 64), workspace=ws, window=far),
             lambda: cache.attend(q, out=rows(2, 1, 4, 64), workspace=ws, max_len=far),
             lambda: cache.read(far, 4, k_out=rows(2, 4, 2, 64), v_out=rows(2, 4, 2, 64)),
             lambda: kv.rope(q, spec, start_pos=far, out=rows(2, 1, 4, 64)),
             lambda: kv.RopeSpec(1.0e4, 64, rot_dim=far), lambda: kv.RopeSpec(1.0e4, 64, orig_context=far),
             lambda: kv.KvCache("bf16", 2, far, 2, 64), lambda: kv.KvCache("bf16", far, 2, 2, 64)]
    for call in calls:
        with pytest.raises(ValueError, match="32 bits"):
            call()
    many = cuda(torch.empty(1, dtype=torch.bfloat16)).expand(abs(far), 1, 64)
    many.is_contiguous = lambda: True
    with pytest.raises(ValueError, match="32 bits"):
        kv.rope(many, spec, out=many)
    for number in (2 ** 31 - 1, 5):
        cache.attend(q, out=rows(2, 1, 4, 64), window=number, workspace=ws)
        kv.rope(q, spec, start_pos=-number, out=rows(2, 1, 4, 64))
    assert [name for name, _ in lib.calls] == ["pds_attention_tree", "pds_rope"] * 2


def test_tensors_that_require_a_gradient_are_refused(lib):
    """The results would lack it without a word."""
    cache, spec = make_cache(), kv.RopeSpec(1.0e4, 64)
    ws = cuda(torch.empty(64, dtype=torch.uint8))
    q, k = rows(2, 1, 4, 64).requires_grad_(), rows(2, 1, 2, 64).requires_grad_()
    plain = rows(2, 1, 2, 64)
    calls = [lambda: kv.rope(q, spec, out=rows(2, 1, 4, 64)), lambda: cache.write(k, plain),
             lambda: cache.write(plain, k),
             lambda: cache.attend(q, out=rows(2, 1, 4, 64), workspace=ws)]
    for call in calls:
        with pytest.raises(ValueError, match="gradient"):
            call()
    assert not lib.calls
    with torch.no_grad():
        for call in calls:
            call()
    assert len(lib.calls) == 4


def test_the_tensors_of_a_cache_cannot_be_replaced():
    """The C ABI's struct holds their addresses: another tensor in their place would not be
    used, and the old one's memory could be gone."""
    cache = make_cache()
    for name in ("k", "v", "k_scale", "v_scale"):
        with pytest.raises(AttributeError):
            setattr(cache, name, torch.zeros_like(cache.k))
    cache.k[0, 0] = 1.0
    assert cache.c.k == cache.k.data_ptr() and cache.c.v == cache.v.data_ptr()
