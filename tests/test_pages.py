"""The paged cache on the host: what the entry points and the PyTorch side refuse before any
device work, and the oracle's definitions."""

import ctypes
import math
import os

import numpy as np
import pytest

from dense_decoder_layer_gb300 import pds
from oracle import decode as D
from oracle import pages as P

torch = pytest.importorskip("torch")

from dense_decoder_layer_gb300 import kv, pages
from test_kv_calls import cuda, lib, make_cache  # noqa: F401 (a fixture)

needs_lib = pytest.mark.skipif(not os.path.exists(pds.LIB_PATH), reason="libpds.so not built")
PTR = 0x10000


def _pages(**kw):
    c = pds.pds_pages(pds.PDS_KV_E4M3, 2, 10, 16, 8, 2, 128, 0, 0, 0, 0, *[PTR] * 9)
    for f, x in kw.items():
        setattr(c, f, x)
    return c


def _calls(lib, c):
    rows = [lib.pds_pages_write(c, None, PTR, PTR, PTR, 1, 0, 0, None, None),
            lib.pds_pages_read(c, PTR, 1, PTR, PTR, None),
            lib.pds_pages_attend(c, None, PTR, 2 * PTR, 4, 0, 0, 0.0, 0, PTR, 1 << 30, None)]
    book = [lib.pds_pages_reserve(c, PTR, 1, PTR, PTR, PTR, None),
            lib.pds_pages_release(c, PTR, None)]
    return rows, book + [lib.pds_pages_slots(c, PTR, PTR, 1, PTR, PTR, PTR, None)]


def _admitted(call):
    """Whether a call got as far as its buffers: no device here, or none of its memory."""
    return call == pds.PDS_ELAUNCH or "memory of the current device" in pds.last_error()


@needs_lib
@pytest.mark.parametrize("kw,want", [
    (dict(format=3), "EINVAL"), (dict(format=-1), "EINVAL"), (dict(reserved=1), "EINVAL"),
    (dict(n_seqs=0), "EINVAL"), (dict(n_pages=0), "EINVAL"), (dict(page_size=-16), "EINVAL"),
    (dict(max_pages=0), "EINVAL"), (dict(n_kv_heads=0), "EINVAL"), (dict(head_dim=96), "DECLINED"),
    (dict(page_size=4), "DECLINED"), (dict(page_size=24), "DECLINED"), (dict(page_size=2048), "DECLINED"),
    (dict(n_seqs=4097), "DECLINED"), (dict(n_kv_heads=1025), "DECLINED"),
    (dict(n_pages=1 << 27), "DECLINED"), (dict(max_pages=(1 << 26) + 1), "DECLINED"),
    (dict(table=None), "EINVAL"), (dict(lens=None), "EINVAL"), (dict(table=PTR + 2), "EINVAL"),
    (dict(held=PTR + 1), "EINVAL"), (dict(n_free=PTR + 3), "EINVAL")])
def test_bad_pools_are_refused_everywhere(kw, want):
    rows, book = _calls(pds.load(), _pages(**kw))
    assert set(rows + book) == {getattr(pds, "PDS_" + want)}
    assert pds.load().pds_pages_release(None, PTR, None) == pds.PDS_EINVAL


@needs_lib
@pytest.mark.parametrize("kw,want", [
    (dict(k=None), "EINVAL"), (dict(v=PTR + 8), "EINVAL"), (dict(k_scale=None), "EINVAL"),
    (dict(v_scale=PTR + 4), "EINVAL"), (dict(page_stride=4096), "EINVAL"),
    (dict(page_stride=4096, row_stride=128, head_stride=64), "EINVAL"),
    (dict(page_stride=4096, row_stride=136, head_stride=2176), "EINVAL"),
    (dict(page_stride=4096 - 128, row_stride=128, head_stride=2048), "EINVAL"),
    (dict(page_stride=1 << 38, row_stride=128, head_stride=2048), "DECLINED")])
def test_bad_rows_of_a_pool_are_refused_where_they_are_used(kw, want):
    rows, book = _calls(pds.load(), _pages(**kw))
    assert set(rows) == {getattr(pds, "PDS_" + want)}
    assert _admitted(pds.load().pds_pages_release(_pages(**kw), PTR, None))


@needs_lib
def test_pages_without_a_book():
    lib, c = pds.load(), _pages(held=None, free_pages=None, n_free=None)
    rows, book = _calls(lib, c)
    assert book[:2] == [pds.PDS_EINVAL] * 2
    assert _admitted(lib.pds_pages_read(c, PTR, 1, PTR, PTR, None))
    assert _admitted(lib.pds_pages_slots(c, PTR, PTR, 1, PTR, PTR, PTR, None))


@needs_lib
def test_bad_arguments_are_refused():
    lib, c, bad = pds.load(), _pages(), pds.PDS_EINVAL
    for args in ((None, 1, PTR, PTR, PTR), (PTR, -1, PTR, PTR, PTR), (PTR, 1, None, PTR, PTR),
                 (PTR, 1, PTR, PTR, None), (PTR + 1, 1, PTR, PTR, PTR), (PTR, 1, PTR, PTR + 2, PTR)):
        assert lib.pds_pages_reserve(c, *args, None) == bad
        if args[4]:  # (starts may be left out there)
            assert lib.pds_pages_slots(c, PTR, *args, None) == bad
    assert lib.pds_pages_slots(c, None, PTR, 1, PTR, PTR, PTR, None) == bad
    assert lib.pds_pages_release(c, None, None) == bad and lib.pds_pages_release(c, PTR + 1, None) == bad
    spec = pds.pds_rope_spec(1.0e4, 0, 0, 0, None, 0.0, 1.0, 0, 32.0, 1.0)
    for args in ((None, None, PTR, PTR, 1, 0, 0, None), (None, PTR, PTR, None, 1, 0, 0, None),
                 (None, PTR + 8, PTR, PTR, 1, 0, 0, None), (None, PTR, PTR, PTR, 0, 0, 0, None),
                 (None, PTR, PTR, PTR, 1, 255, 0, None), (None, PTR, PTR, PTR, 1, 0, 260, None),
                 (spec, PTR, PTR, PTR, 1, 0, 0, None), (None, PTR, PTR, PTR + 2, 1, 0, 0, None)):
        assert lib.pds_pages_write(c, *args, None) == bad
    for args in ((None, 1, PTR, PTR), (PTR, 0, PTR, PTR), (PTR, 1, None, None), (PTR, 1, PTR + 4, PTR)):
        assert lib.pds_pages_read(c, *args, None) == bad
    good = dict(new=None, q=PTR, o=2 * PTR, h=4, qs=0, os=0, cap=0.0, window=0, ws=PTR, n=1 << 30)
    for kw, want in ((dict(q=None), bad), (dict(o=PTR), bad), (dict(h=0), bad), (dict(h=3), pds.PDS_DECLINED),
                     (dict(h=8194), pds.PDS_DECLINED), (dict(cap=-1.0), bad), (dict(cap=math.nan), bad),
                     (dict(cap=math.inf), bad), (dict(window=-1), bad), (dict(ws=None), bad),
                     (dict(ws=PTR + 8), bad), (dict(new=PTR + 2), bad), (dict(qs=500), bad), (dict(os=516), bad),
                     (dict(q=PTR + 2), bad)):
        assert lib.pds_pages_attend(c, *{**good, **kw}.values(), None) == want, kw
    assert lib.pds_pages_attend_workspace_bytes(c, 3) == 0
    assert lib.pds_pages_attend_workspace_bytes(None, 4) == 0


# ------------------------------------------------------ the PyTorch side


def _cache(fmt="bf16", **kw):
    dtype = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int4": torch.uint8}[fmt]
    k = torch.zeros(6, 2, 16, 32 if fmt == "int4" else 64).to(dtype)
    kw.setdefault("k", k)
    kw.setdefault("v", k.clone())
    cache = pages.PagedKvCache(fmt, 3, 6, 16, 4, 2, 64, **kw)
    cache.index = 0
    return cache


def _i32(*x):
    return cuda(torch.tensor(x, dtype=torch.int32))


def test_the_book_starts_with_all_pages_free(lib):  # noqa: F811
    cache = _cache()
    assert cache.free.tolist() == [5, 4, 3, 2, 1, 0] and cache.n_free.tolist() == [6]
    assert cache.held.tolist() == [0, 0, 0] and cache.lens.tolist() == [0, 0, 0]
    own = _cache(table=torch.zeros(3, 4, dtype=torch.int32))
    assert own.held is None and own.free is None and own.n_free is None and own.c.held is None
    cache.lens = torch.tensor([1, 2, 3])
    assert cache.lens.tolist() == [1, 2, 3]
    with pytest.raises(AttributeError):
        cache.table = cache.table.clone()


def test_bad_tensors_of_a_cache_are_refused():
    t = lambda *s: torch.zeros(*s, dtype=torch.int32)
    for kw in (dict(table=t(3, 5)), dict(table=t(3, 4).long()), dict(lens=t(4)), dict(held=t(3)),
               dict(free=t(6)), dict(n_free=t(1)), dict(free=t(5), n_free=t(1)),
               dict(k=torch.zeros(6, 2, 16, 64)), dict(k=torch.zeros(6, 16, 2, 64, dtype=torch.bfloat16)),
               dict(table=t(4, 3).T), dict(v=torch.zeros(6, 16, 2, 64, dtype=torch.bfloat16).transpose(1, 2)),
               dict(k=torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16).expand(6, 2, 16, 64),
                    v=torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16).expand(6, 2, 16, 64))):
        with pytest.raises(ValueError):
            _cache(**kw)
    with pytest.raises(ValueError):
        pages.PagedKvCache("bf16", 2 ** 31, 6, 16, 4, 2, 64, device="cpu")


def test_what_the_calls_hand_over_and_refuse(lib):  # noqa: F811
    cache = _cache("e4m3")
    slots, positions, starts = (cuda(t) for t in (torch.zeros(7, dtype=torch.int32),
                                                  torch.zeros(7, dtype=torch.int32),
                                                  torch.zeros(4, dtype=torch.int32)))
    new = _i32(1, 2, 0)
    assert cache.reserve(new, slots=slots, positions=positions, starts=starts) == (slots, positions, starts)
    assert lib.calls[-1] == ("pds_pages_reserve", (cache.c, new.data_ptr(), 7, slots.data_ptr(),
                                                   positions.data_ptr(), starts.data_ptr(), 0))
    for kw in (dict(), dict(rows=2 ** 31), dict(slots=slots[::2]), dict(slots=slots, positions=starts),
               dict(slots=slots, positions=positions, starts=positions)):
        with pytest.raises(ValueError):
            cache.reserve(new, **kw)
    for bad in (_i32(1, 2), new.long(), torch.zeros(3, dtype=torch.int32)):
        with pytest.raises(ValueError):
            cache.reserve(bad, slots=slots, positions=positions, starts=starts)
        with pytest.raises(ValueError):
            cache.release(bad)
    k = cuda(torch.zeros(7, 2, 64, dtype=torch.bfloat16))
    cache.write(k, k, slots)
    assert lib.calls[-1][1] == (cache.c, None, k.data_ptr(), k.data_ptr(), slots.data_ptr(), 7, 0, 0, None, 0)
    n = len(lib.calls)
    cache.write(k[:0], k[:0], slots[:0])  # no rows, no call
    cache.read(slots[:0], k_out=k[:0], v_out=k[:0])
    assert len(lib.calls) == n
    for args, kw in (((k, k, starts), {}), ((k, k[:6], slots), {}), ((k.float(), k, slots), {}),
                     ((k, k, slots), dict(rope=kv.RopeSpec(1e4, 64))),
                     ((k, k, slots), dict(rope=kv.RopeSpec(1e4, 128), positions=positions)),
                     ((k[:1].expand(7, 2, 64), k, slots), {})):
        with pytest.raises(ValueError):
            cache.write(*args, **kw)
    grad = cuda(torch.zeros(7, 2, 64, dtype=torch.bfloat16).requires_grad_())
    with pytest.raises(ValueError, match="gradient"):
        cache.write(k, grad, slots)
    with pytest.raises(ValueError):
        cache.read(slots, k_out=k[:, :1], v_out=k)
    q, o = (cuda(torch.zeros(3, 4, 64, dtype=torch.bfloat16)) for _ in range(2))
    ws = cuda(torch.zeros(64, dtype=torch.int32))
    assert cache.attend(q, new=new, out=o, workspace=ws) is o
    assert lib.calls[-1][1] == (cache.c, new.data_ptr(), q.data_ptr(), o.data_ptr(), 4, 0, 0, 0.0, 0,
                                ws.data_ptr(), 256, 0)
    for args, kw in (((q[:2],), {}), ((q,), dict(new=starts)), ((q,), dict(window=2 ** 31)),
                     ((q.float(),), {}), ((q,), dict(workspace=torch.zeros(64))), ((q,), dict(workspace=ws[::2]))):
        with pytest.raises(ValueError):
            cache.attend(*args, **{"out": o, "workspace": ws, **kw})
    with pytest.raises(ValueError, match="gradient"):
        cache.attend(cuda(torch.zeros(3, 4, 64, dtype=torch.bfloat16).requires_grad_()), out=o, workspace=ws)


def test_outputs_and_pools_that_require_a_gradient_are_refused(lib):  # noqa: F811
    """A write into them would be recorded by nobody."""
    leaf = lambda *s: cuda(torch.zeros(*s, dtype=torch.bfloat16).requires_grad_())
    plain = lambda *s: cuda(torch.zeros(*s, dtype=torch.bfloat16))
    ws, slots = cuda(torch.zeros(64, dtype=torch.int32)), cuda(torch.zeros(7, dtype=torch.int32))
    cache, flat = _cache(), make_cache()
    spec = kv.RopeSpec(1e4, 64)
    calls = [lambda: cache.attend(plain(3, 4, 64), out=leaf(3, 4, 64), workspace=ws),
             lambda: cache.read(slots, k_out=leaf(7, 2, 64), v_out=plain(7, 2, 64)),
             lambda: cache.read(slots, k_out=plain(7, 2, 64), v_out=leaf(7, 2, 64)),
             lambda: _cache(k=leaf(6, 2, 16, 64)), lambda: _cache(v=leaf(6, 2, 16, 64)),
             lambda: flat.attend(plain(2, 1, 4, 64), out=leaf(2, 1, 4, 64), workspace=ws),
             lambda: flat.read(0, 4, k_out=leaf(2, 4, 2, 64), v_out=plain(2, 4, 2, 64)),
             lambda: flat.read_new(4, k_out=plain(2, 4, 2, 64), v_out=leaf(2, 4, 2, 64)),
             lambda: kv.KvCache("bf16", 2, 16, 2, 64, k=leaf(2, 16, 2, 64), v=plain(2, 16, 2, 64)),
             lambda: kv.rope(plain(7, 2, 64), spec, out=leaf(7, 2, 64))]
    for call in calls:
        with pytest.raises(ValueError, match="gradient"):
            call()
    assert not lib.calls
    with torch.no_grad():
        calls[0](), calls[-1]()
    assert len(lib.calls) == 2


# ----------------------------------------------------------- definitions


def test_a_release_undoes_a_reserve():
    rng = np.random.default_rng(0)
    book = P.Book([[0] * 9] * 4, [0] * 4, rng.permutation(40), 8)
    lens = [0, 7, 8, 30]
    book.reserve(lens, [0] * 4)
    state = [list(p) for p in book.table], list(book.free)
    slots, positions, starts = book.reserve(lens, [9, 1, 0, 20])
    assert starts == [0, 9, 10, 10, 30] and len(set(slots)) == 30
    assert positions[:10] == list(range(9)) + [7] and positions[10:] == list(range(30, 50))
    assert [len(p) for p in book.table] == [2, 1, 1, 7]
    assert slots[9] == book.table[1][0] * 8 + 7
    book.release(lens)
    assert (book.table, book.free) == state
    assert book.reserve(lens, [300, 0, 0, 0]) is None and (book.table, book.free) == state


def test_attention_over_rows_is_the_tree_attention_of_one_token():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((6, 16)), rng.standard_normal((21, 2, 16)), rng.standard_normal((21, 2, 16))
    for window in (0, 1, 5, 40):
        for cap in (0.0, 2.0):
            want, _ = D.tree_attention(q[None], k, v, 20, softcap=cap, window=window)
            got, size, top = P.attend(q, k, v, max(0, 21 - window) if window else 0, 21, cap)
            assert np.allclose(got, want[0], rtol=1e-12, atol=1e-14)
            assert np.all(np.abs(got) <= size * (1 + 1e-12)) and np.all(top <= size.max(-1, keepdims=True) * 9)
    assert not P.attend(q, k, v, 0, 0)[0].any()
