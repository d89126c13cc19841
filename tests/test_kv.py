"""Cached decoding on the host: what the entry points refuse before any device
work, and the oracle's definitions."""

import ctypes
import math
import os

import numpy as np
import pytest

from dense_decoder_layer_gb300 import pds
from oracle import decode as D

needs_lib = pytest.mark.skipif(not os.path.exists(pds.LIB_PATH), reason="libpds.so not built")
PTR = 0x10000


def _cache(**kw):
    c = pds.pds_cache(pds.PDS_KV_E4M3, 2, 64, 2, 128, 0, 0, 0, 0, PTR, PTR, PTR, PTR, PTR)
    for f, x in kw.items():
        setattr(c, f, x)
    return c


def _spec(**kw):
    s = pds.pds_rope_spec(1.0e4, 0, 0, 0, None, 0.0, 1.0, 0, 32.0, 1.0)
    for f, x in kw.items():
        setattr(s, f, x)
    return s


BAD_CACHES = [
    (dict(format=3), "EINVAL"), (dict(format=-1), "EINVAL"), (dict(reserved=1), "EINVAL"),
    (dict(n_seqs=0), "EINVAL"), (dict(capacity=0), "EINVAL"), (dict(n_kv_heads=-1), "EINVAL"),
    (dict(head_dim=96), "DECLINED"), (dict(n_seqs=4097), "DECLINED"), (dict(k=None), "EINVAL"),
    (dict(v=PTR + 8), "EINVAL"), (dict(lens=None), "EINVAL"), (dict(lens=PTR + 2), "EINVAL"),
    (dict(k_scale=None), "EINVAL"), (dict(v_scale=PTR + 1), "EINVAL"),
    (dict(head_stride=128, row_stride=64, seq_stride=64 * 256), "EINVAL"),
    (dict(head_stride=136, row_stride=272, seq_stride=64 * 272), "EINVAL"),
    (dict(head_stride=128), "EINVAL"),
]


@needs_lib
@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_bad_caches_are_refused_everywhere(kw, want):
    lib, c, want = pds.load(), _cache(**kw), getattr(pds, "PDS_" + want)
    assert lib.pds_cache_write(c, None, PTR, PTR, 1, 0, 0, None, None, None) == want
    assert lib.pds_cache_read(c, 0, 1, PTR, PTR, None) == want
    assert lib.pds_attention_tree(c, PTR, PTR, 1, 4, 0, 0, None, 0.0, 0, 0, None, 0, None) == want
    assert lib.pds_cache_write(None, None, PTR, PTR, 1, 0, 0, None, None, None) == pds.PDS_EINVAL


BAD_SPECS = [
    (dict(theta=0.0), "EINVAL"), (dict(theta=math.inf), "EINVAL"), (dict(layout=2), "EINVAL"),
    (dict(rot_dim=-16), "EINVAL"), (dict(rot_dim=144), "EINVAL"), (dict(rot_dim=24), "DECLINED"),
    (dict(mscale=-1.0), "EINVAL"), (dict(scaling=3), "EINVAL"),
    (dict(scaling=1, factor=0.0), "EINVAL"), (dict(scaling=2, factor=2.0), "EINVAL"),
    (dict(scaling=2, factor=2.0, orig_context=64, beta_slow=40.0), "EINVAL"),
    (dict(scaling=2, factor=2.0, orig_context=64, theta=1.0), "EINVAL"),
]


@needs_lib
@pytest.mark.parametrize("kw,want", BAD_SPECS)
def test_bad_rotations_are_refused(kw, want):
    lib, s, want = pds.load(), _spec(**kw), getattr(pds, "PDS_" + want)
    assert lib.pds_rope(s, PTR, PTR, 1, 2, 128, 0, 0, None, 0, 0, None) == want
    assert lib.pds_cache_write(_cache(), s, PTR, PTR, 1, 0, 0, None, None, None) == want


@needs_lib
def test_bad_frequency_factors_are_refused():
    for bad in (0.0, -1.0, math.nan, math.inf):
        arr = (ctypes.c_float * 64)(*([1.0] * 63 + [bad]))
        s = _spec(freq_factors=ctypes.cast(arr, ctypes.POINTER(ctypes.c_float)))
        assert pds.load().pds_rope(s, PTR, PTR, 1, 2, 128, 0, 0, None, 0, 0, None) == pds.PDS_EINVAL


@needs_lib
def test_bad_calls_are_refused():
    lib, c, s = pds.load(), _cache(), _spec()
    E, Dn = pds.PDS_EINVAL, pds.PDS_DECLINED

    def rope(x=PTR, y=PTR, rows=1, heads=2, hd=128, xs=0, ys=0, pos=None):
        return lib.pds_rope(s, x, y, rows, heads, hd, xs, ys, pos, 0, 0, None)
    assert [rope(x=None), rope(y=PTR + 8), rope(rows=0), rope(heads=0), rope(hd=0),
            rope(xs=128, ys=256), rope(xs=260), rope(pos=PTR + 2), rope(xs=-8),
            rope(xs=512)] == [E] * 10
    assert [rope(hd=120), rope(hd=272)] == [Dn] * 2
    assert lib.pds_rope(None, PTR, PTR, 1, 2, 128, 0, 0, None, 0, 0, None) == E

    def write(k=PTR, v=PTR, t=1, ks=0, vs=0, par=None, pos=None):
        return lib.pds_cache_write(c, None, k, v, t, ks, vs, par, pos, None)
    assert [write(k=None), write(v=PTR + 2), write(t=0), write(ks=128), write(vs=260),
            write(par=PTR + 1), write(pos=PTR + 1)] == [E] * 7
    assert write(t=65) == Dn
    c.capacity = 512
    assert write(t=257, par=PTR) == Dn

    def read(first=0, rows=1, k=PTR, v=PTR):
        return lib.pds_cache_read(c, first, rows, k, v, None)
    assert [read(first=-2), read(rows=0), read(k=None, v=None), read(v=PTR + 4)] == [E] * 4
    assert [read(first=512), read(first=1, rows=512), read(first=-1, rows=513)] == [Dn] * 3

    def attend(q=PTR, o=PTR, t=1, h=4, qs=0, os_=0, par=None, cap=0.0, win=0, most=0, ws=None):
        return lib.pds_attention_tree(c, q, o, t, h, qs, os_, par, cap, win, most, ws, 0, None)
    assert [attend(q=None), attend(o=PTR + 8), attend(t=0), attend(h=0), attend(cap=-1.0),
            attend(cap=math.nan), attend(win=-1), attend(most=-1), attend(qs=256),
            attend(os_=516), attend(par=PTR + 2), attend(ws=PTR + 8)] == [E] * 12
    assert [attend(h=3), attend(t=257)] == [Dn] * 2
    c.capacity = 3
    assert attend(t=4) == Dn
    assert pds.last_error().startswith("declined")
    assert [lib.pds_attention_tree_workspace_bytes(x, t, h)
            for x, t, h in ((None, 1, 4), (c, 0, 4), (c, 257, 4), (c, 1, 3))] == [0] * 4


@needs_lib
def test_calls_without_a_device_fail_after_admission():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a CUDA device is present")
    lib = pds.load()
    assert lib.pds_cache_read(_cache(), 0, 1, PTR, PTR, None) == pds.PDS_ELAUNCH
    assert lib.pds_rope(_spec(), PTR, PTR, 1, 2, 128, 0, 0, None, 0, 0, None) == pds.PDS_ELAUNCH
    assert "no CUDA device" in pds.last_error()


def test_row_strides_of_views():
    """The wrapper's reading of a tensor's layout: packed, a slice of a fused projection, a
    transposed view, and what it refuses."""
    torch = pytest.importorskip("torch")
    from dense_decoder_layer_gb300 import kv

    class Cuda:  # a tensor's shape and strides, seen as a device tensor
        def __init__(self, t):
            self.t, self.dtype, self.device, self.shape = t, t.dtype, t.device, t.shape

        def get_device(self):
            return 0

        def stride(self, *a):
            return self.t.stride(*a)

        def is_contiguous(self):
            return self.t.is_contiguous()

    def rows(t, lead=2):
        return kv._rows(Cuda(t), t.shape, lead, 0, "x")
    fused = torch.empty(2, 3, 512, dtype=torch.bfloat16)
    part = fused[..., 128:384].unflatten(-1, (4, 64))
    assert rows(part) == 512
    assert rows(part.contiguous()) == 0
    assert rows(part[:, :1]) == 1536
    for bad in (part.transpose(0, 1), part[..., ::2], part.float()):
        with pytest.raises(ValueError):
            rows(bad)
    with pytest.raises(ValueError):
        kv._rows(Cuda(part), (2, 3, 4, 63), 2, 0, "x")
    with pytest.raises(ValueError):
        kv._rows(Cuda(part), part.shape, 2, 1, "x")


# ------------------------------------------------------------- the oracle


def test_e4m3_grid():
    v = D.e4m3_values()
    assert v[0x7E] == 448 and v[0x01] == 2.0 ** -9 and v[0x38] == 1.0 and v[0xB8] == -1.0
    codes = np.array([c for c in range(256) if c & 127 != 127], np.uint8)
    assert np.array_equal(D.e4m3_round(v[codes]), codes)
    assert D.e4m3_round(np.array([17.0 / 16, 19.0 / 16, 460.0, 2.0 ** -10, 1.5 * 2.0 ** -9]))\
        .tolist() == [0x38, 0x3A, 0x7E, 0x00, 0x02]  # ties to the even code


@pytest.mark.parametrize("fmt", ["e4m3", "int4"])
def test_quantised_rows_stand_for_their_values(fmt):
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((50, 128)) * 10.0 ** rng.integers(-3, 3, (50, 1))).astype(np.float32)
    x[0], x[1], x[2, 5], x[3] = 0, 1e-44, np.inf, np.abs(x[3])
    codes, words = D.quantise(x, fmt)
    y = D.dequantise(codes, words, fmt)
    assert np.all(y[:2] == 0) and np.all(np.isnan(y[2])) and words[2] == 0x7FC00000
    s = (words & np.uint32(0xFFFF0000 if fmt == "int4" else 0xFFFFFFFF)).view(np.float32)[3:, None]
    # e4m3: half a step, 2^-4 of the value or 2^-10 of the scale; int4: half a step, one more where the
    # zero point's and the value's roundings add up past 15, and the scale's own rounding (15 steps, 2^-8)
    tol = np.maximum(np.abs(x[3:]) * 2.0 ** -4, s * 2.0 ** -10) if fmt == "e4m3" else s * (1.5 + 15 / 256)
    assert np.all(np.abs(y[3:] - x[3:]) <= tol * (1 + 1e-6))


def test_tree_attention_of_a_chain_is_causal_attention():
    import oracle
    rng = np.random.default_rng(2)
    q, k, v = (rng.standard_normal(s) for s in ((5, 4, 8), (9, 2, 8), (9, 2, 8)))
    want = oracle.causal_gqa_attention(q, k, v, 4).reshape(5, 4, 8)
    np.testing.assert_allclose(D.tree_attention(q, k, v, 4)[0], want, atol=1e-12)
    # a tree's token is the last one of the chain of its path
    parents = [-1, 0, 0, 1, 2, -2]
    q6, k6, v6 = (rng.standard_normal(s) for s in ((6, 4, 8), (10, 2, 8), (10, 2, 8)))
    o = D.tree_attention(q6, k6, v6, 4, parents, window=5)[0]
    for t, path in enumerate(D.tree_paths(parents)):
        if path:
            rows = [0, 1, 2, 3] + [4 + a for a in path]
            one = D.tree_attention(q6[path], k6[rows], v6[rows], 4, window=5)[0][-1]
            np.testing.assert_allclose(o[t], one, atol=1e-12)
    assert np.all(o[5] == 0)


def test_yarn_keeps_fast_pairs_and_interpolates_slow_ones():
    w = D.scaled_inv_freq(128, 5.0e5)
    y = D.scaled_inv_freq(128, 5.0e5, scaling="yarn", factor=8.0, orig_context=8192)
    assert y[0] == w[0] and np.isclose(y[-1], w[-1] / 8) and np.all(np.diff(y) < 0)
    turns = 8192 * w / (2 * math.pi)
    assert np.all(y[turns > 40] == w[turns > 40])
    t = np.random.default_rng(0).standard_normal((3, 2, 128))
    back = D.rotate(D.rotate(t, [1, 5, 70000], y), [1, 5, 70000], y, inverse=True)
    np.testing.assert_allclose(back, t, atol=1e-9)


@needs_lib
def test_more_heads_than_the_attention_takes_are_declined():
    lib, c = pds.load(), _cache()
    assert lib.pds_attention_tree(c, PTR, PTR, 1, 8194, 0, 0, None, 0.0, 0, 0, None, 0,
                                  None) == pds.PDS_DECLINED
    assert lib.pds_attention_tree_workspace_bytes(c, 1, 8194) == 0


def test_expanded_tensors_are_refused():
    """Rows that share memory have stride 0, which to the C ABI says packed."""
    torch = pytest.importorskip("torch")
    from dense_decoder_layer_gb300 import kv

    class Cuda(torch.Tensor):  # a host tensor that says it is on device 0
        def get_device(self):
            return 0

    one = torch.empty(1, 1, 4, 64, dtype=torch.bfloat16)
    for shape in ((2, 1, 4, 64), (1, 3, 4, 64), (2, 3, 4, 64)):
        with pytest.raises(ValueError, match="overlap"):
            kv._rows(one.expand(shape).as_subclass(Cuda), shape, 2, 0, "x")
    row = torch.empty(1, 1, 1, 64, dtype=torch.bfloat16).expand(2, 8, 4, 64)
    with pytest.raises(ValueError, match="expanded"):
        kv.KvCache("bf16", 2, 8, 4, 64, k=row, v=row, lens=torch.zeros(2, dtype=torch.int32))


@needs_lib
@pytest.mark.parametrize("shape,strides,apart", [
    ((2, 64, 2), (64 * 256, 256, 128), True),        # packed
    ((2, 64, 2), (64 * 256, 128, 64 * 128), True),   # heads first
    ((2, 64, 2), (256, 512, 128), True),             # rows first
    ((2, 64, 2), (64 * 512, 512, 256), True),        # half of wider rows
    ((2, 64, 2), (64 * 256, 128, 128), False),       # a row is the next one's second head
    ((2, 64, 2), (256, 256, 128), False),            # sequences a row apart
    ((2, 64, 2), (64 * 128, 256, 128), False),       # sequences half a cache apart
    ((2, 64, 3), (64 * 256, 256, 128), False),       # a third head in a row of two
    ((1, 64, 2), (0, 256, 128), True), ((1, 1, 2), (0, 128, 128), True),
    ((2, 64, 1), (64 * 128, 128, 128), True),
    ((2, 64, 2), (2 ** 62, 256, 128), False),        # past 64 bits
    ((4096, 64, 2), (2 ** 52, 256, 128), False)])
def test_strides_that_let_rows_overlap_are_refused(shape, strides, apart):
    """(Where nothing is refused the call ends at the missing device, or the missing memory.)"""
    n, cap, hkv = shape
    ss, rs, hs = strides
    c = _cache(n_seqs=n, capacity=cap, n_kv_heads=hkv, seq_stride=ss, row_stride=rs, head_stride=hs)
    lib = pds.load()
    for st in (lib.pds_cache_read(c, 0, 1, PTR, PTR, None),
               lib.pds_cache_write(c, None, PTR, PTR, 1, 0, 0, None, None, None),
               lib.pds_attention_tree(c, PTR, PTR, 1, 2 * hkv, 0, 0, None, 0.0, 0, 0, None, 0, None)):
        assert st != pds.PDS_OK
        assert ("overlap" in pds.last_error()) == (not apart)


def test_a_failed_lookup_of_a_device_is_made_again(tmp_path):
    """facts.h as the calls use it, in a program of its own: the first lookups fail."""
    import shutil
    import subprocess
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    src = tmp_path / "facts.cpp"
    src.write_text("""
        #include "facts.h"
        int main() {
          pds::DeviceFacts facts;
          uint32_t word = 0, *status = nullptr;
          int sms = 0, looked = 0;
          bool good = false;
          auto lookup = [&](uint32_t** s, int* n) { ++looked; *s = &word; *n = good ? 152 : 0; return good; };
          if (facts.get(lookup, &status, &sms) || facts.get(lookup, &status, &sms)) return 1;
          if (status || sms) return 2;
          good = true;
          for (int i = 0; i < 3; ++i)
            if (!facts.get(lookup, &status, &sms) || status != &word || sms != 152) return 3;
          return looked == 3 ? 0 : 4;
        }""")
    csrc = os.path.join(os.path.dirname(pds.__file__), "csrc")
    subprocess.run([cxx, "-std=c++17", "-pthread", "-I", csrc, str(src), "-o", str(tmp_path / "facts")],
                   check=True, timeout=120)
    assert subprocess.run([str(tmp_path / "facts")], timeout=20).returncode == 0


@needs_lib
def test_attention_in_place_is_refused():
    lib, c = pds.load(), _cache()
    assert lib.pds_attention_tree(c, PTR, PTR, 1, 4, 0, 0, None, 0.0, 0, 0, None, 0, None) == pds.PDS_EINVAL
    assert "same buffer" in pds.last_error()
    lib.pds_attention_tree(c, PTR, 2 * PTR, 1, 4, 0, 0, None, 0.0, 0, 0, None, 0, None)
    assert "same buffer" not in pds.last_error()


def test_yarn_by_counting_turns():
    """The ramp's ends found from what they mean, without the closed form: the (real) index of
    the pair that turns beta times within the original context, by bisection of its turns."""
    theta, rot, ctx, factor, fast, slow = 5.0e5, 128, 8192, 8.0, 32.0, 1.0

    def index(beta):
        lo, hi = -64.0, 2.0 * rot
        for _ in range(200):
            mid = (lo + hi) / 2
            turns = ctx * theta ** (-2 * mid / rot) / (2 * math.pi)
            lo, hi = (mid, hi) if turns > beta else (lo, mid)
        return lo
    first, last = max(0, math.floor(index(fast))), min(rot - 1, math.ceil(index(slow)))
    w = D.scaled_inv_freq(rot, theta, scaling="yarn", factor=factor, orig_context=ctx,
                          beta_fast=fast, beta_slow=slow)
    for i in range(rot // 2):
        kept = theta ** (-2 * i / rot)
        part = min(1.0, max(0.0, (i - first) / (last - first)))
        assert abs(w[i] - (kept * (1 - part) + kept / factor * part)) <= 1e-12 * kept
    assert 0 < first < last < rot // 2
