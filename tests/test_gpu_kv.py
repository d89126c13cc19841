"""Cached decoding on the GPU against the float64 definitions: rotary positions,
rows into a quantised cache and back, attention of drafted tokens.

Tolerances, derived before the first run.  A rounding to bf16 is off by at
most 2^-8 of the value.
* pds_rope: one rounding of the result; the turn is exact to 2^-32, its
  conversion, sine and cosine to a few float32 roundings, the two products
  and their sum to three more: in all below 2^-19 of |u| + |w|.
* pds_cache_write without a rotation, pds_cache_read: IEEE float32 operations
  in a fixed order, so equal bit for bit.  With a rotation a code may land on
  the other side of a tie: half a step of the format around the true value.
* attention: P is rounded to bf16 (2^-8 of each weight, so 2^-8 of the
  weighted sum A of |v|), the result once more (2^-8 of |o|); a score is off
  by at most (hd + 8) 2^-23 sum |q k| / sqrt(hd) (float32 sums, the scales and
  the base-2 exponential), which moves A by as much."""

import math

import numpy as np
import pytest

import synth
from oracle import decode as D
from parity import bf16_to_f64

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

EPS = 2.0 ** -8


def _kv():
    from dense_decoder_layer_gb300 import kv
    return kv


def _bf16(x):
    bits = synth.bf16_round(np.ascontiguousarray(x, np.float32))
    t = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).cuda()
    return t, synth.bf16_bits_to_f32(bits).astype(np.float64)


def _normal(rng, *shape, scale=1.0):
    return _bf16((rng.standard_normal(shape) * scale).astype(np.float32))


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _codes(t, fmt):
    """Codes one per element of a cache tensor, and of its scale tensor the words."""
    raw = t.contiguous().view(torch.uint8).cpu().numpy()
    if fmt == "int4":
        return np.stack((raw & 15, raw >> 4), -1).reshape(*raw.shape[:-1], -1)
    return raw


def _words(t):
    return t.contiguous().view(torch.int32).cpu().numpy().view(np.uint32)


# ------------------------------------------------------------------- rope


@pytest.mark.parametrize("layout", ["neox", "norm"])
@pytest.mark.parametrize("rows,heads,hd,rot,scaling", [
    (1, 1, 16, 0, "none"), (1, 32, 64, 0, "none"), (5, 3, 128, 48, "none"), (3, 40, 128, 0, "yarn"),
    (300, 2, 256, 128, "linear"), (257, 5, 80, 16, "yarn"), (2, 70, 128, 0, "none")])
def test_rope(rows, heads, hd, rot, scaling, layout):
    kv = _kv()
    rng = np.random.default_rng(rows + heads)
    x, x64 = _normal(rng, rows, heads, hd)
    ff = None if scaling == "linear" else (1 + rng.random((rot or hd) // 2)).astype(np.float32)
    kw = dict(scaling=scaling, factor=4.0, orig_context=4096)
    spec = kv.RopeSpec(5.0e5, hd, rot, layout, ff, 1.25, **kw)
    omega = D.scaled_inv_freq(rot or hd, 5.0e5, ff, **kw)
    pos = rng.integers(0, 1 << 20, rows)
    pos[0] = 2 ** 31 - 1 if rows > 1 else 7
    pos[-1] = -3 if rows > 2 else pos[-1]
    for inverse in (False, True):
        want = D.rotate(x64, pos, omega, layout, 1.25, inverse)
        size = np.abs(D.rotate(np.abs(x64), 0 * pos, omega, layout, 1.25))
        r = rot or hd
        a, b = ((slice(0, r // 2), slice(r // 2, r)) if layout == "neox"
                else (slice(0, r, 2), slice(1, r, 2)))
        pair = size[..., a] + size[..., b]
        size[..., a] = size[..., b] = pair
        size[..., r:] = 0
        y = kv.rope(x, spec, positions=_i32(pos), inverse=inverse)
        err = np.abs(bf16_to_f64(y) - want)
        # 2^31 turns the float64 angle itself by 2^-53 2^31: below the rest
        assert np.all(err <= EPS * np.abs(want) + 2.0 ** -19 * size)
    z = x.clone()
    assert torch.equal(kv.rope(z, spec, positions=_i32(pos), out=z, inverse=True), y)


def test_rope_strides_positions_and_gradient():
    kv = _kv()
    rng = np.random.default_rng(3)
    fused, f64 = _normal(rng, 4, 3, 5 * 64)
    x = fused[..., 64:256].unflatten(-1, (3, 64))
    spec = kv.RopeSpec(1.0e4, 64)
    before = fused.clone()
    y = kv.rope(x, spec, start_pos=11)
    omega = D.scaled_inv_freq(64, 1.0e4)
    want = D.rotate(f64[..., 64:256].reshape(12, 3, 64), 11 + np.arange(12), omega)
    assert np.all(np.abs(bf16_to_f64(y).reshape(12, 3, 64) - want) <= EPS * np.abs(want) + 2.0 ** -17)
    kv.rope(x, spec, start_pos=11, out=x)  # in place in the middle of a wider row
    assert torch.equal(x.contiguous(), y)
    assert torch.equal(fused[..., :64], before[..., :64])
    assert torch.equal(fused[..., 256:], before[..., 256:])
    # the gradient of sum(g rope(x)) against differences of the definition
    g, g64 = _normal(rng, 12, 3, 64)
    grad = bf16_to_f64(kv.rope(g, spec, start_pos=11, inverse=True))
    d = rng.standard_normal((12, 3, 64))
    x0 = f64[..., 64:256].reshape(12, 3, 64)
    diff = np.sum(g64 * (D.rotate(x0 + d, 11 + np.arange(12), omega) -
                         D.rotate(x0 - d, 11 + np.arange(12), omega))) / 2
    assert abs(np.sum(grad * d) - diff) <= EPS * np.sum(np.abs(grad * d)) + 1e-3


# ----------------------------------------------------------- write and read


LAYOUTS = {"packed": None, "heads_first": (0, 2, 1, 3), "rows_first": (1, 0, 2, 3)}


def _cache(kv, fmt, n, cap, hkv, hd, layout="packed", lens=None):
    dtype, per = {"bf16": (torch.bfloat16, 1), "e4m3": (torch.float8_e4m3fn, 1),
                  "int4": (torch.uint8, 2)}[fmt]
    order = LAYOUTS[layout]
    shape = (n, cap, hkv, hd // per)
    kw = {}
    if order is not None:
        for x in ("k", "v"):
            raw = torch.zeros([shape[i] for i in order], dtype=torch.uint8, device="cuda")\
                if per == 2 else torch.zeros([shape[i] for i in order], device="cuda").to(dtype)
            kw[x] = raw.permute([order.index(i) for i in range(4)])
    return kv.KvCache(fmt, n, cap, hkv, hd, lens=None if lens is None else _i32(lens), **kw)


@pytest.mark.parametrize("layout", list(LAYOUTS))
@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int4"])
@pytest.mark.parametrize("n,t,hkv,hd,lens", [(1, 1, 1, 64, [0]), (3, 5, 3, 128, [0, 11, 35]),
                                             (2, 17, 9, 64, [3, 1])])
def test_write_and_read_are_exact(fmt, n, t, hkv, hd, lens, layout):
    kv = _kv()
    rng = np.random.default_rng(n + t)
    cap = 40
    cache = _cache(kv, fmt, n, cap, hkv, hd, layout, lens)
    for x in (cache.k, cache.v):
        x.copy_(x.view(torch.uint8).fill_(0x5A).view(x.dtype))
    scale = 10.0 ** rng.integers(-4, 4, (n, t, hkv, 1))
    fused = torch.empty(n, t, 3 * hkv * hd, dtype=torch.bfloat16, device="cuda")
    kx, vx = (rng.standard_normal((n, t, hkv, hd)) * scale).astype(np.float32), \
        rng.standard_normal((n, t, hkv, hd)).astype(np.float32)
    kx[0, 0, 0] = 0
    vx[0, -1, 0] = np.abs(vx[0, -1, 0]) + 5   # a row of one sign
    kx[-1, -1, -1, 3] = 1e-39                 # a subnormal among ordinary values
    if fmt != "bf16":
        vx[-1, 0, -1, 7] = np.inf
        kx[0, -1, -1] = 1e-38                 # a scale below the normal range
        vx[0, 0, -1, 0] = np.nan if n == 1 else vx[0, 0, -1, 0]
    (k, k64), (v, v64) = _bf16(kx), _bf16(vx)
    kd = fused[..., :hkv * hd].unflatten(-1, (hkv, hd))
    kd.copy_(k)
    before = [x.clone() for x in (cache.k.view(torch.uint8), cache.v.view(torch.uint8))]
    cache.write(kd, v)
    cache.sync()
    ko, vo = cache.read_new(t)
    cache.sync()
    for x64, got, tensor, words, old in ((k64, ko, cache.k, cache.k_scale, before[0]),
                                         (v64, vo, cache.v, cache.v_scale, before[1])):
        if fmt == "bf16":
            assert np.array_equal(bf16_to_f64(got), x64, equal_nan=True)
        else:
            codes, w = D.quantise(x64.astype(np.float32), fmt)
            have, hw = _codes(tensor, fmt), _words(words)
            for s in range(n):
                at = slice(lens[s], lens[s] + t)
                assert np.array_equal(hw[s][:, at].T, w[s])
                # the sign of a zero is no value
                same = (have[s, at] == codes[s]) | ((fmt == "e4m3") & (have[s, at] & 127 == 0) &
                                                    (codes[s] & 127 == 0))
                assert same.all()
            back = D.dequantise(codes, w, fmt)
            want = synth.bf16_bits_to_f32(synth.bf16_round(back.astype(np.float32)))
            assert np.array_equal(bf16_to_f64(got), want.astype(np.float64), equal_nan=True)
        now = tensor.view(torch.uint8)
        for s in range(n):  # every other row as it was
            for rows in (slice(0, lens[s]), slice(lens[s] + t, cap)):
                assert torch.equal(now[s, rows], old[s, rows])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int4"])
@pytest.mark.parametrize("layout,rot", [("neox", 0), ("norm", 32)])
def test_write_rotates_keys_at_tree_positions(fmt, layout, rot):
    kv = _kv()
    rng = np.random.default_rng(7)
    n, t, hkv, hd, lens = 2, 6, 2, 128, [9, 20]
    parents = [[-1, 0, 0, 1, 3, -2], [-1, -1, 1, 2, 2, 0]]
    spec = kv.RopeSpec(1.0e4, hd, rot, layout)
    omega = D.scaled_inv_freq(rot or hd, 1.0e4)
    cache = _cache(kv, fmt, n, 32, hkv, hd, lens=lens)
    k, k64 = _normal(rng, n, t, hkv, hd)
    v, v64 = _normal(rng, n, t, hkv, hd)
    old = cache.k.view(torch.uint8).clone()
    cache.write(k, v, rope=spec, parents=_i32(parents))
    ko, vo = (bf16_to_f64(x) for x in cache.read_new(t))
    for s in range(n):
        depth = [len(p) - 1 for p in D.tree_paths(parents[s])]
        want = D.rotate(k64[s], [lens[s] + d for d in depth], omega, layout)
        for i, d in enumerate(depth):
            if d < 0:
                assert torch.equal(cache.k.view(torch.uint8)[s, lens[s] + i], old[s, lens[s] + i])
                continue
            err, x = np.abs(ko[s, i] - want[i]), np.abs(want[i])
            top = x.max(-1, keepdims=True)
            # the format's half step (int4: of a scale up to 2 top / 15, and the roundings that
            # test_kv.py derives), the read's bf16 rounding, the rotation's error
            tol = EPS * x if fmt == "bf16" else \
                np.maximum(x * 2.0 ** -4, top / 448 * 2.0 ** -10) * 1.07 + EPS * x if fmt == "e4m3" else \
                (2 * top / 15) * (1.5 + 15 / 256) + EPS * (x + top)
            assert np.all(err <= tol + 2.0 ** -17 * top)
    # positions given: the same rows as a rotation before the write
    pos = rng.integers(0, 1000, (n, t))
    cache.write(k, v, rope=spec, positions=_i32(pos))
    a = cache.read_new(t)[0].clone()
    if fmt == "bf16":
        pre = kv.rope(k, spec, positions=_i32(pos))
        assert torch.equal(a, pre)
    cache.sync()


def test_read_a_range_leaves_the_rest():
    kv = _kv()
    rng = np.random.default_rng(9)
    cache = _cache(kv, "e4m3", 3, 50, 2, 64, lens=[0, 0, 0])
    k, _ = _normal(rng, 3, 50, 2, 64)
    cache.write(k, k)
    full = cache.read_new(50)[0].clone()
    cache.lens.copy_(_i32([0, 13, 50]))
    ko = torch.full((3, 30, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    cache.read(5, 30, k_out=ko)
    for s, live in enumerate((0, 8, 30)):
        assert torch.equal(ko[s, :live], full[s, 5:5 + live])
        assert (ko[s, live:] == 7.0).all()
    cache.sync()


# --------------------------------------------------------------- attention


def _filled(kv, rng, fmt, n, cap, hkv, hd, lens, layout="packed", kscale=1.0):
    """A cache whose `lens` rows hold random values, and those values in float64."""
    cache = _cache(kv, fmt, n, cap, hkv, hd, layout, [0] * n)
    k, k64 = _normal(rng, n, cap, hkv, hd, scale=kscale)
    v, v64 = _normal(rng, n, cap, hkv, hd)
    cache.write(k, v)
    if fmt != "bf16":
        k64, v64 = (D.dequantise(_codes(x, fmt), np.swapaxes(_words(w), 1, 2), fmt)
                    for x, w in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    cache.lens.copy_(_i32(lens))
    return cache, k64, v64


def _check(o, q64, k64, v64, lens, parents=None, softcap=0.0, window=0, seqs=None):
    got = bf16_to_f64(o)
    n, t, h, hd = q64.shape
    for s in range(n) if seqs is None else seqs:
        want, size = D.tree_attention(q64[s], k64[s], v64[s], lens[s],
                                      None if parents is None else parents[s], softcap, window)
        group = h // k64.shape[2]
        seen = np.abs(k64[s, :lens[s] + t])
        reach = max(float(np.nanmax(np.einsum("thd,jhd->thj", np.abs(q64[s][:, i::group]), seen)))
                    for i in range(group))
        slack = (hd + 8) * 2.0 ** -23 * reach / math.sqrt(hd)
        tol = EPS * np.abs(want) + (EPS + 2 * slack) * size * 1.01
        assert np.all(np.isfinite(got[s]))
        assert np.all(np.abs(got[s] - want) <= tol), (s, float(np.max(np.abs(got[s] - want) - tol)))


def _tree(rng, n, t, pad=0):
    p = np.full((n, t), -2)
    for s in range(n):
        used = t - (pad if s % 2 else 0)
        p[s, :used] = [max(-1, i - int(rng.integers(1, 4))) for i in range(used)]
    return p.tolist()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int4"])
@pytest.mark.parametrize("n,t,h,hkv,hd,lens", [
    (1, 1, 1, 1, 64, [0]), (1, 1, 3, 1, 128, [1]), (2, 1, 8, 2, 64, [15, 16]),
    (3, 1, 24, 8, 128, [17, 0, 2048]), (1, 2, 5, 1, 128, [300]), (2, 3, 12, 3, 64, [255, 257]),
    (1, 7, 8, 2, 128, [1000]), (1, 33, 4, 2, 64, [129]), (1, 64, 3, 1, 128, [517]),
    (2, 256, 2, 1, 64, [5, 700]), (1, 40, 16, 2, 128, [777]), (5, 4, 32, 8, 128, [0, 3, 999, 31, 1500])])
def test_chain_attention(fmt, n, t, h, hkv, hd, lens):
    kv = _kv()
    rng = np.random.default_rng(t + h + sum(lens))
    cap = max(lens) + t + 1
    cache, k64, v64 = _filled(kv, rng, fmt, n, cap, hkv, hd, lens)
    q, q64 = _normal(rng, n, t, h, hd, scale=1.5)
    o = cache.attend(q)
    cache.sync()
    _check(o, q64, k64, v64, lens)
    assert torch.equal(o, cache.attend(q))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int4"])
@pytest.mark.parametrize("n,t,h,hkv,hd,lens,softcap,window", [
    (1, 4, 4, 2, 128, [0], 0.0, 0), (2, 9, 6, 2, 64, [100, 31], 0.0, 0),
    (2, 16, 8, 2, 64, [333, 99], 30.0, 128), (3, 21, 8, 4, 128, [700, 0, 64], 5.0, 0),
    (2, 64, 6, 2, 128, [1025, 40], 0.0, 3), (2, 130, 4, 1, 64, [600, 2], 0.0, 100),
    (2, 256, 2, 1, 128, [37, 1], 0.0, 0), (1, 5, 4, 4, 64, [5000], 0.0, 1),
    (2, 12, 40, 2, 128, [2500, 2499], 0.0, 2000)])
def test_tree_attention(fmt, n, t, h, hkv, hd, lens, softcap, window):
    kv = _kv()
    rng = np.random.default_rng(t * h + sum(lens))
    cache, k64, v64 = _filled(kv, rng, fmt, n, max(lens) + t, hkv, hd, lens)
    parents = _tree(rng, n, t, pad=t // 3)
    q, q64 = _normal(rng, n, t, h, hd, scale=1.5)
    for max_len in (0, max(lens)):
        o = cache.attend(q, parents=_i32(parents), softcap=softcap, window=window, max_len=max_len)
        cache.sync()
        _check(o, q64, k64, v64, lens, parents, softcap, window)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int4"])
def test_attention_layouts_strides_and_no_workspace(fmt):
    kv = _kv()
    from dense_decoder_layer_gb300 import pds
    rng = np.random.default_rng(5)
    n, t, h, hkv, hd, lens = 2, 3, 6, 2, 128, [200, 700]
    for layout in ("heads_first", "rows_first"):
        cache, k64, v64 = _filled(kv, rng, fmt, n, 720, hkv, hd, lens, layout)
        fused, f64 = _normal(rng, n, t, 10 * hd)
        q = fused[..., 2 * hd:8 * hd].unflatten(-1, (h, hd))
        q64 = f64[..., 2 * hd:8 * hd].reshape(n, t, h, hd)
        wide = torch.full((n, t, (h + 1) * hd), 3.0, dtype=torch.bfloat16, device="cuda")
        out = wide[..., hd:].unflatten(-1, (h, hd))
        cache.attend(q, out=out)
        _check(out, q64, k64, v64, lens)
        assert (wide[..., :hd] == 3.0).all()
        alone = torch.empty(n, t, h, hd, dtype=torch.bfloat16, device="cuda")
        pds.pds_attention_tree(cache.c, q.data_ptr(), alone.data_ptr(), t, h,
                               torch.cuda.current_stream().cuda_stream, q_stride=10 * hd)
        cache.sync()
        _check(alone, q64, k64, v64, lens)


def test_scores_far_apart_and_long_ranges():
    """Sharp scores (the running maximum moves often), and a range split over every SM."""
    kv = _kv()
    rng = np.random.default_rng(6)
    for fmt, lens, kscale in (("bf16", [3000], 8.0), ("e4m3", [40000], 1.0), ("int4", [9000], 8.0)):
        cache, k64, v64 = _filled(kv, rng, fmt, 1, lens[0] + 8, 1, 128, lens, kscale=kscale)
        q, q64 = _normal(rng, 1, 2, 8, 128, scale=2.0)
        o = cache.attend(q)
        cache.sync()
        _check(o, q64, k64, v64, lens)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int4"])
def test_hidden_rows_may_hold_anything(fmt):
    """Infinities and NaN in rows that a token does not see: behind the sequence's end, in
    a padding token's row, below a window, and in a sibling's row."""
    kv = _kv()
    rng = np.random.default_rng(8)
    n, t, h, hkv, hd, lens, window = 1, 6, 6, 2, 64, [300], 64
    cache, k64, v64 = _filled(kv, rng, fmt, n, 400, hkv, hd, lens)
    parents = [[-1, 0, 0, 1, 2, -2]]
    bad = {"behind": slice(306, 400), "padding": slice(305, 306), "below": slice(0, 230),
           "sibling": slice(302, 303)}
    for rows in bad.values():
        for x, w in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
            if fmt == "bf16":
                x[:, rows] = float("nan")
                x[:, rows, :, ::3] = float("inf")
            elif fmt == "e4m3":
                w[:, :, rows] = float("nan")
            else:
                w[:, :, rows] = 0x7FC00000
    q, q64 = _normal(rng, n, t, h, hd)
    o = cache.attend(q, parents=_i32(parents), window=window)
    cache.sync()
    k64, v64 = np.nan_to_num(k64), np.nan_to_num(v64)
    got = bf16_to_f64(o)
    see_bad = [i for i, p in enumerate(D.tree_paths(parents[0])) if 2 in p]
    assert see_bad == [2, 4] and np.isnan(got[0, see_bad]).all()
    rest = [i for i in range(t) if i not in see_bad]
    want, size = D.tree_attention(q64[0], k64[0], v64[0], 300, parents[0], 0.0, window)
    err = np.abs(got[0] - want)[rest]
    assert np.all(err <= EPS * np.abs(want[rest]) + (EPS + 2.0 ** -10) * size[rest])
    assert np.all(got[0, 5] == 0)


def test_a_row_of_bad_length_or_parent_is_refused_on_the_device():
    from dense_decoder_layer_gb300 import pds
    kv = _kv()
    rng = np.random.default_rng(10)
    cache, k64, v64 = _filled(kv, rng, "e4m3", 3, 64, 2, 64, [10, 62, 20])
    q, q64 = _normal(rng, 3, 4, 4, 64)
    k, _ = _normal(rng, 3, 4, 2, 64)
    out = torch.full_like(q, 9.0)
    for bad in (62, -1, 2 ** 31 - 1):
        cache.lens[1] = bad
        for call in (lambda: cache.attend(q, out=out), lambda: cache.write(k, k),
                     lambda: cache.read_new(4)):
            codes = cache.k.view(torch.uint8)[1].clone()
            call()
            with pytest.raises(pds.PdsError) as e:
                cache.sync()
            assert e.value.status == pds.PDS_EINVAL
            cache.sync()  # reported once
            assert torch.equal(cache.k.view(torch.uint8)[1], codes)
    assert (out[1] == 9.0).all()
    # a bad parent: that token's row is zero, the others' are right
    cache, k64, v64 = _filled(kv, rng, "e4m3", 1, 64, 2, 64, [10])
    for bad in ([-1, 1, 0, 0], [-1, 2, 0, 0], [-1, 2 ** 31 - 1, 0, 0], [-1, -2, 0, 1]):
        o = cache.attend(q[:1], parents=_i32([bad]))
        with pytest.raises(pds.PdsError):
            cache.sync()
        got = bf16_to_f64(o)
        lost = [i for i, p in enumerate(bad) if i == 1 or p == 1]
        fixed = [[p if i not in lost else -2 for i, p in enumerate(bad)]]
        assert np.all(got[0, lost] == 0)
        _check(o, q64[:1], k64, v64, [10], fixed)


def test_captured_step_follows_the_lengths():
    """A decode step (rotate, write, attend, advance) captured once and replayed: lengths live
    on the device, so every replay sees the rows of the ones before.  On a stream of its own."""
    kv = _kv()
    rng = np.random.default_rng(11)
    n, h, hkv, hd, steps = 2, 6, 2, 128, 5
    spec = kv.RopeSpec(1.0e4, hd)
    omega = D.scaled_inv_freq(hd, 1.0e4)
    lens = [700, 14]
    for fmt in ("bf16", "e4m3", "int4"):
        cache, _, _ = _filled(kv, rng, fmt, n, 720, hkv, hd, lens)
        q, k, v = (torch.zeros(n, 1, x, hd, dtype=torch.bfloat16, device="cuda") for x in (h, hkv, hkv))
        qr, o = torch.empty_like(q), torch.empty_like(q)
        cache.workspace(1, h)

        def step():
            kv.rope(q, spec, positions=cache.lens, out=qr)
            cache.write(k, v, rope=spec)
            cache.attend(qr, out=o)
            cache.lens.add_(1)
        stream = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            step()  # warm: kernel attributes
            cache.lens.copy_(_i32(lens))
            stream.synchronize()
            with torch.cuda.graph(graph, stream=stream):
                step()
        for i in range(steps):
            (qn, q64), (kn, _), (vn, _) = (_normal(rng, n, 1, x, hd) for x in (h, hkv, hkv))
            q.copy_(qn), k.copy_(kn), v.copy_(vn)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            now = [x + i for x in lens]
            assert cache.lens.tolist() == [x + 1 for x in now]
            if fmt == "bf16":
                k64, v64 = bf16_to_f64(cache.k), bf16_to_f64(cache.v)
            else:
                k64, v64 = (D.dequantise(_codes(x, fmt), np.swapaxes(_words(w), 1, 2), fmt)
                            for x, w in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
            _check(o, bf16_to_f64(qr), k64, v64, now)
            want = D.rotate(q64[:, 0], now, omega)
            assert np.all(np.abs(bf16_to_f64(qr)[:, 0] - want) <= EPS * np.abs(want) + 2.0 ** -16)
        cache.sync()


def test_a_prefill_cache_serves_drafted_tokens():
    """The bf16 cache of a DenseStack, as it is: attention of a chain over it equals
    pds_attention on the same rows, within both roundings."""
    from dense_decoder_layer_gb300 import pds
    kv = _kv()
    rng = np.random.default_rng(12)
    B, s, H, Hkv, hd = 9, 1000, 24, 8, 128
    rows = s + B
    k, k64 = _normal(rng, rows + 7, Hkv, hd)
    v, v64 = _normal(rng, rows + 7, Hkv, hd)
    q, q64 = _normal(rng, B, H, hd)
    want = torch.empty(B, H * hd, dtype=torch.bfloat16, device="cuda")
    pds.pds_attention(q.data_ptr(), k.data_ptr(), v.data_ptr(), want.data_ptr(), B, s, H, Hkv, hd,
                      torch.cuda.current_stream().cuda_stream)
    cache = kv.KvCache("bf16", 1, rows + 7, Hkv, hd, k=k[None], v=v[None], lens=_i32([s]))
    got = cache.attend(q[None])
    cache.sync()
    _check(got, q64[None], k64[None], v64[None], [s])
    _check(want.view(1, B, H, hd), q64[None], k64[None], v64[None], [s])


def test_drafted_tokens_are_the_tokens_decoded_one_by_one():
    """The whole run: a tree of drafted tokens, of which one path is accepted, gives that
    path's tokens the outputs that decoding them one at a time gives."""
    kv = _kv()
    rng = np.random.default_rng(13)
    h, hkv, hd, length = 6, 2, 128, 333
    spec = kv.RopeSpec(5.0e5, hd, scaling="yarn", factor=4.0, orig_context=4096)
    parents = [-1, 0, 0, 2, 1, 3, 5, 3]
    path = [0, 2, 3, 5, 6]
    for fmt in ("bf16", "e4m3", "int4"):
        tree, _, _ = _filled(kv, rng, fmt, 1, 400, hkv, hd, [length])
        one = kv.KvCache(fmt, 1, 400, hkv, hd, k=tree.k.clone(), v=tree.v.clone(),
                         k_scale=None if fmt == "bf16" else tree.k_scale.clone(),
                         v_scale=None if fmt == "bf16" else tree.v_scale.clone(),
                         lens=tree.lens.clone())
        q, k, v = (_normal(rng, 1, len(parents), x, hd)[0] for x in (h, hkv, hkv))
        depth = _i32([len(p) - 1 for p in D.tree_paths(parents)])
        p = _i32([parents])
        qr = kv.rope(q, spec, positions=length + depth)
        tree.write(k, v, rope=spec, parents=p)
        o = tree.attend(qr, parents=p)
        for i, node in enumerate(path):
            at = slice(node, node + 1)
            q1 = kv.rope(q[:, at], spec, positions=one.lens)
            assert torch.equal(q1, qr[:, at])
            one.write(k[:, at], v[:, at], rope=spec)
            o1 = one.attend(q1)
            # the same weights from differently grouped sums: each side is within its own
            # rounding of P and of the result, on values of size about one
            torch.testing.assert_close(o1.float(), o[:, at].float(), rtol=3 * EPS, atol=4 * EPS)
            one.lens += 1
        # the accepted rows move up; both caches then hold the same rows
        src = torch.tensor(path, device="cuda") + length
        for x in (tree.k, tree.v):
            x.view(torch.uint8)[:, length:length + len(path)] = x.view(torch.uint8)[:, src]
        assert torch.equal(tree.k.view(torch.uint8)[:, :length + len(path)],
                           one.k.view(torch.uint8)[:, :length + len(path)])
        tree.sync()
