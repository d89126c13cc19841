"""Cached decoding where it can go wrong: hidden rows under the tensor-core kernel,
many uneven sequences, scales far apart, queries that are not finite, calls on
two streams, long offsets, many rope rows.  Tolerances as in test_gpu_kv, whose
helpers these tests use; what a test adds to them is derived beside it."""

import numpy as np
import pytest

from oracle import decode as D
from parity import bf16_to_f64
from test_gpu_kv import EPS, _check, _codes, _filled, _i32, _kv, _normal, _tree, _words

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int4"])
@pytest.mark.parametrize("t,h,hkv,hd,window", [(40, 6, 2, 64, 64), (100, 6, 2, 128, 0),
                                               (30, 4, 2, 128, 50)])
def test_hidden_rows_under_many_query_rows(fmt, t, h, hkv, hd, window):
    kv = _kv()
    rng = np.random.default_rng(t)
    length = 300
    cache, k64, v64 = _filled(kv, rng, fmt, 1, 460, hkv, hd, [length])
    parents = [-1, 0, 0] + [int(rng.integers(max(0, i - 6), i)) for i in range(3, t - 1)] + [-2]
    bad = [slice(length + t, 460), slice(length + t - 1, length + t), slice(length + 2, length + 3)]
    if window:
        bad.append(slice(0, length - window))
    for rows in bad:
        for x, w in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
            if fmt == "bf16":
                x[:, rows] = float("nan")
                x[:, rows, :, ::3] = float("-inf")
            elif fmt == "e4m3":
                w[:, :, rows] = float("nan")
                x.view(torch.uint8)[:, rows, :, ::5] = 0x7F
            else:
                w[:, :, rows] = 0x7FC00003
    q, q64 = _normal(rng, 1, t, h, hd)
    o = cache.attend(q, parents=_i32([parents]), window=window)
    cache.sync()
    got = bf16_to_f64(o)[0]
    paths = D.tree_paths(parents)
    see = [i for i, p in enumerate(paths) if 2 in p and (not window or len(p) - p.index(2) <= window)]
    rest = [i for i in range(t - 1) if i not in see]
    assert see and len(rest) > 2 and np.isnan(got[see]).all()
    want, size = D.tree_attention(q64[0], k64[0], v64[0], length, parents, 0.0, window)
    err = np.abs(got - want)[rest]
    assert np.all(err <= EPS * np.abs(want[rest]) + (EPS + 2.0 ** -10) * size[rest])
    assert np.all(got[t - 1] == 0)


@pytest.mark.parametrize("t,h,hkv,hd", [(3, 6, 2, 64), (3, 3, 1, 128), (20, 8, 2, 64), (70, 4, 1, 128)])
def test_infinite_values_reach_the_tokens_that_see_them(t, h, hkv, hd):
    kv = _kv()
    rng = np.random.default_rng(hd + t)
    cache, k64, v64 = _filled(kv, rng, "bf16", 1, 200, hkv, hd, [90])
    cache.v[0, 91, :, 0] = float("inf")
    cache.v[0, 91, :, 1] = float("nan")
    cache.v[0, 91, :, hd - 1] = float("-inf")
    q, q64 = _normal(rng, 1, t, h, hd)
    parents = [-1, -1, 1] + [i - 1 if i % 2 else i - 3 for i in range(3, t)]
    o = bf16_to_f64(cache.attend(q, parents=_i32([parents])))[0]
    cache.sync()
    see = [i for i, p in enumerate(D.tree_paths(parents)) if 1 in p]
    rest = [i for i in range(t) if i not in see]
    v64[0, 91, :, [0, 1, hd - 1]] = 0.0
    want, size = D.tree_attention(q64[0], k64[0], v64[0], 90, parents, 0.0, 0)
    tol = EPS * np.abs(want) + (EPS + 2.0 ** -10) * size
    assert np.all(o[see][..., 0] == np.inf) and np.all(o[see][..., hd - 1] == -np.inf)
    assert np.all(np.isnan(o[see][..., 1]))
    assert np.all(np.abs(o - want)[see][..., 2:hd - 1] <= tol[see][..., 2:hd - 1])
    assert np.all(np.abs(o - want)[rest] <= tol[rest])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int4"])
@pytest.mark.parametrize("n,t,h,hkv,hd,most", [(70, 1, 8, 4, 128, 1500), (45, 9, 6, 2, 64, 900),
                                               (33, 20, 8, 4, 128, 700), (4, 2, 4, 1, 64, 900),
                                               (90, 1, 2, 2, 64, 3000)])
def test_many_uneven_sequences(fmt, n, t, h, hkv, hd, most):
    kv = _kv()
    rng = np.random.default_rng(n + t)
    lens = (rng.random(n) ** 3 * most).astype(int).tolist()
    lens[0], lens[n // 2], lens[-1] = 0, most, 1
    cache, k64, v64 = _filled(kv, rng, fmt, n, most + t + 5, hkv, hd, lens)
    parents = _tree(rng, n, t, pad=t // 2) if t > 2 else None
    q, q64 = _normal(rng, n, t, h, hd)
    o = cache.attend(q, parents=None if parents is None else _i32(parents), max_len=most)
    cache.sync()
    _check(o, q64, k64, v64, lens, parents, seqs=[0, 1, n // 2, n - 2, n - 1])


@pytest.mark.parametrize("lens,bad", [([700, 1999], 1), ([2001, 300], 0), ([-5, 1996], 0)])
def test_a_length_that_does_not_fit_among_short_ranges(lens, bad):
    from dense_decoder_layer_gb300 import pds
    kv = _kv()
    rng = np.random.default_rng(21)
    cache, k64, v64 = _filled(kv, rng, "e4m3", 2, 2000, 2, 64, lens)
    q, q64 = _normal(rng, 2, 4, 4, 64)
    out = torch.full_like(q, 9.0)
    cache.attend(q, out=out)
    with pytest.raises(pds.PdsError):
        cache.sync()
    assert (out[bad] == 9.0).all()
    _check(out, q64, k64, v64, lens, seqs=[1 - bad])


@pytest.mark.parametrize("fmt", ["e4m3", "int4"])
@pytest.mark.parametrize("t", [3, 40])
def test_scales_far_apart(fmt, t):
    """V scales over 2^20.  P times a V scale is held in fp16 in a unit that gives the largest
    scale so far 64 to 128, and a row's weights sum to at least one: below fp16's normal
    range a product is off by 2^-25 / 64 of the largest scale, times the code."""
    kv = _kv()
    rng = np.random.default_rng(t)
    length, h, hkv, hd = 500, 4, 2, 64
    cap = length + t
    cache, _, _ = _filled(kv, rng, fmt, 1, cap, hkv, hd, [length])
    scale = np.exp2(rng.uniform(-10, 10, (1, hkv, cap))).astype(np.float32)
    bits = torch.from_numpy(scale).cuda().view(torch.int32)
    if fmt == "e4m3":
        cache.v_scale.view(torch.int32).copy_(bits)
    else:
        cache.v_scale.copy_((bits & -65536) | (cache.v_scale & 15))
    k64, v64 = (D.dequantise(_codes(x, fmt), np.swapaxes(_words(w), 1, 2), fmt)
                for x, w in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    q, q64 = _normal(rng, 1, t, h, hd)
    got = bf16_to_f64(cache.attend(q))[0]
    cache.sync()
    want, size = D.tree_attention(q64[0], k64[0], v64[0], length, None, 0.0, 0)
    floor = cap * 2.0 ** -31 * scale.max() * {"e4m3": 448, "int4": 15}[fmt]
    assert np.all(np.abs(got - want) <= EPS * np.abs(want) + (EPS + 2.0 ** -10) * size + floor)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int4"])
@pytest.mark.parametrize("t", [3, 20, 70])
def test_a_query_that_is_not_finite_spoils_its_own_row_only(fmt, t):
    kv = _kv()
    rng = np.random.default_rng(t)
    cache, k64, v64 = _filled(kv, rng, fmt, 1, 700, 2, 128, [600])
    q, q64 = _normal(rng, 1, t, 8, 128)
    q[0, 0, 0, 5], q[0, 1, 3, 100], q[0, 2, 7, :] = float("nan"), float("inf"), float("-inf")
    got = bf16_to_f64(cache.attend(q))[0]
    cache.sync()
    want, size = D.tree_attention(q64[0], k64[0], v64[0], 600, None, 0.0, 0)
    good = np.ones((t, 8), bool)
    good[[0, 1, 2], [0, 3, 7]] = False
    assert np.isnan(got[0, 0]).all()
    tol = EPS * np.abs(want) + (EPS + 2.0 ** -10) * size
    assert np.all(np.abs(got - want)[good] <= tol[good])


def test_streams_with_a_workspace_each():
    kv = _kv()
    rng = np.random.default_rng(31)
    cache, k64, v64 = _filled(kv, rng, "e4m3", 2, 6100, 2, 128, [6000, 2500])
    jobs = []
    for t in (1, 7, 40):
        for _ in range(2):
            q, _ = _normal(rng, 2, t, 8, 128)
            jobs.append((q, cache.attend(q).clone(), torch.empty_like(cache.workspace(t, 8))))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    outs = [torch.empty_like(q) for q, _, _ in jobs]
    for _ in range(10):
        for (q, _, ws), out, stream in zip(jobs, outs, streams):
            cache.attend(q, out=out, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for out, (_, want, _) in zip(outs, jobs))
    cache.sync()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_offsets_past_32_bits(fmt):
    """Eight sequences of 300000 rows of 8 x 128: 2.5e9 values of K and of V."""
    kv = _kv()
    rng = np.random.default_rng(41)
    n, cap, t, hkv, hd, keep = 8, 300000, 2, 8, 128, 200
    cache = kv.KvCache(fmt, n, cap, hkv, hd)
    (k, k64), (v, v64) = _normal(rng, n, keep, hkv, hd), _normal(rng, n, keep, hkv, hd)
    cache.lens.fill_(cap - keep)
    cache.write(k, v)
    cache.lens.fill_(cap)
    back = cache.read(cap - keep, keep)
    cache.sync()
    if fmt == "bf16":
        assert torch.equal(back[0], k) and torch.equal(back[1], v)
    else:  # an e4m3 step is at most 2^-4 of the value or 2^-10 of the scale, then bf16
        for x, y in zip(back, (k64, v64)):
            err = np.abs(bf16_to_f64(x) - y)
            assert np.all(err <= (2.0 ** -4 + EPS) * np.abs(y) + 2.0 ** -10 / 448 * np.abs(y).max() * 1.01)
        k64, v64 = (bf16_to_f64(x) for x in back)
    for tokens in (t, 20):
        cache.lens.fill_(cap - tokens)
        q, q64 = _normal(rng, n, tokens, 16, hd)
        o = bf16_to_f64(cache.attend(q, window=100))
        cache.sync()
        for s in (0, n - 1):
            want, size = D.tree_attention(q64[s], k64[s], v64[s], keep - tokens, None, 0.0, 100)
            # (the rows read back are themselves rounded once: 2^-8 of K, V)
            slack = 2.0 ** -10 if fmt == "bf16" else 2.0 ** -4
            assert np.all(np.abs(o[s] - want) <= EPS * np.abs(want) + (EPS + slack) * size)


@pytest.mark.parametrize("layout", ["neox", "norm"])
@pytest.mark.parametrize("rows,heads,hd,rot", [(2049, 3, 64, 0), (2048, 1, 16, 0), (4097, 5, 80, 48),
                                               (2051, 9, 256, 256)])
def test_many_rope_rows(rows, heads, hd, rot, layout):
    kv = _kv()
    rng = np.random.default_rng(rows)
    x, x64 = _normal(rng, rows, heads, hd)
    spec = kv.RopeSpec(1.0e4, hd, rot, layout)
    y = kv.rope(x, spec, start_pos=77)
    want = D.rotate(x64, 77 + np.arange(rows), D.scaled_inv_freq(rot or hd, 1.0e4), layout)
    err = np.abs(bf16_to_f64(y) - want)
    assert np.all(err <= EPS * np.abs(want) + 2.0 ** -19 * 2 * np.abs(x64).max())
    wide = torch.zeros(rows, heads + 2, hd, dtype=torch.bfloat16, device="cuda")
    wide[:, 1:-1] = x
    kv.rope(wide[:, 1:-1], spec, start_pos=77, out=wide[:, 1:-1])
    assert torch.equal(wide[:, 1:-1], y)
    assert (wide[:, 0] == 0).all() and (wide[:, -1] == 0).all()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int4"])
def test_keys_alone_or_values_alone_are_read(fmt):
    from dense_decoder_layer_gb300 import pds
    kv = _kv()
    rng = np.random.default_rng(51)
    cache, _, _ = _filled(kv, rng, fmt, 2, 40, 3, 64, [37, 5])
    k, v = cache.read(3, 30)
    stream = torch.cuda.current_stream().cuda_stream
    for i, want in enumerate((k, v)):
        out = torch.zeros_like(want)
        ptr = [None, None]
        ptr[i] = out.data_ptr()
        assert pds.load().pds_cache_read(cache.c, 3, 30, *ptr, stream) == pds.PDS_OK
        cache.sync()
        assert torch.equal(out, want)


@pytest.mark.parametrize("fmt,n,t,h,hkv,hd,length", [
    ("bf16", 1, 256, 256, 16, 64, 300), ("e4m3", 1, 256, 200, 50, 64, 700),
    ("int4", 1, 1, 400, 400, 64, 600), ("bf16", 2, 2, 340, 340, 64, 900),
    ("e4m3", 2, 200, 160, 8, 128, 400)])
def test_more_heads_and_rows_than_run_at_once(fmt, n, t, h, hkv, hd, length):
    """One sequence alone fills the GPU more than once: its ranges are not cut."""
    kv = _kv()
    rng = np.random.default_rng(h)
    lens = [length, length // 3][:n]
    cache, k64, v64 = _filled(kv, rng, fmt, n, length + t + 2, hkv, hd, lens)
    q, q64 = _normal(rng, n, t, h, hd)
    o = cache.attend(q)
    cache.sync()
    # the last kv head and the first, and within them two query heads
    g = h // hkv
    for kvh in (0, hkv - 1):
        heads = [kvh * g, kvh * g + g - 1] if g > 1 else [kvh * g]
        part = slice(kvh, kvh + 1)
        _check(o[:, :, heads], q64[:, :, heads], k64[:, :, part], v64[:, :, part], lens)
    assert torch.equal(o, cache.attend(q))


def test_turns_are_correct_to_float32():
    """A key that is 1 in one channel becomes (cos, sin): the e4m3 row's scale is the larger of
    the two, at least 2^-1/2, over 448.  0.76 units in the last place of a value below 1 are
    1.08 2^-24 of it, the division rounds once more: in all below 2.25 2^-24."""
    kv = _kv()
    rng = np.random.default_rng(61)
    t, hd = 250, 64
    k = torch.zeros(1, t, hd // 2, hd, dtype=torch.bfloat16, device="cuda")
    for i in range(hd // 2):
        k[:, :, i, i] = 1.0
    pos = rng.integers(0, 2 ** 31, t)
    pos[:20] = np.arange(20)
    cache = kv.KvCache("e4m3", 1, t, hd // 2, hd)
    spec = kv.RopeSpec(5.0e5, hd)
    cache.write(k, k, rope=spec, positions=_i32(pos[None]))
    cache.sync()
    angle = np.outer(pos.astype(np.longdouble), D.scaled_inv_freq(hd, 5.0e5).astype(np.longdouble))
    want = np.maximum(np.abs(np.cos(angle)), np.abs(np.sin(angle))) / 448
    got = cache.k_scale[0].T.cpu().numpy().astype(np.float64)
    err = np.abs(got / want - 1)
    near = pos < 2 ** 16  # there the float64 frequencies themselves are exact enough
    assert np.all(err[near] <= 2.25 * 2.0 ** -24)
    assert np.all(err <= 2.25 * 2.0 ** -24 + 2.0 ** 31 * 2.0 ** -52)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int4"])
@pytest.mark.parametrize("n,t,h,hkv,hd,window", [(170, 1, 4, 2, 64, 0), (80, 3, 8, 4, 128, 0),
                                                 (45, 20, 8, 4, 64, 0), (400, 1, 1, 1, 128, 0),
                                                 (90, 9, 8, 4, 64, 500)])
def test_a_few_long_sequences_among_many(fmt, n, t, h, hkv, hd, window):
    """More sequences than run at once: the long ones are cut, the one that does not fit is not
    served, the others are right."""
    from dense_decoder_layer_gb300 import pds
    kv = _kv()
    rng = np.random.default_rng(n)
    cap = 5000
    lens = rng.integers(0, 60, n)
    lens[[1, n - 3]] = 4900, 2777
    lens[n // 2] = 5000 - t
    bad = n // 3
    lens[bad] = cap - t + 1
    lens = lens.tolist()
    cache = kv.KvCache(fmt, n, cap, hkv, hd)
    k, k64 = _normal(rng, 1, cap, hkv, hd)
    v, v64 = _normal(rng, 1, cap, hkv, hd)
    cache.write(k.expand(n, -1, -1, -1).contiguous(), v.expand(n, -1, -1, -1).contiguous())
    if fmt != "bf16":
        k64, v64 = (D.dequantise(_codes(x[:1], fmt), np.swapaxes(_words(w[:1]), 1, 2), fmt)
                    for x, w in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    cache.lens.copy_(_i32(lens))
    q, q64 = _normal(rng, n, t, h, hd)
    out = torch.full_like(q, 9.0)
    cache.attend(q, out=out, window=window)
    with pytest.raises(pds.PdsError):
        cache.sync()
    assert (out[bad] == 9.0).all()
    k64, v64 = (np.broadcast_to(x, (n, *x.shape[1:])) for x in (k64, v64))
    _check(out, q64, k64, v64, lens, window=window,
           seqs=[0, 1, bad - 1, bad + 1, n // 2, n - 3, n - 2, n - 1])
    again = torch.full_like(q, 9.0)
    cache.attend(q, out=again, window=window)
    assert torch.equal(out, again)
    with pytest.raises(pds.PdsError):
        cache.sync()


def test_rotations_called_in_turn_keep_to_their_own_numbers():
    """A rotation that was made before may be used again, and only for a call that names all of its numbers:
    each variant differs from the base in one of them and is called right behind it, with a refused call
    between, forward and back, by rope, by the contiguous and by the paged write."""
    kv = _kv()
    from dense_decoder_layer_gb300 import pages, pds
    rng = np.random.default_rng(41)
    base = dict(theta=5.0e5, head_dim=128, rot_dim=0, layout="neox", freq_factors=None, mscale=1.25,
                scaling="yarn", factor=4.0, orig_context=4096, beta_fast=32.0, beta_slow=1.0)
    ff = (1 + rng.random(64)).astype(np.float32)
    # (one with the number that makes the two scalings alike otherwise)
    variants = [dict(theta=4.0e5), dict(layout="norm"), dict(rot_dim=64), dict(freq_factors=ff), dict(mscale=0.0),
                dict(scaling="linear"), dict(scaling="none"), dict(factor=8.0), dict(orig_context=1024),
                dict(beta_fast=16.0), dict(beta_slow=4.0), dict(head_dim=64)]
    rows, heads = 40, 2
    pos = rng.integers(1, 1 << 20, rows)
    x = {hd: _normal(rng, rows, heads, hd) for hd in (64, 128)}

    def check(kw):
        hd, rot = kw["head_dim"], kw["rot_dim"] or kw["head_dim"]
        spec = kv.RopeSpec(*[kw[f] for f in ("theta", "head_dim", "rot_dim", "layout", "freq_factors", "mscale")],
                           **{f: kw[f] for f in ("scaling", "factor", "orig_context", "beta_fast", "beta_slow")})
        omega = D.scaled_inv_freq(rot, kw["theta"], kw["freq_factors"], kw["scaling"], kw["factor"],
                                  kw["orig_context"], kw["beta_fast"], kw["beta_slow"])
        t, t64 = x[hd]
        most = 2 * np.abs(t64).max() * max(1.0, kw["mscale"])
        for inverse in (False, True):
            want = D.rotate(t64, pos, omega, kw["layout"], kw["mscale"] or 1.0, inverse)
            got = bf16_to_f64(kv.rope(t, spec, positions=_i32(pos), inverse=inverse))
            assert np.all(np.abs(got - want) <= EPS * np.abs(want) + 2.0 ** -19 * most), (kw, inverse)
        turned = kv.rope(t, spec, positions=_i32(pos))
        flat = kv.KvCache("bf16", 1, rows, heads, hd)
        flat.write(t[None], t[None], rope=spec, positions=_i32(pos))
        paged = pages.PagedKvCache("bf16", 1, 5, 8, 1, heads, hd)
        paged.write(t, t, torch.arange(rows, dtype=torch.int32, device="cuda"), rope=spec, positions=_i32(pos))
        assert torch.equal(flat.k[0], turned) and torch.equal(paged.k.transpose(1, 2).reshape(turned.shape), turned)
        return got if hd == 128 else None

    first = check(base)
    for change in variants:
        other = check({**base, **change})
        # (a call that took the base's rotation would be seen)
        assert other is None or np.abs(other - first).max() > 0.1, change
        with pytest.raises(pds.PdsError):
            kv.rope(x[128][0], kv.RopeSpec(**{**base, "factor": -1.0}), positions=_i32(pos))
        assert np.array_equal(check(base), first)
