"""Cached decoding with values far from the ordinary.  Tolerances as in test_gpu_kv,
whose helpers these tests use; what a test adds to them is derived beside it."""

import math

import numpy as np
import pytest

from oracle import decode as D
from parity import bf16_to_f64
from test_gpu_kv import EPS, _bf16, _codes, _filled, _i32, _kv, _normal, _words

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _scales(cache):
    """V's scales, float64 [n, Hkv, capacity]."""
    w = cache.v_scale.view(torch.int32)
    return (w & -65536 if cache.fmt == "int4" else w).view(torch.float32).double().cpu().numpy()


def _close(cache, o, q64, k64, v64, length, parents=None, softcap=0.0, window=0, rows=None):
    """One sequence's rows (all, or those listed) against the definition: test_gpu_kv's
    tolerance, and over codes what fp16 drops.  A weight times its V scale is held in a
    unit that gives the largest scale so far at least 64; below fp16's normal range it is off
    by 2^-25 of that unit, and a row's weights sum to at least one: n 2^-31 of the largest scale
    times the largest code for n keys."""
    got = bf16_to_f64(o)[0]
    want, size = D.tree_attention(q64[0], k64[0], v64[0], length, parents, softcap, window)
    t, h, hd = got.shape
    group = h // k64.shape[2]
    floor = 0.0
    if cache.fmt != "bf16":
        scale = _scales(cache)[0][:, :length + t]
        top = np.repeat(scale.max(-1), group)[None, :, None]
        floor = (length + t) * 2.0 ** -31 * top * {"e4m3": 448, "int4": 15}[cache.fmt]
    reach = np.abs(q64[0]) @ np.ones(hd) * np.abs(k64[0, :length + t]).max()
    slack = (hd + 8) * 2.0 ** -23 * reach / math.sqrt(hd)
    tol = EPS * np.abs(want) + (EPS + 2 * slack[..., None]) * size * 1.01 + floor
    rows = range(t) if rows is None else rows
    assert np.isfinite(got[rows]).all()
    assert np.all((np.abs(got - want) <= tol)[rows]), float(np.max((np.abs(got - want) - tol)[rows]))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int4"])
@pytest.mark.parametrize("t,h,hkv,hd", [(3, 4, 2, 128), (40, 4, 2, 128), (100, 6, 2, 64)])
def test_large_finite_queries_take_the_best_key(fmt, t, h, hkv, hd):
    """Scores so large that one key has all the weight, wherever it leads by more than the
    scores' float32 rounding and by 40 besides (e^-40 is nothing next to a rounding).  Its
    weight is rounded to bf16, its sum is not, and the result is rounded once more."""
    kv = _kv()
    rng = np.random.default_rng(t)
    length = 400
    cache, k64, v64 = _filled(kv, rng, fmt, 1, length + t, hkv, hd, [length])
    k, v = k64[0], v64[0]
    for size in (3e4, 1e7, 1e8, 4e8, 1e9, 1e10, 1e12, 1e20, 1e30, 1e35):
        q, q64 = _normal(rng, 1, t, h, hd, scale=size)
        o = bf16_to_f64(cache.attend(q))[0]
        cache.sync()
        decided = 0
        for i in range(t):
            rows = length + i + 1
            for head in range(h):
                g, x = head // (h // hkv), q64[0, i, head]
                z = k[:rows, g] @ x / math.sqrt(hd)
                reach = (np.abs(k[:rows, g]) @ np.abs(x)).max()
                slack = (hd + 8) * 2.0 ** -23 * reach / math.sqrt(hd)
                top, second = np.sort(z)[:-3:-1]
                assert np.isfinite(o[i, head]).all()
                if top - second > 2 * slack + 40:
                    decided += 1
                    want = v[z.argmax(), g]
                    assert np.all(np.abs(o[i, head] - want) <=
                                  2 * EPS * np.abs(want) + 2.0 ** -30 * np.abs(v).max())
        assert decided > 0.8 * t * h


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int4"])
@pytest.mark.parametrize("t", [3, 40, 150])
def test_scores_far_apart_under_few_and_many_rows(fmt, t):
    kv = _kv()
    rng = np.random.default_rng(t + 1)
    cache, k64, v64 = _filled(kv, rng, fmt, 1, 1500 + t, 2, 128, [1500], kscale=8.0)
    q, q64 = _normal(rng, 1, t, 4, 128, scale=2.0)
    o = cache.attend(q)
    cache.sync()
    _close(cache, o, q64, k64, v64, 1500)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int4"])
@pytest.mark.parametrize("t,h", [(6, 6), (40, 4), (100, 6)])
def test_queries_of_padding_tokens_may_hold_anything(fmt, t, h):
    kv = _kv()
    rng = np.random.default_rng(t)
    cache, k64, v64 = _filled(kv, rng, fmt, 1, 500 + t, 2, 64, [500])
    parents = [[-1] + [int(rng.integers(max(-1, i - 5), i)) for i in range(1, t)]]
    pad = [t - 1, t - 2, t // 2]
    for i in pad:
        parents[0] = [(-2 if j == i else -1 if p == i else p) for j, p in enumerate(parents[0])]
    q, q64 = _normal(rng, 1, t, h, 64)
    for fill in (1e8, 1e10, 1e20, 3e38, float("inf"), float("nan"), None):
        if fill is None:  # bits as they come
            bits = rng.integers(-2 ** 15, 2 ** 15, (len(pad), h, 64)).astype(np.int16)
            q[0, pad] = torch.from_numpy(bits).cuda().view(torch.bfloat16)
        else:
            q[0, pad] = _bf16(fill * np.sign(rng.standard_normal((len(pad), h, 64))))[0]
        o = cache.attend(q, parents=_i32(parents))
        cache.sync()
        assert (o[0, pad] == 0).all()
        _close(cache, o, q64, k64, v64, 500, parents[0],
               rows=[i for i in range(t) if i not in pad])

@pytest.mark.parametrize("fmt", ["e4m3", "int4"])
@pytest.mark.parametrize("t,h,hkv,hd,softcap", [(2, 4, 2, 128, 0.0), (5, 4, 2, 64, 20.0), (12, 4, 2, 128, 0.0),
                                                (40, 4, 2, 64, 0.0), (70, 8, 2, 128, 20.0)])
def test_query_rows_far_apart_do_not_touch_each_other(fmt, t, h, hkv, hd, softcap):
    """Live rows of one block whose sizes differ by up to 2^126: each is as exact as alone."""
    kv = _kv()
    rng = np.random.default_rng(t + hd)
    cache, k64, v64 = _filled(kv, rng, fmt, 1, 300 + t, hkv, hd, [300])
    size = 10.0 ** rng.choice([-8, -2, 0, 0, 0, 1, 3], (1, t, h, 1))
    for big in (1.0, 1e4, 1e12, 1e30):
        scale = size.copy()
        scale[0, ::3, 1] = big
        q, q64 = _normal(rng, 1, t, h, hd)
        q, q64 = _bf16(q64 * scale)
        o = cache.attend(q, softcap=softcap)
        cache.sync()
        # rows of size 1 and below; for larger ones the scores' own rounding decides
        small = (scale[0, :, :, 0] <= 1.0)
        got = bf16_to_f64(o)[0]
        assert np.isfinite(got).all()
        want, size_v = D.tree_attention(q64[0], k64[0], v64[0], 300, None, softcap, 0)
        reach = np.abs(q64[0]).sum(-1) * np.abs(k64).max()
        slack = (hd + 8) * 2.0 ** -23 * reach / math.sqrt(hd)
        floor = (300 + t) * 2.0 ** -31 * _scales(cache).max() * {"e4m3": 448, "int4": 15}[fmt]
        # a capped score: c - 2 c / (e + 1) is off by some 2^-21 c
        cap = softcap * 2.0 ** -21
        tol = EPS * np.abs(want) + (EPS + 2 * (slack[..., None] + cap)) * size_v * 1.01 + floor
        assert np.all((np.abs(got - want) <= tol)[small])


def _products_close(cache, o, q64, k64, v64, length, parents, rows, window=0):
    """Rows of one sequence over codes, each measured by what it sees itself: test_gpu_kv's
    tolerance, and 2^-27 of the row's largest product of a weight and a V scale, times the
    largest code, per key (fp16's smallest step is 2^-24, off by half of it, and a row's largest
    product is held as 4 or more)."""
    got = bf16_to_f64(o)[0]
    t, h, hd = got.shape
    group = h // k64.shape[2]
    scale = _scales(cache)[0]
    paths = D.tree_paths(range(-1, t - 1) if parents is None else parents)
    for i in rows:
        keys = np.array(list(range(length)) + [length + a for a in paths[i]])
        pos = np.array(list(range(length)) + [length + a for a in range(len(paths[i]))])
        keys = keys[pos > pos[-1] - window] if window else keys
        for head in range(h):
            g, x = head // group, q64[0, i, head]
            z = k64[0, keys, g] @ x / math.sqrt(hd)
            w = np.exp(z - z.max())
            w /= w.sum()
            want, size = w @ v64[0, keys, g], w @ np.abs(v64[0, keys, g])
            slack = (hd + 8) * 2.0 ** -23 * (np.abs(k64[0, keys, g]) @ np.abs(x)).max() / math.sqrt(hd)
            floor = len(keys) * 2.0 ** -27 * (w * scale[g, keys]).max() * {"e4m3": 448, "int4": 15}[cache.fmt]
            tol = EPS * np.abs(want) + (EPS + 2 * slack) * size * 1.01 + floor
            assert np.all(np.abs(got[i, head] - want) <= tol), (i, head)


def _set_scale(cache, rows, value):
    """V's scale words of some rows; their codes as they are."""
    if cache.fmt == "e4m3":
        cache.v_scale[:, :, rows] = value
    else:
        bits = int(np.float32(value).view(np.int32)) & -65536
        cache.v_scale[:, :, rows] = (cache.v_scale[:, :, rows] & 15) | bits


def _values(cache):
    from test_gpu_kv import _codes, _words
    return (D.dequantise(_codes(x, cache.fmt), np.swapaxes(_words(w), 1, 2), cache.fmt)
            for x, w in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))


BIG = [2.0 ** 33, 2.0 ** 70, 3.0e38]


@pytest.mark.parametrize("fmt", ["e4m3", "int4"])
@pytest.mark.parametrize("t,h,hkv,hd,length", [(3, 4, 2, 128, 300), (12, 4, 2, 64, 300), (40, 4, 2, 64, 300),
                                               (100, 6, 2, 128, 310), (20, 4, 2, 128, 2000)])
def test_large_scales_that_a_row_does_not_see(fmt, t, h, hkv, hd, length):
    """Below the window, in a padding token's row, in the row of a token with a bad parent
    (which the write refuses), in a sibling's."""
    from dense_decoder_layer_gb300 import pds
    kv = _kv()
    rng = np.random.default_rng(t)
    window = 90
    for big in BIG:
        cache, _, _ = _filled(kv, rng, fmt, 1, length + t, hkv, hd, [length])
        parents = [-1, 0, 0] + [int(rng.integers(max(0, i - 6), i)) for i in range(3, t)]
        bad, pad = (t - 1, t - 2) if t > 5 else (None, None)
        if bad:
            parents[bad], parents[pad] = t + 3, -2
        for rows in [slice(0, length - window), slice(length + 2, length + 3)] + \
                ([slice(length + t - 2, length + t)] if bad else []):
            _set_scale(cache, rows, big)
        k64, v64 = _values(cache)
        q, q64 = _normal(rng, 1, t, h, hd)
        o = cache.attend(q, parents=_i32([parents]), window=window)
        if bad:
            with pytest.raises(pds.PdsError):
                cache.sync()
            parents[bad] = -2
        else:
            cache.sync()
        paths = D.tree_paths(parents)
        rest = [i for i, p in enumerate(paths) if p and 2 not in p]
        assert len(rest) > 1
        _products_close(cache, o, q64, k64, v64, length, parents, rest, window)


@pytest.mark.parametrize("fmt", ["e4m3", "int4"])
@pytest.mark.parametrize("t,h,hkv,hd", [(1, 2, 1, 128), (3, 4, 2, 128), (12, 4, 2, 64), (40, 4, 2, 64),
                                        (100, 4, 2, 128)])
def test_large_scales_of_keys_with_hardly_any_weight(fmt, t, h, hkv, hd):
    """Visible keys whose scale is far above the others' and whose weight is as far below: the
    largest product decides, wherever such keys lie."""
    kv = _kv()
    rng = np.random.default_rng(t + hd)
    length = 600
    for big, place in ((2.0 ** 20, 5), (2.0 ** 40, 300), (2.0 ** 60, 599), (2.0 ** 36, slice(64, 520, 57))):
        cache, _, _ = _filled(kv, rng, fmt, 1, length + t, hkv, hd, [length])
        base = rng.standard_normal(hd)
        base *= 8 / np.linalg.norm(base)
        q, q64 = _bf16(base + 0.3 * rng.standard_normal((1, t, h, hd)))
        k, _ = _normal(rng, 1, length + t, hkv, hd)
        if isinstance(place, int):
            place = slice(place, place + 1)
        k[:, place] = _bf16(-8.0 * base)[0]
        v, _ = _normal(rng, 1, length + t, hkv, hd)
        cache.lens.zero_()
        cache.write(k, v)
        cache.lens.fill_(length)
        _set_scale(cache, place, big)
        k64, v64 = _values(cache)
        o = cache.attend(q)
        cache.sync()
        _products_close(cache, o, q64, k64, v64, length, None, range(t))


@pytest.mark.parametrize("fmt", ["e4m3", "int4"])
@pytest.mark.parametrize("t,h,hkv,hd", [(1, 2, 1, 128), (12, 4, 2, 64), (40, 4, 2, 64), (140, 4, 2, 128)])
def test_scales_over_sixty_powers_of_two(fmt, t, h, hkv, hd):
    kv = _kv()
    rng = np.random.default_rng(t + 7)
    length = 500
    for spread in (10, 30):
        cache, _, _ = _filled(kv, rng, fmt, 1, length + t, hkv, hd, [length])
        scale = np.exp2(rng.uniform(-spread, spread, (1, hkv, length + t))).astype(np.float32)
        scale[0, :, ::7] = 0  # rows of zeros among them
        bits = torch.from_numpy(scale).cuda().view(torch.int32)
        if fmt == "e4m3":
            cache.v_scale.view(torch.int32).copy_(bits)
        else:
            cache.v_scale.copy_((bits & -65536) | (cache.v_scale & 15))
        k64, v64 = _values(cache)
        q, q64 = _normal(rng, 1, t, h, hd, scale=3.0)
        o = cache.attend(q)
        cache.sync()
        _products_close(cache, o, q64, k64, v64, length, None, range(t))


@pytest.mark.parametrize("fmt", ["e4m3", "int4"])
@pytest.mark.parametrize("t,place", [(1, 128), (1, 384), (40, 64), (40, 192)])
def test_large_scores_that_are_neighbours(fmt, t, place):
    """Two keys whose scores, around 2^27 in powers of two, are one or a few float32 apart (16
    each), the larger one met later: its weight is not 2^16.  A token's result is some mean of the
    two values, whichever way the scores are rounded."""
    kv = _kv()
    hd, length = 128, 512
    for step in range(24):
        cache = kv.KvCache(fmt, 1, length + t, 1, hd)
        k = torch.zeros(1, length + t, 1, hd, dtype=torch.bfloat16, device="cuda")
        k[0, [0, place], 0, 0] = 448.0 if fmt == "e4m3" else 15.0
        v = torch.ones_like(k)
        v[0, place] = 3.0
        cache.write(k, v)
        cache.lens.fill_(length)
        # the later key's scale: float32 steps up where the format has them, else K's first
        # channel stays and the second adds the difference
        q = torch.zeros(1, t, 1, hd, dtype=torch.bfloat16, device="cuda")
        q[..., 0] = (2.0 ** 27 * (1 + step / 24)) / (0.1275 * float(k[0, 0, 0, 0]))
        if fmt == "e4m3":
            cache.k_scale.view(torch.int32)[0, 0, place] += 1 + step % 3
        else:
            k[0, place, 0, 1] = 1.0
            q[..., 1] = 16.0 * (1 + step % 3) / 0.1275
            cache.lens.zero_()
            cache.write(k, v)
            cache.lens.fill_(length)
        o = cache.attend(q)
        cache.sync()
        got = bf16_to_f64(o)
        assert np.all((got >= 1 - EPS) & (got <= 3 * (1 + EPS))), (step, got.min(), got.max())


def test_as_many_rope_rows_as_32_bits_count():
    """2^31 - 1 rows of one 16-wide head, in place; positions past 32 bits at their end."""
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 69 GB")
    kv = _kv()
    n = 2 ** 31 - 1
    x = torch.empty(n, 1, 16, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(0)
    at = [0, 1, 2 ** 30 - 1, 2 ** 30, n - 2, n - 1]
    _, want = _normal(rng, len(at), 1, 16)
    for i, j in enumerate(at):
        x[j] = torch.from_numpy(want[i]).to("cuda", torch.bfloat16)
    spec = kv.RopeSpec(1.0e4, 16)
    kv.rope(x, spec, start_pos=3, out=x)
    got = bf16_to_f64(torch.stack([x[j] for j in at]))
    want = D.rotate(want, [3 + j for j in at], D.scaled_inv_freq(16, 1.0e4))
    # float64 angles of positions around 2^31 are themselves off by 2^-22
    assert np.all(np.abs(got - want) <= EPS * np.abs(want) + 2.0 ** -16)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int4"])
@pytest.mark.parametrize("t,h,hkv,hd", [(1, 3, 1, 128), (5, 4, 2, 64), (40, 4, 2, 64), (100, 6, 2, 128)])
def test_any_softcap(fmt, t, h, hkv, hd):
    """Caps far above the scores leave them as they are; far below, all are the cap."""
    kv = _kv()
    rng = np.random.default_rng(t + hd)
    cache, k64, v64 = _filled(kv, rng, fmt, 1, 300 + t, hkv, hd, [300])
    q, q64 = _normal(rng, 1, t, h, hd, scale=3.0)
    for softcap in (1.0e-3, 0.5, 10.0, 60.0, 70.0, 1.0e3, 1.0e5, 1.0e8, 1.0e30, 3.0e38):
        o = cache.attend(q, softcap=softcap)
        cache.sync()
        _close(cache, o, q64, k64, v64, 300, softcap=softcap)
    # without one: within the same distance of the same values (a cap of 3e38 moves them by
    # less than 1e-70), so the two calls differ by two such tolerances at most
    _close(cache, cache.attend(q), q64, k64, v64, 300, softcap=3.0e38)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int4"])
def test_accepted_rows_that_moved_up_are_the_rows_decoded_one_by_one(fmt):
    """Codes and scale words: afterwards the two caches give the same bits."""
    kv = _kv()
    rng = np.random.default_rng(71)
    h, hkv, hd, length = 6, 2, 128, 333
    spec = kv.RopeSpec(5.0e5, hd)
    parents, path = [-1, 0, 0, 2, 1, 3, 5, 3], [0, 2, 3, 5, 6]
    tree, _, _ = _filled(kv, rng, fmt, 1, 400, hkv, hd, [length])
    words = [] if fmt == "bf16" else [tree.k_scale, tree.v_scale]
    one = kv.KvCache(fmt, 1, 400, hkv, hd, k=tree.k.clone(), v=tree.v.clone(), lens=tree.lens.clone(),
                     k_scale=words[0].clone() if words else None,
                     v_scale=words[1].clone() if words else None)
    k, v = (_normal(rng, 1, len(parents), hkv, hd)[0] for _ in range(2))
    tree.write(k, v, rope=spec, parents=_i32([parents]))
    for node in path:
        one.write(k[:, node:node + 1], v[:, node:node + 1], rope=spec)
        one.lens += 1
    src = torch.tensor(path, device="cuda") + length
    to = slice(length, length + len(path))
    for x in (tree.k, tree.v):
        x.view(torch.uint8)[:, to] = x.view(torch.uint8)[:, src]
    for x in words:
        x[:, :, to] = x[:, :, src]
    tree.lens += len(path)
    for x, y in zip(tree.read(0, 338), one.read(0, 338)):
        assert torch.equal(x, y)
    q, _ = _normal(rng, 1, 3, h, hd)
    k, v = (_normal(rng, 1, 3, hkv, hd)[0] for _ in range(2))
    for cache in (tree, one):
        cache.write(k, v, rope=spec)
    assert torch.equal(tree.attend(q), one.attend(q))
    tree.sync()


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("fmt", ["e4m3", "int4"])
def test_codes_of_rows_of_every_magnitude(fmt, paged):
    """Codes and scale words are the definition's, bit for bit: rows from below the smallest scale to
    bf16's largest numbers, some with values that lie on the borders between codes, where the scale is a power of
    two (halfway between neighbours of the e4m3 grid, or between whole numbers)."""
    kv, hd, hkv = _kv(), 64, 8
    rng = np.random.default_rng(31)
    powers = np.repeat(np.arange(-133, 127), 4)
    n = len(powers)
    x = rng.standard_normal((2, n, hkv, hd))
    x /= np.abs(x).max(-1, keepdims=True)
    x *= 1 + 0.99 * rng.random((2, n, hkv, 1))
    if fmt == "e4m3":
        grid = D.e4m3_values()[:127]
        borders = np.concatenate(((grid[1:] + grid[:-1]) / 2, grid))
        most, unit = 448.0, 2.0 ** -8
    else:
        borders = np.arange(-8, 23) / 2
        most, unit = 11.0, 2.0 ** -3
    rows = rng.choice(borders, (2, n, 2, hd)) * (rng.choice([-1, 1], (2, n, 2, hd)) if fmt == "e4m3" else 1)
    rows[..., 0] = most
    if fmt == "int4":
        rows[..., 1] = -4.0
    x[:, :, :2] = rows * unit
    x = np.ldexp(x, powers[None, :, None, None])
    (k, k64), (v, v64) = (_bf16(y.astype(np.float32)) for y in x)
    if paged:
        from dense_decoder_layer_gb300 import pages
        cache = pages.PagedKvCache(fmt, 1, n // 8, 8, 1, hkv, hd)
        cache.write(k, v, torch.arange(n, dtype=torch.int32, device="cuda"))
        flat = lambda t: t.transpose(1, 2).reshape(n, hkv, *t.shape[3:])
    else:
        cache = kv.KvCache(fmt, 1, n, hkv, hd)
        for at in range(0, n, 256):  # (at most 256 tokens a call)
            cache.lens.fill_(at)
            cache.write(k[None, at:at + 256], v[None, at:at + 256])
        flat = lambda t: t[0] if t.dim() == 4 else t[0].T
    cache.sync()
    for x64, codes, words in ((k64, cache.k, cache.k_scale), (v64, cache.v, cache.v_scale)):
        want, w = D.quantise(x64.astype(np.float32), fmt)
        assert np.array_equal(_words(flat(words)), w)
        have = _codes(flat(codes), fmt)
        same = (have == want) | ((fmt == "e4m3") & (have & 127 == 0) & (want & 127 == 0))  # (a zero's sign)
        assert same.all()
        assert (w >> 23 == 0).any() and ((w >> 23 > 0) & (w >> 23 < 67)).any() and (w >> 23 > 240).any()
