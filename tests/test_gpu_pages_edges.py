"""The paged cache at its edges: values far apart or not finite, offsets beyond 32 bits, large
batches, streams, captured steps, and the operators in a run beside the contiguous cache.

Tolerances as in test_gpu_pages.py; where two ways of the same sum are compared, the sum of both."""

import math

import numpy as np
import pytest

from oracle import pages as P
from parity import bf16_to_f64
from test_gpu_kv import _bf16, _i32, _normal
from test_gpu_pages import FORMATS, _cache, _check, _filled, _mods, _raw, _values

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BUSY = 50_000_000  # cycles that a stream is kept busy for, some 25 ms


def _write_all(cache, lens, k, v):
    slots, _, _ = cache.slots(_i32([0] * len(lens)), _i32(lens), rows=sum(lens))
    cache.write(k, v, slots)
    cache.sync()


@pytest.mark.parametrize("fmt", FORMATS)
def test_values_that_are_not_finite_stay_with_their_sequence_and_head(fmt):
    rng = np.random.default_rng(1)
    lens, new = [300, 40, 129], [1, 1, 1]
    total = [301, 41, 130]
    cache = _cache(fmt, lens, new, 16, 2, 128)
    k = rng.standard_normal((sum(total), 2, 128)).astype(np.float32)
    v = rng.standard_normal((sum(total), 2, 128)).astype(np.float32)
    k[150, 0, 5] = np.nan        # the first sequence's first kv head
    v[301 + 3, 1, 7] = np.inf    # the second's second
    _write_all(cache, total, _bf16(k)[0], _bf16(v)[0])
    q, q64 = _normal(rng, 3, 8, 128)
    bad = q.clone()
    bad[2, 6, 100] = float("inf")  # one head of the third
    values = _values(cache, total)
    o = cache.attend(bad)
    cache.sync()
    got = bf16_to_f64(o)
    assert np.isnan(got[0, :4]).all() and np.isfinite(got[0, 4:]).all()
    assert np.isfinite(got[1, :4]).all() and not np.isfinite(got[1, 4:]).all(-1).any()
    assert np.isnan(got[2, 6]).any() and np.isfinite(np.delete(got[2], 6, 0)).all()
    # what is finite is right
    clean = [tuple(np.where(np.isfinite(x), x, 0) for x in kv) for kv in values]
    ok = torch.from_numpy(np.isfinite(got).all(-1)).cuda()
    ref = cache.attend(q)
    assert torch.equal(o[ok], ref[ok])
    for s, h in ((0, slice(4, 8)), (1, slice(0, 4)), (2, slice(0, 8))):
        want, size, _ = P.attend(q64[s], *clean[s], 0, total[s])
        assert np.all(np.abs(bf16_to_f64(ref)[s, h] - want[h]) <= 2.0 ** -7 * size[h] + 1e-6)


@pytest.mark.parametrize("group,hd", [(3, 128), (8, 64)])
@pytest.mark.parametrize("extra", [0, 4000])
@pytest.mark.parametrize("where", ["last", "tile", "first", "both"])
def test_scores_of_minus_infinity_weigh_nothing(where, extra, group, hd):
    """A part of a cut sequence may hold only rows that weigh nothing: the others make the result, whichever
    schedule cuts it (clusters over a narrow table, equal shares over a wide one).

    |o| and the weighted sum of |v| that the errors are measured by are both below `size`: 2^-8 of it for the
    result's rounding, and less than that for the scores (sums of |q k| below 400, times 136 2^-23 twice)
    and the weights (2^-16)."""
    rng = np.random.default_rng(21)
    hkv, lens = 8, [1024, 130]
    cache = _cache("bf16", lens, [1, 1], 16, hkv, hd, extra=extra)
    total = [x + 1 for x in lens]
    k = rng.standard_normal((sum(total), hkv, hd)).astype(np.float32)
    v = rng.standard_normal((sum(total), hkv, hd)).astype(np.float32)
    rows = {"last": [1024], "tile": range(256, 384), "first": range(128), "both": [*range(512), 1024]}[where]
    k[list(rows), :, 5] = -np.inf
    _write_all(cache, total, _bf16(k)[0], _bf16(v)[0])
    q = rng.standard_normal((2, hkv * group, hd)).astype(np.float32)
    q[:, :, 5] = np.abs(q[:, :, 5]) + 0.1
    q, q64 = _bf16(q)
    got = bf16_to_f64(cache.attend(q))
    cache.sync()
    for s, kv in enumerate(_values(cache, total)):
        want, size, _ = P.attend(q64[s], *kv, 0, total[s])
        assert np.isfinite(want).all()
        assert np.all(np.abs(got[s] - want) <= 2.0 ** -7 * size)


@pytest.mark.parametrize("fmt", ["e4m3", "int4"])
@pytest.mark.parametrize("spread", [0, 20, 60, -60])
def test_scales_far_apart(fmt, spread):
    """V rows of magnitudes 2^spread apart, in and out of sight; K rows so that the small ones count."""
    rng = np.random.default_rng(2)
    lens, hd = [700, 130], 64
    total = [701, 131]
    cache = _cache(fmt, lens, [1, 1], 8, 1, hd)
    k = rng.standard_normal((sum(total), 1, hd)) * 0.5
    v = rng.standard_normal((sum(total), 1, hd))
    up = np.zeros(sum(total))
    up[::7] = spread
    up[0] = 0
    v *= np.exp2(up)[:, None, None]
    v[5] = 0  # rows of zeros, seen by everyone
    _write_all(cache, total, _bf16(k.astype(np.float32))[0], _bf16(v.astype(np.float32))[0])
    q, q64 = _normal(rng, 2, 5, hd)
    for window in (0, 3):
        o = cache.attend(q, window=window)
        cache.sync()
        _check(fmt, o, q64, _values(cache, total), lens, [1, 1], window=window)


@pytest.mark.parametrize("fmt", ["e4m3", "int4"])
@pytest.mark.parametrize("group,hd", [(3, 128), (8, 64)])
@pytest.mark.parametrize("extra", [0, 4000])
@pytest.mark.parametrize("power", [-100, -40, 0, 60, 100])
def test_rows_of_zeros_before_small_and_large_scales(fmt, power, extra, group, hd):
    """V rows of zeros at a sequence's start, over whole tiles and between tiles, the others' scales close
    together but far from 1: what a row of zeros is taken for goes by theirs."""
    rng = np.random.default_rng(22)
    hkv, lens = 2, [1100, 300, 3, 640]
    total = [x + 1 for x in lens]
    cache = _cache(fmt, lens, [1] * 4, 16, hkv, hd, extra=extra)
    k = rng.standard_normal((sum(total), hkv, hd)) * 0.2
    v = rng.standard_normal((sum(total), hkv, hd)) * 2.0 ** power
    at = np.cumsum([0] + total)
    for s, rows in enumerate(([0, 1, *range(256, 700)], range(290), [0], [*range(130), *range(200, 390), 640])):
        v[at[s] + np.array(rows)] = 0
    v[at[3] + 150, 0] = 0  # and in one head only
    _write_all(cache, total, _bf16(k.astype(np.float32))[0], _bf16(v.astype(np.float32))[0])
    q, q64 = _normal(rng, 4, hkv * group, hd)
    values = _values(cache, total)
    assert all((np.abs(x[1]).max() > 2.0 ** power) for x in values)
    for window in (0, 200):
        o = cache.attend(q, window=window)
        cache.sync()
        _check(fmt, o, q64, values, lens, [1] * 4, window=window)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("scale", [1e-6, 30.0])
def test_flat_and_steep_scores(fmt, scale):
    rng = np.random.default_rng(3)
    lens, new = [1000, 257], [1, 1]
    cache, values = _filled(fmt, rng, lens, new, 32, 2, 128, kscale=1.0)
    q, q64 = _normal(rng, 2, 6, 128, scale=scale)
    o = cache.attend(q)
    cache.sync()
    _check(fmt, o, q64, values, lens, new)


@pytest.mark.parametrize("fmt", FORMATS)
def test_the_largest_weight_in_any_place(fmt):
    """One key far above the others, first, last, at a tile's or a page's edge: its row comes out."""
    rng = np.random.default_rng(4)
    n, hd = 9, 128
    lens = [600] * n
    cache, values = _filled(fmt, rng, lens, [1] * n, 16, 1, hd)
    q, q64 = _normal(rng, n, 2, hd, scale=0.1)
    for s, row in enumerate((0, 1, 15, 16, 127, 128, 511, 599, 600)):
        k, v = values[s]
        for h in range(2):
            x = 40 * k[row, 0] / np.abs(k[row, 0]).max()
            q[s, h], _ = _bf16(x.astype(np.float32))
            q64[s, h] = bf16_to_f64(q[s, h])
    o = cache.attend(q)
    cache.sync()
    _check(fmt, o, q64, values, lens, [1] * n)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("order", ["heads", "rows"])
def test_pools_beyond_32_bits(fmt, order):
    """Pages at the far end of a pool of more than 2^32 bytes."""
    rng = np.random.default_rng(5)
    hkv, hd, page = 8, 128, 64
    n_pages = {"bf16": 1 << 16, "e4m3": 1 << 17, "int4": 1 << 17}[fmt]  # 8 GiB, 4 for int4 and e4m3 8
    _, pages = _mods()
    from test_gpu_pages import _pool
    k, v = _pool(fmt, n_pages, page, hkv, hd, order)
    lens = [500, 63]
    table = np.full((2, 8), -1)
    far = n_pages - 1 - np.arange(9)
    table[0, :8], table[1, 0] = far[:8], far[8]
    cache = pages.PagedKvCache(fmt, 2, n_pages, page, 8, hkv, hd, k=k, v=v, table=_i32(table), lens=_i32(lens))
    total = [x + 1 for x in lens]
    kx, _ = _normal(rng, sum(total), hkv, hd)
    vx, _ = _normal(rng, sum(total), hkv, hd)
    _write_all(cache, total, kx, vx)
    # the same rows in a small pool
    small = _cache(fmt, lens, [1, 1], page, hkv, hd, order)
    _write_all(small, total, kx, vx)
    q, q64 = _normal(rng, 2, 16, hd)
    assert torch.equal(cache.attend(q), small.attend(q))
    slots, _, _ = cache.slots(_i32([0, 0]), _i32(total), rows=sum(total))
    there, _, _ = small.slots(_i32([0, 0]), _i32(total), rows=sum(total))
    assert all(torch.equal(x, y) for x, y in zip(cache.read(slots), small.read(there)))
    cache.sync()
    assert (_raw(cache.k)[:n_pages - 9] == 0).all()


@pytest.mark.parametrize("n,h,hkv,hd,fmt", [(4096, 2, 1, 64, "e4m3"), (1500, 4, 2, 128, "bf16"),
                                            (300, 40, 2, 64, "int4"), (33, 8, 8, 128, "e4m3")])
def test_many_sequences(n, h, hkv, hd, fmt):
    rng = np.random.default_rng(n)
    lens = [int(x) for x in rng.integers(0, 40, n)]
    lens[n // 2] = 5000  # one that is cut
    new = [int(x) for x in rng.integers(0, 2, n)]
    new[n // 2] = 1
    cache, values = _filled(fmt, rng, lens, new, 8, hkv, hd)
    q, q64 = _normal(rng, n, h, hd)
    o = cache.attend(q, new=_i32(new))
    cache.sync()
    _check(fmt, o, q64, values, lens, new)


def test_all_idle():
    for n in (1, 5, 100):
        cache = _cache("e4m3", [30] * n, [0] * n, 8, 2, 64)
        q, _ = _normal(np.random.default_rng(0), n, 4, 64)
        o = torch.full_like(q, 7.0)
        assert (cache.attend(q, new=_i32([0] * n), out=o) == 0).all()
        slots, positions, starts = cache.reserve(_i32([0] * n), rows=0)
        assert slots.numel() == 0 and (starts == 0).all()
        cache.sync()


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_serving_run_beside_the_contiguous_cache(fmt):
    """Prompts let in, decode steps, sequences that end and others in their places: the same rows, and the
    same attention, as in a contiguous cache per request."""
    kv, pages = _mods()
    rng = np.random.default_rng(8)
    n, hkv, h, hd, page = 5, 2, 6, 64, 8
    cache = pages.PagedKvCache(fmt, n, 40, page, 16, hkv, hd)
    spec = kv.RopeSpec(1.0e4, hd)
    flat = [None] * n

    def step(new, fresh):
        lens = cache.lens.tolist()
        for s in fresh:
            flat[s] = kv.KvCache(fmt, 1, page * 16, hkv, hd)
        rows = sum(new) + 2
        slots, positions, starts = cache.reserve(_i32(new), rows=rows)
        k, k64 = _normal(rng, rows, hkv, hd)
        v, _ = _normal(rng, rows, hkv, hd)
        x, _ = _normal(rng, rows, h, hd)
        kv.rope(x, spec, positions=positions, out=x)
        cache.write(k, v, slots, rope=spec, positions=positions)
        at = starts.tolist()
        q = torch.zeros(n, h, hd, dtype=torch.bfloat16, device="cuda")
        want = torch.zeros_like(q)
        for s in range(n):
            if not new[s]:
                continue
            part = slice(at[s], at[s + 1])
            q[s] = x[at[s + 1] - 1]
            flat[s].write(k[part][None], v[part][None], rope=spec)
            # the contiguous cache takes the tokens one after the other: its last one sees all
            o = flat[s].attend(x[part][None])
            want[s] = o[0, -1]
            flat[s].lens += new[s]
        got = cache.attend(q, new=_i32(new))
        cache.lens += _i32(new)
        cache.sync()
        a, b = bf16_to_f64(got), bf16_to_f64(want)
        # (the contiguous one's weights are rounded to bf16 or fp16: 2^-8 of |v|, whose largest is below 8)
        assert np.all(np.abs(a - b) <= 2.0 ** -8 * (np.abs(a) + np.abs(b)) + 2.0 ** -8 * 8)
        now = cache.lens.tolist()
        for s in range(n):
            if now[s]:
                there, _, _ = cache.slots(_i32([0] * n), _i32([now[s] if i == s else 0 for i in range(n)]),
                                          rows=now[s])
                for x1, x2 in zip(cache.read(there), flat[s].read(0, now[s])):
                    assert torch.equal(x1.view(torch.int16), x2[0].view(torch.int16))

    def end(gone):
        keep = cache.lens.clone()
        keep[gone] = 0
        cache.release(keep)
        cache.lens = keep

    step([5, 0, 17, 1, 30], fresh=range(n))
    step([1, 1, 1, 1, 1], fresh=[])
    end([2, 4])
    step([1, 9, 3, 1, 60], fresh=[2, 4])
    for _ in range(9):
        step([1] * n, fresh=[])
    end([0, 1, 2, 3, 4])
    assert int(cache.n_free) == 40 and sorted(cache.free.tolist()) == list(range(40))


def test_a_prefix_in_pages_goes_on_in_a_stack():
    """A prompt's rows, kept in pages layer by layer, gathered by slot into another stack's contiguous
    caches: its next tokens are those of the stack that made the rows, bit for bit."""
    import synth
    from dense_decoder_layer_gb300.stack import DenseStack
    _, pages = _mods()
    dims = synth.Dims(2, 512, 8, 2, 64, 1536, 100, 0, 1.0e4)
    layers, _, _, hidden = synth.draw_workload(dims)
    more = np.random.default_rng(51).standard_normal((30, dims.d_model)).astype(np.float32)
    first, second = (DenseStack(dims, 200, 100) for _ in range(2))
    for stack in (first, second):
        stack.load_layers(layers)
    first.prefill(torch.from_numpy(hidden), 0)
    first.sync()
    hkv, hd, rows = dims.n_kv_heads, dims.head_dim, hidden.shape[0]
    for l in range(dims.n_layers):
        # (one book could serve all layers; another request's pages lie between)
        cache = pages.PagedKvCache("bf16", 2, 40, 16, 10, hkv, hd)
        slots, _, _ = cache.reserve(_i32([23, 0]), rows=23)
        cache.lens = _i32([23, 0])
        slots, _, _ = cache.reserve(_i32([0, rows]), rows=rows)
        cache.write(*first.rows(l, 0, rows), slots)
        there, _, _ = cache.slots(_i32([0, 0]), _i32([0, rows]), rows=rows)
        cache.read(there, k_out=second.rows(l, 0, rows)[0], v_out=second.rows(l, 0, rows)[1])
        cache.sync()
        assert torch.equal(first.k_cache[l][:rows], second.k_cache[l][:rows])
    a, b = (stack.prefill(torch.from_numpy(more), rows) for stack in (first, second))
    assert torch.equal(a, b) and a.abs().max() > 0
    for l in range(dims.n_layers):
        for x, y in zip(first.rows(l, rows, 30), second.rows(l, rows, 30)):
            assert torch.equal(x, y)


# ------------------------------------------------------- streams and graphs


def test_calls_on_another_stream():
    rng = np.random.default_rng(9)
    lens, new = [3000, 100], [1, 1]
    cache, values = _filled("e4m3", rng, lens, new, 16, 8, 128)
    q, q64 = _normal(rng, 2, 32, 128)
    want = cache.attend(q)
    slots, _, _ = cache.slots(_i32([0, 0]), _i32([3001, 101]), rows=3102)
    back = cache.read(slots)
    first, count = _i32([0, 0]), _i32([3001, 101])
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    junk = torch.empty_like(q).fill_(7.0)  # behind the sleep, as memory that may come back
    del junk
    o = cache.attend(q, stream=stream)
    there, _, _ = cache.slots(first, count, rows=3102, stream=stream)
    got = cache.read(there, stream=stream)
    stream.synchronize()
    assert torch.equal(o, want) and torch.equal(there, slots)
    assert all(torch.equal(a, b) for a, b in zip(got, back))
    torch.cuda.synchronize()
    assert cache.workspace(32).data_ptr() != cache.workspace(32, stream=stream).data_ptr()
    cache.sync()


def test_two_streams_at_once():
    rng = np.random.default_rng(10)
    lens, new = [5000, 4000, 300], [1, 1, 1]
    cache, _ = _filled("bf16", rng, lens, new, 16, 8, 128)
    streams = [torch.cuda.Stream() for _ in range(2)]
    qs = [_normal(rng, 3, 32, 128)[0] for _ in range(2)]
    want = [cache.attend(q) for q in qs]
    outs = [torch.empty_like(q) for q in qs]
    torch.cuda.synchronize()
    for _ in range(50):
        for q, o, s in zip(qs, outs, streams):
            cache.attend(q, out=o, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    cache.sync()


@pytest.mark.parametrize("max_pages", [40, 4000])
@pytest.mark.parametrize("fmt", FORMATS)
def test_captured_steps(fmt, max_pages):
    """A decode step with all lengths on the device, captured once and replayed while the sequences grow
    over page borders; beside it another cache's graph on another stream.  Tables for short and for long
    sequences: cut over clusters, and over all blocks."""
    kv, pages = _mods()
    rng = np.random.default_rng(11)
    n, hkv, h, hd, page, steps = 4, 8, 32, 128, 8, 20
    spec = kv.RopeSpec(1.0e4, hd)
    ones = _i32([1] * n)
    data = [[_normal(rng, n, x, hd)[0] for x in (hkv, hkv, h)] for _ in range(steps)]

    def make():
        cache = pages.PagedKvCache(fmt, n, 64, page, max_pages, hkv, hd)
        cache.reserve(_i32([1, 0, 0, 0]), rows=1)
        start = _i32([3, 0, 60, 17])
        slots, positions, _ = cache.reserve(start, rows=80)
        k, v = (_bf16(np.random.default_rng(5 + i).standard_normal((80, hkv, hd)).astype(np.float32))[0]
                for i in range(2))
        cache.write(k, v, slots, rope=spec, positions=positions)
        cache.lens = start
        return cache

    def body(cache, k, v, q):
        slots, positions, _ = cache.reserve(ones, rows=n)
        kv.rope(q, spec, positions=positions, out=q)
        cache.write(k, v, slots, rope=spec, positions=positions)
        o = cache.attend(q, new=ones)
        cache.lens += ones
        return o

    eager = make()
    want = [body(eager, k.clone(), v.clone(), q.clone()) for k, v, q in data]
    eager.sync()
    runs = []
    for _ in range(2):
        cache = make()
        static = [torch.zeros_like(x) for x in data[0]]
        lens = cache.lens.clone()
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):  # once outside of a capture
            body(cache, *static)
        torch.cuda.synchronize()
        cache.release(lens)
        cache.lens = lens
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            o = body(cache, *static)
        runs.append((cache, static, graph, o, stream))
    torch.cuda.synchronize()
    for i in range(steps):
        for cache, static, graph, o, stream in runs:
            with torch.cuda.stream(stream):
                for to, x in zip(static, data[i]):
                    to.copy_(x)
                graph.replay()
        torch.cuda.synchronize()
        for cache, static, graph, o, stream in runs:
            assert torch.equal(o, want[i]), i
    for cache, *_ in runs:
        assert torch.equal(cache.lens, eager.lens) and torch.equal(cache.held, eager.held)
        cache.sync()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_two_graphs_of_one_cache_at_once(fmt):
    rng = np.random.default_rng(12)
    lens = [9000, 8000, 300]
    cache, _ = _filled(fmt, rng, lens, [1, 1, 1], 16, 8, 128)
    qs = [_normal(rng, 3, 32, 128)[0] for _ in range(2)]
    want = [cache.attend(q) for q in qs]
    graphs, outs = [], []
    for q in qs:
        stream = torch.cuda.Stream()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            outs.append(cache.attend(q))
        graphs.append((g, stream))
    torch.cuda.synchronize()
    for _ in range(30):
        for g, stream in graphs:
            with torch.cuda.stream(stream):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    cache.sync()


def test_a_window_over_pages_given_back():
    """Rows before every window are nobody's: their pages' entries may be anything."""
    rng = np.random.default_rng(13)
    for fmt in FORMATS:
        lens = [700, 129]
        cache, values = _filled(fmt, rng, lens, [1, 1], 16, 2, 64)
        cache.table[0, :(701 - 100) // 16] = -1
        q, q64 = _normal(rng, 2, 4, 64)
        o = cache.attend(q, window=100)
        cache.sync()
        _check(fmt, o, q64, values, lens, [1, 1], window=100)


def test_device_that_is_not_current_and_wrong_devices():
    _, pages = _mods()
    cache = _cache("bf16", [5], [1], 8, 1, 64)
    q, _ = _normal(np.random.default_rng(0), 1, 2, 64)
    with pytest.raises(ValueError):
        cache.attend(q.cpu())
    with pytest.raises(ValueError):
        cache.attend(q, new=torch.ones(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        cache.reserve(_i32([1]), slots=torch.zeros(1, dtype=torch.int32))
    if torch.cuda.device_count() > 1:
        with torch.cuda.device(1):
            assert cache.attend(q).device.index == 0
