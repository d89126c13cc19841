"""Cached decoding on streams other than the current one, and in captured graphs that
run at the same time."""

import numpy as np
import pytest

from test_gpu_kv import _filled, _i32, _kv, _normal

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BUSY = 50_000_000  # cycles that the current stream is kept busy for, some 25 ms


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_read_on_another_stream_makes_its_outputs_there(fmt):
    kv = _kv()
    cache, _, _ = _filled(kv, np.random.default_rng(1), fmt, 2, 300, 2, 64, [300, 200])
    want = cache.read(0, 300)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    got = cache.read(0, 300, stream=stream)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    cache.sync()


def test_outputs_are_not_memory_that_the_current_stream_still_uses():
    kv = _kv()
    rng = np.random.default_rng(2)
    cache, _, _ = _filled(kv, rng, "e4m3", 1, 6100, 2, 128, [6000])
    spec = kv.RopeSpec(1.0e4, 128)
    q, _ = _normal(rng, 1, 3, 8, 128)
    calls = [lambda **kw: cache.attend(q, **kw), lambda **kw: kv.rope(q, spec, start_pos=5, **kw)]
    for call in calls:
        want = call()
        torch.cuda.synchronize()
        for _ in range(3):  # (the second time the stream has memory of its own)
            stream = torch.cuda.Stream()
            torch.cuda._sleep(BUSY)
            old = torch.empty_like(q)
            old.fill_(7.0)  # behind the sleep
            del old
            got = call(stream=stream)
            torch.cuda.synchronize()
            assert torch.equal(got, want)
    n = cache.workspace(3, 8).numel()
    old = torch.empty(n, dtype=torch.uint8, device="cuda")
    there = old.data_ptr()
    del old
    stream = torch.cuda.Stream()
    assert cache.workspace(3, 8, stream=stream).data_ptr() != there
    cache.sync()


def test_calls_of_one_shape_on_two_streams():
    kv = _kv()
    rng = np.random.default_rng(3)
    cache, _, _ = _filled(kv, rng, "e4m3", 2, 6100, 2, 128, [6000, 2500])
    streams = [torch.cuda.Stream() for _ in range(4)]
    for t in (1, 40):
        qs = [_normal(rng, 2, t, 8, 128)[0] for _ in streams]
        wants = [cache.attend(q) for q in qs]
        assert len({cache.workspace(t, 8, stream=s).data_ptr() for s in streams}) == len(streams)
        torch.cuda.synchronize()
        for _ in range(20):
            outs = [cache.attend(q, stream=s) for q, s in zip(qs, streams)]
            with torch.cuda.stream(streams[0]):
                again = cache.attend(qs[0])
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(outs + [again], wants + [wants[0]]))
    cache.sync()


def test_captured_graphs_that_run_at_the_same_time():
    """Two graphs of the same cache and shape, and eager calls beside them."""
    kv = _kv()
    rng = np.random.default_rng(4)
    cache, _, _ = _filled(kv, rng, "e4m3", 2, 6100, 2, 128, [6000, 2500])
    for t in (1, 40):
        qs = [_normal(rng, 2, t, 8, 128)[0] for _ in range(3)]
        wants = [cache.attend(q) for q in qs]
        eager, outs, graphs = torch.cuda.Stream(), [], []
        torch.cuda.synchronize()
        with torch.cuda.stream(eager):
            cache.attend(qs[2])
        for q in qs[:2]:
            graph, out = torch.cuda.CUDAGraph(), torch.empty_like(q)
            with torch.cuda.graph(graph, stream=eager):
                for _ in range(3):
                    cache.attend(q, out=out)
            graphs.append(graph), outs.append(out)
        streams = [torch.cuda.Stream() for _ in graphs]
        for _ in range(20):
            for graph, stream in zip(graphs, streams):
                with torch.cuda.stream(stream):
                    graph.replay()
            with torch.cuda.stream(eager):
                last = cache.attend(qs[2])
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(outs + [last], wants))
    cache.sync()


def test_lengths_still_move_between_replays():
    """The graph's own workspace serves any lengths up to max_len."""
    kv = _kv()
    rng = np.random.default_rng(5)
    cache, _, _ = _filled(kv, rng, "bf16", 3, 3000, 2, 64, [10, 10, 10])
    q, _ = _normal(rng, 3, 2, 4, 64)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(q)
    cache.attend(q)
    with torch.cuda.graph(graph):
        cache.attend(q, out=out)
    for lens in ([10, 0, 2000], [2998, 2998, 2998], [1, 700, 30]):
        cache.lens.copy_(_i32(lens))
        graph.replay()
        want = cache.attend(q)
        assert torch.equal(out, want)
    cache.sync()
