"""Cached decoding on streams other than the current one."""

import numpy as np
import pytest

from test_gpu_kv import _filled, _kv, _normal

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
    cache.sync()
