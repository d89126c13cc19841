"""What the kernels' sources have to keep to, read as text on the host."""

import pathlib
import re

import pytest

CSRC = pathlib.Path(__file__).parents[1] / "dense_decoder_layer_gb300" / "csrc"
SOURCES = sorted(p.name for p in CSRC.glob("*.cu*"))


def _closing(text, at, pair):
    """Index behind the bracket that closes the one at `at`."""
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == pair[0]) - (text[i] == pair[1])
        if depth == 0:
            return i + 1
    raise AssertionError("unbalanced " + pair)


def _kernels(text):
    """(name, parameters, body) of every kernel that a source defines."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"\b__global__\b", text):
        head = re.compile(r"(?:__launch_bounds__\s*(?P<bounds>\()|(?P<name>\w+)\s*(?P<params>\())")
        at = m.end()
        while True:
            h = head.search(text, at)
            if h.group("name") and h.group("name") != "__launch_bounds__":
                break
            at = _closing(text, text.index("(", h.start()), "()")
        params_end = _closing(text, h.start("params"), "()")
        body = text[params_end:]
        if not body.lstrip().startswith("{"):
            continue  # a declaration
        at = text.index("{", params_end)
        yield h.group("name"), text[h.start("params"):params_end], text[at:_closing(text, at, "{}")]


def test_the_reader_of_sources_finds_the_kernels():
    found = {name for s in SOURCES for name, _, _ in _kernels((CSRC / s).read_text())}
    assert {"rope_kernel", "cache_write_kernel", "cache_read_kernel", "pages_scan_kernel", "pages_write_kernel",
            "pages_read_kernel", "pages_attn_kernel", "pages_join_kernel", "norm_prep_kernel"} <= found


@pytest.mark.parametrize("source", SOURCES)
def test_kernels_that_start_early_promise_no_unchanging_memory(source):
    """A kernel that waits for the one before it (griddepcontrol.wait) starts while that one still writes.
    A pointer to const declared __restrict__ says that nothing changes the memory while the kernel runs, so that
    its loads may pass the wait: it is not true here."""
    for name, params, body in _kernels((CSRC / source).read_text()):
        if "grid_dep_wait" in body:
            assert not re.search(r"const\s+\w+\s*\*\s*__restrict__", params), name
