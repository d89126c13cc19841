"""PyTorch-side owner of a paged decoding cache: one pool of pages for many sequences,
tables and slot maps made on the GPU, rows in and out by slot, and attention of one new
token per sequence.

Every step runs in ``libpds.so`` through :mod:`.pds` (the section on the paged cache in
``include/pds.h`` says what each call computes).  A step of a serving batch, prompts and
single tokens together, all lengths on the device::

    cache = pages.PagedKvCache("e4m3", n_seqs=64, n_pages=4096, page_size=16, max_pages=512,
                               n_kv_heads=8, head_dim=128)
    slots, positions, starts = cache.reserve(new, rows=n_rows)   # new: int32 [n_seqs]
    kv.rope(q, spec, positions=positions, out=q)                 # q, k, v: the new rows, packed
    cache.write(k, v, slots, rope=spec, positions=positions)
    o = cache.attend(last_q, new=new)                            # one token per sequence
    cache.lens += new
    cache.release(keep)                                          # finished sequences: keep 0, lens 0

A call with ``stream`` does what it would do under ``torch.cuda.stream(stream)``:
what it allocates belongs to that stream, its inputs have to be ready there and to be
kept until it is done with them.  The calls record no gradients and refuse tensors that
require one.
"""

from __future__ import annotations

import torch

from . import kv, pds
from .kv import FORMATS, _call, _index, _int32, _need, _new, _no_gradient, _rows

_I32 = torch.int32


class PagedKvCache:
    """One layer's K/V rows of ``n_seqs`` sequences in ``n_pages`` pages of ``page_size`` rows (8,
    16, 32 ... 1024), at most ``max_pages`` of them per sequence.

    ``fmt`` is one of :class:`kv.KvCache`'s: "bf16", "e4m3" or "int4".  Tensors may be given: ``k``,
    ``v`` [n_pages, n_kv_heads, page_size, head_dim] (bfloat16, float8_e4m3fn, or uint8 with
    head_dim/2 bytes), in any order of pages, heads and rows whose channels are contiguous;
    ``k_scale``, ``v_scale`` contiguous [n_pages, n_kv_heads, page_size] (float32 for e4m3, int32 for
    int4); and, int32 and contiguous, ``table`` [n_seqs, max_pages], ``held`` [n_seqs] pages
    of each sequence, ``lens`` [n_seqs] rows before the new ones, ``free`` [n_pages] and ``n_free``
    [1]: the pages that no sequence has are free[:n_free], taken from the end.  Without them
    nobody has a page.  A program with tables of its own gives ``table`` and does without
    ``reserve`` and ``release``.

    ``max_pages`` bounds the sequences' lengths, and the attention is laid out for what it allows:
    a table no wider than needed serves few short sequences up to 2.4 us faster.
    """

    def __init__(self, fmt, n_seqs, n_pages, page_size, max_pages, n_kv_heads, head_dim,
                 device="cuda", k=None, v=None, k_scale=None, v_scale=None, table=None, held=None,
                 lens=None, free=None, n_free=None):
        self.fmt = fmt
        for name, x in (("n_seqs", n_seqs), ("n_pages", n_pages), ("page_size", page_size),
                        ("max_pages", max_pages), ("n_kv_heads", n_kv_heads), ("head_dim", head_dim)):
            setattr(self, name, _int32(int(x), name))
        given = next((t for t in (k, table) if t is not None), None)
        self.device = torch.device(device) if given is None else given.device
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.index = self.device.index
        dtype, per_byte = {"bf16": (torch.bfloat16, 1), "e4m3": (torch.float8_e4m3fn, 1),
                           "int4": (torch.uint8, 2)}[fmt]
        rows = (self.n_pages, self.n_kv_heads, self.page_size, self.head_dim // per_byte)
        words = {"bf16": None, "e4m3": torch.float32, "int4": torch.int32}[fmt]

        def have(t, shape, dtype, what, packed=True):
            if t is None:
                return torch.zeros(shape, dtype=dtype, device=self.device)
            _need(t.dtype == dtype and tuple(t.shape) == tuple(shape) and t.device == self.device,
                  f"{what}: {dtype} {tuple(shape)} on {self.device}")
            _no_gradient(t, what)
            _need(t.is_contiguous() if packed else t.stride(-1) == 1, f"{what}: layout")
            return t

        k, v = have(k, rows, dtype, "k", False), have(v, rows, dtype, "v", False)
        packed = k.is_contiguous() and v.is_contiguous()
        _need(packed or k.stride() == v.stride(), "k and v: the same strides")
        _need(packed or any(k.stride()[:3]), "k and v: rows of their own (an expanded tensor?)")
        if words is not None:
            k_scale = have(k_scale, rows[:3], words, "k_scale")
            v_scale = have(v_scale, rows[:3], words, "v_scale")
        else:
            k_scale = v_scale = None
        _need((free is None) == (n_free is None), "free and n_free: both or neither")
        _need(free is not None or table is not None or held is None, "held: with a table")
        booked = table is None or free is not None  # else the table is the caller's to keep
        table = have(table, (self.n_seqs, self.max_pages), _I32, "table")
        lens = have(lens, (self.n_seqs,), _I32, "lens")
        if booked or held is not None:
            held = have(held, (self.n_seqs,), _I32, "held")
        if booked:
            if free is None:
                free = torch.arange(self.n_pages - 1, -1, -1, dtype=_I32, device=self.device)
                n_free = torch.full((1,), self.n_pages, dtype=_I32, device=self.device)
            free = have(free, (self.n_pages,), _I32, "free")
            n_free = have(n_free, (1,), _I32, "n_free")
        self._tensors = k, v, k_scale, v_scale, table, held, free, n_free
        self._lens = lens
        page, head, row, _ = (0, 0, 0, 0) if packed else k.stride()

        def ptr(t):
            return None if t is None else t.data_ptr()

        self.c = pds.pds_pages(
            FORMATS[fmt], self.n_seqs, self.n_pages, self.page_size, self.max_pages, self.n_kv_heads,
            self.head_dim, 0, page * per_byte, row * per_byte, head * per_byte, ptr(k), ptr(v),
            ptr(k_scale), ptr(v_scale), ptr(table), ptr(held), ptr(lens), ptr(free), ptr(n_free))
        self._ws = {}  # attention workspace by (heads, stream)

    # The kernels have these tensors' addresses: they can be written to, not replaced.
    k = property(lambda self: self._tensors[0], doc="The K rows.")
    v = property(lambda self: self._tensors[1], doc="The V rows.")
    k_scale = property(lambda self: self._tensors[2], doc="K's scale words (None: bf16).")
    v_scale = property(lambda self: self._tensors[3], doc="V's scale words (None: bf16).")
    table = property(lambda self: self._tensors[4], doc="Pages of each sequence.")
    held = property(lambda self: self._tensors[5], doc="How many it has (None: tables of the caller's own).")
    free = property(lambda self: self._tensors[6], doc="Pages that no sequence has, in [:n_free].")
    n_free = property(lambda self: self._tensors[7], doc="How many these are.")

    @property
    def lens(self):
        """Rows of each sequence before its new ones (int32, on the device); assigning copies into it."""
        return self._lens

    @lens.setter
    def lens(self, value):
        if value is not self._lens:
            self._lens.copy_(value)

    def _map(self, rows, slots, positions, starts):
        rows = slots.numel() if rows is None else rows
        return (_int32(rows, "rows"), _index(slots, rows, self.index, "slots"),
                _index(positions, rows, self.index, "positions"),
                _index(starts, self.n_seqs + 1, self.index, "starts"))

    def _made(self, rows, stream):
        return _new(torch.empty, _int32(rows, "rows"), self.device, stream, _I32)

    def reserve(self, new, rows=None, slots=None, positions=None, starts=None, stream=None):
        """Pages for ``new`` [n_seqs] (int32) rows behind each sequence's ``lens``, and where
        these rows are: (slots, positions, starts), rows packed in the order of the sequences,
        ``starts`` [n_seqs + 1] the first of each.  ``rows`` (or the size of ``slots``) bounds their
        number; entries behind the last row are -1 and position 0."""
        _need(rows is not None or slots is not None, "rows: how many there may be, or slots to fill")
        if slots is None:
            slots = self._made(rows, stream)
        if positions is None:
            positions = self._made(slots.numel(), stream)
        if starts is None:
            starts = self._made(self.n_seqs + 1, stream)
        args = self._map(rows, slots, positions, starts)
        _call(pds.load().pds_pages_reserve, self.index, stream, self.c,
              _index(new, self.n_seqs, self.index, "new"), *args)
        return slots, positions, starts

    def slots(self, first, count, rows=None, slots=None, positions=None, starts=None, stream=None):
        """The same map of rows ``first`` .. ``first + count - 1`` (int32 [n_seqs]) that the
        sequences have; ``positions`` and ``starts`` are filled where they are given (else None)."""
        _need(rows is not None or slots is not None, "rows: how many there may be, or slots to fill")
        if slots is None:
            slots = self._made(rows, stream)
        args = self._map(rows, slots, positions, starts)
        _call(pds.load().pds_pages_slots, self.index, stream, self.c,
              _index(first, self.n_seqs, self.index, "first"),
              _index(count, self.n_seqs, self.index, "count"), *args)
        return slots, positions, starts

    def release(self, keep, stream=None):
        """Give back the pages behind each sequence's first ``keep`` [n_seqs] (int32) rows."""
        _call(pds.load().pds_pages_release, self.index, stream, self.c,
              _index(keep, self.n_seqs, self.index, "keep"))

    def write(self, k, v, slots, rope=None, positions=None, stream=None):
        """Store the rows [rows, n_kv_heads, head_dim] (bf16) at ``slots`` (int32, -1: left out), K
        rotated by ``rope`` (a :class:`kv.RopeSpec`) at ``positions``."""
        _no_gradient(k, "k"), _no_gradient(v, "v")
        rows = k.shape[0]
        shape = (rows, self.n_kv_heads, self.head_dim)
        ks, vs = _rows(k, shape, 1, self.index, "k"), _rows(v, shape, 1, self.index, "v")
        if rope is not None:
            if rope.head_dim != self.head_dim:
                raise ValueError(f"rope: heads of {rope.head_dim} channels, the cache's have {self.head_dim}")
            _need(positions is not None, "positions: a rotation needs them")
        at = _index(slots, rows, self.index, "slots")
        positions = _index(positions, rows, self.index, "positions")
        if rows:
            _call(pds.load().pds_pages_write, self.index, stream, self.c, None if rope is None else rope.c,
                  k.data_ptr(), v.data_ptr(), at, _int32(rows, "rows"), ks, vs, positions)

    def read(self, slots, k_out=None, v_out=None, stream=None):
        """(K, V) rows at ``slots`` (int32) as bf16 [rows, n_kv_heads, head_dim]; those of the slot
        -1 are left as they are (zero in a new tensor)."""
        rows = slots.numel()
        shape = (rows, self.n_kv_heads, self.head_dim)
        if k_out is None:
            k_out = _new(torch.zeros, shape, self.device, stream)
        if v_out is None:
            v_out = _new(torch.zeros, shape, self.device, stream)
        _no_gradient(k_out, "k_out"), _no_gradient(v_out, "v_out")
        if _rows(k_out, shape, 0, self.index, "k_out") or _rows(v_out, shape, 0, self.index, "v_out"):
            raise ValueError("k_out, v_out: contiguous tensors")
        at = _index(slots, rows, self.index, "slots")
        if rows:
            _call(pds.load().pds_pages_read, self.index, stream, self.c, at, _int32(rows, "rows"),
                  k_out.data_ptr(), v_out.data_ptr())
        return k_out, v_out

    def _workspace_bytes(self, n_heads):
        with torch.cuda.device(self.device):
            return pds.pds_pages_attend_workspace_bytes(self.c, n_heads)

    def workspace(self, n_heads, stream=None):
        """The attention's workspace for this many heads on a stream (the current one), made on
        first use and shared by the calls with as many heads on that stream."""
        if stream is None:
            stream = torch.cuda.current_stream(self.device)
        key = (n_heads, stream.cuda_stream)
        ws = self._ws.get(key)
        if ws is None:
            ws = _new(torch.empty, self._workspace_bytes(n_heads), self.device, stream, torch.uint8)
            self._ws[key] = ws
        return ws

    def _own_workspace(self, n_heads, stream):
        """One for this call alone if its stream is being captured, from the graph's
        memory: a graph may be replayed beside other work on any stream.  Else None."""
        if not kv._captures(self.index, stream):
            return None
        return _new(torch.empty, self._workspace_bytes(n_heads), self.device, stream, torch.uint8)

    def attend(self, q, new=None, out=None, softcap=0.0, window=0, stream=None, workspace=None):
        """Attention of one token per sequence, the last of its ``new`` [n_seqs] (int32; None: 1
        each) written rows: queries ``q`` [n_seqs, heads, head_dim] (bf16, rotated) over all its
        rows, with ``window`` the last so many.  A sequence without a new row gets zeros.  Without
        ``workspace`` the calls on a stream share one, and in a captured graph each has
        its own from the graph's memory."""
        _, heads, _ = shape = q.shape
        device = self.index
        if shape[0] != self.n_seqs or shape[2] != self.head_dim:
            raise ValueError(f"q: [{self.n_seqs}, heads, {self.head_dim}], not {tuple(shape)}")
        _no_gradient(q, "q")
        if out is None:
            out = _new(torch.empty, shape, self.device, stream)
        else:
            _no_gradient(out, "out")
        qs, os_ = _rows(q, shape, 1, device, "q"), _rows(out, shape, 1, device, "out")
        if workspace is None:
            raw = kv._raw_stream(device) if stream is None else stream.cuda_stream
            if raw and (stream is not None or kv._current_device() != device or kv._is_capturing()):
                workspace = self._own_workspace(heads, stream)  # (stream 0 is not captured)
            if workspace is None:
                workspace = self._ws.get((heads, raw))
            if workspace is None:
                workspace = self.workspace(heads, stream)
        elif workspace.get_device() != device or not workspace.is_contiguous():
            raise ValueError(f"workspace: a contiguous tensor on cuda:{device}")
        _call(pds.load().pds_pages_attend, device, stream, self.c, _index(new, self.n_seqs, device, "new"),
              q.data_ptr(), out.data_ptr(), heads, qs, os_, softcap, _int32(window, "window"),
              workspace.data_ptr(), workspace.nbytes)
        return out

    def sync(self, stream=None):
        """Wait for the stream; raises PdsError where a call on this device, of any stream and any
        cache, met a number that it could not serve (reported once)."""
        _call(pds.load().pds_component_sync, self.index, stream)
