"""PyTorch-side owner of a decoding cache: rotary positions, quantised K/V rows
and attention of drafted tokens over them.

Every step runs in ``libpds.so`` through :mod:`.pds` (the section on cached
decoding in ``include/pds.h`` says what each call computes).  ``KvCache``
keeps the cache tensors of one layer, the sequences' lengths and the
attention's workspace alive and hands their pointers to the C ABI.

A decode step with drafted tokens::

    spec = kv.RopeSpec(5.0e5, head_dim=128)
    cache = kv.KvCache("e4m3", n_seqs=4, capacity=8192, n_kv_heads=8, head_dim=128)
    kv.rope(q, spec, positions=positions, out=q)
    cache.write(k, v, rope=spec, parents=parents)
    o = cache.attend(q, parents=parents)
    cache.lens += accepted            # after the accepted rows are in place

A call with ``stream`` does what it would do under ``torch.cuda.stream(stream)``:
what it allocates belongs to that stream, its inputs have to be ready there and to be
kept until it is done with them.
The calls record no gradients and refuse tensors that require one.
"""

from __future__ import annotations

import ctypes

import torch

from . import pds

FORMATS = {"bf16": pds.PDS_KV_BF16, "e4m3": pds.PDS_KV_E4M3, "int4": pds.PDS_KV_INT4}
LAYOUTS = {"neox": pds.PDS_ROPE_NEOX, "norm": pds.PDS_ROPE_NORM}
SCALINGS = {"none": pds.PDS_ROPE_UNSCALED, "linear": pds.PDS_ROPE_LINEAR,
            "yarn": pds.PDS_ROPE_YARN}


# A decode step's call is a few microseconds of GPU work, so the wrappers keep
# to a few cheap attribute reads: device and stream by index, the shape
# compared as a whole, strides looked at only for tensors that are not packed.
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream
_is_capturing = torch._C._cuda_isCurrentStreamCapturing
_BF16, _I32 = torch.bfloat16, torch.int32


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _int32(x, what):
    """x, which the C ABI takes in 32 bits (ctypes would drop the others)."""
    if not -2**31 <= x < 2**31:
        raise ValueError(f"{what}: {x} does not fit 32 bits")
    return x


def _no_gradient(t, what, instead=""):
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{what} requires a gradient, which this call does not record: detach it or "
                         f"call under torch.no_grad(){instead}")


def _rows(t, shape, n_lead, device, what):
    """Element stride (0: packed) between consecutive rows of a bf16 tensor of `shape`: its
    first `n_lead` sizes count rows, which are contiguous and evenly spaced."""
    if t.dtype != _BF16 or t.get_device() != device or t.shape != shape:
        raise ValueError(f"{what}: a bf16 tensor {tuple(shape)} on cuda:{device}, not {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    if t.is_contiguous():
        return 0
    strides = t.stride()
    width = 1
    for size, stride in zip(reversed(shape[n_lead:]), reversed(strides[n_lead:])):
        _need(size == 1 or stride == width, f"{what}: a row's heads and channels must be contiguous")
        width *= size
    step, count = None, 1
    for size, stride in zip(reversed(shape[:n_lead]), reversed(strides[:n_lead])):
        if size > 1:
            step = stride // count if step is None else step
            _need(stride == step * count, f"{what}: rows must be evenly spaced")
            _need(step >= width, f"{what}: rows must not overlap (an expanded tensor?)")
        count *= size
    return width if step is None else step


def _index(t, rows, device, what):
    if t is None:
        return None
    if t.dtype != _I32 or t.get_device() != device or t.numel() != rows or not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous int32 tensor of {rows} values on cuda:{device}")
    return t.data_ptr()


def _new(make, shape, device, stream, dtype=_BF16):
    """make(shape) on the stream that the call is for."""
    index = stream.device_index if stream is not None else None
    if stream is None or stream.cuda_stream == _raw_stream(index):
        return make(shape, dtype=dtype, device=device)
    if _current_device() != index:
        with torch.cuda.stream(stream):
            return make(shape, dtype=dtype, device=device)
    before = torch.cuda.current_stream(index)  # (a tenth of the context's microseconds)
    torch.cuda.set_stream(stream)
    try:
        return make(shape, dtype=dtype, device=device)
    finally:
        torch.cuda.set_stream(before)


def _call(fn, device, stream, *args):
    """fn(*args, stream) with the tensors' device current."""
    if stream is not None and stream.device_index != device:
        raise ValueError(f"stream: one of cuda:{stream.device_index}, the tensors are on cuda:{device}")
    if _current_device() == device:
        st = fn(*args, _raw_stream(device) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(device):
            st = fn(*args, _raw_stream(device) if stream is None else stream.cuda_stream)
    if st:
        pds.check(st)


class RopeSpec:
    """A rotation (``pds_rope_spec``): ``layout`` "neox" or "norm", ``rot_dim`` the
    rotated channels (0: the whole head), ``freq_factors`` optional per pair,
    ``scaling`` "none", "linear" (``factor``) or "yarn" (all four)."""

    def __init__(self, theta, head_dim, rot_dim=0, layout="neox", freq_factors=None, mscale=0.0,
                 scaling="none", factor=1.0, orig_context=0, beta_fast=32.0, beta_slow=1.0):
        self.head_dim = int(head_dim)
        arr = None
        if freq_factors is not None:
            pairs = (int(rot_dim) or self.head_dim) // 2
            _need(len(freq_factors) == pairs, f"freq_factors: {pairs} values, one per rotated pair")
            arr = (ctypes.c_float * pairs)(*[float(f) for f in freq_factors])
        self._factors = arr
        self.c = pds.pds_rope_spec(theta, LAYOUTS[layout], _int32(rot_dim, "rot_dim"),
                                   SCALINGS[scaling],
                                   ctypes.cast(arr, ctypes.POINTER(ctypes.c_float)) if arr else None,
                                   mscale, factor, _int32(orig_context, "orig_context"), beta_fast,
                                   beta_slow)


def rope(x, spec, positions=None, start_pos=0, out=None, inverse=False, stream=None):
    """The rows of ``x`` [..., heads, head_dim] (bf16) turned at ``positions`` (int32, one per
    row) or ``start_pos + row``; ``out`` may be ``x``.  ``inverse`` turns back: it is the gradient,
    which a caller takes by that call (an ``x`` that requires one is refused)."""
    shape = x.shape
    heads, hd = shape[-2], shape[-1]
    if hd != spec.head_dim:
        raise ValueError(f"x: heads of {hd} channels, the spec's have {spec.head_dim}")
    _no_gradient(x, "x", "; the gradient is rope(..., inverse=True) of the result's")
    if out is None:
        out = _new(torch.empty, shape, x.device, stream)
    device, lead = x.get_device(), len(shape) - 2
    xs = _rows(x, shape, lead, device, "x")
    ys = xs if out is x else _rows(out, shape, lead, device, "out")
    n = x.numel()
    if n:
        rows = _int32(n // (heads * hd), "x: its rows")
        _call(pds.load().pds_rope, device, stream, spec.c, x.data_ptr(), out.data_ptr(), rows,
              heads, hd, xs, ys, _index(positions, rows, device, "positions"),
              _int32(start_pos, "start_pos"), inverse)
    return out


class KvCache:
    """One layer's K/V rows of ``n_seqs`` sequences, ``capacity`` rows each.

    ``fmt`` is "bf16", "e4m3" (a byte per channel) or "int4" (half a byte); the
    latter two with a scale word per row and head.  Tensors may be given: ``k``,
    ``v`` [n_seqs, capacity, n_kv_heads, head_dim] (bfloat16, float8_e4m3fn, or
    uint8 with head_dim/2 bytes), in any order of rows and heads whose
    channels are contiguous; ``k_scale``, ``v_scale`` contiguous [n_seqs,
    n_kv_heads, capacity] (float32 for e4m3, int32 for int4); ``lens`` int32
    [n_seqs], the cached rows of each sequence, which the calls never change.
    """

    def __init__(self, fmt, n_seqs, capacity, n_kv_heads, head_dim, device="cuda", k=None, v=None,
                 k_scale=None, v_scale=None, lens=None):
        self.fmt, self.n_seqs, self.capacity = fmt, int(n_seqs), int(capacity)
        self.n_kv_heads, self.head_dim = int(n_kv_heads), int(head_dim)
        for name in ("n_seqs", "capacity", "n_kv_heads", "head_dim"):
            _int32(getattr(self, name), name)
        self.device = torch.device(device) if k is None else k.device
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.index = self.device.index
        dtype, self.per_byte = {"bf16": (torch.bfloat16, 1), "e4m3": (torch.float8_e4m3fn, 1),
                                "int4": (torch.uint8, 2)}[fmt]
        shape = (self.n_seqs, self.capacity, self.n_kv_heads, self.head_dim // self.per_byte)
        words = (self.n_seqs, self.n_kv_heads, self.capacity)
        word = {"bf16": None, "e4m3": torch.float32, "int4": torch.int32}[fmt]

        def have(t, shape, dtype, what, packed):
            if t is None:
                return torch.zeros(shape, dtype=dtype, device=self.device)
            _need(t.dtype == dtype and tuple(t.shape) == tuple(shape) and t.device == self.device,
                  f"{what}: {dtype} {tuple(shape)} on {self.device}")
            _need(t.is_contiguous() if packed else t.stride(-1) == 1, f"{what}: layout")
            return t

        k, v = have(k, shape, dtype, "k", False), have(v, shape, dtype, "v", False)
        packed = k.is_contiguous() and v.is_contiguous()
        _need(packed or k.stride() == v.stride(), "k and v: the same strides")
        _need(packed or any(k.stride()[:3]), "k and v: rows of their own (an expanded tensor?)")
        if word is not None:
            k_scale = have(k_scale, words, word, "k_scale", True)
            v_scale = have(v_scale, words, word, "v_scale", True)
        else:
            k_scale = v_scale = None
        self._tensors = k, v, k_scale, v_scale
        self._lens = have(lens, (self.n_seqs,), torch.int32, "lens", True)
        seq, row, head, _ = (0, 0, 0, 0) if packed else k.stride()
        self.c = pds.pds_cache(
            FORMATS[fmt], self.n_seqs, self.capacity, self.n_kv_heads, self.head_dim, 0,
            seq * self.per_byte, row * self.per_byte, head * self.per_byte, k.data_ptr(), v.data_ptr(),
            k_scale.data_ptr() if word is not None else None,
            v_scale.data_ptr() if word is not None else None, self._lens.data_ptr())
        self._ws = {}  # attention workspace by (tokens, heads, stream)

    # The kernels have these tensors' addresses: they can be written to, not replaced.
    k = property(lambda self: self._tensors[0], doc="The K rows.")
    v = property(lambda self: self._tensors[1], doc="The V rows.")
    k_scale = property(lambda self: self._tensors[2], doc="K's scale words (None: bf16).")
    v_scale = property(lambda self: self._tensors[3], doc="V's scale words (None: bf16).")

    @property
    def lens(self):
        """Cached rows of each sequence (int32, on the device); assigning copies into it."""
        return self._lens

    @lens.setter
    def lens(self, value):
        if value is not self._lens:
            self._lens.copy_(value)

    def _workspace_bytes(self, n_tokens, n_heads):
        with torch.cuda.device(self.device):
            return pds.pds_attention_tree_workspace_bytes(self.c, n_tokens, n_heads)

    def workspace(self, n_tokens, n_heads, stream=None):
        """The attention's workspace for this many tokens and heads on a stream (the current
        one), made on first use and shared by the calls of that shape on that stream."""
        if stream is None:
            stream = torch.cuda.current_stream(self.device)
        key = (n_tokens, n_heads, stream.cuda_stream)
        ws = self._ws.get(key)
        if ws is None:
            ws = _new(torch.empty, self._workspace_bytes(n_tokens, n_heads), self.device, stream,
                      torch.uint8)
            self._ws[key] = ws
        return ws

    def _own_workspace(self, n_tokens, n_heads, stream):
        """One for this call alone if the current stream is being captured, from the graph's
        memory: a graph may be replayed beside other work on any stream.  Else None."""
        with torch.cuda.device(self.index):
            if not _is_capturing():
                return None
        return _new(torch.empty, self._workspace_bytes(n_tokens, n_heads), self.device, stream,
                    torch.uint8)

    def write(self, k, v, rope=None, parents=None, positions=None, stream=None):
        """Store new rows [n_seqs, n_tokens, n_kv_heads, head_dim] (bf16) behind the cached
        ones, K rotated by ``rope`` (a :class:`RopeSpec`) at the tokens' positions."""
        _no_gradient(k, "k"), _no_gradient(v, "v")
        t, device = k.shape[1], self.index
        shape = (self.n_seqs, t, self.n_kv_heads, self.head_dim)
        ks, vs = _rows(k, shape, 2, device, "k"), _rows(v, shape, 2, device, "v")
        if rope is not None and rope.head_dim != self.head_dim:
            raise ValueError(f"rope: heads of {rope.head_dim} channels, the cache's have {self.head_dim}")
        rows = self.n_seqs * t
        _call(pds.load().pds_cache_write, device, stream, self.c, None if rope is None else rope.c,
              k.data_ptr(), v.data_ptr(), t, ks, vs, _index(parents, rows, device, "parents"),
              _index(positions, rows, device, "positions"))

    def read(self, first_row, rows, k_out=None, v_out=None, stream=None):
        """(K, V) rows ``first_row ...`` as bf16 [n_seqs, rows, n_kv_heads, head_dim]; rows that
        a sequence does not have are left as they are (zero in a new tensor)."""
        shape = (self.n_seqs, rows, self.n_kv_heads, self.head_dim)
        if k_out is None:
            k_out = _new(torch.zeros, shape, self.device, stream)
        if v_out is None:
            v_out = _new(torch.zeros, shape, self.device, stream)
        if _rows(k_out, shape, 0, self.index, "k_out") or _rows(v_out, shape, 0, self.index, "v_out"):
            raise ValueError("k_out, v_out: contiguous tensors")
        _call(pds.load().pds_cache_read, self.index, stream, self.c,
              _int32(first_row, "first_row"), _int32(rows, "rows"),
              k_out.data_ptr(), v_out.data_ptr())
        return k_out, v_out

    def read_new(self, rows, k_out=None, v_out=None, stream=None):
        """(K, V) of the ``rows`` tokens that the last write stored."""
        return self.read(pds.PDS_AT_LENS, rows, k_out, v_out, stream)

    def attend(self, q, out=None, parents=None, softcap=0.0, window=0, max_len=0, stream=None,
               workspace=None):
        """Attention of the written tokens' queries ``q`` [n_seqs, n_tokens, heads, head_dim]
        (bf16, rotated) over the cache and each other; ``parents`` int32 [n_seqs, n_tokens]
        makes them a tree, without it they are a chain.  Without ``workspace`` the calls of a shape on a
        stream share one, and in a captured graph each has its own from the graph's memory."""
        _, t, heads, _ = shape = q.shape
        device = self.index
        if shape[0] != self.n_seqs or shape[3] != self.head_dim:
            raise ValueError(f"q: [{self.n_seqs}, tokens, heads, {self.head_dim}], not {tuple(shape)}")
        _no_gradient(q, "q")
        if out is None:
            out = _new(torch.empty, shape, self.device, stream)
        qs, os_ = _rows(q, shape, 2, device, "q"), _rows(out, shape, 2, device, "out")
        if workspace is None:
            raw = _raw_stream(device) if stream is None else stream.cuda_stream
            if raw and (_current_device() != device or _is_capturing()):
                workspace = self._own_workspace(t, heads, stream)  # (stream 0 is not captured)
            if workspace is None:
                workspace = self._ws.get((t, heads, raw))
            if workspace is None:
                workspace = self.workspace(t, heads, stream)
        elif workspace.get_device() != device or not workspace.is_contiguous():
            raise ValueError(f"workspace: a contiguous tensor on cuda:{device}")
        _call(pds.load().pds_attention_tree, device, stream, self.c, q.data_ptr(), out.data_ptr(),
              t, heads, qs, os_, _index(parents, self.n_seqs * t, device, "parents"), softcap,
              _int32(window, "window"), _int32(max_len, "max_len"), workspace.data_ptr(), workspace.nbytes)
        return out

    def sync(self, stream=None):
        """Wait for the stream; raises PdsError where a call on this device, of any stream and any
        cache, met a length or a parent that it could not serve (reported once)."""
        _call(pds.load().pds_component_sync, self.index, stream)
