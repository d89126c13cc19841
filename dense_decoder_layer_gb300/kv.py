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
"""

from __future__ import annotations

import ctypes

import torch

from . import pds

FORMATS = {"bf16": pds.PDS_KV_BF16, "e4m3": pds.PDS_KV_E4M3, "int4": pds.PDS_KV_INT4}
LAYOUTS = {"neox": pds.PDS_ROPE_NEOX, "norm": pds.PDS_ROPE_NORM}
SCALINGS = {"none": pds.PDS_ROPE_UNSCALED, "linear": pds.PDS_ROPE_LINEAR,
            "yarn": pds.PDS_ROPE_YARN}


def _stream(stream, device):
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return s.cuda_stream


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _rows(t, lead, tail, what):
    """Element stride between consecutive rows of a bf16 tensor [*lead, *tail]
    whose rows are contiguous and evenly spaced."""
    _need(t.dtype == torch.bfloat16 and t.is_cuda, f"{what}: a bf16 CUDA tensor")
    _need(t.shape == (*lead, *tail), f"{what}: shape {tuple(t.shape)}, not {(*lead, *tail)}")
    if t.is_contiguous():
        return 0
    width = 1
    for size, stride in zip(reversed(tail), reversed(t.stride()[len(lead):])):
        _need(size == 1 or stride == width, f"{what}: a row's heads and channels must be contiguous")
        width *= size
    step, count = None, 1
    for size, stride in zip(reversed(lead), reversed(t.stride()[:len(lead)])):
        if size > 1:
            step = stride // count if step is None else step
            _need(stride == step * count, f"{what}: rows must be evenly spaced")
        count *= size
    return width if step is None else step


def _index(t, shape, device, what):
    if t is None:
        return None
    _need(t.dtype == torch.int32 and t.device == device and t.is_contiguous() and
          tuple(t.shape) == tuple(shape), f"{what}: a contiguous int32 tensor {tuple(shape)} on {device}")
    return t.data_ptr()


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
        self.c = pds.pds_rope_spec(theta, LAYOUTS[layout], rot_dim, SCALINGS[scaling],
                                   ctypes.cast(arr, ctypes.POINTER(ctypes.c_float)) if arr else None,
                                   mscale, factor, orig_context, beta_fast, beta_slow)


def rope(x, spec, positions=None, start_pos=0, out=None, inverse=False, stream=None):
    """The rows of ``x`` [..., heads, head_dim] (bf16) turned at ``positions`` (int32, one per
    row) or ``start_pos + row``; ``out`` may be ``x``.  ``inverse`` turns back (the gradient)."""
    lead, (heads, hd) = x.shape[:-2], x.shape[-2:]
    _need(hd == spec.head_dim, f"x: heads of {hd} channels, the spec's have {spec.head_dim}")
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    _need(out.device == x.device, "out: on the device of x")
    xs, ys = _rows(x, lead, (heads, hd), "x"), _rows(out, lead, (heads, hd), "out")
    rows = 1
    for n in lead:
        rows *= n
    if positions is not None:
        positions = positions.reshape(-1)
    if rows and heads:
        with torch.cuda.device(x.device):
            pds.pds_rope(spec.c, x.data_ptr(), out.data_ptr(), rows, heads, hd,
                         _stream(stream, x.device), xs, ys,
                         _index(positions, (rows,), x.device, "positions"), start_pos, inverse)
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
        self.device = torch.device(device) if k is None else k.device
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
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

        self.k, self.v = have(k, shape, dtype, "k", False), have(v, shape, dtype, "v", False)
        _need(self.k.stride() == self.v.stride(), "k and v: the same strides")
        self.k_scale = self.v_scale = None
        if word is not None:
            self.k_scale = have(k_scale, words, word, "k_scale", True)
            self.v_scale = have(v_scale, words, word, "v_scale", True)
        self.lens = have(lens, (self.n_seqs,), torch.int32, "lens", True)
        seq, row, head, _ = (0, 0, 0, 0) if self.k.is_contiguous() else self.k.stride()
        self.c = pds.pds_cache(
            FORMATS[fmt], self.n_seqs, self.capacity, self.n_kv_heads, self.head_dim, 0,
            seq * self.per_byte, row * self.per_byte, head * self.per_byte, self.k.data_ptr(),
            self.v.data_ptr(), self.k_scale.data_ptr() if word is not None else None,
            self.v_scale.data_ptr() if word is not None else None, self.lens.data_ptr())
        self._ws = {}  # attention workspace by (tokens, heads)

    def workspace(self, n_tokens, n_heads):
        """The attention's workspace for this many tokens and heads, made on first use and
        shared by the calls of that shape (so: one stream at a time)."""
        ws = self._ws.get((n_tokens, n_heads))
        if ws is None:
            with torch.cuda.device(self.device):
                n = pds.pds_attention_tree_workspace_bytes(self.c, n_tokens, n_heads)
            ws = torch.empty(n, dtype=torch.uint8, device=self.device)
            self._ws[n_tokens, n_heads] = ws
        return ws

    def write(self, k, v, rope=None, parents=None, positions=None, stream=None):
        """Store new rows [n_seqs, n_tokens, n_kv_heads, head_dim] (bf16) behind the cached
        ones, K rotated by ``rope`` (a :class:`RopeSpec`) at the tokens' positions."""
        tail = (self.n_kv_heads, self.head_dim)
        t = k.shape[1]
        ks, vs = _rows(k, (self.n_seqs, t), tail, "k"), _rows(v, (self.n_seqs, t), tail, "v")
        _need(k.device == self.device and v.device == self.device, "k, v: on the cache's device")
        _need(rope is None or rope.head_dim == self.head_dim, "rope: for this head_dim")
        with torch.cuda.device(self.device):
            pds.pds_cache_write(self.c, None if rope is None else rope.c, k.data_ptr(),
                                v.data_ptr(), t, _stream(stream, self.device), ks, vs,
                                _index(parents, (self.n_seqs, t), self.device, "parents"),
                                _index(positions, (self.n_seqs, t), self.device, "positions"))

    def read(self, first_row, rows, k_out=None, v_out=None, stream=None):
        """(K, V) rows ``first_row ...`` as bf16 [n_seqs, rows, n_kv_heads, head_dim]; rows that
        a sequence does not have are left as they are (zero in a new tensor)."""
        shape = (self.n_seqs, rows, self.n_kv_heads, self.head_dim)
        out = []
        for t in (k_out, v_out):
            if t is None:
                t = torch.zeros(shape, dtype=torch.bfloat16, device=self.device)
            _need(t.dtype == torch.bfloat16 and tuple(t.shape) == shape and t.is_contiguous() and
                  t.device == self.device, f"output: contiguous bf16 {shape} on {self.device}")
            out.append(t)
        with torch.cuda.device(self.device):
            pds.pds_cache_read(self.c, first_row, rows, out[0].data_ptr(), out[1].data_ptr(),
                               _stream(stream, self.device))
        return tuple(out)

    def read_new(self, rows, k_out=None, v_out=None, stream=None):
        """(K, V) of the ``rows`` tokens that the last write stored."""
        return self.read(pds.PDS_AT_LENS, rows, k_out, v_out, stream)

    def attend(self, q, out=None, parents=None, softcap=0.0, window=0, max_len=0, stream=None,
               workspace=None):
        """Attention of the written tokens' queries ``q`` [n_seqs, n_tokens, heads, head_dim]
        (bf16, rotated) over the cache and each other; ``parents`` int32 [n_seqs, n_tokens]
        makes them a tree, without it they are a chain."""
        t, heads = q.shape[1], q.shape[2]
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        _need(q.device == self.device and out.device == self.device, "q, out: on the cache's device")
        lead, tail = (self.n_seqs, t), (heads, self.head_dim)
        qs, os_ = _rows(q, lead, tail, "q"), _rows(out, lead, tail, "out")
        if workspace is None:
            workspace = self.workspace(t, heads)
        with torch.cuda.device(self.device):
            pds.pds_attention_tree(self.c, q.data_ptr(), out.data_ptr(), t, heads,
                                   _stream(stream, self.device), qs, os_,
                                   _index(parents, (self.n_seqs, t), self.device, "parents"),
                                   softcap, window, max_len, workspace.data_ptr(),
                                   workspace.numel())
        return out

    def sync(self, stream=None):
        """Wait for the stream; raises PdsError where a call met a length or a parent that it
        could not serve."""
        with torch.cuda.device(self.device):
            st = pds.pds_component_sync(_stream(stream, self.device))
        if st != pds.PDS_OK:
            raise pds.PdsError(st, pds.last_error())
