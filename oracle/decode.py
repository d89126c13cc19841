"""Definitions of the cached-decoding operators in float64 numpy: scaled RoPE
frequencies, the quantised row formats, and attention of a tree of drafted
tokens over a cache.  Plain loops over sequences, heads and tokens; the
quantisers also have the float32 form the format is defined by (bit for bit)."""

from __future__ import annotations

import math

import numpy as np

from .stack import rope_inv_freq


def scaled_inv_freq(rot_dim, theta, freq_factors=None, scaling="none", factor=1.0,
                    orig_context=0, beta_fast=32.0, beta_slow=1.0):
    """Angular frequency per pair of a rotation stretched for a long context."""
    w = rope_inv_freq(rot_dim, theta, freq_factors)
    if scaling == "none":
        return w
    if scaling == "linear":
        return w / factor

    def edge(beta):  # the pair that turns beta times within the original context
        return rot_dim * math.log(orig_context / (2 * math.pi * beta)) / (2 * math.log(theta))

    lo, hi = max(0, math.floor(edge(beta_fast))), min(rot_dim - 1, math.ceil(edge(beta_slow)))
    ramp = np.clip((np.arange(rot_dim // 2) - lo) / max(hi - lo, 1e-3), 0, 1)
    return w * ((1 - ramp) + ramp / factor)


def rotate(t, positions, omega, layout="neox", mscale=1.0, inverse=False):
    """Heads of ``t[n, heads, hd]`` turned by ``positions[n] * omega``."""
    half = len(omega)
    rot = 2 * half
    ang = np.asarray(positions, np.float64)[:, None] * omega
    c, s = mscale * np.cos(ang)[:, None], mscale * np.sin(ang)[:, None] * (-1 if inverse else 1)
    out = np.array(t, np.float64)
    a, b = ((slice(0, half), slice(half, rot)) if layout == "neox"
            else (slice(0, rot, 2), slice(1, rot, 2)))
    u, w = np.array(out[..., a]), np.array(out[..., b])
    out[..., a], out[..., b] = u * c - w * s, u * s + w * c
    return out


def e4m3_values():
    """The value of each of the 256 codes (1-4-3, bias 7; 0x7f and 0xff are NaN)."""
    out = np.empty(256)
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[code] = math.nan if code & 127 == 127 else -v if code & 128 else v
    return out


def e4m3_round(x):
    """Codes of the grid values nearest to ``x`` (ties to even), |x| <= 464."""
    mag = e4m3_values()[:127]
    a = np.abs(np.asarray(x, np.float64))
    hi = np.clip(np.searchsorted(mag, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - mag[lo], mag[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(a >= mag[126], 126, code)
    return (code + 128 * np.signbit(x)).astype(np.uint8)


def quantise(x, fmt):
    """(codes uint8, scale words uint32) of float32 rows ``x[..., hd]`` as the formats
    define them; 4-bit codes one per byte."""
    x = np.asarray(x, np.float32)
    tiny = np.finfo(np.float32).tiny
    finite = np.isfinite(x).all(-1)
    x = np.where(finite[..., None], x, np.float32(0))
    if fmt == "e4m3":
        s = np.abs(x).max(-1) / np.float32(448)
        s = np.where(s >= tiny, s, np.float32(0)).astype(np.float32)
        safe = np.where(s > 0, s, np.float32(1))[..., None]
        codes = np.where(s[..., None] > 0, e4m3_round(x / safe), 0).astype(np.uint8)
        words = s.view(np.uint32)
    else:
        hi, lo = np.maximum(x.max(-1), 0), np.minimum(x.min(-1), 0)
        s = bf16_round(hi / np.float32(15) - lo / np.float32(15))
        s = np.where(s >= tiny, s, np.float32(0)).astype(np.float32)
        safe = np.where(s > 0, s, np.float32(1))
        z = np.clip(np.rint(-lo / safe), 0, 15)
        codes = np.clip(np.rint(x / safe[..., None]) + z[..., None], 0, 15)
        codes = np.where(s[..., None] > 0, codes, 0).astype(np.uint8)
        z = np.where(s > 0, z, 0)
        words = s.view(np.uint32) | z.astype(np.uint32)
    return codes, np.where(finite, words, np.uint32(0x7FC00000)).astype(np.uint32)


def bf16_round(x):
    """float32 rounded to bf16 (nearest even), as float32."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000
    return b.astype(np.uint32).view(np.float32)


def dequantise(codes, words, fmt):
    """The values the codes stand for, float64."""
    words = np.ascontiguousarray(words, np.uint32)
    if fmt == "e4m3":
        return e4m3_values()[codes] * words.view(np.float32).astype(np.float64)[..., None]
    s = (words & np.uint32(0xFFFF0000)).view(np.float32).astype(np.float64)
    return (codes.astype(np.float64) - (words & 15)[..., None]) * s[..., None]


def tree_paths(parents):
    """Per token the list of its ancestors from the root down, itself last; [] for padding."""
    paths = []
    for t, p in enumerate(parents):
        if p < -1:
            paths.append([])
        elif p == -1:
            paths.append([t])
        else:
            assert p < t and paths[p], "a parent is an earlier token"
            paths.append(paths[p] + [t])
    return paths


def tree_attention(q, k, v, length, parents=None, softcap=0.0, window=0):
    """One sequence: ``q[T, H, hd]`` over ``k, v[>= length + T, Hkv, hd]``.  Returns
    (o[T, H, hd], the sums of weight |v| that o's error is measured by)."""
    T, H, hd = q.shape
    group = H // k.shape[1]
    o, size = np.zeros((T, H, hd)), np.zeros((T, H, hd))
    for t, path in enumerate(tree_paths(range(-1, T - 1) if parents is None else parents)):
        if not path:
            continue
        rows = list(range(length)) + [length + a for a in path]
        pos = np.array(list(range(length)) + [length + i for i in range(len(path))])
        if window:
            rows = [r for r, p in zip(rows, pos) if p > pos[-1] - window]
        for h in range(H):
            z = k[rows, h // group] @ q[t, h] / math.sqrt(hd)
            if softcap:
                z = softcap * np.tanh(z / softcap)
            w = np.exp(z - z.max())
            w /= w.sum()
            o[t, h] = w @ v[rows, h // group]
            size[t, h] = w @ np.abs(v[rows, h // group])
    return o, size
