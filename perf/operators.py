"""The cached-decoding operators: rotary positions, the write and the read of a
quantised K/V cache, and attention of drafted tokens over it.

``run`` computes one operator, either as plain torch operations in 32 bits
(``own`` false) or through the framework's entry points (``own`` true).  The
cases are real sizes: the head shapes are those of the Llama-style stacks
this repository serves (24/8 x 128, 32/8 x 128, 32/8 x 64), the cached
lengths those of its decode and long-prefix workloads (2048 to 32768 rows).

A case's fields: ``op`` (rope, write, read, attend), ``format`` of the cache
(bf16, e4m3, int4), ``n_seqs`` sequences of ``tokens`` new rows over
``len_min`` to ``len_max`` cached rows (evenly spread), ``heads``,
``kv_heads``, ``head_dim``; for attend whether the tokens form a ``tree``
(else a chain), ``softcap`` and ``window``; for rope and write the rotation
(``layout``, ``rot_dim``, ``scaling``) and for rope ``inverse``.
"""

import math

import torch

own = False

DEV = "cuda"
THETA = 5.0e5
YARN = dict(factor=8.0, orig_context=8192, beta_fast=32.0, beta_slow=1.0)


def _case(op, **kw):
    c = dict(op=op, format="bf16", n_seqs=1, tokens=1, heads=32, kv_heads=8, head_dim=128,
             len_min=0, len_max=0, tree=False, softcap=0.0, window=0, layout="neox", rot_dim=0,
             scaling="none", inverse=False)
    c.update(kw)
    return c


def listed():
    return [
        # the queries of one decode step of the 1B-shaped stack: pure latency
        _case("rope", name="rope-decode", tokens=1, heads=32, head_dim=64, len_min=2048,
              len_max=2048),
        # the queries of a long prompt under a context stretched by YaRN
        _case("rope", name="rope-prompt-yarn", tokens=8192, heads=32, head_dim=128,
              scaling="yarn", len_min=24576, len_max=24576),
        # one decode step of eight sequences into a 4-bit cache (and the new rows read back)
        _case("write", name="write-decode-int4", format="int4", n_seqs=8, tokens=1, len_min=100,
              len_max=2048),
        # a prompt's K/V rows rotated and quantised to e4m3 on their way into the cache
        _case("write", name="write-prompt-e4m3", format="e4m3", tokens=2048, len_min=2048,
              len_max=2048),
        # an e4m3 prefix read back for the prefill kernels
        _case("read", name="read-e4m3", format="e4m3", len_min=8192, len_max=8192),
        # ragged 4-bit prefixes of four sequences, 64-wide heads
        _case("read", name="read-int4-ragged", format="int4", n_seqs=4, head_dim=64, len_min=777,
              len_max=4097),
        # one decode step over a bf16 cache: the 3B-shaped decode workload
        _case("attend", name="attend-1-bf16", heads=24, len_min=2048, len_max=2048),
        # a serving batch of single tokens over ragged e4m3 caches
        _case("attend", name="attend-batch-e4m3", format="e4m3", n_seqs=16, len_min=100,
              len_max=8192),
        # 64 drafted tokens over a 32k-row 4-bit cache
        _case("attend", name="attend-tree64-int4", format="int4", tokens=64, heads=24, tree=True,
              len_min=32768, len_max=32768),
        # a small drafted tree over short windowed contexts, 64-wide heads, capped scores
        _case("attend", name="attend-tree16-window", n_seqs=2, tokens=16, head_dim=64, tree=True,
              softcap=30.0, window=128, len_min=99, len_max=333),
        # drafted trees of four sequences over long bf16 caches
        _case("attend", name="attend-tree32-bf16", n_seqs=4, tokens=32, heads=24, tree=True,
              len_min=8192, len_max=16384),
        # a chunk of a prompt over what is cached of it already
        _case("attend", name="attend-chunk256-e4m3", format="e4m3", tokens=256, len_min=8192,
              len_max=8192),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["rope", "write", "read", "attend", "attend", "attend"])
        hd = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 4, 8])
        c = _case(op, kv_heads=hkv, heads=hkv * rng.choice([1, 2, 3, 4, 5, 8]), head_dim=hd,
                  n_seqs=_log(rng, 1, 32), format=rng.choice(["bf16", "e4m3", "int4"]))
        c["len_max"] = _log(rng, 1, 32768)
        c["len_min"] = rng.choice([0, c["len_max"] // 3, c["len_max"]])
        if op in ("rope", "write"):
            c["tokens"] = _log(rng, 1, 2048)
            c["layout"] = rng.choice(["neox", "norm"])
            c["rot_dim"] = rng.choice([0, 0, hd // 2])
            c["scaling"] = rng.choice(["none", "linear", "yarn"])
            c["inverse"] = op == "rope" and rng.random() < 0.3
        if op == "attend":
            c["tokens"] = rng.choice([1, _log(rng, 1, 256)])
            c["tree"] = c["tokens"] > 1 and rng.random() < 0.7
            c["softcap"] = rng.choice([0.0, 0.0, 30.0])
            c["window"] = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
        if op != "write" and op != "attend" and op != "read":
            c["format"] = "bf16"
        if op == "read" and c["format"] == "bf16":
            c["format"] = "e4m3"
        if _cost(c) <= top:
            return c


def _lens(c):
    n, lo, hi = c["n_seqs"], c["len_min"], c["len_max"]
    return [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _row_bytes(c):  # one head's K or V row in the cache
    hd = c["head_dim"]
    return {"bf16": 2 * hd, "e4m3": hd + 4, "int4": hd // 2 + 4}[c["format"]]


def work(c):
    n, t, h, hkv, hd = c["n_seqs"], c["tokens"], c["heads"], c["kv_heads"], c["head_dim"]
    if c["op"] == "rope":
        return {"bytes": n * t * (4 * h * hd + 4), "flops": 3 * n * t * h * hd}
    if c["op"] == "write":
        back = 4 * hd if c["format"] == "int4" else 0
        return {"bytes": n * t * hkv * (4 * hd + 2 * _row_bytes(c) + back),
                "flops": 6 * n * t * hkv * hd}
    if c["op"] == "read":
        rows = sum(_lens(c))
        return {"bytes": rows * hkv * (4 * hd + 2 * _row_bytes(c)), "flops": 2 * rows * hkv * hd}
    w = c["window"]
    seen = sum(min(x, w) if w else x for x in _lens(c)) + n * t
    pairs = sum(t * (min(x, w) if w else x) for x in _lens(c)) + n * t
    return {"bytes": seen * hkv * 2 * _row_bytes(c) + 4 * n * t * h * hd, "flops": 4 * pairs * h * hd}


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50)


# ------------------------------------------------------------------ inputs


def _quantise(x, fmt):
    """(codes, scale words) of x[..., hd] float32; a scale word per row and head."""
    if fmt == "e4m3":
        s = x.abs().amax(-1) / 448.0
        q = torch.where(s[..., None] > 0, x / s[..., None], torch.zeros_like(x))
        return q.to(torch.float8_e4m3fn), s
    lo, hi = x.amin(-1).clamp(max=0.0), x.amax(-1).clamp(min=0.0)
    s = (hi / 15.0 - lo / 15.0).to(torch.bfloat16).float()
    safe = torch.where(s > 0, s, torch.ones_like(s))
    z = torch.round(-lo / safe).clamp(0, 15)
    q = (torch.round(x / safe[..., None]) + z[..., None]).clamp(0, 15).to(torch.uint8)
    words = s.view(torch.int32) | z.to(torch.int32)
    return q[..., 0::2] | (q[..., 1::2] << 4), words


def _dequantise(codes, words, fmt, dtype=torch.float32):
    if fmt == "bf16":
        return codes.to(dtype)
    if fmt == "e4m3":
        return codes.to(dtype) * words.to(dtype)[..., None]
    q = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).to(dtype)
    z = (words & 15).to(dtype)
    s = (words & -65536).view(torch.float32).to(dtype)
    return (q - z[..., None]) * s[..., None]


def _tree(n, t, g):
    """Parents of a drafted tree per sequence: -1 for a root, -2 for the padding
    behind a sequence's last node (every other sequence is a quarter shorter)."""
    i = torch.arange(t, device=DEV)
    back = torch.randint(1, 5, (n, t), device=DEV, generator=g)
    p = (i - back).clamp(min=-1)
    used = torch.where(torch.arange(n, device=DEV) % 2 == 1, t - t // 4, t)
    return torch.where(i < used[:, None], p, torch.full_like(p, -2)).to(torch.int32).contiguous()


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    n, t, h, hkv, hd = c["n_seqs"], c["tokens"], c["heads"], c["kv_heads"], c["head_dim"]
    lens = torch.tensor(_lens(c), dtype=torch.int32, device=DEV)

    def normal(*shape):
        return torch.randn(*shape, device=DEV, generator=g)

    s = {"case": dict(c), "lens": lens}
    if c["op"] == "rope":
        s["x"] = normal(n * t, h, hd).bfloat16()
        s["pos"] = (lens[:, None] + torch.arange(t, device=DEV, dtype=torch.int32)).reshape(-1)
        s["y"] = torch.empty_like(s["x"])
        return s
    # K has a few strong channels, as trained models have
    strength = torch.where(torch.rand(hkv, hd, device=DEV, generator=g) < 0.05, 4.0, 1.0)
    cap = c["len_max"] + t + 3
    if c["op"] == "write":
        s["k_new"] = (normal(n, t, hkv, hd) * strength).bfloat16()
        s["v_new"] = normal(n, t, hkv, hd).bfloat16()
        rows = n * cap
        s["k"], s["ks"] = _packed(torch.zeros(rows, hkv, hd, device=DEV), c["format"], n)
        s["v"], s["vs"] = _packed(torch.zeros(rows, hkv, hd, device=DEV), c["format"], n)
        s["k_out"] = torch.zeros(n, t, hkv, hd, device=DEV, dtype=torch.bfloat16)
        s["v_out"] = torch.zeros_like(s["k_out"])
        return s
    s["k"], s["ks"] = _packed(normal(n * cap, hkv, hd) * strength, c["format"], n)
    s["v"], s["vs"] = _packed(normal(n * cap, hkv, hd), c["format"], n)
    if c["op"] == "read":
        s["k_out"] = torch.zeros(n, c["len_max"], hkv, hd, device=DEV, dtype=torch.bfloat16)
        s["v_out"] = torch.zeros_like(s["k_out"])
        return s
    s["q"] = (1.5 * normal(n, t, h, hd)).bfloat16()
    s["o"] = torch.empty_like(s["q"])
    s["parents"] = _tree(n, t, g) if c["tree"] else None
    return s


def _packed(x, fmt, n):
    """The cache tensors of x[n * cap, Hkv, hd]: codes [n, cap, Hkv, ...], scale words [n, Hkv, cap]."""
    if fmt == "bf16":
        return x.bfloat16().unflatten(0, (n, -1)), None
    q, s = _quantise(x, fmt)
    return q.unflatten(0, (n, -1)), s.unflatten(0, (n, -1)).transpose(1, 2).contiguous()


# -------------------------------------------------------- the plain forms


def _omega(c, dtype=torch.float64):
    rot = c["rot_dim"] or c["head_dim"]
    i = torch.arange(rot // 2, device=DEV, dtype=dtype)
    w = THETA ** (-2.0 * i / rot)
    if c["scaling"] == "linear":
        return w / YARN["factor"]
    if c["scaling"] == "yarn":
        def edge(beta):
            return rot * math.log(YARN["orig_context"] / (2 * math.pi * beta)) / (2 * math.log(THETA))
        lo = max(0, math.floor(edge(YARN["beta_fast"])))
        hi = min(rot - 1, math.ceil(edge(YARN["beta_slow"])))
        r = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return w * ((1 - r) + r / YARN["factor"])
    return w


def _rotate(x, pos, c):
    """x[rows, heads, hd] float32 turned at its rows' positions (angles in 64 bits)."""
    rot = c["rot_dim"] or c["head_dim"]
    a = pos.double()[:, None] * _omega(c)[None, :]
    cos, sin = a.cos().float()[:, None], a.sin().float()[:, None]
    if c["inverse"]:
        sin = -sin
    if c["layout"] == "neox":
        u, w = x[..., : rot // 2], x[..., rot // 2:rot]
        y = torch.cat((u * cos - w * sin, u * sin + w * cos), dim=-1)
    else:
        u, w = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((u * cos - w * sin, u * sin + w * cos), dim=-1).flatten(-2)
    return torch.cat((y, x[..., rot:]), dim=-1)


def _ancestors(s):
    """(seen[n, t, t], depth[n, t], used[n, t]): which nodes a node sees (itself and its ancestors)."""
    c, p = s["case"], s.get("parents")
    n, t = c["n_seqs"], c["tokens"]
    if p is None:
        seen = torch.ones(t, t, device=DEV).tril().expand(n, t, t)
        used = torch.ones(n, t, dtype=torch.bool, device=DEV)
    else:
        used = p >= -1
        step = (p[:, :, None] == torch.arange(t, device=DEV)) & used[:, :, None]
        seen = step.float() + torch.eye(t, device=DEV)
        for _ in range(max(1, t - 1).bit_length()):
            seen = (seen @ seen).clamp(max=1.0)
    return seen > 0, (seen > 0).sum(-1) - 1, used


def _visible(s, width):
    """Boolean [n, t, width]: the cache rows a token sees."""
    c, lens = s["case"], s["lens"].long()
    n, t = c["n_seqs"], c["tokens"]
    seen, depth, used = _ancestors(s)
    j = torch.arange(width, device=DEV)
    pre = (j < lens[:, None])[:, None].expand(n, t, width)
    at = (lens[:, None] + torch.arange(t, device=DEV))[:, None].expand(n, t, t)
    vis = pre.clone().scatter_(2, at, seen)
    if c["window"]:
        pos = lens[:, None] + depth
        row = j.expand(n, width).clone().scatter_(1, at[:, 0], pos)
        vis &= row[:, None] > (pos - c["window"])[:, :, None]
    return vis & used[..., None]


def _attend(s, dtype):
    c = s["case"]
    n, t, h, hkv, hd = c["n_seqs"], c["tokens"], c["heads"], c["kv_heads"], c["head_dim"]
    width = c["len_max"] + t
    words = [None if w is None else w.transpose(1, 2)[:, :width] for w in (s["ks"], s["vs"])]
    k = _dequantise(s["k"][:, :width], words[0], c["format"], dtype)
    v = _dequantise(s["v"][:, :width], words[1], c["format"], dtype)
    q = s["q"].to(dtype).unflatten(2, (hkv, -1)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    z = (q @ k.permute(0, 2, 3, 1)) / math.sqrt(hd)
    if c["softcap"]:
        z = c["softcap"] * torch.tanh(z / c["softcap"])
    vis = _visible(s, width).repeat_interleave(h // hkv, dim=1)[:, None]
    z = z.masked_fill_(~vis, -math.inf)
    m = z.amax(-1, keepdim=True)
    e = z.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    o = (e @ v.permute(0, 2, 1, 3)) / e.sum(-1, keepdim=True).clamp_(min=1e-30)
    return o.unflatten(2, (t, -1)).permute(0, 2, 1, 3, 4).flatten(2, 3)


def _new_rows(s):
    """Indices (sequence, row) [n, t] of a write's new rows."""
    c = s["case"]
    at = s["lens"].long()[:, None] + torch.arange(c["tokens"], device=DEV)
    return torch.arange(c["n_seqs"], device=DEV)[:, None], at


def _written(s, k, v):
    """What a write case returns: the whole cache of an 8- or 16-bit format (the
    values its codes stand for, and the scales), a 4-bit one's new rows read back."""
    if s["case"]["format"] == "int4":
        return {"k": s["k_out"] if k is None else k, "v": s["v_out"] if v is None else v}
    out = {"k": s["k"], "v": s["v"]}
    if s["ks"] is not None:
        out.update(k_scale=s["ks"], v_scale=s["vs"])
    return out


def _plain(s):
    c = s["case"]
    if c["op"] == "rope":
        return _rotate(s["x"].float(), s["pos"], c).bfloat16()
    if c["op"] == "write":
        b, at = _new_rows(s)
        k = _rotate(s["k_new"].float().flatten(0, 1), at.flatten(), c).view_as(s["k_new"])
        v = s["v_new"].float()
        if c["format"] == "bf16":
            s["k"][b, at], s["v"][b, at] = k.bfloat16(), v.bfloat16()
            return _written(s, None, None)
        for x, codes, words in ((k, s["k"], s["ks"]), (v, s["v"], s["vs"])):
            q, w = _quantise(x, c["format"])
            codes.view(torch.uint8)[b, at] = q.view(torch.uint8)
            words.transpose(1, 2)[b, at] = w
        if c["format"] != "int4":
            return _written(s, None, None)
        back = [_dequantise(s[x][b, at], s[x + "s"].transpose(1, 2)[b, at], "int4").bfloat16()
                for x in ("k", "v")]
        return _written(s, *back)
    if c["op"] == "read":
        rows = c["len_max"]
        live = (torch.arange(rows, device=DEV) < s["lens"][:, None])[..., None, None]
        return tuple(torch.where(live, _dequantise(s[x][:, :rows], s[x + "s"].transpose(1, 2)[:, :rows],
                                                   c["format"]), 0.0).bfloat16() for x in ("k", "v"))
    return _attend(s, torch.float32).bfloat16()


# --------------------------------------------------- the framework's calls


def _framework(s):
    c = s["case"]
    if "handle" not in s:  # what a program makes once and keeps
        from dense_decoder_layer_gb300 import kv

        spec = kv.RopeSpec(THETA, head_dim=c["head_dim"], rot_dim=c["rot_dim"], layout=c["layout"],
                           scaling=c["scaling"], **YARN)
        cache = None
        if c["op"] != "rope":
            cache = kv.KvCache(c["format"], c["n_seqs"], s["k"].shape[1], c["kv_heads"],
                               c["head_dim"], k=s["k"], v=s["v"], k_scale=s["ks"],
                               v_scale=s["vs"], lens=s["lens"])
        s["handle"] = (kv, spec, cache)
    kv, spec, cache = s["handle"]
    if c["op"] == "rope":
        return kv.rope(s["x"], spec, positions=s["pos"], out=s["y"], inverse=c["inverse"])
    if c["op"] == "write":
        cache.write(s["k_new"], s["v_new"], rope=spec)
        if c["format"] != "int4":
            return _written(s, None, None)
        k, v = cache.read_new(c["tokens"], k_out=s["k_out"], v_out=s["v_out"])
        return _written(s, k, v)
    if c["op"] == "read":
        return cache.read(0, c["len_max"], k_out=s["k_out"], v_out=s["v_out"])
    return cache.attend(s["q"], out=s["o"], parents=s["parents"], softcap=c["softcap"],
                        window=c["window"], max_len=c["len_max"])


def run(state):
    if own:
        return _framework(state)
    return _plain(state)


# ------------------------------------------------------ 64 bits, apart


def _exact_rope(x, pos, c):
    x = x.double()
    y = x.clone()
    rot = c["rot_dim"] or c["head_dim"]
    half = rot // 2
    sign = -1.0 if c["inverse"] else 1.0
    turn = torch.polar(torch.ones(pos.numel(), half, device=DEV, dtype=torch.float64),
                       sign * torch.outer(pos.double(), _omega(c)))[:, None]
    first = slice(0, half) if c["layout"] == "neox" else slice(0, rot, 2)
    second = slice(half, rot) if c["layout"] == "neox" else slice(1, rot, 2)
    z = torch.complex(x[..., first], x[..., second]) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_e4m3(x):
    """(value on the e4m3 grid, scale) in 64 bits, ties to even."""
    s = x.abs().amax(-1) / 448
    y = x / torch.where(s > 0, s, torch.ones_like(s))[..., None]
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / step) * step).clamp(-448, 448), s


def _exact_int4(x):
    lo, hi = x.amin(-1).clamp(max=0), x.amax(-1).clamp(min=0)
    s = ((hi - lo) / 15).bfloat16().double()
    s1 = torch.where(s > 0, s, torch.ones_like(s))
    z = torch.round(-lo / s1)
    q = (torch.round(x / s1[..., None]) + z[..., None]).clamp(0, 15)
    return (q - z[..., None]) * s[..., None]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "rope":
        return _exact_rope(s["x"], s["pos"], c)
    if c["op"] == "read":
        out = []
        for x in ("k", "v"):
            y = torch.zeros(s["k_out"].shape, device=DEV, dtype=torch.float64)
            for b, length in enumerate(_lens(c)):
                words = s[x + "s"][b].T[:length]
                y[b, :length] = _dequantise(s[x][b, :length], words, c["format"], torch.float64)
            out.append(y)
        return tuple(out)
    if c["op"] == "write":
        t, out = c["tokens"], {}
        for x in ("k", "v"):
            new = s[x + "_new"].double()
            vals = torch.zeros(s["k"].shape[:2] + new.shape[2:], device=DEV, dtype=torch.float64)
            scales = torch.zeros(new.shape[0], new.shape[2], s["k"].shape[1], device=DEV,
                                 dtype=torch.float64)
            back = torch.zeros_like(new)
            for b, length in enumerate(_lens(c)):
                y = new[b]
                if x == "k":
                    y = _exact_rope(y, length + torch.arange(t, device=DEV), c)
                if c["format"] == "bf16":
                    vals[b, length:length + t] = y
                elif c["format"] == "e4m3":
                    q, sc = _exact_e4m3(y)
                    vals[b, length:length + t] = q
                    scales[b, :, length:length + t] = sc.T
                else:
                    back[b] = _exact_int4(y)
            out[x] = back if c["format"] == "int4" else vals
            if c["format"] == "e4m3":
                out[x + "_scale"] = scales
        return out
    # attention, sequence by sequence and token by token of the tree
    n, t, h, hkv, hd = c["n_seqs"], c["tokens"], c["heads"], c["kv_heads"], c["head_dim"]
    parents = None if s["parents"] is None else s["parents"].tolist()
    o = torch.zeros(n, t, h, hd, device=DEV, dtype=torch.float64)
    for b, length in enumerate(_lens(c)):
        part = {}
        for x in ("k", "v"):
            words = None if s[x + "s"] is None else s[x + "s"][b].T[:length + t]
            part[x] = _dequantise(s[x][b, :length + t], words, c["format"], torch.float64)
        paths, mask = [], torch.zeros(t, length + t, dtype=torch.bool)
        for i in range(t):
            up = i - 1 if parents is None else parents[b][i]
            paths.append([] if up < -1 else ([i] if up == -1 else paths[up] + [i]))
            if not paths[i]:
                continue
            pos = length + len(paths[i]) - 1
            first = max(0, pos - c["window"] + 1) if c["window"] else 0
            mask[i, first:length] = True
            for depth, a in enumerate(paths[i]):
                mask[i, length + a] = length + depth >= first
        mask = mask.to(DEV)
        live = mask.any(-1)
        for head in range(h):
            kv = head // (h // hkv)
            z = s["q"][b, :, head].double() @ part["k"][:, kv].T / math.sqrt(hd)
            if c["softcap"]:
                z = c["softcap"] * torch.tanh(z / c["softcap"])
            p = torch.softmax(z.masked_fill(~mask, -math.inf), dim=-1)
            o[b, live, head] = (p[live] @ part["v"][:, kv])
    return o
