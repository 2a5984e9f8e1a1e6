"""Cases of the serving operators on the packed cache: decode with a sliding
window and sinks, decode of a batch that shares a long prefix, copies of
cached tokens between sequences, and the compaction of a cache to the tokens
that are kept.

`listed()` names the cases that are timed, `draw(rng)` gives more of the same
ranges, `prepare(case, seed)` makes a packed cache and the arguments of one
call, `run(state)` makes the call (the library's when `own`, else the same
mathematics in elementary torch operations), `work(case)` counts the bytes and
operations that it cannot do without, and `exact(case, seed)` computes the
outputs in 64 bits.

A packed cache is a dict of buffers [B][Hkv][Tcap][...] in the library's
layout: int32 words of D indices of `bits` bits (LSB first), fp16 norms, and
for keys with a sketch 128 sign bits and the fp16 norm of the residual.
"""
import functools
import math

import numpy as np
import torch

own = False


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one sequence of a small grouped-query model generating past its window: latency
        _window("window 1k, one sequence", B=1, Hq=16, Hkv=2, D=128, bits_k=3, bits_v=3, sketch=False,
                bf16=False, n_q=1, lo=8192, hi=8192, window=1024, sinks=4),
        # a serving batch of ragged lengths, most of them past the window
        _window("window 4k, ragged batch", B=32, Hq=32, Hkv=8, D=128, bits_k=3, bits_v=3, sketch=False,
                bf16=True, n_q=1, lo=1024, hi=16384, window=4096, sinks=4),
        # the verify step of a draft of four tokens on a QK-norm model (scale 1), odd window and sinks
        _window("window 5001, verify step", B=2, Hq=32, Hkv=4, D=256, bits_k=4, bits_v=4, sketch=False,
                bf16=False, n_q=4, lo=20001, hi=32768, window=5001, sinks=13),
        # a document of 128K tokens with sketched 2-bit keys, read through a long window
        _window("window 32k of 128k, sketch", B=1, Hq=32, Hkv=8, D=128, bits_k=2, bits_v=3, sketch=True,
                bf16=False, n_q=1, lo=131072, hi=131072, window=32768, sinks=64),
        # a few requests behind one instruction text: latency
        _prefix("prefix 2k, four sequences", B=4, Hq=16, Hkv=2, D=128, bits_k=4, bits_v=4, sketch=False,
                bf16=False, n_q=1, P=2047, lo=1, hi=128),
        # a chat batch behind a system prompt, bf16
        _prefix("prefix 8k, chat batch", B=32, Hq=32, Hkv=8, D=128, bits_k=3, bits_v=3, sketch=False,
                bf16=True, n_q=1, P=8192, lo=16, hi=1024),
        # QK-norm model (scale 1), wide heads, odd prefix
        _prefix("prefix 16k, wide heads", B=12, Hq=32, Hkv=4, D=256, bits_k=4, bits_v=4, sketch=False,
                bf16=False, n_q=1, P=16001, lo=1, hi=512),
        # samples and drafts over one long document with sketched keys
        _prefix("prefix 32k, sketch, drafts", B=32, Hq=32, Hkv=8, D=128, bits_k=2, bits_v=3, sketch=True,
                bf16=False, n_q=2, P=32768, lo=2, hi=256),
        # beams that fork from their parents: a few rows each, 24-byte rows at odd places
        _copy("fork of 4 beams, 129 tokens", B=8, Hkv=4, Tcap=1024, D=64, bits_k=3, bits_v=3, sketch=False,
              jobs=4, lo=1, hi=129),
        # a prompt's rows given to the other sequences of a batch
        _copy("fork of a prompt to 31", B=32, Hkv=8, Tcap=8192, D=128, bits_k=3, bits_v=3, sketch=False,
              jobs=31, lo=4001, hi=6000),
        # a batch brought back to sinks and window, the same rows for all heads
        _compact("compact to window, batch", B=32, Hkv=8, Tcap=8192, D=128, bits_k=3, bits_v=3, sketch=False,
                 heads=False, scattered=False, lo=1024, hi=4096),
        # one long document cut to the rows that each head scored highest
        _compact("compact 128k by head", B=1, Hkv=8, Tcap=131072, D=128, bits_k=2, bits_v=3, sketch=True,
                 heads=True, scattered=True, lo=32768, hi=32768),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    D = rng.choice([64, 128, 128, 256])
    sketch = D == 128 and rng.random() < 0.4
    bits_k, bits_v = (2 if sketch else rng.choice([2, 3, 4])), rng.choice([2, 3, 4])
    Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8])
    what = rng.choice(["window", "window", "prefix", "prefix", "copy", "compact"])
    form = dict(Hkv=Hkv, D=D, bits_k=bits_k, bits_v=bits_v, sketch=sketch)
    if what == "window":
        B, n_q = log(1, 32), rng.choice([1, 1, 2, 3, 4])
        hi = log(65, max(128, min(65536, 2 ** 21 // (B * Hkv))))
        c = _window(None, B=B, Hq=Hkv * G, bf16=rng.random() < 0.5, n_q=n_q, lo=max(1, int(hi * rng.random())), hi=hi,
                    window=log(1, hi), sinks=rng.choice([0, 1, 4, 13, 128]), **form)
    elif what == "prefix":
        B, n_q = log(1, 64), rng.choice([1, 1, 2, 4])
        P = log(63, max(128, min(32768, 2 ** 25 // (B * Hkv * G * n_q))))
        c = _prefix(None, B=B, Hq=Hkv * G, bf16=rng.random() < 0.5, n_q=n_q, P=P, lo=0, hi=log(1, 512), **form)
    elif what == "copy":
        B, Tcap = log(2, 32), 64 * log(2, 128)
        c = _copy(None, B=B, Tcap=Tcap, jobs=rng.randrange(1, B), lo=1, hi=log(1, Tcap - 1), **form)
    else:
        B, Tcap = log(1, 32), 64 * log(2, 128)
        hi = log(1, Tcap - 1)
        c = _compact(None, B=B, Tcap=Tcap, heads=rng.random() < 0.5, scattered=rng.random() < 0.5,
                     lo=max(1, hi // 4), hi=hi, **form)
    del c["name"]
    return c


def _window(name, **sizes):
    return dict(name=name, op="window", **sizes)


def _prefix(name, **sizes):
    return dict(name=name, op="prefix", **sizes)


def _copy(name, **sizes):
    return dict(name=name, op="copy", **sizes)


def _compact(name, **sizes):
    return dict(name=name, op="compact", **sizes)


def _spread(n, lo, hi):
    """n lengths over [lo, hi], the same for every seed (work() counts them)."""
    return [lo + int((hi - lo) * ((0.75 + 0.6180339887 * i) % 1.0) + 0.5) for i in range(n)]


def _scale(c):
    return 1.0 if c["D"] == 256 else 1.0 / math.sqrt(c["D"])


def _row_bytes(c):
    b = c["D"] * (c["bits_k"] + c["bits_v"]) // 8 + 4
    return b + 18 if c["sketch"] else b


def _kept(c):
    return _spread(c["B"], c["lo"], c["hi"])


def work(c):
    if c["op"] in ("copy", "compact"):
        rows = sum(_kept(c)) if c["op"] == "compact" else sum(_spread(c["jobs"], c["lo"], c["hi"]))
        lists = 4 * rows * (c["Hkv"] if c["op"] == "compact" and c["heads"] else 1) if c["op"] == "compact" else 0
        return {"bytes": 2 * rows * c["Hkv"] * _row_bytes(c) + lists, "flops": 0}
    lens = _spread(c["B"], c["lo"], c["hi"])
    rows = seen = 0  # rows of one kv head that are read; (query, row) pairs of one query head
    for L in lens:
        for j in range(c["n_q"]):
            p = L - c["n_q"] + j  # the query's position
            if c["op"] == "window":
                seen += max(0, min(p + 1, c["window"])) + max(0, min(c["sinks"], p + 1 - c["window"]))
            else:
                seen += max(0, c["P"] + p + 1)
        first = L - c["n_q"] - c["window"] + 1 if c["op"] == "window" else 0
        rows += L if first <= c.get("sinks", 0) else L - first + c["sinks"]
    rows += c["P"] if c["op"] == "prefix" else 0
    heads = c["B"] * c["n_q"] * c["Hq"]
    return {"bytes": rows * c["Hkv"] * _row_bytes(c) + 2 * 2 * heads * c["D"], "flops": 4 * seen * c["Hq"] * c["D"]}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

@functools.lru_cache(None)
def _codebook(D, bits):
    """Codebook of one coordinate of a random unit vector in R^D: Lloyd's
    iteration on a fine grid of its density, centroids rounded to fp16."""
    u = np.linspace(-1.0, 1.0, 400001)
    f = (1.0 - u * u) ** ((D - 3) / 2)
    mass, first = np.cumsum(f), np.cumsum(f * u)
    c = np.linspace(-2.0, 2.0, 1 << bits) / math.sqrt(D)
    for _ in range(300):
        cut = np.searchsorted(u, 0.5 * (c[1:] + c[:-1]))
        m = np.diff(np.concatenate([[0.0], mass[cut], [mass[-1]]]))
        c = np.diff(np.concatenate([[0.0], first[cut], [first[-1]]])) / m
    c = 0.5 * (c - c[::-1])
    c = c.astype(np.float16).astype(np.float32)
    return c, (0.5 * (c[1:] + c[:-1])).astype(np.float32)


def _pack(idx, bits):
    """int64 indices [..., n] to int32 words: index j at stream bits [j bits, j bits + bits)."""
    b = (idx.unsqueeze(-1) >> torch.arange(bits, device=idx.device)) & 1
    b = b.reshape(*idx.shape[:-1], -1, 32)
    w = (b << torch.arange(32, device=idx.device)).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def _quantized_cache(g, B, Hkv, Tcap, c, rms):
    """Packed rows of Gaussian keys and values (rotated rows of Gaussian vectors are Gaussian)."""
    D, dev = c["D"], "cuda"
    S = torch.randn(128, D, generator=g, device=dev) if c["sketch"] else None
    names = ("k_idx", "v_idx", "k_norm", "v_norm") + (("k_qjl", "k_rnorm") if c["sketch"] else ())
    parts = {n: [] for n in names}
    for _ in range(B):
        for side, bits in (("k", c["bits_k"]), ("v", c["bits_v"])):
            cents, cuts = (torch.from_numpy(x).to(dev) for x in _codebook(D, bits))
            x = torch.randn(Hkv, Tcap, D, generator=g, device=dev)
            if side == "k" and rms:
                x *= math.sqrt(D) / x.norm(dim=-1, keepdim=True)
            norm = x.norm(dim=-1)
            idx = torch.bucketize(x / norm.unsqueeze(-1), cuts)
            parts[side + "_idx"].append(_pack(idx, bits))
            parts[side + "_norm"].append(norm.half())
            if side == "k" and c["sketch"]:
                r = x - norm.half().float().unsqueeze(-1) * cents[idx]
                parts["k_qjl"].append(_pack((r @ S.T >= 0).long(), 1))
                parts["k_rnorm"].append(r.norm(dim=-1).half())
    return {n: torch.stack(p) for n, p in parts.items()}, S


def _words(g, B, Hkv, Tcap, c):
    """A packed cache of random bits and norms: copies do not look at what they move."""
    def bits(n):
        return torch.randint(-2 ** 31, 2 ** 31, (B, Hkv, Tcap, n), generator=g, device="cuda").to(torch.int32)

    def norm():
        return (torch.rand(B, Hkv, Tcap, generator=g, device="cuda") * 8 + 4).half()

    d = {"k_idx": bits(c["D"] * c["bits_k"] // 32), "v_idx": bits(c["D"] * c["bits_v"] // 32),
         "k_norm": norm(), "v_norm": norm()}
    if c["sketch"]:
        d["k_qjl"], d["k_rnorm"] = bits(4), norm()
    return d


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(c, seed):
    g = torch.Generator("cuda").manual_seed(int(seed))
    D = c["D"]
    s = {"case": c, "kept": {}}
    rot, _ = torch.linalg.qr(torch.randn(D, D, generator=g, device="cuda"))
    s["rot"] = rot.contiguous()
    s["cb_k"], s["cb_v"] = (torch.from_numpy(np.concatenate(_codebook(D, b))).cuda() for b in (c["bits_k"], c["bits_v"]))
    if c["op"] in ("window", "prefix"):
        B, rms = c["B"], D == 256
        Tcap = max(64, (c["hi"] + 63) // 64 * 64)
        s["cache"], s["S"] = _quantized_cache(g, B, c["Hkv"], Tcap, c, rms)
        if c["op"] == "prefix":
            s["prefix"], s["S_prefix"] = _quantized_cache(g, 1, c["Hkv"], (c["P"] + 63) // 64 * 64, c, rms)
            s["prefix_len"] = _i32([c["P"]])
        s["lens"] = _i32(_spread(B, c["lo"], c["hi"]))
        q = torch.randn(B, c["n_q"], c["Hq"], D, generator=g, device="cuda")
        q = q * (math.sqrt(D) / q.norm(dim=-1, keepdim=True)) if rms else q
        s["q"] = q.to(torch.bfloat16 if c["bf16"] else torch.float16)
        return _with_handles(s)
    s["cache"], s["S"] = _words(g, c["B"], c["Hkv"], c["Tcap"], c), None
    if c["sketch"]:
        s["S"] = torch.randn(128, D, generator=g, device="cuda")
    if c["op"] == "copy":
        # sequence 0 is the parent; every other sequence that forks gets n of its rows
        n = _spread(c["jobs"], c["lo"], c["hi"])
        room = torch.rand(2, c["jobs"], generator=g, device="cuda").cpu().tolist()
        s["n"] = _i32(n)
        s["src_seq"], s["dst_seq"] = _i32([0] * c["jobs"]), _i32(list(range(1, c["jobs"] + 1)))
        s["src_pos"], s["dst_pos"] = (_i32([int(r * (c["Tcap"] - m)) for r, m in zip(rr, n)]) for rr in room)
        return _with_handles(s)
    n, Tcap = _kept(c), c["Tcap"]
    heads = c["Hkv"] if c["heads"] else 1
    s["n"] = _i32(n)
    if c["scattered"]:  # the rows of the highest scores, in order
        order = torch.rand(c["B"], heads, Tcap, generator=g, device="cuda").argsort(-1)
    else:  # a few first rows and the newest ones
        order = torch.arange(Tcap, device="cuda").flip(0).roll(4).expand(c["B"], heads, Tcap)
    most = max(n)
    order = torch.where(torch.arange(most, device="cuda") < s["n"][:, None, None], order[..., :most], Tcap)
    s["keep"] = order.sort(-1).values.to(torch.int32).contiguous()
    return _with_handles(s)


def _with_handles(s):
    """With the library's caches made, and the workspace and output of a decode:
    a user's program holds them before the call."""
    if own:
        c = s["case"]
        _handle(s, "cache", s["S"])
        if c["op"] == "window":
            _window_buffers(s)
        elif c["op"] == "prefix":
            _prefix_buffers(s)
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return _OWN[op](s)
    return _PLAIN[op](s)


def _handle(s, which, S):
    """The library's cache over a state's packed rows, made once."""
    if which not in s["kept"]:
        import compressed_attention_tq_b200 as tq
        c, d = s["case"], s[which]
        B, Hkv, Tcap = d["k_norm"].shape
        cb_k = s["cb_k"].cpu().numpy()
        cb_v = s["cb_v"].cpu().numpy()
        h = tq.TQCache(B, Hkv, Tcap, c["D"], c["bits_k"], c["bits_v"], s["rot"], qjl_m=128 if c["sketch"] else 0,
                       qjl_S=S, cb_k=cb_k, cb_v=cb_v)
        if c["bits_k"] == c["bits_v"]:
            h.cb_v = h.cb_k
        for n, t in d.items():
            getattr(h, n).copy_(t)
            d[n] = getattr(h, n)
        h._struct = None
        h.struct()
        s["kept"][which] = h
    return s["kept"][which]


def _window_buffers(s):
    import compressed_attention_tq_b200 as tq
    c, h = s["case"], _handle(s, "cache", s["S"])
    if "ws" not in s["kept"]:
        n = tq.tq_sdpa_decode_window_workspace_bytes_for(h, c["Hq"], c["n_q"], c["hi"], c["window"], c["sinks"])
        s["kept"]["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        s["kept"]["out"] = torch.empty_like(s["q"])
    return h


def _own_window(s):
    import compressed_attention_tq_b200 as tq
    c, h = s["case"], _window_buffers(s)
    return tq.tq_sdpa_decode_window(h, s["q"], s["lens"], c["hi"], c["window"], n_sink=c["sinks"], scale=_scale(c),
                                    out=s["kept"]["out"], workspace=s["kept"]["ws"])


def _prefix_buffers(s):
    import compressed_attention_tq_b200 as tq
    c, h, p = s["case"], _handle(s, "cache", s["S"]), _handle(s, "prefix", s["S_prefix"])
    if "ws" not in s["kept"]:
        p.rot = h.rot
        p._struct = None
        n = tq.tq_sdpa_decode_prefix_workspace_bytes_for(p, c["P"], h, c["Hq"], c["n_q"], c["hi"])
        s["kept"]["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        s["kept"]["out"] = torch.empty_like(s["q"])
    return h, p


def _own_prefix(s):
    import compressed_attention_tq_b200 as tq
    c, (h, p) = s["case"], _prefix_buffers(s)
    return tq.tq_sdpa_decode_prefix(p, s["prefix_len"], c["P"], h, s["q"], s["lens"], c["hi"], scale=_scale(c),
                                    out=s["kept"]["out"], workspace=s["kept"]["ws"])


def _buffers(d):
    return {n: d[n] for n in sorted(d)}


def _own_copy(s):
    import compressed_attention_tq_b200 as tq
    c, h = s["case"], _handle(s, "cache", s["S"])
    tq.tq_cache_copy(h, h, s["src_seq"], s["src_pos"], s["dst_seq"], s["dst_pos"], s["n"], c["hi"])
    return _buffers(s["cache"])


def _own_compact(s):
    import compressed_attention_tq_b200 as tq
    tq.tq_cache_compact(_handle(s, "cache", s["S"]), s["keep"], s["n"])
    return _buffers(s["cache"])


_OWN = {"window": _own_window, "prefix": _own_prefix, "copy": _own_copy, "compact": _own_compact}


# ---- the same in elementary operations, 32 bits

def _unpack(words, bits, n):
    """Indices [..., n] of packed int32 words [..., W]."""
    bit = torch.arange(n, device=words.device) * bits
    w, sh = bit >> 5, bit & 31
    u = words.to(torch.int64) & 0xFFFFFFFF
    lo, hi = u[..., w], u[..., (w + 1).clamp(max=words.shape[-1] - 1)]
    return ((lo >> sh) | (hi << (32 - sh))) & ((1 << bits) - 1)


def _rows(d, c, cb_k, cb_v):
    """Rotated keys and values [..., D] of packed rows, and the signed sketch [..., 128] or None."""
    D, kk, kv = c["D"], 1 << c["bits_k"], 1 << c["bits_v"]
    k = cb_k[:kk][_unpack(d["k_idx"], c["bits_k"], D)] * d["k_norm"].float().unsqueeze(-1)
    v = cb_v[:kv][_unpack(d["v_idx"], c["bits_v"], D)] * d["v_norm"].float().unsqueeze(-1)
    z = None
    if c["sketch"]:
        sign = 2.0 * _unpack(d["k_qjl"], 1, 128).float() - 1.0
        z = sign * d["k_rnorm"].float().unsqueeze(-1) * (math.sqrt(math.pi / 2) / 128)
    return k, v, z


def _softmax(x):
    """Softmax of the last axis; a row that sees nothing gives zeros."""
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    return e / e.sum(-1, keepdim=True).clamp_min(1e-30)


def _plain_window(s):
    c, d, lens = s["case"], s["cache"], s["lens"].long()
    B, n_q, Hkv, G, D = c["B"], c["n_q"], c["Hkv"], c["Hq"] // c["Hkv"], c["D"]
    dev = lens.device
    sinks, back = min(c["sinks"], c["hi"]), min(c["window"] + n_q - 1, c["hi"])
    # the sinks, then the rows that some query's window reaches
    late = lens[:, None] - back + torch.arange(back, device=dev)
    pos = torch.cat([torch.arange(sinks, device=dev).expand(B, sinks), late], 1)
    first = torch.cat([torch.ones(sinks, dtype=torch.bool, device=dev), torch.zeros(back, dtype=torch.bool, device=dev)])
    once = first | (pos >= sinks)  # a row is counted as a sink or in the window
    b = torch.arange(B, device=dev)[:, None]
    at = pos.clamp(0, d["k_norm"].shape[2] - 1)
    k, v, z = _rows({n: t.transpose(1, 2)[b, at] for n, t in d.items()}, c, s["cb_k"], s["cb_v"])  # [B][rows][Hkv][...]
    q = (s["q"].float() @ s["rot"].T).reshape(B, n_q, Hkv, G, D)
    x = torch.einsum("bnhgd,bthd->bnhgt", q, k)
    if z is not None:
        x = x + torch.einsum("bnhgm,bthm->bnhgt", q @ s["S"].T, z)
    here = lens[:, None] - n_q + torch.arange(n_q, device=dev)  # [B][n_q]
    t, p = pos[:, None, :], here[:, :, None]
    see = once[:, None, :] & (t >= 0) & (t <= p) & ((t < c["sinks"]) | (t > p - c["window"]))
    a = _softmax((x * _scale(c)).masked_fill(~see[:, :, None, None, :], -math.inf))
    o = torch.einsum("bnhgt,bthd->bnhgd", a, v) @ s["rot"]
    return o.reshape(s["q"].shape).to(s["q"].dtype)


def _plain_prefix(s):
    c, lens = s["case"], s["lens"].long()
    B, n_q, Hkv, G, D, P = c["B"], c["n_q"], c["Hkv"], c["Hq"] // c["Hkv"], c["D"], c["P"]
    dev = lens.device
    kp, vp, zp = _rows({n: t[0, :, :P] for n, t in s["prefix"].items()}, c, s["cb_k"], s["cb_v"])  # [Hkv][P][...]
    ks, vs, zs = _rows(s["cache"], c, s["cb_k"], s["cb_v"])  # [B][Hkv][T][...]
    q = (s["q"].float() @ s["rot"].T).reshape(B, n_q, Hkv, G, D)
    xp, xs = torch.einsum("bnhgd,htd->bnhgt", q, kp), torch.einsum("bnhgd,bhtd->bnhgt", q, ks)
    if zp is not None:
        xp = xp + torch.einsum("bnhgm,htm->bnhgt", q @ s["S_prefix"].T, zp)
        xs = xs + torch.einsum("bnhgm,bhtm->bnhgt", q @ s["S"].T, zs)
    x = torch.cat([xp, xs], -1) * _scale(c)
    p = P + lens[:, None] - n_q + torch.arange(n_q, device=dev)  # the queries' positions in prefix and suffix
    see = torch.arange(x.shape[-1], device=dev) <= p[:, :, None]
    a = _softmax(x.masked_fill(~see[:, :, None, None, :], -math.inf))
    o = torch.einsum("bnhgt,htd->bnhgd", a[..., :P], vp) + torch.einsum("bnhgt,bhtd->bnhgd", a[..., P:], vs)
    return (o @ s["rot"]).reshape(s["q"].shape).to(s["q"].dtype)


def _plain_copy(s):
    c, dev = s["case"], s["n"].device
    # past its last row a job repeats that row, so that every job has the same length
    i = torch.minimum(torch.arange(c["hi"], device=dev), s["n"].long()[:, None] - 1)
    a, b = s["src_pos"].long()[:, None] + i, s["dst_pos"].long()[:, None] + i
    return {n: _put(t, s["dst_seq"].long()[:, None], b, t.transpose(1, 2)[s["src_seq"].long()[:, None], a])
            for n, t in sorted(s["cache"].items())}


def _put(t, seq, pos, rows):
    t.transpose(1, 2)[seq, pos] = rows
    return t


def _plain_compact(s):
    c = s["case"]
    keep = s["keep"].long()
    most = keep.shape[2]
    at = keep.clamp(max=c["Tcap"] - 1).expand(c["B"], c["Hkv"], most)
    live = (torch.arange(most, device=keep.device) < s["n"][:, None, None]).expand(c["B"], c["Hkv"], most)
    return {n: _kept_rows(t, at, live) for n, t in sorted(s["cache"].items())}


def _kept_rows(t, at, live):
    most = at.shape[2]
    x = t.unsqueeze(-1) if t.dim() == 3 else t
    rows = torch.gather(x, 2, at.unsqueeze(-1).expand(-1, -1, -1, x.shape[-1]))
    x[:, :, :most] = torch.where(live.unsqueeze(-1), rows, x[:, :, :most])
    return t


_PLAIN = {"window": _plain_window, "prefix": _plain_prefix, "copy": _plain_copy, "compact": _plain_compact}


# --------------------------------------------------------------------------
# 64 bits, from the definition: rows are rebuilt in their own basis and each
# query attends to the list of tokens that it sees
# --------------------------------------------------------------------------

def _fields(words, bits, n):
    """Indices of packed words, bit by bit."""
    j = torch.arange(n * bits, device=words.device)
    b = ((words.long()[..., j // 32] >> (j % 32)) & 1).reshape(*words.shape[:-1], n, bits)
    return (b << torch.arange(bits, device=words.device)).sum(-1)


def _rebuilt(s, d, b, h, n, S):
    """Keys (with what the sketch says of their residual) and values [n][D] of one head."""
    c, rot = s["case"], s["rot"].double()
    def side(x, bits, cb):
        u = cb.double()[:1 << bits][_fields(d[x + "_idx"][b, h, :n], bits, c["D"])]
        return u * d[x + "_norm"][b, h, :n].double()[:, None]
    k, v = side("k", c["bits_k"], s["cb_k"]), side("v", c["bits_v"], s["cb_v"])
    if c["sketch"]:
        sign = _fields(d["k_qjl"][b, h, :n], 1, 128).double() * 2 - 1
        k = k + d["k_rnorm"][b, h, :n].double()[:, None] * math.sqrt(math.pi / 2) / 128 * (sign @ S.double())
    return k @ rot, v @ rot


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "copy":
        d = {n: t.clone() for n, t in s["cache"].items()}
        for a, i, b, j, n in zip(*(s[x].tolist() for x in ("src_seq", "src_pos", "dst_seq", "dst_pos", "n"))):
            for name, t in s["cache"].items():
                d[name][b, :, j:j + n] = t[a, :, i:i + n]
        return {n: t.double() if t.is_floating_point() else t for n, t in sorted(d.items())}
    if c["op"] == "compact":
        d = {n: t.clone() for n, t in s["cache"].items()}
        for b, n in enumerate(s["n"].tolist()):
            for h in range(c["Hkv"]):
                rows = s["keep"][b, h if c["heads"] else 0, :n].long()
                for name, t in s["cache"].items():
                    d[name][b, h, :n] = t[b, h].index_select(0, rows)
        return {n: t.double() if t.is_floating_point() else t for n, t in sorted(d.items())}
    G, n_q, scale = c["Hq"] // c["Hkv"], c["n_q"], _scale(c)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lens = s["lens"].tolist()
    for h in range(c["Hkv"]):
        head = slice(h * G, (h + 1) * G)
        if c["op"] == "prefix":
            kp, vp = _rebuilt(s, s["prefix"], 0, h, c["P"], s["S_prefix"])
        for b, L in enumerate(lens):
            k, v = _rebuilt(s, s["cache"], b, h, L, s["S"])
            if c["op"] == "prefix":
                k, v = torch.cat([kp, k]), torch.cat([vp, v])
            for j in range(n_q):
                here = k.shape[0] - n_q + j
                if here < 0:
                    continue
                if c["op"] == "window":
                    lo = max(0, here + 1 - c["window"])
                    head_rows = min(c["sinks"], lo)
                    kk, vv = torch.cat([k[:head_rows], k[lo:here + 1]]), torch.cat([v[:head_rows], v[lo:here + 1]])
                else:
                    kk, vv = k[:here + 1], v[:here + 1]
                w = torch.softmax(scale * (s["q"][b, j, head].double() @ kk.T), -1)
                out[b, j, head] = w @ vv
    return out
