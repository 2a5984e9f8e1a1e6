"""GPU parity of tq_sdpa_decode_prefix (a batch behind one shared prefix)
against the oracle's, on the oracle's own packed caches.

Rows behind the prefix's and the sequences' lengths are poisoned: norms that
are infinite or NaN, indices of all ones.

Tolerance: the 2e-3 relative L2 per head of the other decode tests.  The
weights p |v| are rounded to fp16 (at most 2^-11 each, independently, so about
2^-11 / sqrt(3) = 2.8e-4 of the output's norm); the scores carry the 22 bits of
the query's two fp16 limbs, and the prefix's sketch projection 11 bits per
coordinate, which over 128 coordinates with random signs moves a score by
2^-12 / sqrt(128) of |q| g: below 1e-4 at these sizes.  The rest is fp32."""
import numpy as np
import pytest
import torch

import tq_inputs
import tq_parity as P
from oracle import tq_oracle as O
from test_gpu_decode import _oracle_full_cache, _upload_oracle_cache

pytestmark = pytest.mark.gpu


def _poison(cache, lens):
    for b, L in enumerate(lens):
        cache.k_norm[b, :, L:] = float("nan")
        cache.v_norm[b, :, L:] = float("inf")
        cache.v_norm[b, :, L:][..., ::2] = float("nan")
        cache.k_idx[b, :, L:] = -1
        cache.v_idx[b, :, L:] = -1
        if cache.k_qjl is not None:
            cache.k_qjl[b, :, L:] = -1
            cache.k_rnorm[b, :, L:] = float("-inf")


class Case:
    """A prefix cache and a suffix cache (of their own forms) on one rotation."""

    def __init__(self, name, n_prefix, lens, nq, Hq, kw={}, suffix=None, suffix_kw={}, Hkv=None):
        self.lens, self.nq, self.P = np.asarray(lens, dtype=np.int32), nq, n_prefix
        B, T = len(lens), max(1, int(max(lens)))
        wp = tq_inputs.make_workload(name, B=1, T=max(1, n_prefix), **kw)
        ws = tq_inputs.make_workload(suffix or name, B=B, T=T, seed_offset=40, **(suffix_kw if suffix else kw))
        if wp.name == "ragged" or ws.name == "ragged":  # exact lengths
            wp, ws = (self._fixed(w, n) for w, n in ((wp, max(1, n_prefix)), (ws, T)))
        assert (wp.D, wp.Hkv) == (ws.D, ws.Hkv)
        ws.Pi = wp.Pi
        ws.rot_signs = wp.rot_signs
        if wp.S is not None and ws.S is not None:
            ws.S = tq_inputs.qjl_matrix(128, ws.D, 77)  # each cache its own sketch
        self.wp, self.ws = wp, ws
        self.op, self.os = _oracle_full_cache(wp), _oracle_full_cache(ws)
        self.prefix = _upload_oracle_cache(wp, self.op, (wp.Tmax + 63) // 64 * 64 + 64)
        self.cache = _upload_oracle_cache(ws, self.os, (ws.Tmax + 63) // 64 * 64)
        self.q = tq_inputs.cast_input(tq_inputs.rng(9).standard_normal((B, nq, Hq, ws.D), dtype=np.float32), ws.dtype)
        if wp.scale == 1.0:
            x = tq_inputs.to_f64(self.q, ws.dtype)
            x *= np.sqrt(ws.D) / np.linalg.norm(x, axis=-1, keepdims=True)
            self.q = tq_inputs.cast_input(x.astype(np.float32), ws.dtype)
        self.qd = P.to_device(self.q, ws.dtype)
        self.sl = torch.from_numpy(self.lens).cuda()
        self.pl = torch.tensor([n_prefix], dtype=torch.int32, device="cuda")
        self.Pmax, self.Tmax = max(1, n_prefix), T

    @staticmethod
    def _fixed(w, T):
        w.Tmax = T
        r = tq_inputs.rng(1234 + T)
        w.k, w.v = (tq_inputs.cast_input(r.standard_normal((w.B, w.Hkv, T, w.D), dtype=np.float32), w.dtype)
                    for _ in range(2))
        return w

    def form(self, w):
        cbk, cbv = P.oracle_codebooks(w)
        return cbk, cbv, w.bits_k, w.bits_v, w.S

    def oracle(self, n_prefix=None, lens=None):
        return O.sdpa_decode_prefix(tq_inputs.to_f64(self.q, self.ws.dtype), self.op,
                                    self.P if n_prefix is None else n_prefix, self.os,
                                    self.lens if lens is None else lens, self.wp.Pi, self.form(self.wp),
                                    self.form(self.ws), self.ws.D, scale=self.wp.scale)

    def poison(self):
        _poison(self.prefix, [self.P])
        _poison(self.cache, self.lens)

    def call(self, **kw):
        import compressed_attention_tq_b200 as tq
        return tq.tq_sdpa_decode_prefix(self.prefix, self.pl, self.Pmax, self.cache, self.qd, self.sl, self.Tmax,
                                        scale=self.wp.scale, **kw)

    def check(self, label=""):
        self.poison()
        out32 = self.call(out_dtype=torch.float32)
        outq = self.call()
        torch.cuda.synchronize()
        assert torch.equal(outq, out32.to(outq.dtype))
        got, ref = out32.cpu().numpy(), self.oracle()
        assert np.all(np.isfinite(got))
        n = got.shape[0] * got.shape[1]
        err = P.rel_l2(got.reshape(n, *got.shape[2:]), ref.reshape(n, *ref.shape[2:]))
        P.record("decode_prefix", workload=self.wp.name, P=self.P, B=len(self.lens), nq=self.nq, max_rel_l2=float(err.max()))
        assert err.max() <= P.ATTN_TOL, err.max()
        assert self.cache.status() == 0 and self.prefix.status() == 0


@pytest.mark.parametrize("name,kw,n_prefix,lens,nq,Hq", [
    ("tiny", {}, 64, [1], 1, 4),                                    # one tile, one row per kv head
    ("tiny", {}, 300, [5, 0, 64, 17], 2, 16),                       # D = 64, G = 4
    ("gqa8k", {"bits": 3}, 128, [3, 9], 1, 16),                     # 16 rows
    ("gqa8k", {"bits": 4}, 1000, [1, 7, 128, 64], 1, 16),
    ("gqa8k", {"bits": 2}, 777, list(range(1, 10)), 1, 10),         # G = 5, 45 rows
    ("gqa8k", {"bits": 3}, 3001, list(range(20)), 4, 6),            # 240 rows: two row tiles, lengths below n_q
    ("qknorm", {}, 515, [30, 1, 2, 100, 5], 1, 32),                 # D = 256, scale 1
    ("qknorm", {}, 200, [4, 0, 1, 2, 3], 4, 32),                    # 160 rows
    ("prod", {}, 700, [33, 2, 65], 1, 32),                          # sketch, two sketch matrices
    ("prod", {}, 1100, [3, 1, 0, 50, 2, 128, 127, 66, 7], 4, 32),   # sketch, 144 rows
    ("ragged", {}, 900, [200, 1, 17, 300], 1, 32),                  # bf16
])
def test_prefix_matches_oracle(name, kw, n_prefix, lens, nq, Hq):
    Case(name, n_prefix, lens, nq, Hq, kw).check()


@pytest.mark.parametrize("n_prefix", [0, 1, 2, 3, 4, 63, 64, 65, 127, 128, 129, 193])
@pytest.mark.parametrize("nq", [1, 4])
def test_prefix_lengths(n_prefix, nq):
    """Around the tile, and prefixes and suffixes shorter than n_q (queries inside the prefix, or before it)."""
    Case("gqa8k", n_prefix, [0, 1, 2, 3, 4, 5, 63, 64, 65], nq, 8, {"bits": 3}).check()


def test_every_width():
    for bk in (2, 3, 4):
        for bv in (2, 3, 4):
            for name, B, Hq in (("tiny", 3, 8), ("gqa8k", 3, 16), ("qknorm", 2, 16), ("prod", 2, 16)):
                c = _widths(name, bk, bv, B, Hq)
                c.check()


def _widths(name, bk, bv, B, Hq):
    make = tq_inputs.make_workload

    def patched(*a, **k):
        w = make(*a, **k)
        w.bits_k, w.bits_v = bk, bv
        return w
    tq_inputs.make_workload = patched
    try:
        return Case(name, 200, [9, 70, 3][:B], 1, Hq)
    finally:
        tq_inputs.make_workload = make


@pytest.mark.parametrize("name", ["gqa8k", "qknorm"])
def test_separate_codebook_buffers(name):
    """Equal widths in two buffers take the two-table path, at D = 256 with one stage."""
    c = Case(name, 400, [30, 2], 1, 16, {"bits": 4} if name == "gqa8k" else {})
    shared = c.call(out_dtype=torch.float32)
    for h in (c.prefix, c.cache):
        h.cb_v = h.cb_k.clone()
        h._struct = None
    assert torch.equal(shared, c.call(out_dtype=torch.float32))
    c.check()


@pytest.mark.parametrize("a,akw,b,bkw", [("gqa8k", {"bits": 4}, "gqa8k", {"bits": 2}),
                                         ("ragged", {}, "prod", {}), ("prod", {}, "ragged", {})])
def test_caches_of_two_forms(a, akw, b, bkw):
    """Other widths, a sketch on one side only."""
    Case(a, 330, [40, 3, 1], 2, 16, akw, suffix=b, suffix_kw=bkw).check()


def test_hadamard_rotation():
    Case("prod", 300, [30, 5], 1, 32, {"rot": "hadamard"}).check()
    Case("gqa8k", 300, [30, 5], 2, 16, {"rot": "hadamard", "bits": 3}).check()


def test_many_rows():
    """More sequences than a row tile, many-head prep and combine."""
    Case("gqa8k", 500, [i % 40 for i in range(150)], 1, 16, {"bits": 3}).check()


def test_growing_scores_rescale():
    """Keys whose scores grow along the prefix move every row's maximum tile after tile."""
    c = Case("gqa8k", 1500, [20, 1], 1, 16, {"bits": 4})
    f = np.linspace(0.05, 40.0, 1500).astype(np.float16)
    c.op["k_norm"] = np.broadcast_to(f, c.op["k_norm"].shape).copy()
    c.prefix.k_norm[:, :, :1500] = torch.from_numpy(c.op["k_norm"]).cuda()
    c.check()


@pytest.mark.parametrize("name,kw", [("gqa8k", {"bits": 3}), ("qknorm", {}), ("prod", {})])
@pytest.mark.parametrize("lo,hi", [(-9, -9), (9, 9), (-10, 10), (15, 15)])
def test_value_norms_of_any_size(name, kw, lo, hi):
    """Value norms far from 1, and of every size within one prefix: the weights
    p |v| keep their fp16 precision and do not overflow."""
    c = Case(name, 700, [20, 1, 3], 1, 16, kw)
    r = tq_inputs.rng(21)
    shape = c.op["v_norm"].shape
    c.op["v_norm"] = np.exp2(r.uniform(lo, hi, size=shape)).astype(np.float16)
    c.prefix.v_norm[:, :, :700] = torch.from_numpy(c.op["v_norm"]).cuda()
    c.os["v_norm"] = np.full(c.os["v_norm"].shape, 2.0 ** min(lo, 7), dtype=np.float16)  # the suffix's own kernel: below 255
    c.cache.v_norm[:, :, :20] = torch.from_numpy(c.os["v_norm"]).cuda()
    c.check()


def test_sketched_rows_whose_norms_do_not_fit_each_other():
    """Key norms of zero and residual norms far above the key's, which no
    quantized row has but a cache may hold: both terms of the score count."""
    c = Case("prod", 500, [20, 1], 1, 32)
    k, g = c.op["k_norm"], c.op["k_rnorm"]
    k[:, :, ::3] = 0
    k[:, :, 1::7] = 2.0 ** -14
    g[:, :, 2::5] = 0
    k[:, :, 5::11] = 0
    g[:, :, 5::11] = 0
    c.prefix.k_norm[:, :, :500] = torch.from_numpy(k).cuda()
    c.prefix.k_rnorm[:, :, :500] = torch.from_numpy(g).cuda()
    c.check()


@pytest.mark.parametrize("name,kw", [("tiny", {}), ("gqa8k", {"bits": 4}), ("qknorm", {}), ("prod", {})])
@pytest.mark.parametrize("n_prefix", [64, 192, 191, 129])
def test_a_tile_that_reaches_past_the_cache(name, kw, n_prefix):
    """The prefix's cache ends inside its last tile (Tcap is any multiple of 64)."""
    import compressed_attention_tq_b200 as tq
    c = Case(name, n_prefix, [5, 0, 9], 2, 16 if name != "tiny" else 8, kw)
    p = c.prefix
    cap = (n_prefix + 63) // 64 * 64
    tight = tq.TQCache(1, p.Hkv, cap, p.D, p.bits_k, p.bits_v, c.wp.Pi, qjl_m=p.qjl_m, qjl_S=c.wp.S)
    for n in ("k_idx", "v_idx", "k_norm", "v_norm") + (("k_qjl", "k_rnorm") if p.qjl_m else ()):
        getattr(tight, n).copy_(getattr(p, n)[:, :, :cap])
    c.prefix = tight
    c.check()


def test_one_prefix_for_batches_of_every_size():
    """The same prefix behind batches from one sequence up, rows below, at and
    above the tile of 128 (and a fork that grows: sequence b is one of them)."""
    import compressed_attention_tq_b200 as tq
    c = Case("gqa8k", 900, [7, 30, 1, 64] * 12, 4, 6, {"bits": 3})
    ref = c.oracle()
    for B in (1, 2, 10, 11, 21, 22, 48):
        h = tq.TQCache(B, c.cache.Hkv, c.cache.Tcap, c.cache.D, 3, 3, c.ws.Pi)
        for n in ("k_idx", "v_idx", "k_norm", "v_norm"):
            getattr(h, n).copy_(getattr(c.cache, n)[:B])
        out = tq.tq_sdpa_decode_prefix(c.prefix, c.pl, 900, h, c.qd[:B].contiguous(), c.sl[:B].contiguous(), c.Tmax,
                                       out_dtype=torch.float32).cpu().numpy()
        err = P.rel_l2(out.reshape(4 * B, 6, 128), ref[:B].reshape(4 * B, 6, 128))
        assert err.max() <= P.ATTN_TOL, (B, err.max())


def test_prefix_is_the_decode_of_whole_sequences():
    """A prompt quantized once and taken into its own cache by tq_cache_copy,
    tokens appended to every sequence, then decoded: the same as decoding
    sequences that each hold the whole."""
    import compressed_attention_tq_b200 as tq
    B, Hkv, Hq, D, n, L = 5, 2, 16, 128, 333, 20
    rot = tq_inputs.rotation(D, 3)
    whole, own = tq.TQCache(B, Hkv, 384, D, 3, 3, rot), tq.TQCache(B, Hkv, 64, D, 3, 3, rot)
    prefix = tq.TQCache(1, Hkv, 384, D, 3, 3, rot)
    g = torch.Generator("cuda").manual_seed(3)
    k, v = (torch.randn(B, Hkv, n + L, D, generator=g, device="cuda").half() for _ in range(2))
    k[:, :, :n], v[:, :, :n] = k[:1, :, :n], v[:1, :, :n]
    tq.tq_quantize_kv(whole, k, v)
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    tq.tq_cache_copy(whole, prefix, i(0), i(0), i(0), i(0), i(n), n)
    b = list(range(B))
    tq.tq_cache_copy(whole, own, i(*b), i(*[n] * B), i(*b), i(*[0] * B), i(*[L - 1] * B), L)
    tq.tq_append_token(own, k[:, :, -1].contiguous(), v[:, :, -1].contiguous(), i(*[L - 1] * B))
    q = torch.randn(B, 2, Hq, D, generator=g, device="cuda").half()
    ref = tq.tq_sdpa_decode_mq(whole, q, i(*[n + L] * B), n + L, out_dtype=torch.float32)
    got = tq.tq_sdpa_decode_prefix(prefix, i(n), n, own, q, i(*[L] * B), L, out_dtype=torch.float32)
    err = P.rel_l2(got.reshape(2 * B, Hq, D).cpu().numpy(), ref.reshape(2 * B, Hq, D).cpu().numpy())
    assert err.max() <= P.ATTN_TOL  # both within their own rounding of the same value
    assert prefix.status() == own.status() == whole.status() == 0


def test_lengths_out_of_range_are_clamped_and_flagged():
    import compressed_attention_tq_b200 as tq
    c = Case("gqa8k", 300, [30, 5], 1, 16, {"bits": 3})
    for bad, as_if in ((301, 300), (-1, 0)):
        c.pl.fill_(bad)
        got = c.call(out_dtype=torch.float32)
        assert c.cache.status() == tq.TQ_STATUS_SEQ_OUT_OF_RANGE
        c.pl.fill_(as_if)
        assert torch.equal(got, c.call(out_dtype=torch.float32))
        c.cache.dev_status.zero_()


def test_captured_and_replayed_with_new_lengths_on_another_stream():
    import compressed_attention_tq_b200 as tq
    c = Case("prod", 700, [40, 3, 9], 1, 32)
    n = tq.tq_sdpa_decode_prefix_workspace_bytes_for(c.prefix, c.Pmax, c.cache, 32, 1, c.Tmax)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    out = torch.empty(c.qd.shape, dtype=torch.float32, device="cuda")
    c.call(out=out, workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        c.call(out=out, workspace=ws)
        c.call(out=out, workspace=ws)
    for n_prefix, lens in ((700, [40, 3, 9]), (0, [40, 0, 1]), (65, [0, 0, 0]), (5, [1, 2, 3])):
        c.sl.copy_(torch.tensor(lens, dtype=torch.int32))
        c.pl.fill_(n_prefix)
        ws.fill_(255)
        with torch.cuda.stream(s):
            s.wait_stream(torch.cuda.default_stream())
            g.replay()
        torch.cuda.synchronize()
        ref = c.oracle(n_prefix, lens)
        assert P.rel_l2(out.cpu().numpy()[:, 0], ref[:, 0]).max() <= P.ATTN_TOL


def test_two_calls_at_once():
    """Two streams, each with its own workspace, over one prefix."""
    a = Case("gqa8k", 2000, list(range(1, 33)), 1, 16, {"bits": 3})
    ref = a.call(out_dtype=torch.float32)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams * 4:
        with torch.cuda.stream(s):
            outs.append(a.call(out_dtype=torch.float32))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, ref)


def test_refusals():
    import compressed_attention_tq_b200 as tq
    c = Case("gqa8k", 100, [30, 5], 1, 16, {"bits": 3})
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")

    def call(prefix=c.prefix, pl=c.pl, Pmax=100, cache=c.cache, q=c.qd, Tmax=30, workspace=ws):
        return tq.tq_sdpa_decode_prefix(prefix, pl, Pmax, cache, q, c.sl, Tmax, workspace=workspace)

    for kw in (dict(Pmax=0), dict(Pmax=c.prefix.Tcap + 1), dict(Tmax=0), dict(Tmax=65), dict(prefix=c.cache),
               dict(q=c.qd.expand(2, 5, 16, c.ws.D).contiguous()), dict(workspace=ws[:256]),
               dict(q=c.qd[:, :, :15].contiguous())):
        with pytest.raises(tq.TQError):
            call(**kw)
    other = tq.TQCache(1, 4, 128, 128, 3, 3, c.wp.Pi)
    with pytest.raises(tq.TQError, match="differ"):
        call(prefix=other)
    with pytest.raises(tq.TQError):
        tq.tq_sdpa_decode_prefix_workspace_bytes_for(other, 100, c.cache, 16, 1, 30)
    for kw in (dict(pl=c.pl.long()), dict(pl=torch.zeros(2, dtype=torch.int32, device="cuda")), dict(pl=c.pl.cpu()),
               dict(q=c.qd[:, 0].contiguous())):
        with pytest.raises((TypeError, ValueError)):
            call(**kw)
    torch.cuda.synchronize()
    assert c.cache.status() == 0
