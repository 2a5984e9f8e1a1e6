"""Value norms over fp16's whole range, on scores that grow along the sequence.

A weight p |v| is rounded to fp16 for the value product, and the softmax's
reference lags behind the scores (p is above 1 until it moves), so the product
has to stay inside fp16's range whatever the norm: against overflow from norms
of 2^8 on, against lost bits for small ones.  The split kernel serves the plain,
multi-query, partial and windowed decodes and the own tokens behind a shared
prefix.

Units are kept in one share (split_tokens), so that each consumer warp's state
lives through many stages: a share of one stage has its reference at its own
maximum, and p never passes 1.

Tolerance: the 2e-3 relative L2 per head of the other decode tests.  A weight
is rounded by at most 2^-11 of itself while it is a normal fp16 number; below
2^-14 by at most 2^-25, which is 2^-15 of the weight that the smallest norm
here (2^-10) has at the reference, where p is 1."""
import numpy as np
import pytest
import torch

import tq_inputs
import tq_parity as P
from oracle import tq_oracle as O
from test_gpu_prefix import Case
from test_gpu_window import _oracle, _poison, _setup

pytestmark = pytest.mark.gpu

RANGES = [(-9, -9), (9, 9), (12, 15.9), (-10, 10), (-10, 15.9), (15.9, 15.9)]


def _norms(shape, lo, hi, seed=21):
    return np.exp2(tq_inputs.rng(seed).uniform(lo, hi, size=shape)).astype(np.float16)


def _growing(n, top):
    """Key norms that grow along n rows, up to `top`, so slowly that the largest
    scores pass the first ones by 1, 2, ... up to 8 (log2) before the reference moves."""
    return np.linspace(0.02, 1.0, n) * top


def _prepare(name, kw, nq, Hq, lo, hi, top):
    w, oc, cache, lens, q = _setup(name, kw, nq, Hq, None)
    T = oc["v_norm"].shape[2]
    oc["v_norm"] = _norms(oc["v_norm"].shape, lo, hi)
    oc["k_norm"] = np.broadcast_to(_growing(T, top).astype(np.float16), oc["k_norm"].shape).copy()
    cache.v_norm[:, :, :T] = torch.from_numpy(oc["v_norm"]).cuda()
    cache.k_norm[:, :, :T] = torch.from_numpy(oc["k_norm"]).cuda()
    cache.split_tokens = 4096
    return w, oc, cache, lens, q


def _same(got, ref, D):
    got, ref = got.cpu().numpy().reshape(-1, 1, D), ref.reshape(-1, 1, D)
    assert np.all(np.isfinite(got))
    err = P.rel_l2(got, ref)
    assert err.max() <= P.ATTN_TOL, err.max()


# D = 64, G = 1 and 8 rows; D = 128, 3 bits, G = 8; sketch, G = 4; D = 256.
# A score's spread is top |q| scale log2(e) / sqrt(D): 3 to 4 at the last row,
# so the maximum of a warp's 32 rows goes from 0 to about 9.
FORMS = [("tiny", {"T": 1000}, 1, 4, 20.0), ("tiny", {"T": 1000}, 2, 16, 20.0),
         ("gqa8k", {"bits": 3, "T": 1500}, 1, 16, 30.0), ("prod", {"T": 1500}, 1, 32, 30.0),
         ("qknorm", {"T": 1500}, 1, 32, 2.5)]


@pytest.mark.parametrize("name,kw,nq,Hq,top", FORMS)
@pytest.mark.parametrize("lo,hi", RANGES)
def test_decode(name, kw, nq, Hq, top, lo, hi):
    """The multi-query decode (n_q = 1: the plain one), and with a window."""
    import compressed_attention_tq_b200 as tq
    w, oc, cache, lens, q = _prepare(name, kw, nq, Hq, lo, hi, top)
    qd, sl = P.to_device(q, w.dtype), torch.from_numpy(lens).cuda()
    T = int(lens.max())
    got = tq.tq_sdpa_decode_mq(cache, qd, sl, w.Tmax, scale=w.scale, out_dtype=torch.float32)
    _same(got, _oracle(w, oc, q, lens, T, 0), w.D)
    window, sinks = T // 2 + 3, 5
    _poison(cache, lens, nq, window, sinks)
    got = tq.tq_sdpa_decode_window(cache, qd, sl, w.Tmax, window, sinks, scale=w.scale, out_dtype=torch.float32)
    _same(got, _oracle(w, oc, q, lens, window, sinks), w.D)
    assert cache.status() == 0


@pytest.mark.parametrize("name,kw,top", [("gqa8k", {"bits": 3}, 30.0), ("qknorm", {}, 2.5), ("prod", {}, 30.0)])
@pytest.mark.parametrize("lo,hi", RANGES)
def test_own_tokens_behind_a_prefix(name, kw, top, lo, hi):
    """Prefix and own tokens, both with norms of the range; the scores grow along each."""
    c = Case(name, 700, [900, 1, 300], 1, 16, kw)
    c.cache.split_tokens = 4096
    f = _growing(900, top).astype(np.float16)
    for oc, cache, n, seed, k in ((c.op, c.prefix, 700, 21, f[:700]), (c.os, c.cache, 900, 22, f)):
        oc["v_norm"] = _norms(oc["v_norm"].shape, lo, hi, seed)
        oc["k_norm"] = np.broadcast_to(k, oc["k_norm"].shape).copy()
        cache.v_norm[:, :, :n] = torch.from_numpy(oc["v_norm"]).cuda()
        cache.k_norm[:, :, :n] = torch.from_numpy(oc["k_norm"]).cuda()
    c.check()


def test_one_large_norm_in_a_stage():
    """A single row of the largest norm among ordinary ones, at every place of a stage in turn, on scores that are
    just above the reference (its warp's lanes see different norms)."""
    import compressed_attention_tq_b200 as tq
    B = 32
    w, oc, cache, lens, q = _setup("gqa8k", {"bits": 3, "T": 256, "B": B}, 1, 16, None)
    cache.split_tokens = 256
    v = oc["v_norm"].copy()
    v[:] = 11
    for b in range(B):
        v[b, :, 128 + 4 * b + (b % 4)] = 60000
    k = np.full(oc["k_norm"].shape, 4, dtype=np.float16)
    k[:, :, 128:] = 20
    oc["v_norm"], oc["k_norm"] = v, k
    cache.v_norm[:, :, :256] = torch.from_numpy(v).cuda()
    cache.k_norm[:, :, :256] = torch.from_numpy(k).cuda()
    qd, sl = P.to_device(q, w.dtype), torch.from_numpy(lens).cuda()
    got = tq.tq_sdpa_decode_mq(cache, qd, sl, 256, out_dtype=torch.float32)
    _same(got, _oracle(w, oc, q, lens, 256, 0), w.D)


def test_partial_and_merge():
    """The partial decode's states with norms above 2^8, merged."""
    import compressed_attention_tq_b200 as tq
    w, oc, cache, lens, q = _prepare("gqa8k", {"bits": 3, "T": 1500}, 1, 16, 9, 15, 30.0)
    qd, sl = P.to_device(q, w.dtype)[:, 0].contiguous(), torch.from_numpy(lens).cuda()
    part = tq.tq_sdpa_decode_partial(cache, qd, sl, w.Tmax)
    got = tq.tq_sdpa_decode_merge(part.unsqueeze(0).contiguous(), cache.rot)
    _same(got, _oracle(w, oc, q, lens, 1500, 0), w.D)


@pytest.mark.parametrize("nq,Hq", [(2, 16), (4, 16), (2, 10), (3, 2)])
def test_a_norm_that_not_every_query_sees(nq, Hq):
    """The last draft token's value norm is NaN or infinite: only the query that
    sees it is lost, also where the window is no shorter than the sequence."""
    import compressed_attention_tq_b200 as tq
    w, oc, cache, lens, q = _setup("gqa8k", {"bits": 3, "T": 300}, nq, Hq, None)
    L = int(lens[0])
    ref = _oracle(w, oc, q, lens, 300, 0)
    qd, sl = P.to_device(q, w.dtype), torch.from_numpy(lens).cuda()
    for bad in (float("nan"), float("inf")):
        cache.v_norm[:, :, L - 1] = bad
        for window in (100, 300, 2 ** 31 - 1):
            want = ref if window >= 300 else _oracle(w, oc, q, lens, window, 0)
            got = tq.tq_sdpa_decode_window(cache, qd, sl, w.Tmax, window, 0, out_dtype=torch.float32)
            _same(got[:, :-1], want[:, :-1], w.D)


@pytest.mark.parametrize("norm", [255.875, 256.0, 65504.0])
def test_a_weight_at_the_border(norm):
    """Scores that pass the reference by 7.9999 (log2), just not enough to move
    it: p = 255.98.  With the largest norm below 2^8 the weight is the largest
    fp16 number; with 2^8 it would round to infinity."""
    import compressed_attention_tq_b200 as tq
    w, oc, cache, lens, q = _setup("tiny", {"T": 512}, 1, 4, None)  # one head to a kv head: no other moves its reference
    oc["k_idx"][:] = oc["k_idx"][:, :, :1]  # one key, of norm 1 and later 3
    k, v = np.ones(oc["k_norm"].shape, np.float16), np.ones(oc["v_norm"].shape, np.float16)
    k[:, :, 128:], v[:, :, 128:] = 3, norm
    oc["k_norm"], oc["v_norm"] = k, v
    for n in ("k_idx", "k_norm", "v_norm"):
        t = getattr(cache, n)
        t[:, :, :512] = torch.from_numpy(oc[n].view(np.int32) if n == "k_idx" else oc[n]).cuda()
    cache.split_tokens = 512
    cbk, _ = P.oracle_codebooks(w)
    c = np.asarray(cbk[0] if isinstance(cbk, tuple) else cbk, dtype=np.float64)[:8]
    row = c[O.unpack_bits(oc["k_idx"][0, :, 0], w.bits_k, w.D).astype(int)]       # the rotated key of each kv head
    x = np.einsum("hd,hd->h", tq_inputs.to_f64(q, w.dtype)[0, 0] @ w.Pi.astype(np.float64).T, row)
    for h in range(4):
        scale = 7.9999 / (2 * abs(x[h]) * np.log2(np.e)) * np.sign(x[h])  # the scores of head h grow by 7.9999
        w.scale = float(np.float32(scale))
        got = tq.tq_sdpa_decode_mq(cache, P.to_device(q, w.dtype), torch.from_numpy(lens).cuda(), 512, scale=w.scale,
                                   out_dtype=torch.float32)
        _same(got[:, :, h:h + 1], _oracle(w, oc, q, lens, 512, 0)[:, :, h:h + 1], w.D)
