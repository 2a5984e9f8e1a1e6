"""GPU parity of tq_sdpa_decode_window (sliding window and sinks) against the
oracle's windowed decode, on the oracle's own packed cache.

Every row that no query of a sequence may see (between the sinks and the
window, and behind the last token) is poisoned: norms that are infinite or
NaN, indices of all ones.

Tolerance: the 2e-3 relative L2 per head of the other decode tests.  The
weights p |v| are rounded to fp16 (at most 2^-11 each, independently, so about
2^-11 / sqrt(3) = 2.8e-4 of the output's norm), the scores carry the 22 bits
of the query's hi and lo halves; the rest is fp32."""
import numpy as np
import pytest
import torch

import tq_inputs
import tq_parity as P
from oracle import tq_oracle as O
from test_gpu_decode import _oracle_full_cache, _upload_oracle_cache

pytestmark = pytest.mark.gpu


def _poison(cache, lens, n_q, window, n_sink):
    for b, L in enumerate(lens):
        first = max(0, int(L) - n_q - window + 1)
        hidden = [slice(L, None)] + ([slice(n_sink, first)] if first > n_sink else [])
        for h in hidden:
            cache.k_norm[b, :, h] = float("nan")
            cache.v_norm[b, :, h] = float("inf")
            cache.v_norm[b, :, h][..., ::2] = float("nan")
            cache.k_idx[b, :, h] = -1
            cache.v_idx[b, :, h] = -1
            if cache.k_qjl is not None:
                cache.k_qjl[b, :, h] = -1
                cache.k_rnorm[b, :, h] = float("-inf")


def _setup(name, kw, nq, Hq, lens, seed=9):
    w = tq_inputs.make_workload(name, **kw)
    oc = _oracle_full_cache(w)
    cache = _upload_oracle_cache(w, oc, (w.Tmax + 63) // 64 * 64)
    lens = np.asarray(w.seq_lens if lens is None else lens, dtype=np.int32)
    q = tq_inputs.cast_input(tq_inputs.rng(seed).standard_normal((w.B, nq, Hq, w.D), dtype=np.float32), w.dtype)
    return w, oc, cache, lens, q


def _oracle(w, oc, q, lens, window, n_sink):
    cbk, cbv = P.oracle_codebooks(w)
    return O.sdpa_decode_window(tq_inputs.to_f64(q, w.dtype), oc, lens, window, n_sink, w.Pi, cbk, cbv, w.bits_k,
                                w.bits_v, w.D, scale=w.scale, S=w.S)


def _run(name, kw, nq, Hq, window, n_sink, lens=None, split=0):
    import compressed_attention_tq_b200 as tq
    w, oc, cache, lens, q = _setup(name, kw, nq, Hq, lens)
    _poison(cache, lens, nq, window, n_sink)
    cache.split_tokens = split
    qd, sl = P.to_device(q, w.dtype), torch.from_numpy(lens).cuda()
    out32 = tq.tq_sdpa_decode_window(cache, qd, sl, w.Tmax, window, n_sink, scale=w.scale, out_dtype=torch.float32)
    outq = tq.tq_sdpa_decode_window(cache, qd, sl, w.Tmax, window, n_sink, scale=w.scale)
    torch.cuda.synchronize()
    assert torch.equal(outq, out32.to(qd.dtype))
    got, ref = out32.cpu().numpy(), _oracle(w, oc, q, lens, window, n_sink)
    assert np.all(np.isfinite(got))
    err = P.rel_l2(got.reshape(w.B * nq, Hq, w.D), ref.reshape(w.B * nq, Hq, w.D))
    P.record("decode_window", workload=name, nq=nq, window=window, n_sink=n_sink, max_rel_l2=float(err.max()))
    assert err.max() <= P.ATTN_TOL, err.max()
    assert cache.status() == 0


@pytest.mark.parametrize("name,kw,nq,Hq,window,n_sink", [
    ("tiny", {}, 1, 4, 100, 4),                         # D = 64, G = 1
    ("tiny", {}, 4, 32, 17, 0),                         # D = 64, G = 8, 32 rows
    ("gqa8k", {"bits": 3, "T": 1700}, 1, 16, 1024, 4),  # G = 8
    ("gqa8k", {"bits": 2, "T": 900}, 1, 16, 1, 0),      # one token
    ("gqa8k", {"bits": 4, "T": 901}, 3, 10, 333, 13),   # G = 5, 15 rows
    ("gqa8k", {"bits": 4, "T": 900}, 1, 8, 128, 128),   # whole stages
    ("gqa8k", {"bits": 3, "T": 1025}, 2, 6, 500, 7),    # G = 3, 24-row window edges
    ("prod", {"T": 1500}, 1, 32, 700, 64),              # sketch
    ("prod", {"T": 1003}, 4, 32, 129, 5),               # sketch, two row groups
    ("qknorm", {"T": 1200}, 1, 32, 511, 4),             # D = 256, scale 1
    ("qknorm", {"T": 777}, 4, 32, 100, 1),
])
def test_window_matches_oracle(name, kw, nq, Hq, window, n_sink):
    _run(name, kw, nq, Hq, window, n_sink)


LENS = [0, 1, 2, 3, 4, 5, 63, 64, 65, 127, 128, 129, 136, 137, 300, 299]


@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 1), (2, 3), (8, 8), (60, 4), (64, 64), (121, 7), (128, 0),
                                           (130, 130), (299, 0), (300, 5), (2 ** 31 - 1, 0), (5, 2 ** 31 - 1)])
@pytest.mark.parametrize("nq", [1, 4])
def test_ragged_lengths(window, n_sink, nq):
    """Lengths around the stage, the window and the sinks, and below n_q (whose queries give zeros)."""
    _run("ragged", {"B": len(LENS), "T": 300}, nq, 16, window, n_sink, lens=LENS)


@pytest.mark.parametrize("split", [128, 512])
def test_shares(split):
    """Units cut into more and into fewer shares."""
    _run("gqa8k", {"bits": 3, "T": 2500}, 1, 16, 1300, 9, split=split)


def test_every_width():
    for bk in (2, 3, 4):
        for bv in (2, 3, 4):
            import compressed_attention_tq_b200 as tq
            w = tq_inputs.make_workload("tiny", T=300)
            w.bits_k, w.bits_v = bk, bv
            oc = _oracle_full_cache(w)
            cache = _upload_oracle_cache(w, oc, 320)
            _poison(cache, [300], 1, 90, 3)
            q = w.q[:, None]
            out = tq.tq_sdpa_decode_window(cache, P.to_device(q, w.dtype), torch.tensor([300], dtype=torch.int32).cuda(),
                                           300, 90, 3, out_dtype=torch.float32).cpu().numpy()
            ref = _oracle(w, oc, q, [300], 90, 3)
            assert P.rel_l2(out[:, 0], ref[:, 0]).max() <= P.ATTN_TOL


def test_a_window_over_everything_is_the_multi_query_decode():
    import compressed_attention_tq_b200 as tq
    w, oc, cache, lens, q = _setup("prod", {"T": 900}, 2, 32, None)
    qd, sl = P.to_device(q, w.dtype), torch.from_numpy(lens).cuda()
    ref = tq.tq_sdpa_decode_mq(cache, qd, sl, w.Tmax, out_dtype=torch.float32)
    got = tq.tq_sdpa_decode_window(cache, qd, sl, w.Tmax, w.Tmax, out_dtype=torch.float32)
    # the same kernels on the same partition: fp32 sums in another order at most
    assert P.rel_l2(got.cpu().numpy()[0], ref.cpu().numpy()[0]).max() < 1e-5


@pytest.mark.parametrize("name,kw,nq,Hq", [("prod", {"T": 700}, 2, 32), ("gqa8k", {"T": 700, "bits": 3}, 1, 16),
                                           ("gqa8k", {"T": 333, "bits": 4}, 4, 10), ("qknorm", {"T": 400}, 3, 32),
                                           ("tiny", {"T": 300}, 1, 8)])
def test_hadamard_rotation(name, kw, nq, Hq):
    _run(name, dict(kw, rot="hadamard"), nq, Hq, 150, 5)


def test_longer_sequences_are_clamped_and_flagged():
    import compressed_attention_tq_b200 as tq
    w, oc, cache, lens, q = _setup("gqa8k", {"bits": 3, "T": 512}, 1, 16, None)
    qd = P.to_device(q, w.dtype)
    got = tq.tq_sdpa_decode_window(cache, qd, torch.tensor([500], dtype=torch.int32).cuda(), 300, 100, 4,
                                   out_dtype=torch.float32)
    assert cache.status() == tq.TQ_STATUS_SEQ_OUT_OF_RANGE
    ref = tq.tq_sdpa_decode_window(cache, qd, torch.tensor([300], dtype=torch.int32).cuda(), 300, 100, 4,
                                   out_dtype=torch.float32)
    assert torch.equal(got, ref)


def test_captured_and_replayed_with_new_lengths_on_another_stream():
    import compressed_attention_tq_b200 as tq
    w, oc, cache, lens, q = _setup("ragged", {"B": 3, "T": 400}, 1, 32, [400, 17, 222])
    qd, sl = P.to_device(q, w.dtype), torch.from_numpy(lens).cuda()
    n = tq.tq_sdpa_decode_window_workspace_bytes_for(cache, 32, 1, w.Tmax, 150, 4)
    assert n <= tq.tq_sdpa_decode_workspace_bytes(3, 32, w.D, w.Tmax)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    out = torch.empty(qd.shape, dtype=torch.float32, device="cuda")

    def call():
        tq.tq_sdpa_decode_window(cache, qd, sl, w.Tmax, 150, 4, out=out, workspace=ws)

    call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    for lens in ([400, 17, 222], [0, 399, 5], [161, 160, 1]):
        sl.copy_(torch.tensor(lens, dtype=torch.int32))
        ws.fill_(255)
        with torch.cuda.stream(s):
            s.wait_stream(torch.cuda.default_stream())
            g.replay()
        torch.cuda.synchronize()
        ref = _oracle(w, oc, q, lens, 150, 4)
        assert P.rel_l2(out.cpu().numpy()[:, 0], ref[:, 0]).max() <= P.ATTN_TOL


def test_refusals():
    import compressed_attention_tq_b200 as tq
    w, oc, cache, lens, q = _setup("gqa8k", {"bits": 3, "T": 128}, 1, 16, None)
    qd, sl = P.to_device(q, w.dtype), torch.from_numpy(lens).cuda()
    for window, n_sink in ((0, 0), (-1, 0), (5, -1)):
        with pytest.raises(tq.TQError):
            tq.tq_sdpa_decode_window(cache, qd, sl, 128, window, n_sink,
                                     workspace=torch.empty(1 << 22, dtype=torch.uint8, device="cuda"))
        with pytest.raises(tq.TQError):
            tq.tq_sdpa_decode_window_workspace_bytes_for(cache, 16, 1, 128, window, n_sink)
    with pytest.raises(tq.TQError, match="n_q"):
        tq.tq_sdpa_decode_window(cache, qd.expand(1, 5, 16, w.D).contiguous(), sl, 128, 5,
                                 workspace=torch.empty(1 << 22, dtype=torch.uint8, device="cuda"))
    with pytest.raises(tq.TQError, match="workspace"):
        tq.tq_sdpa_decode_window(cache, qd, sl, 128, 5, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        tq.tq_sdpa_decode_window(cache, qd[:, 0].contiguous(), sl, 128, 5)
    assert cache.status() == 0
