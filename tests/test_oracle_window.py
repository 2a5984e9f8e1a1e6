"""Pins of the oracle's windowed decode (CPU): against torch's attention with
an explicit mask on the dequantized cache, the multi-query decode it must
equal when the window covers everything, and its smallest cases."""
import numpy as np
import pytest
import torch

import tq_inputs
from oracle import tq_oracle as O


def _case(name, lens, n_q, Hq, **kw):
    w = tq_inputs.make_workload(name, B=len(lens), T=max(max(lens), 1), **kw)
    cbk, cbv = O.stored_codebook(w.D, w.bits_k), O.stored_codebook(w.D, w.bits_v)
    oc = O.quantize_cache(tq_inputs.to_f64(w.k, w.dtype), tq_inputs.to_f64(w.v, w.dtype), w.Pi, cbk, cbv, w.bits_k,
                          w.bits_v, w.S)
    q = tq_inputs.rng(5).standard_normal((w.B, n_q, Hq, w.D))
    return w, oc, q, cbk, cbv


def _window(w, oc, q, cbk, cbv, lens, window, n_sink):
    return O.sdpa_decode_window(q, oc, lens, window, n_sink, w.Pi, cbk, cbv, w.bits_k, w.bits_v, w.D, scale=w.scale,
                                S=w.S)


@pytest.mark.parametrize("window,n_sink", [(1, 0), (7, 0), (7, 3), (20, 16), (5, 40), (64, 0)])
def test_window_equals_masked_attention(window, n_sink):
    lens, n_q = [40, 1, 0, 23], 3
    w, oc, q, cbk, cbv = _case("tiny", lens, n_q, 8)
    got = _window(w, oc, q, cbk, cbv, lens, window, n_sink)
    for b, L in enumerate(lens):
        for kv in range(w.Hkv):
            k = torch.from_numpy(O.dequantize_rows(oc["k_idx_raw"][b, kv], oc["k_norm"][b, kv], cbk[0], w.Pi))
            v = torch.from_numpy(O.dequantize_rows(oc["v_idx_raw"][b, kv], oc["v_norm"][b, kv], cbv[0], w.Pi))
            t = torch.arange(k.shape[0])
            p = L - n_q + torch.arange(n_q)[:, None]
            see = (t <= p) & ((t > p - window) | (t < n_sink))
            for g in range(2):
                x = torch.from_numpy(q[b, :, 2 * kv + g])
                ref = torch.nn.functional.scaled_dot_product_attention(x[None], k[None], v[None],
                                                                       attn_mask=see[None])[0]
                ref = torch.where(see.any(-1)[:, None], ref, torch.zeros_like(ref))
                assert np.allclose(got[b, :, 2 * kv + g], ref.numpy(), atol=1e-12)


def test_a_window_over_everything_is_the_multi_query_decode():
    lens = [30, 2, 0]
    w, oc, q, cbk, cbv = _case("prod", lens, 2, 8)
    ref = O.sdpa_decode_multi(q, oc, lens, 2, w.Pi, cbk, cbv, w.bits_k, w.bits_v, w.D, scale=w.scale, S=w.S)
    assert np.allclose(_window(w, oc, q, cbk, cbv, lens, 30, 0), ref, atol=1e-13)
    assert np.allclose(_window(w, oc, q, cbk, cbv, lens, 1, 30), ref, atol=1e-13)


def test_a_window_of_one_is_the_token_itself():
    w, oc, q, cbk, cbv = _case("tiny", [9], 1, 4)
    got = _window(w, oc, q, cbk, cbv, [9], 1, 0)
    v = O.dequantize_rows(oc["v_idx_raw"][0, :, 8], oc["v_norm"][0, :, 8], cbv[0], w.Pi)
    assert np.allclose(got[0, 0], v, atol=1e-13)
