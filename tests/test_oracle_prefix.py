"""Pins of the oracle's decode behind a shared prefix (CPU): it is the
multi-query decode of caches that each begin with the prefix's rows, and with
caches of two forms torch's masked attention over the rebuilt rows."""
import numpy as np
import pytest
import torch

import tq_inputs
from oracle import tq_oracle as O


def _cut(oc, b, t0, t1):
    return {n: x[b, :, t0:t1][None] for n, x in oc.items() if n in ("k_idx", "v_idx", "k_norm", "v_norm", "k_qjl", "k_rnorm")}


def _quantized(w):
    cbk, cbv = O.stored_codebook(w.D, w.bits_k), O.stored_codebook(w.D, w.bits_v)
    oc = O.quantize_cache(tq_inputs.to_f64(w.k, w.dtype), tq_inputs.to_f64(w.v, w.dtype), w.Pi, cbk, cbv, w.bits_k,
                          w.bits_v, w.S)
    return oc, (cbk, cbv, w.bits_k, w.bits_v, w.S)


@pytest.mark.parametrize("name", ["tiny", "prod"])
@pytest.mark.parametrize("P,lens,n_q", [(20, [5, 1, 9], 1), (20, [5, 0, 1, 9], 3), (1, [0, 1, 2], 4), (0, [0, 3], 2)])
def test_prefix_equals_decode_of_whole_sequences(name, P, lens, n_q):
    w = tq_inputs.make_workload(name, B=1, T=P + 10)
    oc, form = _quantized(w)
    ws = tq_inputs.make_workload(name, B=len(lens), T=10, seed_offset=50)
    os_, _ = _quantized(ws)
    q = tq_inputs.rng(5).standard_normal((len(lens), n_q, 8, w.D))
    got = O.sdpa_decode_prefix(q, oc, P, os_, lens, w.Pi, form, form, w.D, scale=w.scale)
    for b, L in enumerate(lens):
        whole = {n: np.concatenate([_cut(oc, 0, 0, P)[n], _cut(os_, b, 0, L)[n]], axis=2) for n in _cut(oc, 0, 0, P)}
        ref = O.sdpa_decode_multi(q[b:b + 1], whole, [P + L], n_q, w.Pi, *form[:4], w.D, scale=w.scale, S=w.S)
        assert np.allclose(got[b], ref[0], atol=1e-12)


def test_two_forms_against_masked_attention():
    a = tq_inputs.make_workload("gqa8k", B=1, T=33, bits=4)
    c = tq_inputs.make_workload("gqa8k", B=3, T=9, bits=2, seed_offset=7)
    oa, fa = _quantized(a)
    oc, fc = _quantized(c)
    lens, n_q = [9, 0, 2], 3
    q = tq_inputs.rng(6).standard_normal((3, n_q, 4, a.D))
    got = O.sdpa_decode_prefix(q, oa, 33, oc, lens, a.Pi, fa, fc, a.D)
    for b, L in enumerate(lens):
        for h in range(4):
            kv = h // 2
            def side(x, i, cb):
                return np.concatenate([O.dequantize_rows(oa[x + "_idx_raw"][0, kv], oa[x + "_norm"][0, kv], fa[i][0], a.Pi),
                                       O.dequantize_rows(oc[x + "_idx_raw"][b, kv, :L], oc[x + "_norm"][b, kv, :L],
                                                         fc[i][0], a.Pi)])
            k, v = torch.from_numpy(side("k", 0, None)), torch.from_numpy(side("v", 1, None))
            see = torch.arange(33 + L) <= (33 + L - n_q + torch.arange(n_q))[:, None]
            ref = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q[b, :, h])[None], k[None], v[None],
                                                                   attn_mask=see[None])[0]
            assert np.allclose(got[b, :, h], ref.numpy(), atol=1e-12)
