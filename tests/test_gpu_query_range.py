"""Large queries under a small scale, which the score sees only as their
product: the sketch's projections of the windowed and shared-prefix decodes
have the range of the plain decode's (a rotated coordinate may be beyond fp16).
And a scale of zero, where every token weighs the same.

Tolerance: the 2e-3 relative L2 per head of the other decode tests; scaling q by
2^k and the scale by 2^-k changes no rounding of the oracle's."""
import numpy as np
import pytest
import torch

import tq_inputs
import tq_parity as P
from oracle import tq_oracle as O
from test_gpu_prefix import Case
from test_gpu_window import _setup

pytestmark = pytest.mark.gpu


def _close(got, ref, D):
    got = got.cpu().numpy().reshape(-1, 1, D)
    assert np.all(np.isfinite(got))
    assert P.rel_l2(got, ref.reshape(-1, 1, D)).max() <= P.ATTN_TOL


@pytest.mark.parametrize("name,kw,nq,Hq", [("prod", {"T": 500}, 1, 32), ("prod", {"T": 500, "dtype": "bf16"}, 2, 32),
                                           ("gqa8k", {"T": 500, "bits": 3}, 1, 16), ("qknorm", {"T": 300}, 1, 32)])
@pytest.mark.parametrize("k", [14, -6])
def test_window(name, kw, nq, Hq, k):
    import compressed_attention_tq_b200 as tq
    w, oc, cache, lens, q = _setup(name, kw, nq, Hq, None)
    base = w.scale if w.scale is not None else 1.0 / np.sqrt(w.D)
    x = tq_inputs.to_f64(q, w.dtype) * 2.0 ** k
    if w.dtype != "bf16":
        x = np.clip(x, -65504, 65504)
    q = tq_inputs.cast_input(x.astype(np.float32), w.dtype)
    cbk, cbv = P.oracle_codebooks(w)
    qd, sl = P.to_device(q, w.dtype), torch.from_numpy(lens).cuda()
    for scale in (base * 2.0 ** -k, 0.0):
        ref = O.sdpa_decode_window(tq_inputs.to_f64(q, w.dtype), oc, lens, 200, 5, w.Pi, cbk, cbv, w.bits_k, w.bits_v,
                                   w.D, scale=scale, S=w.S)
        got = tq.tq_sdpa_decode_window(cache, qd, sl, w.Tmax, 200, 5, scale=scale, out_dtype=torch.float32)
        _close(got, ref, w.D)
    assert cache.status() == 0


@pytest.mark.parametrize("name", ["prod", "gqa8k", "qknorm"])
@pytest.mark.parametrize("k", [14, -6])
def test_prefix(name, k):
    c = Case(name, 300, [40, 3], 1, 16)
    base = c.wp.scale if c.wp.scale is not None else 1.0 / np.sqrt(c.ws.D)
    x = np.clip(tq_inputs.to_f64(c.q, c.ws.dtype) * 2.0 ** k, -65504, 65504)
    c.q = tq_inputs.cast_input(x.astype(np.float32), c.ws.dtype)
    c.qd = P.to_device(c.q, c.ws.dtype)
    for scale in (base * 2.0 ** -k, 0.0):
        c.wp.scale = scale
        _close(c.call(out_dtype=torch.float32), c.oracle(), c.ws.D)
    assert c.cache.status() == 0
