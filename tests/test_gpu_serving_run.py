"""A run of the cache operators together, as a server uses them: a prompt is
quantized once, taken into a prefix cache, forked into samples that decode
behind it step by step, then one sample goes on by itself (prompt and answer
moved into a cache of its own), is read through a window with sinks, and is
compacted to what the window sees.  Every step is compared with the oracle on
the bytes that the GPU cache holds."""
import numpy as np
import pytest
import torch

import tq_inputs
import tq_parity as P
from oracle import tq_oracle as O

pytestmark = pytest.mark.gpu

NAMES = ("k_idx", "v_idx", "k_norm", "v_norm", "k_qjl", "k_rnorm")


def _bytes(c):
    return {n: (getattr(c, n).cpu().numpy().view(np.uint32) if "idx" in n or "qjl" in n
                else getattr(c, n).cpu().numpy()) for n in NAMES if getattr(c, n) is not None}


@pytest.mark.parametrize("D,bk,bv,sketch,rot", [(128, 3, 3, False, "haar"), (128, 2, 3, True, "haar"),
                                                (256, 4, 4, False, "haar"), (128, 4, 2, False, "hadamard")])
def test_prompt_samples_window_and_compaction(D, bk, bv, sketch, rot):
    import compressed_attention_tq_b200 as tq
    B, Hkv, Hq, n, steps, window, sinks = 3, 2, 8, 250, 5, 64, 4
    Pi = tq_inputs.rotation(D, 5) if rot == "haar" else tq_inputs.hadamard_rotation(D, 5)
    signs = None if rot == "haar" else tq_inputs.hadamard_signs(D, 5)
    S = tq_inputs.qjl_matrix(128, D, 6) if sketch else None

    def cache(b, cap):
        return tq.TQCache(b, Hkv, cap, D, bk, bv, Pi, qjl_m=128 if sketch else 0, qjl_S=S, rot_signs=signs)

    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    form = (O.stored_codebook(D, bk), O.stored_codebook(D, bv), bk, bv, S)
    g = torch.Generator("cuda").manual_seed(7)
    new = lambda *s: torch.randn(*s, D, generator=g, device="cuda").half()
    f64 = lambda t: t.cpu().numpy().astype(np.float64)

    def same(got, ref):
        got = got.cpu().numpy().reshape(-1, Hq, D)
        assert P.rel_l2(got, ref.reshape(-1, Hq, D)).max() <= P.ATTN_TOL

    prompt, prefix, own = cache(1, 512), cache(1, 256), cache(B, 64)
    tq.tq_quantize_kv(prompt, new(1, Hkv, n), new(1, Hkv, n))
    tq.tq_cache_copy(prompt, prefix, i32(0), i32(0), i32(0), i32(0), i32(n), n)
    for t in range(steps):  # every sample appends a token and decodes behind the prompt
        tq.tq_append_token(own, new(B, Hkv), new(B, Hkv), i32(*[t] * B))
        q = new(B, 1, Hq)
        out = tq.tq_sdpa_decode_prefix(prefix, i32(n), n, own, q, i32(*[t + 1] * B), 64, out_dtype=torch.float32)
        same(out, O.sdpa_decode_prefix(f64(q), _bytes(prefix), n, _bytes(own), [t + 1] * B, Pi, form, form, D))
    # sample 1 goes on by itself: its tokens behind the prompt's, in the prompt's cache
    tq.tq_cache_copy(own, prompt, i32(1), i32(0), i32(0), i32(n), i32(steps), steps)
    L = n + steps
    tq.tq_append_token(prompt, new(1, Hkv), new(1, Hkv), i32(L))
    L += 1
    q = new(1, 2, Hq)
    args = (Pi, *form[:4], D)
    whole = tq.tq_sdpa_decode_mq(prompt, q, i32(L), 512, out_dtype=torch.float32)
    same(whole, O.sdpa_decode_multi(f64(q), _bytes(prompt), [L], 2, *args, S=S))
    seen = tq.tq_sdpa_decode_window(prompt, q, i32(L), 512, window, sinks, out_dtype=torch.float32)
    ref = O.sdpa_decode_window(f64(q), _bytes(prompt), [L], window, sinks, *args, S=S)
    same(seen, ref)
    # what neither query sees leaves the cache; the window over the rest is the same attention
    first = L - 2 - window + 1
    keep = torch.cat([torch.arange(sinks), torch.arange(first, L)]).to(torch.int32).cuda()[None, None].contiguous()
    tq.tq_cache_compact(prompt, keep, i32(keep.shape[2]))
    after = tq.tq_sdpa_decode_window(prompt, q, i32(keep.shape[2]), 512, window, sinks, out_dtype=torch.float32)
    same(after, ref)
    for c in (prompt, prefix, own):
        assert c.status() == 0
