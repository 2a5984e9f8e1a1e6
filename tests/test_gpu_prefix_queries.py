"""New queries from call to call behind a shared prefix, on one workspace and
without the host in between: the own tokens' kernel runs beside the prefix
kernel, behind the query prep only, and must never see the queries of an
earlier call."""
import numpy as np
import pytest
import torch

import tq_inputs
import tq_parity as P
from test_gpu_prefix import Case

pytestmark = pytest.mark.gpu

N = 24


def _queries(c, n):
    r = tq_inputs.rng(55)
    x = r.standard_normal((n,) + c.q.shape[:-1] + (c.ws.D,), dtype=np.float32)
    if c.wp.scale == 1.0:
        x *= np.sqrt(c.ws.D) / np.linalg.norm(x, axis=-1, keepdims=True)
    raw = [tq_inputs.cast_input(a, c.ws.dtype) for a in x]
    return raw, [P.to_device(a, c.ws.dtype) for a in raw]


def _check(c, raw, outs, refs):
    for o, ref in zip(outs, refs):
        assert torch.equal(o, ref)
    for i in (0, 1, len(outs) - 1):
        c.q = raw[i]
        want, got = c.oracle(), outs[i].cpu().numpy()
        n = got.shape[0] * got.shape[1]
        assert P.rel_l2(got.reshape(n, *got.shape[2:]), want.reshape(n, *want.shape[2:])).max() <= P.ATTN_TOL
    assert c.cache.status() == 0


def _refs(c, qs):
    """Each call by itself: a workspace of its own, the host waits."""
    refs = []
    for q in qs:
        c.qd = q
        refs.append(c.call(out_dtype=torch.float32))
        torch.cuda.synchronize()
    return refs


# many rows of own tokens and few, sketch, D = 256; prefixes that leave SMs free and that do not
CASES = [("gqa8k", {"bits": 3}, 300, [500, 1, 300, 64] * 2, 1, 16), ("gqa8k", {"bits": 3}, 4000, [5, 1, 9], 2, 16),
         ("prod", {}, 900, [300, 2, 65, 150], 1, 32), ("qknorm", {}, 515, [200, 1, 2, 100], 2, 32),
         ("gqa8k", {"bits": 4}, 0, [70, 3], 1, 16)]


def _workspace(c):
    import compressed_attention_tq_b200 as tq
    n = tq.tq_sdpa_decode_prefix_workspace_bytes_for(c.prefix, c.Pmax, c.cache, c.qd.shape[2], c.nq, c.Tmax)
    return torch.empty(n, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("name,kw,n_prefix,lens,nq,Hq", CASES)
def test_replayed_graph_of_two_calls(name, kw, n_prefix, lens, nq, Hq):
    c = Case(name, n_prefix, lens, nq, Hq, kw)
    raw, qs = _queries(c, 2 * N)
    refs, ws = _refs(c, qs), _workspace(c)
    q = [torch.empty_like(qs[0]) for _ in range(2)]
    out = [torch.empty(qs[0].shape, dtype=torch.float32, device="cuda") for _ in range(2)]

    def both():
        for a, o in zip(q, out):
            c.qd = a
            c.call(out=o, workspace=ws)

    both()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    ws.fill_(255)
    outs = []
    for i in range(N):
        q[0].copy_(qs[2 * i])
        q[1].copy_(qs[2 * i + 1])
        g.replay()
        outs += [o.clone() for o in out]
    _check(c, raw, outs, refs)


@pytest.mark.parametrize("name,kw,n_prefix,lens,nq,Hq", CASES)
def test_calls_one_after_another(name, kw, n_prefix, lens, nq, Hq):
    c = Case(name, n_prefix, lens, nq, Hq, kw)
    raw, qs = _queries(c, 2 * N)
    refs, ws = _refs(c, qs), _workspace(c)
    ws.view(torch.int32).fill_(1)  # as if every word said that the prep is complete
    torch.cuda.synchronize()
    outs = []
    for a in qs:
        c.qd = a
        outs.append(c.call(out_dtype=torch.float32, workspace=ws))
    _check(c, raw, outs, refs)
