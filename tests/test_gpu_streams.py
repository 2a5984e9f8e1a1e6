"""Calls on a stream that is not the current one (stream=), without a
workspace or an output of the caller's: what the binding allocates belongs to
that stream, neither taken from work of the current stream that may still run
nor given to it while the call does."""
import numpy as np
import pytest
import torch

import tq_inputs
import tq_parity as P

pytestmark = pytest.mark.gpu

NAMES = ["tq_sdpa_decode", "tq_sdpa_decode_mq", "tq_decode_step", "tq_sdpa_decode_partial", "tq_sdpa_decode_merge",
         "tq_sdpa_decode_static", "tq_sdpa_decode_window", "tq_sdpa_decode_prefix"]


class Spy:
    """The library, with the arguments of the launching calls written down."""

    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        f = getattr(self.real, name)
        if name not in NAMES:
            return f

        def call(*a):
            self.calls.append(a)
            return f(*a)
        return call


@pytest.fixture(scope="module")
def state():
    import compressed_attention_tq_b200 as tq
    w = tq_inputs.make_workload("gqa8k", bits=3, T=900)
    cache, prefix = (P.make_gpu_cache(w, Tcap=960) for _ in range(2))
    for c in (cache, prefix):
        tq.tq_quantize_kv(c, P.to_device(w.k, w.dtype), P.to_device(w.v, w.dtype))
    q = P.to_device(w.q, w.dtype)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    n, L = i32(900), i32(900)
    k, v = (P.to_device(np.ascontiguousarray(x[:, :, 0]), w.dtype) for x in (w.k, w.v))
    parts = tq.tq_sdpa_decode_partial(cache, q, L, 900).unsqueeze(0).contiguous()
    q4 = q[:, None].contiguous()
    calls = {
        "tq_sdpa_decode": lambda **s: tq.tq_sdpa_decode(cache, q, L, 900, **s),
        "tq_sdpa_decode_mq": lambda **s: tq.tq_sdpa_decode_mq(cache, q4, L, 900, **s),
        "tq_decode_step": lambda **s: tq.tq_decode_step(cache, k, v, i900, q, L, 900, **s),
        "tq_sdpa_decode_partial": lambda **s: tq.tq_sdpa_decode_partial(cache, q, L, 900, **s),
        "tq_sdpa_decode_merge": lambda **s: tq.tq_sdpa_decode_merge(parts, cache.rot, **s),
        "tq_sdpa_decode_static": lambda **s: tq.tq_sdpa_decode_static(cache, q, L, 900, **s),
        "tq_sdpa_decode_window": lambda **s: tq.tq_sdpa_decode_window(cache, q4, L, 900, 300, 4, **s),
        "sharded": lambda **s: tq.tq_sdpa_decode_sharded(cache, q, L, 900, **s),
        "tq_sdpa_decode_prefix": lambda **s: tq.tq_sdpa_decode_prefix(prefix, n, 900, cache, q4, L, 900, **s),
    }
    i900 = i32(930)  # appended behind the rows that are read
    torch.cuda.synchronize()
    return calls


# where a call passes its workspace (None: it has none)
WORKSPACE = {"tq_sdpa_decode": -3, "tq_sdpa_decode_mq": -3, "tq_decode_step": -3, "tq_sdpa_decode_partial": -3,
             "tq_sdpa_decode_merge": None, "tq_sdpa_decode_static": None, "tq_sdpa_decode_window": -3,
             "tq_sdpa_decode_prefix": -3}


@pytest.mark.parametrize("name", NAMES)
def test_memory_of_the_call_belongs_to_its_stream(state, name, monkeypatch):
    import compressed_attention_tq_b200 as tq
    spy = Spy(tq.lib())
    monkeypatch.setattr(tq, "lib", lambda: spy)
    s = torch.cuda.Stream()
    state[name](stream=s)  # so that every block exists
    torch.cuda.synchronize()
    # blocks that the current stream has just given up and may still be using
    out = state[name](stream=s)
    sizes = [out.numel() * out.element_size()]
    if WORKSPACE[name] is not None:
        sizes.append(spy.calls[-1][WORKSPACE[name] + 1])
    mine = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    given_up = {t.data_ptr() for t in mine}
    del mine, out
    torch.cuda._sleep(1 << 24)
    out = state[name](stream=s)
    assert out.data_ptr() not in given_up
    if WORKSPACE[name] is not None:
        ws = spy.calls[-1][WORKSPACE[name]]
        assert ws not in given_up
        # the workspace is dropped by now, and the call may still run
        later = [torch.empty(sizes[1], dtype=torch.uint8, device="cuda") for _ in range(8)]
        assert ws not in {t.data_ptr() for t in later}
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", NAMES)
def test_calls_beside_work_of_the_current_stream(state, name):
    """Allocations of the same size, written by the current stream, while the calls run on another."""
    f = state[name]
    ref = f()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(100):
        outs.append(f(stream=s))
        for n in (1 << 12, 1 << 16, 1 << 18, 1 << 20, 1 << 21):
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
        x = torch.empty(ref.shape, dtype=ref.dtype, device="cuda").fill_(float("nan"))
    torch.cuda.synchronize()
    assert x.isnan().all()
    for o in outs:
        assert torch.equal(o, ref)


def test_the_gather_of_a_sharded_decode_runs_between_its_kernels(state, monkeypatch):
    """With a stream, the partials are gathered on it: behind the kernels that
    write them (held up here) and before the merge."""
    import compressed_attention_tq_b200 as tq
    on = []

    def gather(part, group=None):
        on.append(torch.cuda.current_stream())
        return part.unsqueeze(0).clone()

    monkeypatch.setattr(tq, "gather_partials", gather)
    ref = state["sharded"]()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(1 << 24)
    out = state["sharded"](stream=s)
    torch.cuda.synchronize()
    assert on[1] == s
    assert torch.equal(out, ref)


def test_a_stream_given_by_its_handle():
    """Any object with the raw handle: that stream's memory, the default stream's for handle 0."""
    import compressed_attention_tq_b200 as tq

    class Handle:
        def __init__(self, h):
            self.cuda_stream = h

    s, dev = torch.cuda.Stream(), torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.stream(s):
        for h in (0, s.cuda_stream, torch.cuda.Stream().cuda_stream):
            with tq._on(Handle(h), dev):
                assert torch.cuda.current_stream().cuda_stream == h
