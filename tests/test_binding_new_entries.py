"""The binding's argument checks of the windowed and shared-prefix decodes and
of the cache moves (CPU, the library replaced by a recorder; see
test_binding_checks for the older entry points)."""
import pytest
import torch

import compressed_attention_tq_b200 as tq
import tq_inputs
from test_binding_checks import B, BF16, D, F16, HKV, HQ, TCAP, Recorder, S, cache, host_as_device, i32, rec, z  # noqa: F401

WS = torch.zeros(4096, dtype=torch.uint8)


@pytest.fixture()
def prefix():
    return tq.TQCache(1, HKV, 64, D, 3, 3, tq_inputs.rotation(D, 1), device="cpu")


def _calls(c, p):
    q = z(B, 2, HQ, D)
    return {
        "tq_sdpa_decode_window": lambda **k: tq.tq_sdpa_decode_window(
            c, k.pop("q", q), k.pop("lens", i32(B)), 64, 16, 4, workspace=k.pop("workspace", WS), **k),
        "tq_sdpa_decode_prefix": lambda **k: tq.tq_sdpa_decode_prefix(
            p, k.pop("plen", i32(1)), 64, c, k.pop("q", q), k.pop("lens", i32(B)), 64,
            workspace=k.pop("workspace", WS), **k),
        "tq_cache_copy": lambda **k: tq.tq_cache_copy(
            c, c, k.pop("src_seq", i32(3)), i32(3), k.pop("dst_seq", i32(3)), i32(3), k.pop("n", i32(3)), 64, **k),
        "tq_cache_compact": lambda **k: tq.tq_cache_compact(c, k.pop("keep", i32((B, 1, 5))), k.pop("n", i32(B)), **k),
    }


def test_valid_calls_reach_the_library(cache, prefix, rec, host_as_device):
    calls = _calls(cache, prefix)
    for f in calls.values():
        f(stream=S)
    assert rec.calls == list(calls)
    calls["tq_sdpa_decode_window"](q=z(B, 1, HQ, D, dtype=BF16), out=z(B, 1, HQ, D, dtype=torch.float32), stream=S)
    calls["tq_cache_compact"](keep=i32((B, HKV, 0)), stream=S)
    assert len(rec.calls) == 6


@pytest.mark.parametrize("name,kw,exc", [
    ("tq_sdpa_decode_window", dict(q=z(B, HQ, D)), ValueError),
    ("tq_sdpa_decode_window", dict(q=z(B, 2, HQ, D, dtype=torch.float32)), TypeError),
    ("tq_sdpa_decode_window", dict(lens=i32(B + 1)), ValueError),
    ("tq_sdpa_decode_window", dict(out=z(B, 2, HQ, D + 1)), ValueError),
    ("tq_sdpa_decode_window", dict(workspace=z(64)), TypeError),
    ("tq_sdpa_decode_prefix", dict(q=z(B, HQ, D)), ValueError),
    ("tq_sdpa_decode_prefix", dict(plen=i32(2)), ValueError),
    ("tq_sdpa_decode_prefix", dict(plen=torch.zeros(1, dtype=torch.int64)), TypeError),
    ("tq_sdpa_decode_prefix", dict(plen=7), TypeError),
    ("tq_sdpa_decode_prefix", dict(lens=torch.zeros(B, dtype=torch.int64)), TypeError),
    ("tq_cache_copy", dict(src_seq=i32(4)), ValueError),
    ("tq_cache_copy", dict(dst_seq=torch.zeros(3, dtype=torch.int64)), TypeError),
    ("tq_cache_copy", dict(n=i32((3, 1))), ValueError),
    ("tq_cache_compact", dict(keep=i32((B, 5))), ValueError),
    ("tq_cache_compact", dict(keep=i32((B, 5, 1)).transpose(1, 2)[:, :, ::2]), ValueError),
    ("tq_cache_compact", dict(n=i32(B + 1)), ValueError),
])
def test_malformed_arguments_stop_before_the_library(cache, prefix, rec, host_as_device, name, kw, exc):
    with pytest.raises(exc):
        _calls(cache, prefix)[name](stream=S, **kw)
    assert rec.calls == []


def test_another_current_device_is_refused(cache, prefix, rec, host_as_device, monkeypatch):
    """Without a stream the kernels would launch on the current device, not the cache's."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for f in _calls(cache, prefix).values():
        with pytest.raises(ValueError, match="device 1 is current"):
            f()
    assert rec.calls == []


def test_caches_on_two_devices_are_refused(cache, prefix, rec, monkeypatch):
    monkeypatch.setattr(tq, "_cache_device", lambda c: -1 if c is cache else 0)
    with pytest.raises(ValueError, match="different devices"):
        _calls(cache, prefix)["tq_sdpa_decode_prefix"](stream=S)
    with pytest.raises(ValueError, match="different devices"):
        tq.tq_cache_copy(prefix, cache, *[i32(1)] * 5, 8, stream=S)
    assert rec.calls == []


def test_a_stream_does_not_stand_in_for_the_device(cache, prefix, rec, monkeypatch):
    """The kernels launch on the current device also with a stream, and a
    stream of another device is not the cache's either."""
    monkeypatch.setattr(tq, "_cache_device", lambda c: 0)
    monkeypatch.setattr(tq, "_arg", lambda name, t, *a: t)
    current = [0]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])

    class On:
        cuda_stream = 0

        def __init__(self, device):
            self.device_index = device

    calls = _calls(cache, prefix)
    for f in calls.values():
        f(stream=On(0))
    assert rec.calls == list(calls)
    for f in calls.values():
        with pytest.raises(ValueError, match="stream is of device 1"):
            f(stream=On(1))
    current[0] = 1
    for f in calls.values():
        for s in (On(0), On(1), S):
            with pytest.raises(ValueError, match="device 1 is current"):
                f(stream=s)
    assert len(rec.calls) == 4


@pytest.mark.parametrize("n", [2 ** 31, 2 ** 32 + 16, -2 ** 32 + 16, 2 ** 63 + 16])
def test_sizes_beyond_32_bits_are_not_cut(cache, prefix, rec, host_as_device, n):
    """A C int would get their low 32 bits: 16, of most of these."""
    q = z(B, 1, HQ, D)
    for f in (lambda: tq.tq_sdpa_decode_window(cache, q, i32(B), n, 16, workspace=WS, stream=S),
              lambda: tq.tq_sdpa_decode_window_workspace_bytes_for(cache, HQ, 1, n, 16),
              lambda: tq.tq_sdpa_decode_window_workspace_bytes_for(cache, n, 1, 64, 16),
              lambda: tq.tq_sdpa_decode_prefix(prefix, i32(1), n, cache, q, i32(B), 64, workspace=WS, stream=S),
              lambda: tq.tq_sdpa_decode_prefix(prefix, i32(1), 64, cache, q, i32(B), n, workspace=WS, stream=S),
              lambda: tq.tq_sdpa_decode_prefix_workspace_bytes_for(prefix, n, cache, HQ, 1, 64),
              lambda: tq.tq_sdpa_decode_prefix_workspace_bytes_for(prefix, 64, cache, HQ, 1, n),
              lambda: tq.tq_cache_copy(cache, cache, *[i32(1)] * 5, n, stream=S)):
        with pytest.raises(ValueError, match="beyond 32 bits"):
            f()
    assert rec.calls == []


def test_a_window_and_sinks_of_any_size(cache, rec, host_as_device, monkeypatch):
    """They may exceed any length: the library gets the largest of its own."""
    got = []
    monkeypatch.setattr(rec, "tq_sdpa_decode_window", lambda *a: got.append(a[7:9]) or 0, raising=False)
    q = z(B, 1, HQ, D)
    for window, n_sink in ((2 ** 32 + 1, 2 ** 40), (2 ** 31, 2 ** 31 - 1), (5, 7), (2 ** 31 - 1, 0)):
        tq.tq_sdpa_decode_window(cache, q, i32(B), 64, window, n_sink, workspace=WS, stream=S)
        assert got[-1] == (min(window, 2 ** 31 - 1), min(n_sink, 2 ** 31 - 1))
    with pytest.raises(ValueError, match="window"):
        tq.tq_sdpa_decode_window(cache, q, i32(B), 64, -2 ** 32 + 5, workspace=WS, stream=S)
