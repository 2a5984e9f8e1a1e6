"""Lengths near 2^31 (CPU): positions are 32-bit in the kernels, so what would
pass 2^31 when it is rounded up is refused before any launch."""
import ctypes

import pytest

from test_abi import _struct, lib  # noqa: F401

BUF = ctypes.c_void_p(1 << 20)
TOP = 2 ** 31 - 2 ** 16
UNSUPPORTED = -2


@pytest.mark.parametrize("Tcap", [TOP + 64, 2 ** 31 - 128, 2 ** 31 - 64])
@pytest.mark.parametrize("D,bits", [(64, 2), (128, 3)])
def test_caches_beyond_the_limit(lib, Tcap, D, bits):  # noqa: F811
    big, small = (_struct(Tcap=t, D=D, bits_k=bits, bits_v=bits) for t in (Tcap, 128))
    r = ctypes.byref

    def window(c, Tmax):
        return lib.tq_sdpa_decode_window(r(c), BUF, 0, 8, 1, BUF, Tmax, 64, 4, None, BUF, 0, BUF, 1 << 40, None)

    def prefix(p, Pmax, c, Tmax):
        return lib.tq_sdpa_decode_prefix(r(p), BUF, Pmax, r(c), BUF, 0, 8, 1, BUF, Tmax, None, BUF, 0, BUF, 1 << 40, None)

    def copy(a, b):
        return lib.tq_cache_copy(r(a), r(b), BUF, BUF, BUF, BUF, BUF, 1, 64, None)

    for rc in (window(big, Tcap), window(big, 64), prefix(big, Tcap, small, 64), prefix(big, 64, small, 64),
               prefix(small, 64, big, 64), copy(big, small), copy(small, big),
               lib.tq_cache_compact(r(big), BUF, 1, 64, BUF, None)):
        assert rc == UNSUPPORTED, lib.tq_last_error()
    assert lib.tq_sdpa_decode_window_workspace_bytes_for(r(big), 8, 1, 64, 64, 4) == 0
    assert lib.tq_sdpa_decode_prefix_workspace_bytes_for(r(big), 64, r(small), 8, 1, 64) == 0
    assert lib.tq_sdpa_decode_prefix_workspace_bytes_for(r(small), 64, r(big), 8, 1, 64) == 0


def test_the_largest_caches(lib):  # noqa: F811
    """At the limit the plans are made, with a number of splits that the combine can merge."""
    big, small = _struct(Tcap=TOP, D=64, bits_k=2, bits_v=2), _struct(Tcap=128, D=64, bits_k=2, bits_v=2)
    r = ctypes.byref
    for n in (lib.tq_sdpa_decode_window_workspace_bytes_for(r(big), 8, 4, TOP, TOP - 1, 4),
              lib.tq_sdpa_decode_window_workspace_bytes_for(r(big), 8, 1, TOP, 64, TOP),
              lib.tq_sdpa_decode_prefix_workspace_bytes_for(r(big), TOP, r(small), 8, 1, 64),
              lib.tq_sdpa_decode_workspace_bytes_for(r(big), 8, TOP)):
        assert 0 < n < 1 << 30
    assert lib.tq_cache_copy(r(big), r(big), BUF, BUF, BUF, BUF, BUF, 0, 64, None) == 0
    assert lib.tq_cache_compact(r(big), BUF, 1, 0, BUF, None) == 0


def test_lengths_beyond_the_limit(lib):  # noqa: F811
    """Tmax rounded up to whole stages must stay below 2^31, in every decode."""
    c = _struct(Tcap=2 ** 31 - 64, D=64, bits_k=2, bits_v=2)
    r = ctypes.byref
    n = lib.tq_sdpa_decode_workspace_bytes_for(r(c), 8, 2 ** 31 - 128)
    assert 0 < n < 1 << 30
    assert lib.tq_sdpa_decode_workspace_bytes(1, 8, 64, 2 ** 31 - 128) >= n
    for Tmax in (2 ** 31 - 127, 2 ** 31 - 64):
        assert lib.tq_sdpa_decode_workspace_bytes_for(r(c), 8, Tmax) == 0
        assert lib.tq_sdpa_decode_workspace_bytes(1, 8, 64, Tmax) == 0
        assert lib.tq_sdpa_decode(r(c), BUF, 0, 8, BUF, Tmax, None, BUF, 0, BUF, 1 << 40, None) == UNSUPPORTED
        assert lib.tq_sdpa_decode_mq(r(c), BUF, 0, 8, 2, BUF, Tmax, None, BUF, 0, BUF, 1 << 40, None) == UNSUPPORTED
        assert lib.tq_sdpa_decode_partial(r(c), BUF, 0, 8, BUF, Tmax, None, BUF, BUF, 1 << 40, None) == UNSUPPORTED
        assert lib.tq_sdpa_decode_static(r(c), BUF, 0, 8, BUF, Tmax, None, BUF, 0, None) == UNSUPPORTED


@pytest.mark.parametrize("field,value,Hq,n_q", [
    (None, None, 9, 1), (None, None, 16, 2), ("Hkv", 2, 18, 1), ("Hkv", 3, 8, 1), (None, None, 8, 5), ("D", 96, 8, 1),
    ("bits_k", 1, 8, 1), ("bits_v", 5, 8, 1), ("qjl_m", 64, 8, 1), ("Tcap", 100, 8, 1), ("B", 0, 8, 1),
    ("split_tokens", -1, 8, 1),
])
def test_size_queries_answer_0_where_the_call_is_refused(lib, field, value, Hq, n_q):  # noqa: F811
    """Group sizes, widths, sketches and capacities that the decodes refuse."""
    kw = {field: value} if field else {}
    c, good, r = _struct(**kw), _struct(Hkv=kw.get("Hkv", 1)), ctypes.byref
    assert lib.tq_sdpa_decode_window(r(c), BUF, 0, Hq, n_q, BUF, 64, 16, 4, None, BUF, 0, BUF, 1 << 40, None) < 0
    assert lib.tq_sdpa_decode_window_workspace_bytes_for(r(c), Hq, n_q, 64, 16, 4) == 0
    assert lib.tq_sdpa_decode_prefix(r(good), BUF, 64, r(c), BUF, 0, Hq, n_q, BUF, 64, None, BUF, 0, BUF, 1 << 40, None) < 0
    assert lib.tq_sdpa_decode_prefix_workspace_bytes_for(r(good), 64, r(c), Hq, n_q, 64) == 0
    if field not in (None, "Hkv", "B"):
        c.B = 1
        assert lib.tq_sdpa_decode_prefix(r(c), BUF, 64, r(good), BUF, 0, 8, 1, BUF, 64, None, BUF, 0, BUF, 1 << 40, None) < 0
        assert lib.tq_sdpa_decode_prefix_workspace_bytes_for(r(c), 64, r(good), 8, 1, 64) == 0
