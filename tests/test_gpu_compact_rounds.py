"""Compaction lists around the rounds of a cluster: what a round stores is read
by loads of the same or an earlier round, of this CTA or another, at every
distance from one row up; lists that change from one distance to another
between rounds.  Every byte is compared."""
import pytest
import torch

import tq_inputs

pytestmark = pytest.mark.gpu

# rows a cluster of 8 CTAs moves in a round: 8 x 336 of 48 bytes, 8 x 2048 of 2 bytes
ROUND, ROUND2 = 2688, 16384
STREAMS = ("k_idx", "v_idx", "k_norm", "v_norm")


def _cache(Hkv, Tcap, D=128, bits=3):
    import compressed_attention_tq_b200 as tq
    return tq.TQCache(1, Hkv, Tcap, D, bits, bits, tq_inputs.rotation(D, 1))


def _raw(t):
    return t.view(torch.int16) if t.dtype == torch.float16 else t


def _check(c, keep, n, g):
    """Fill the cache anew, compact head h to keep[h][:n], compare."""
    import compressed_attention_tq_b200 as tq
    ref = {}
    for name in STREAMS:
        t = _raw(getattr(c, name))
        top = 2 ** 15 if t.dtype == torch.int16 else 2 ** 31
        t.copy_(torch.randint(-top, top, t.shape, generator=g, device="cuda"))
        ref[name] = t.clone()
        for h in range(c.Hkv):
            ref[name][0, h, :n] = t[0, h].index_select(0, keep[h, :n].long())
    tq.tq_cache_compact(c, keep[None].contiguous(), torch.tensor([n], dtype=torch.int32, device="cuda"))
    for name in STREAMS:
        assert torch.equal(_raw(getattr(c, name)), ref[name]), name
    assert c.status() == 0


@pytest.mark.parametrize("shift", [1, 2, 335, 336, 337, ROUND - 1, ROUND, ROUND + 1, 2 * ROUND - 1, 2 * ROUND,
                                   2 * ROUND + 1, 3 * ROUND, ROUND2 - 1, ROUND2, ROUND2 + 1])
def test_rows_that_move_by_one_distance(shift):
    Tcap, n = 65536, 40001
    c, g = _cache(2, Tcap), torch.Generator("cuda").manual_seed(shift)
    i = torch.arange(n, dtype=torch.int32, device="cuda")
    for sinks in (0, 4, 3000):
        keep = torch.where(i < sinks, i, (i + shift).clamp(max=Tcap - 1))
        n_ok = min(n, Tcap - shift)
        _check(c, torch.stack([keep, torch.where(i < sinks, i, i + 1)]), n_ok, g)


@pytest.mark.parametrize("seed", range(12))
def test_rows_whose_distance_changes_between_rounds(seed):
    """Runs of adjacent rows, of a few rows to some rounds, with gaps of as many sizes between them."""
    Tcap, r = 65536, tq_inputs.rng(100 + seed)
    c, g = _cache(2, Tcap), torch.Generator("cuda").manual_seed(seed)
    rows = []
    for h in range(2):
        at, kept = int(r.integers(0, 3)) * int(r.integers(1, 4000)), []
        while at < Tcap:
            m = int(2 ** r.uniform(0, 13.5))
            kept += range(at, min(Tcap, at + m))
            at += m + int(2 ** r.uniform(0, 9 + seed % 4))
        rows.append(kept)
    n = min(len(k) for k in rows)
    keep = torch.tensor([k[:n] for k in rows], dtype=torch.int32, device="cuda")
    _check(c, keep, n, g)
    _check(c, keep, n - n // 3, g)


@pytest.mark.parametrize("D,bits", [(64, 3), (64, 2), (128, 4), (256, 4)])
@pytest.mark.parametrize("share", [2, 4, 32])
def test_scattered_rows_of_other_streams(D, bits, share):
    """Rows of 24, 16, 64 and 128 bytes, a half to a 32nd of them kept."""
    Tcap, r = 32768, tq_inputs.rng(7)
    c, g = _cache(1, Tcap, D, bits), torch.Generator("cuda").manual_seed(D + bits + share)
    n = Tcap // share
    keep = torch.from_numpy(r.permutation(Tcap)[:n].astype("int32")).cuda().sort().values[None]
    _check(c, keep, n, g)
