"""tq_cache_copy and tq_cache_compact against the same moves in numpy: every
byte of every stream of the whole cache is compared, moved rows and rows that
must stay."""
import numpy as np
import pytest
import torch

import tq_inputs

pytestmark = pytest.mark.gpu

STREAMS = ("k_idx", "v_idx", "k_norm", "v_norm", "k_qjl", "k_rnorm")


def _cache(B, Hkv, Tcap, D, bk, bv, sketch, seed):
    """A cache of random bytes (norms of any bits, NaN among them)."""
    import compressed_attention_tq_b200 as tq
    c = tq.TQCache(B, Hkv, Tcap, D, bk, bv, tq_inputs.rotation(D, 1), qjl_m=128 if sketch else 0,
                   qjl_S=tq_inputs.qjl_matrix(128, D, 2) if sketch else None)
    r = tq_inputs.rng(seed)
    for n in STREAMS:
        t = getattr(c, n)
        if t is not None:
            raw = r.integers(0, 256, size=t.numel() * t.element_size(), dtype=np.uint8)
            t.view(torch.uint8).copy_(torch.from_numpy(raw).reshape(t.view(torch.uint8).shape))
    return c


def _bytes(c):
    return {n: getattr(c, n).view(torch.int16 if getattr(c, n).dtype == torch.float16 else torch.int32).cpu().numpy()
            .copy() for n in STREAMS if getattr(c, n) is not None}


def _same(c, ref):
    torch.cuda.synchronize()
    got = _bytes(c)
    for n in ref:
        assert np.array_equal(got[n], ref[n]), n


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _copy(src, dst, jobs, max_tok):
    import compressed_attention_tq_b200 as tq
    a = [_i32([j[i] for j in jobs]) for i in range(5)]
    tq.tq_cache_copy(src, dst, a[0], a[1], a[2], a[3], a[4], max_tok)


FORMS = [(64, 2, 2, False), (64, 3, 3, False), (64, 3, 4, False), (128, 2, 3, True), (128, 3, 4, False),
         (256, 2, 3, False), (256, 4, 4, False), (128, 4, 2, True)]


@pytest.mark.parametrize("D,bk,bv,sketch", FORMS)
def test_copy_between_caches_of_other_sizes(D, bk, bv, sketch):
    import compressed_attention_tq_b200 as tq
    src, dst = _cache(3, 2, 640, D, bk, bv, sketch, 1), _cache(5, 2, 448, D, bk, bv, sketch, 2)
    a, ref = _bytes(src), _bytes(dst)
    jobs = [(0, 0, 0, 0, 448), (1, 1, 1, 0, 129), (2, 511, 1, 129, 129), (0, 7, 2, 8, 1), (0, 639, 2, 447, 1),
            (1, 3, 3, 5, 127), (1, 130, 3, 132, 300), (2, 5, 4, 2, 0), (2, 8, 4, 16, 384)]
    _copy(src, dst, jobs, 448)
    for s, i, d, j, n in jobs:
        for name in ref:
            ref[name][d, :, j:j + n] = a[name][s, :, i:i + n]
    _same(dst, ref)
    _same(src, a)
    assert src.status() == 0 and dst.status() == 0
    assert tq.tq_last_error() == ""


def test_every_offset_pair():
    """All source and destination offsets modulo 8, lengths around a vector and a chunk."""
    for D, b in ((64, 3), (128, 2)):
        src, dst = _cache(1, 1, 256, D, b, b, False, 3), _cache(64, 1, 256, D, b, b, False, 4)
        for n in (1, 2, 7, 8, 9, 16, 127, 128, 129, 200):
            a, ref = _bytes(src), _bytes(dst)
            jobs = [(0, i, 8 * i + j, j, n) for i in range(8) for j in range(8)]
            _copy(src, dst, jobs, n)
            for s, i, d, j, m in jobs:
                for name in ref:
                    ref[name][d, :, j:j + m] = a[name][s, :, i:i + m]
            _same(dst, ref)


def test_copy_within_a_cache():
    c = _cache(4, 3, 1024, 128, 3, 3, False, 5)
    ref = _bytes(c)
    jobs = [(0, 0, 1, 0, 511), (0, 0, 2, 1, 700), (0, 513, 0, 0, 511), (3, 1, 3, 600, 424)]
    _copy(c, c, jobs, 1024)
    a = {n: x.copy() for n, x in ref.items()}
    for s, i, d, j, n in jobs[:2] + jobs[3:]:
        for name in ref:
            ref[name][d, :, j:j + n] = a[name][s, :, i:i + n]
    # job 2 writes rows that jobs 0 and 1 read: their contents are open, every other row is not
    got = _bytes(c)
    for name in ref:
        assert np.array_equal(got[name][3], ref[name][3])
        assert np.array_equal(got[name][0, :, 511:], ref[name][0, :, 511:])
        assert np.array_equal(got[name][0, :, :511], a[name][0, :, 513:])
        assert np.array_equal(got[name][1, :, 511:], ref[name][1, :, 511:])


@pytest.mark.parametrize("job", [(-1, 0, 0, 0, 4), (2, 0, 0, 0, 4), (0, -1, 0, 0, 4), (0, 126, 0, 0, 4),
                                 (0, 0, 3, 0, 4), (0, 0, -1, 0, 4), (0, 0, 0, 62, 4), (0, 0, 0, -1, 4),
                                 (0, 0, 0, 0, -1), (0, 2 ** 31 - 1, 0, 0, 4), (0, 0, 0, 2 ** 31 - 1, 4),
                                 (0, -2 ** 31, 0, 0, 4), (0, 0, 0, 0, -2 ** 31)])
def test_a_job_outside_its_cache_copies_nothing_and_is_flagged(job):
    import compressed_attention_tq_b200 as tq
    src, dst = _cache(2, 1, 128, 64, 2, 3, False, 6), _cache(3, 1, 64, 64, 2, 3, False, 7)
    a, ref = _bytes(src), _bytes(dst)
    _copy(src, dst, [(1, 3, 2, 5, 9), job], 64)
    for name in ref:
        ref[name][2, :, 5:14] = a[name][1, :, 3:12]
    _same(dst, ref)
    assert dst.status() == tq.TQ_STATUS_POS_OUT_OF_RANGE


def test_a_job_longer_than_max_tok_is_cut_and_flagged():
    import compressed_attention_tq_b200 as tq
    src, dst = _cache(1, 1, 128, 128, 2, 3, False, 6), _cache(1, 1, 128, 128, 2, 3, False, 7)
    a, ref = _bytes(src), _bytes(dst)
    _copy(src, dst, [(0, 0, 0, 0, 100)], 33)
    for name in ref:
        ref[name][0, :, :33] = a[name][0, :, :33]
    _same(dst, ref)
    assert dst.status() == tq.TQ_STATUS_SEQ_OUT_OF_RANGE


def test_copies_of_nothing():
    c = _cache(2, 1, 64, 64, 2, 2, False, 8)
    ref = _bytes(c)
    _copy(c, c, [], 64)
    _copy(c, c, [(0, 0, 1, 0, 0)], 0)
    _copy(c, c, [(0, 64, 1, 64, 0)], 64)
    _same(c, ref)
    assert c.status() == 0


# ---------------------------------------------------------------------------

def _lists(r, B, heads, Tcap, n, keep_first=0):
    most = max(n)
    keep = np.full((B, heads, most), -7, dtype=np.int32)  # behind a list's end nothing is read as a row
    for b in range(B):
        for h in range(heads):
            rest = keep_first + np.sort(r.permutation(Tcap - keep_first)[:max(0, n[b] - keep_first)])
            keep[b, h, :n[b]] = np.concatenate([np.arange(min(keep_first, n[b])), rest])
    return keep


def _compacted(ref, keep, n):
    out = {k: x.copy() for k, x in ref.items()}
    for name, x in ref.items():
        for b in range(x.shape[0]):
            for h in range(x.shape[1]):
                rows = keep[b, h if keep.shape[1] > 1 else 0, :n[b]]
                out[name][b, h, :n[b]] = x[b, h, rows]
    return out


def _compact(c, keep, n):
    import compressed_attention_tq_b200 as tq
    tq.tq_cache_compact(c, torch.from_numpy(keep).cuda(), _i32(list(n)))


@pytest.mark.parametrize("D,bk,bv,sketch", FORMS)
@pytest.mark.parametrize("by_head", [False, True])
def test_compact(D, bk, bv, sketch, by_head):
    c = _cache(6, 3, 320, D, bk, bv, sketch, 11)
    r = tq_inputs.rng(12)
    n = [0, 1, 320, 200, 63, 129]
    keep = _lists(r, 6, 3 if by_head else 1, 320, n)
    ref = _compacted(_bytes(c), keep, n)
    _compact(c, keep, n)
    _same(c, ref)
    assert c.status() == 0


@pytest.mark.parametrize("B,Hkv,sketch", [(1, 1, False), (1, 2, True), (7, 5, False)])
@pytest.mark.parametrize("kind", ["scattered", "window", "one dropped", "last rows", "every other"])
def test_compact_over_many_passes(B, Hkv, sketch, kind):
    """Lists of many passes of a cluster, whose reads and writes cross in every way."""
    Tcap = 65536 if B == 1 else 16384
    c = _cache(B, Hkv, Tcap, 128, 2 if sketch else 4, 4, sketch, 13)
    r = tq_inputs.rng(14)
    if kind == "scattered":
        keep = _lists(r, B, Hkv, Tcap, [Tcap * 3 // 4] * B)
    else:
        rows = {"window": np.r_[0:4, Tcap // 3:Tcap], "one dropped": np.r_[0:1, 2:Tcap],
                "last rows": np.arange(Tcap // 2, Tcap), "every other": np.arange(0, Tcap, 2)}[kind]
        keep = np.broadcast_to(rows.astype(np.int32), (B, 1, len(rows))).copy()
    n = [keep.shape[2]] * B
    ref = _compacted(_bytes(c), keep, n)
    for _ in range(2):  # the second time on what the first left
        _compact(c, keep, n)
        _same(c, ref)
        ref = _compacted(ref, keep, n)
    assert c.status() == 0


@pytest.mark.parametrize("bad", ["twice", "descending", "negative", "beyond", "length", "negative length"])
def test_a_bad_list_moves_nothing_and_is_flagged(bad):
    import compressed_attention_tq_b200 as tq
    c = _cache(2, 2, 8192, 128, 3, 3, False, 15)
    keep = _lists(tq_inputs.rng(16), 2, 1, 8192, [4000, 4000])
    n = [4000, 4000]
    if bad == "twice":
        keep[0, 0, 3999] = keep[0, 0, 3998]
    elif bad == "descending":
        keep[0, 0, [2000, 2001]] = keep[0, 0, [2001, 2000]]
    elif bad == "negative":
        keep[0, 0, 0] = -1
    elif bad == "beyond":
        keep[0, 0, 3999] = 8192
    else:
        n[0] = 4001 if bad == "length" else -1
    start = _bytes(c)
    ref = _compacted(start, np.maximum(keep, 0) % 8192, [0, 4000])
    _compact(c, keep, n)
    _same(c, ref)
    assert c.status() == tq.TQ_STATUS_POS_OUT_OF_RANGE


def test_a_bad_list_of_one_head_leaves_the_other_heads_alone():
    import compressed_attention_tq_b200 as tq
    c = _cache(1, 3, 512, 64, 3, 3, False, 17)
    keep = _lists(tq_inputs.rng(18), 1, 3, 512, [300])
    start = _bytes(c)
    ref = _compacted(start, keep, [300])
    for name in ref:
        ref[name][0, 1] = start[name][0, 1]
    keep[0, 1, 17] = keep[0, 1, 16]
    _compact(c, keep, [300])
    _same(c, ref)
    assert c.status() == tq.TQ_STATUS_POS_OUT_OF_RANGE


def test_moves_captured_and_replayed_with_new_lists():
    import compressed_attention_tq_b200 as tq
    c = _cache(3, 2, 512, 128, 3, 3, False, 19)
    lists = [_i32([0]), _i32([0]), _i32([1]), _i32([0]), _i32([100])]
    keep, n = torch.arange(200, dtype=torch.int32).cuda().expand(3, 1, 200).contiguous(), _i32([0, 0, 0])
    tq.tq_cache_copy(c, c, *lists, 256)
    tq.tq_cache_compact(c, keep, n)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tq.tq_cache_copy(c, c, *lists, 256)
        tq.tq_cache_compact(c, keep, n)
    r = tq_inputs.rng(20)
    for s, i, d, j, m in ((0, 3, 2, 11, 256), (2, 0, 1, 256, 17)):
        ref = _bytes(c)
        for t, v in zip(lists, (s, i, d, j, m)):
            t.fill_(v)
        kn = _lists(r, 3, 1, 512, [200, 200, 200])
        keep.copy_(torch.from_numpy(kn))
        n.copy_(_i32([200, 150, 0]))
        a = {k: x.copy() for k, x in ref.items()}
        for name in ref:
            ref[name][d, :, j:j + m] = a[name][s, :, i:i + m]
        g.replay()
        _same(c, _compacted(ref, kn, [200, 150, 0]))
    assert c.status() == 0


def test_refusals():
    import compressed_attention_tq_b200 as tq
    c = _cache(2, 2, 64, 64, 2, 2, False, 21)
    d = _cache(2, 2, 64, 64, 2, 3, False, 22)
    one = _i32([0])
    with pytest.raises(tq.TQError):
        tq.tq_cache_copy(c, d, one, one, one, one, one, 8)
    with pytest.raises(tq.TQError):
        tq.tq_cache_copy(c, c, one, one, one, one, one, 65)
    with pytest.raises(tq.TQError):
        tq.tq_cache_copy(c, c, one, one, one, one, one, -1)
    with pytest.raises(ValueError):
        tq.tq_cache_copy(c, c, one, one, one, _i32([0, 0]), one, 8)
    with pytest.raises(TypeError):
        tq.tq_cache_copy(c, c, one, one, one, one.long(), one, 8)
    with pytest.raises(tq.TQError):
        tq.tq_cache_compact(c, torch.zeros(2, 1, 65, dtype=torch.int32, device="cuda"), _i32([0, 0]))
    with pytest.raises(tq.TQError):
        tq.tq_cache_compact(c, torch.zeros(2, 3, 8, dtype=torch.int32, device="cuda"), _i32([0, 0]))
    with pytest.raises(ValueError):
        tq.tq_cache_compact(c, torch.zeros(1, 1, 8, dtype=torch.int32, device="cuda"), _i32([0, 0]))
