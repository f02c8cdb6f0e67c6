"""GPU tests of scored attention at the edges of its contract."""
import math

import numpy as np
import pytest

from gpu_helpers import require_gpu
from paged_helpers import random_case, widen
from paged_kv_cache_127_gb300 import synth
from scored_helpers import assert_rows_close
from test_gpu_scored import call_chunk, call_decode, chunk_case, ref_chunk, ref_decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gpu():
    return require_gpu()


# Logits of std `scale * 8`, up to five times that: with these (scale, cap) a warp takes each form of the cap.
# Caps of more than 55 have a running maximum for bf16 too.
CAPS = [(0.1, 0.0), (0.1, 30.0), (0.1, 6.0), (0.1, 1.0), (1.0, 60.0), (1.0, 20.0), (-0.1, 5.0)]


def assert_nan_where(got, ref, nan, dtype, E, vmax):
    """NaN in the (row, head) pairs of `nan`, every element of them, and nowhere else."""
    assert np.isnan(got[nan]).all(), f"{int((~np.isnan(got[nan])).sum())} finite results of a NaN score"
    assert_rows_close(got[~nan], ref[~nan], dtype, dtype, E, vmax)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("scale,cap", CAPS)
def test_decode_scored_nan_score_under_a_cap(gpu, dtype, scale, cap):
    torch, pa = gpu
    rng = synth.make_rng(8000)
    Hq, Hkv, B = 8, 2, 16
    q, K, V, kc, vc, tables, lens = random_case(rng, dtype, 4, Hq, Hkv, 64, B, [90, 40, 700, 33])
    case = (q, kc, vc, tables, lens)
    for opts in (dict(cap=cap), dict(cap=cap, slopes=np.full(Hq, 0.01)), dict(cap=cap, window=50)):
        ref, w, E, vmax = ref_decode(case, dtype, scale, opts)
        q1, k1 = q.copy(), kc.copy()
        q1[1, 3, 5] = synth.nan_value(dtype)                     # one query head: KV head 0
        k1[tables[2][690 // B], 1, 690 % B, 7] = synth.nan_value(dtype)   # one visible key of KV head 1
        nan = np.zeros((4, Hq), bool)
        nan[1, 3] = nan[2, 4:] = True
        sums = torch.zeros(4, Hkv, tables.shape[1] * B, device="cuda")
        got = call_decode(torch, pa, (q1, k1, vc, tables, lens), dtype, dtype, scale, opts, sums=sums)
        assert_nan_where(got, ref, nan, dtype, E, vmax)
        have = sums.cpu().numpy().astype(np.float64)
        for s in range(4):
            for h in range(Hkv):
                seen = w[s][h] > 0
                if (s, h) in ((1, 0), (2, 1)):
                    assert np.isnan(have[s, h, :int(lens[s])][seen]).all()
                else:
                    np.testing.assert_allclose(have[s, h, :int(lens[s])], w[s][h], rtol=3 * E + 2.0 ** -20, atol=1e-30)
                assert (have[s, h, :int(lens[s])][~seen] == 0).all() and (have[s, h, int(lens[s]):] == 0).all()
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("nq", [5, 80, 130])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("scale,cap", CAPS)
def test_chunk_scored_nan_score_under_a_cap(gpu, dtype, scale, cap, nq):
    torch, pa = gpu
    rng = synth.make_rng(8010 + nq)
    Hq, Hkv, B = 8, 2, 16
    lens = [nq + 200, nq, nq + 61]
    case, qs = chunk_case(rng, dtype, Hq, Hkv, 64, B, lens, [nq] * 3)
    q, kc, vc, tables, lens = case
    for opts in (dict(cap=cap), dict(cap=cap, slopes=np.full(Hq, 0.01))):
        ref, E, vmax = ref_chunk(case, qs, dtype, scale, opts)
        q1, k1 = q.copy(), kc.copy()
        q1[int(qs[1]) + 3, 2] = synth.nan_value(dtype)           # a whole query row, and one element of another
        q1[int(qs[0]) + 1, 6, 0] = synth.nan_value(dtype)
        k1[tables[2][1], 1, 4, 9] = synth.nan_value(dtype)       # position 20: every row of the chunk sees it
        nan = np.zeros((len(q), Hq), bool)
        nan[int(qs[1]) + 3, 2] = nan[int(qs[0]) + 1, 6] = True
        nan[int(qs[2]):, 4:] = True
        got = call_chunk(torch, pa, (q1, k1, vc, tables, lens), qs, dtype, dtype, scale, opts)
        assert_nan_where(got, ref, nan, dtype, E, vmax)
    assert pa.pa_device_errors(clear=True) == 0


def hide_unseen(case, qs, opts, dtype):
    """NaN in the keys and values of every position that is in no row's range, holes between ranges too."""
    q, kc, vc, tables, lens = case
    B = kc.shape[2]
    holes = 0
    for s, n in enumerate(lens):
        n, rows = int(n), range(int(qs[s]), int(qs[s + 1]))
        seen = np.zeros(n, bool)
        for i in rows:
            seen[max(0, opts["key_begin"][i]):max(0, min(n, opts["key_end"][i]))] = True
        at = np.nonzero(seen)[0]
        holes += int((~seen[at.min():at.max()]).sum()) if len(at) else 0
        for j in np.nonzero(~seen)[0]:
            for c in (kc, vc):
                c[tables[s][j // B], :, j % B] = synth.nan_value(dtype)
    return holes


def ranges_with_holes(rng, kind, lens, nq):
    begin, end = [], []
    for n, m in zip(lens, nq):
        cuts = np.sort(rng.integers(0, n + 1, 6))
        for t in range(m):
            if kind == "two":            # one of two places, by row
                b, e = ((0, 10), (n - 17, n))[t * 7 // 3 % 2]
            elif kind == "last":         # every row but one at the front
                b, e = (n - 5, n - 2) if t == m - 1 else (3, 21)
            elif kind == "empty":        # rows that see nothing between rows that do
                b, e = ((1, 9), (5, 5), (n, 3), (n - 9, n), (7, 7))[t % 5]
            else:                        # pieces of the context at random, some empty
                k = int(rng.integers(0, 5))
                b, e = int(cuts[k]), int(cuts[k]) + int(rng.integers(0, max(1, (cuts[k + 1] - cuts[k]) * 2 // 3) + 1))
            begin.append(b)
            end.append(e)
    return dict(key_begin=begin, key_end=end)


@pytest.mark.parametrize("path", ["short", "long", "tiles"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind", ["two", "last", "empty", "random"])
@pytest.mark.parametrize("D,B,G", [(64, 16, 1), (128, 32, 8), (128, 16, 4)])
def test_chunk_scored_holes_between_ranges(gpu, D, B, G, kind, dtype, path):
    torch, pa = gpu
    rng = synth.make_rng(8100 + D + B + G + len(kind) + len(path))
    Hkv = {1: 4, 4: 8, 8: 1}[G]
    nq = {"short": [1, 5, 8, 7], "long": [33, 70, 9, 64], "tiles": [300, 129, 5, 257]}[path]
    lens = [n + int(x) for n, x in zip(nq, (150, 333, 40, 90))]
    for more in (dict(), dict(cap=4.0), dict(slopes=np.full(G * Hkv, 0.05))):
        case, qs = chunk_case(rng, dtype, G * Hkv, Hkv, D, B, lens, nq)
        opts = dict(ranges_with_holes(rng, kind, lens, nq), **more)
        clean = (case[0], case[1].copy(), case[2].copy(), case[3], case[4])
        assert hide_unseen(case, qs, opts, dtype) > 0
        ref, E, vmax = ref_chunk(clean, qs, dtype, 0.2, opts)
        got = call_chunk(torch, pa, case, qs, dtype, dtype, 0.2, opts, psize=[0, 4 * B][len(more)])
        assert_rows_close(got, ref, dtype, dtype, E, vmax)
    assert pa.pa_device_errors(clear=True) == 0


def test_chunk_scored_holes_in_a_plan_of_many_blocks(gpu):
    # more row blocks than the plan keeps in shared memory: its other way over the masks
    torch, pa = gpu
    rng = synth.make_rng(8190)
    Hq, Hkv, D, B, S = 8, 1, 64, 16, 420
    nq = [int(x) for x in rng.integers(1, 34, S)]
    lens = [n + int(x) for n, x in zip(nq, rng.integers(20, 120, S))]
    case, qs = chunk_case(rng, "bf16", Hq, Hkv, D, B, lens, nq)
    opts = ranges_with_holes(rng, "random", lens, nq)
    clean = (case[0], case[1].copy(), case[2].copy(), case[3], case[4])
    assert hide_unseen(case, qs, opts, "bf16") > 0
    ref, E, vmax = ref_chunk(clean, qs, "bf16", 0.2, opts)
    for max_q in (34, 170):           # two blocks of a sequence at most, and six: 840 and 2520 in all
        assert_rows_close(call_chunk(torch, pa, case, qs, "bf16", "f32", 0.2, opts, max_q=max_q), ref, "bf16", "f32", E, vmax)
    assert pa.pa_device_errors(clear=True) == 0


# Two f16 parts keep a weight to 2^-22 relative, and to 2^-25 absolute in units in which the largest is 2^lift: lift 15,
# or 7 in the long chunks, whose maximum may lag by 8.  Against weights of 2^-26 of the largest that is 2^(1 - lift).
def tail_error(z, lift):
    return 2.0 ** -22 * z + 2.0 ** -22 + 2.0 ** -21 + 2.0 ** (1 - lift) + 64 * 2.0 ** -24


@pytest.mark.parametrize("dominant_last", [False, True])
@pytest.mark.parametrize("opts", [dict(), dict(cap=300.0), dict(slopes=[0.0] * 4)])
@pytest.mark.parametrize("nq", [0, 3, 70])
def test_scored_f16_tail_of_small_weights(gpu, nq, opts, dominant_last):
    """One key of weight near 1 and value 0, thousands at about 2^-26 and value 1: their mass is the result."""
    torch, pa = gpu
    Hq, Hkv, D, B, n = 4, 1, 64, 32, 8192
    n_rows = max(nq, 1)
    f16 = np.float16
    q = np.zeros((n_rows, Hq, D), f16)
    q[..., 0] = 4.5
    N = n // B
    kc, vc = np.zeros((N, Hkv, B, D), f16), np.ones((N, Hkv, B, D), f16)
    at = n - n_rows if dominant_last else 3          # seen by every row
    kc[at // B, 0, at % B, 0] = 4.0
    vc[at // B, 0, at % B] = 0.0
    tables, lens = np.arange(N, dtype=np.int32)[None], np.array([n], np.int32)
    case = (q, kc, vc, tables, lens)
    scale, cap = 1.0, opts.get("cap", 0.0)
    z = 18.0 if not cap else cap * math.tanh(18.0 / cap)
    keys = np.array([n - n_rows + t + 1 for t in range(n_rows)], np.float64)   # that row t sees
    small = (keys - 1) * math.exp(-z)
    ref = small / (1.0 + small)
    if nq == 0:
        got = call_decode(torch, pa, case, "f16", "f32", scale, opts, psize=n)
    else:
        got = call_chunk(torch, pa, case, np.array([0, nq], np.int32), "f16", "f32", scale, opts, psize=n)
    E = tail_error(z, 7 if nq * Hq >= 64 else 15) + (cap * 2.0 ** -21 if cap else 0.0)
    assert (np.abs(got - ref[:, None, None]) <= 2.5 * E * ref[:, None, None]).all(), \
        f"worst {np.abs(got / ref[:, None, None] - 1).max():.3e} of {2.5 * E:.3e}"
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("cap,sign", [(55.0, 1.0), (55.0, -1.0), (50.0, 1.0), (30.0, 1.0), (60.0, 1.0)])
@pytest.mark.parametrize("nq", [0, 5, 80])
def test_scored_values_up_to_the_stated_bound(gpu, nq, cap, sign):
    """Values of magnitudes up to 2^57 (and in decode, short chunks and with wider caps up to 2^100) with every logit near the
    cap, where weights relative to a constant are largest, or near minus the cap, where they are smallest."""
    torch, pa = gpu
    rng = synth.make_rng(8300 + nq)
    Hq, Hkv, D, B, n = 8, 2, 128, 16, 3000
    top = 57 if nq * (Hq // Hkv) >= 64 and cap <= 55.0 else 100
    N = -(-n // B)
    rows = max(nq, 1)
    q = synth.to_storage(np.abs(rng.normal(size=(rows, Hq, D))).astype(np.float32), "bf16")
    kc = synth.to_storage((sign * np.abs(rng.normal(size=(N, Hkv, B, D)))).astype(np.float32), "bf16")
    vc = synth.to_storage((rng.uniform(0.5, 1.0, (N, Hkv, B, D)) * rng.choice([-1.0, 1.0], (N, Hkv, B, D))).astype(np.float32)
                          * np.float32(2.0 ** (top - 1)), "bf16")
    assert np.abs(widen(vc, "bf16")).max() < 2.0 ** top
    case = (q, kc, vc, np.arange(N, dtype=np.int32)[None], np.array([n], np.int32))
    opts = dict(cap=cap)
    if nq == 0:
        ref, _, E, vmax = ref_decode(case, "bf16", 2.0, opts)
        got = call_decode(torch, pa, case, "bf16", "f32", 2.0, opts)
    else:
        qs = np.array([0, nq], np.int32)
        ref, E, vmax = ref_chunk(case, qs, "bf16", 2.0, opts)
        got = call_chunk(torch, pa, case, qs, "bf16", "f32", 2.0, opts)
    assert_rows_close(got, ref, "bf16", "f32", E, vmax)
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_short_chunks_of_warps_with_few_rows_or_none(gpu, dtype):
    """Eight heads' warps over two row tiles of which the second has no token, or only ones that see nothing, beside rows that see
    every key: what the others do not see may be NaN, and their results are their own."""
    torch, pa = gpu
    rng = synth.make_rng(8400)
    Hq, Hkv, D, B = 16, 4, 128, 16
    nq = [8, 3, 4, 5, 8, 1]
    lens = [500, 330, 290, 1000, 260, 70]
    case, qs = chunk_case(rng, dtype, Hq, Hkv, D, B, lens, nq)
    begin, end = [], []
    for s, (n, m) in enumerate(zip(lens, nq)):
        for t in range(m):
            empty = (s == 0 and t >= 4) or (s == 4 and t < 5) or (s == 3 and t == 2)
            begin.append(n if empty else 96 if s == 4 else 0)
            end.append(0 if empty else n - m + t + 1)
    opts = dict(key_begin=begin, key_end=end, cap=5.0)
    clean = (case[0], case[1].copy(), case[2].copy(), case[3], case[4])
    hide_unseen(case, qs, opts, dtype)
    q = case[0].copy()
    for s, n in enumerate(lens):            # a row that sees nothing may hold anything
        for t in range(nq[s]):
            if begin[int(qs[s]) + t] >= end[int(qs[s]) + t]:
                q[int(qs[s]) + t] = synth.nan_value(dtype)
    ref, E, vmax = ref_chunk(clean, qs, dtype, 0.2, opts)
    for max_q in (8, 15):
        got = call_chunk(torch, pa, (q,) + case[1:], qs, dtype, "f32", 0.2, opts, max_q=max_q)
        assert_rows_close(got, ref, dtype, "f32", E, vmax)
        assert (got[np.array(begin) >= np.array(end)] == 0).all()
    assert pa.pa_device_errors(clear=True) == 0
