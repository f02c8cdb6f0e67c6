"""GPU tests of pa_decode_scored and pa_chunk_scored against plain fp64
references; the tolerances are derived in scored_helpers."""
import itertools
import math

import numpy as np
import pytest

from gpu_helpers import require_gpu, to_dev, to_host, torch_dtype
from paged_helpers import random_case, widen
from paged_kv_cache_127_gb300 import synth
from scored_helpers import assert_rows_close, gather, ranges, scored_rows, values, weight_error

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gpu():
    return require_gpu()


def i32(torch, a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def out_host(out):
    return out.float().cpu().numpy().astype(np.float64)


def make(pa, torch, opts):
    slopes = opts.get("slopes")
    return pa.make_score(softcap=opts.get("cap", 0.0), window=opts.get("window", 0),
                         slopes=None if slopes is None else torch.tensor(slopes, dtype=torch.float32).cuda(),
                         key_begin=i32(torch, opts.get("key_begin")), key_end=i32(torch, opts.get("key_end")))


def call_decode(torch, pa, case, dtype, out_dtype, scale, opts, psize=0, sums=None, rows=None, fill=7.0, score="make"):
    q, kc, vc, tables, lens = case
    S, Hq, D = q.shape
    N, Hkv, B, _ = kc.shape
    dims = pa.make_dims(S, Hq, Hkv, D, B, N, tables.shape[1], psize, dtype)
    out = torch.full((S, Hq, D), fill, dtype=torch_dtype(torch, out_dtype), device="cuda")
    need = pa.pa_decode_scored_workspace_bytes(dims, sums is not None)
    ws = torch.full((max(need, 256),), 0xff, dtype=torch.uint8, device="cuda")
    pa.pa_decode_scored(dims, make(pa, torch, opts) if score == "make" else score, to_dev(torch, q, dtype),
                        to_dev(torch, kc, dtype), to_dev(torch, vc, dtype), i32(torch, tables), i32(torch, lens), scale,
                        out, ws, key_sums=sums, sum_rows=i32(torch, rows))
    torch.cuda.synchronize()
    return out_host(out)


def ref_decode(case, dtype, scale, opts):
    """(out, per-sequence weights summed over each KV head's query heads, E, max |v|)"""
    q, kc, vc, tables, lens = case
    S, Hq, D = q.shape
    B, Hkv = kc.shape[2], kc.shape[1]
    q64 = widen(q, dtype)
    out, sums, worst, vmax = np.zeros((S, Hq, D)), [], 0.0, 0.0
    for s in range(S):
        n = int(lens[s])
        b, e = ranges([n - 1], n, [s], opts.get("window", 0), opts.get("key_begin"), opts.get("key_end"))
        K, V = gather(kc, tables[s], n, B, dtype), gather(vc, tables[s], n, B, dtype)
        o, w, d = scored_rows(q64[s:s + 1], K, V, [n - 1], b, e, scale, opts.get("cap", 0.0), opts.get("slopes"))
        out[s] = o[0]
        sums.append(w[0].reshape(Hkv, Hq // Hkv, n).sum(1))
        worst = max(worst, d)
        if b[0] < e[0]:
            vmax = max(vmax, np.abs(V[b[0]:e[0]]).max())
    return out, sums, weight_error(dtype, worst, int(max(lens, default=0))), vmax


def hide(case, opts, dtype, tables, lens, rows_of=None):
    """NaN in the keys and values of every position that no row of a sequence sees."""
    q, kc, vc, tables, lens = case
    B = kc.shape[2]
    nan = synth.nan_value(dtype)
    for s, n in enumerate(lens):
        n = int(n)
        rows = [s] if rows_of is None else rows_of[s]
        pos = [n - 1] if rows_of is None else list(range(n - len(rows), n))
        if not len(rows):
            continue
        b, e = ranges(pos, n, rows, opts.get("window", 0), opts.get("key_begin"), opts.get("key_end"))
        seen = np.zeros(n, bool)
        live = b < e
        if live.any():
            seen[int(b[live].min()):int(e[live].max())] = True
        for j in np.nonzero(~seen)[0]:
            kc[tables[s][j // B], :, j % B] = nan
            vc[tables[s][j // B], :, j % B] = nan


def decode_options(rng, S, Hq, lens):
    lens = np.asarray(lens, np.int64)
    slopes = 2.0 ** (-8.0 * (np.arange(Hq) + 1) / Hq)
    begin = np.array([int(rng.integers(-3, n + 2)) for n in lens])
    end = np.array([int(rng.integers(-2, n + 5)) for n in lens])
    return [dict(), dict(cap=5.0), dict(window=37), dict(slopes=slopes), dict(key_begin=begin),
            dict(key_begin=begin, key_end=end, cap=20.0), dict(window=100, slopes=slopes, cap=3.0, key_begin=begin)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,B,G", [(64, 16, 1), (64, 32, 8), (128, 16, 4), (128, 32, 2)])
def test_decode_scored_options(gpu, dtype, D, B, G):
    torch, pa = gpu
    rng = synth.make_rng(7000 + D + B + G + len(dtype))
    Hkv = {1: 4, 2: 6, 4: 8, 8: 1}[G]
    lens = [0, 1, 2, 15, 16, 17, B + 3, 200, 531, 64]
    q, K, V, kc, vc, tables, lens = random_case(rng, dtype, len(lens), G * Hkv, Hkv, D, B, lens)
    scale = 3.0 / math.sqrt(D)
    for k, opts in enumerate(decode_options(rng, len(lens), G * Hkv, lens)):
        case = (q, kc.copy(), vc.copy(), tables, lens)
        hide(case, opts, dtype, tables, lens)
        ref, _, E, vmax = ref_decode(case, dtype, scale, opts)
        for out_dtype, psize in itertools.product({"f32", dtype}, [0, B, 4 * B][k % 2:]):
            got = call_decode(torch, pa, case, dtype, out_dtype, scale, opts, psize)
            assert_rows_close(got, ref, dtype, out_dtype, E, vmax)
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,D,B", [(8, 2, 64, 16), (8, 8, 128, 32), (8, 1, 128, 16), (12, 6, 64, 32)])
def test_decode_scored_key_sums(gpu, dtype, Hq, Hkv, D, B):
    torch, pa = gpu
    rng = synth.make_rng(7100 + Hq + Hkv + D + B)
    lens = [0, 1, 70, 333, 17, 600]
    q, K, V, kc, vc, tables, lens = random_case(rng, dtype, len(lens), Hq, Hkv, D, B, lens)
    S, cap = len(lens), tables.shape[1] * B
    cols = cap + 8
    rows = np.array([3, 0, 8, 5, 1, 2])
    slopes = 2.0 ** (-8.0 * (np.arange(Hq) + 1) / Hq)
    for opts in (dict(), dict(cap=6.0, slopes=slopes), dict(window=50), dict(key_begin=np.array([0, 1, 3, 50, 17, 299]))):
        for psize in (0, B):
            start = rng.random((9, Hkv, cols)).astype(np.float32)
            sums = torch.from_numpy(start).cuda()
            case = (q, kc.copy(), vc.copy(), tables, lens)
            hide(case, opts, dtype, tables, lens)
            ref, w, E, vmax = ref_decode(case, dtype, 1 / math.sqrt(D), opts)
            got = call_decode(torch, pa, case, dtype, "f32", 1 / math.sqrt(D), opts, psize, sums, rows)
            assert_rows_close(got, ref, dtype, "f32", E, vmax)
            want = start.astype(np.float64)
            tol = np.zeros_like(want)
            for s in range(S):
                want[rows[s], :, :int(lens[s])] += w[s]
                tol[rows[s], :, :int(lens[s])] = 2.5 * E * w[s]
            have = sums.cpu().numpy().astype(np.float64)
            # one rounding of the addition, and of the sum over the group's heads
            assert (np.abs(have - want) <= tol + 2.0 ** -21 * np.abs(want) * (tol > 0)).all()
    # with no rows, sequence s uses row s; the same call twice adds twice
    sums = torch.zeros(S, Hkv, cap, device="cuda")
    case = (q, kc, vc, tables, lens)
    for _ in range(2):
        call_decode(torch, pa, case, dtype, "f32", 1 / math.sqrt(D), {}, 0, sums)
    _, w, E, _ = ref_decode(case, dtype, 1 / math.sqrt(D), {})
    for s in range(S):
        np.testing.assert_allclose(sums[s].cpu().numpy()[:, :int(lens[s])], 2 * w[s], rtol=3 * E + 2.0 ** -20, atol=1e-30)
        assert (sums[s, :, int(lens[s]):] == 0).all()
    assert pa.pa_device_errors(clear=True) == 0


def call_chunk(torch, pa, case, qs, dtype, out_dtype, scale, opts, max_q=None, psize=0, fill=7.0):
    q, kc, vc, tables, lens = case
    T, Hq, D = q.shape
    N, Hkv, B, _ = kc.shape
    max_q = int(max(1, np.diff(qs).max(initial=1))) if max_q is None else max_q
    dims = pa.make_dims(len(lens), Hq, Hkv, D, B, N, tables.shape[1], psize, dtype)
    out = torch.full((T, Hq, D), fill, dtype=torch_dtype(torch, out_dtype), device="cuda")
    ws = torch.full((max(pa.pa_chunk_scored_workspace_bytes(dims, T, max_q), 256),), 0xff, dtype=torch.uint8, device="cuda")
    pa.pa_chunk_scored(dims, make(pa, torch, opts), to_dev(torch, q, dtype), to_dev(torch, kc, dtype), to_dev(torch, vc, dtype),
                       i32(torch, tables), i32(torch, lens), i32(torch, qs), scale, out, max_q, ws)
    torch.cuda.synchronize()
    return out_host(out)


def ref_chunk(case, qs, dtype, scale, opts):
    q, kc, vc, tables, lens = case
    q64 = widen(q, dtype)
    out, worst, vmax = np.zeros(q.shape), 0.0, 0.0
    B = kc.shape[2]
    for s, n in enumerate(lens):
        n, rows = int(n), np.arange(qs[s], qs[s + 1])
        if not len(rows):
            continue
        pos = np.arange(n - len(rows), n)
        b, e = ranges(pos, n, rows, opts.get("window", 0), opts.get("key_begin"), opts.get("key_end"))
        K, V = gather(kc, tables[s], n, B, dtype), gather(vc, tables[s], n, B, dtype)
        out[rows], _, d = scored_rows(q64[rows], K, V, pos, b, e, scale, opts.get("cap", 0.0), opts.get("slopes"))
        worst = max(worst, d)
        live = b < e
        if live.any():
            vmax = max(vmax, np.abs(V[int(b[live].min()):int(e[live].max())]).max())
    return out, weight_error(dtype, worst, int(max(lens, default=0))), vmax


def chunk_case(rng, dtype, Hq, Hkv, D, B, lens, nq):
    _, K, V, kc, vc, tables, lens = random_case(rng, dtype, len(lens), Hq, Hkv, D, B, lens)
    qs = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
    return (values(rng, (int(qs[-1]), Hq, D), 1.0, dtype), kc, vc, tables, lens), qs


def chunk_options(rng, lens, nq, Hq):
    """Masks as packed documents, a prefix, a window, ranges at random (some empty) and combinations."""
    slopes = 2.0 ** (-8.0 * (np.arange(Hq) + 1) / Hq)
    docs, prefix, lo, hi = [], [], [], []
    for n, m in zip(lens, nq):
        for pos in range(n - m, n):
            docs.append(pos - pos % 45)
            prefix.append(max(pos + 1, min(n, n - m // 2)))
            lo.append(int(rng.integers(-2, pos + 3)))
            hi.append(int(rng.integers(-2, n + 4)))
    return [dict(), dict(cap=4.0), dict(window=30), dict(slopes=slopes), dict(key_begin=docs, cap=30.0),
            dict(key_end=prefix, slopes=slopes), dict(key_begin=lo, key_end=hi),
            dict(window=1, cap=2.0), dict(key_begin=docs, key_end=prefix, window=64, slopes=slopes, cap=10.0)]


@pytest.mark.parametrize("path", ["short", "long"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,B,G", [(64, 16, 1), (64, 32, 8), (128, 16, 4), (128, 32, 2)])
def test_chunk_scored_options(gpu, dtype, D, B, G, path):
    torch, pa = gpu
    rng = synth.make_rng(7200 + D + B + G + len(path))
    Hkv = {1: 4, 2: 6, 4: 2, 8: 1}[G]
    nq = [1, B + 3, 33, 70, 0, 7] if path == "long" else [1, 5, 3, 6, 0, 7]
    lens = [1, B + 3, 200, 430, 40, 7]
    case0, qs = chunk_case(rng, dtype, G * Hkv, Hkv, D, B, lens, nq)
    scale = 2.0 / math.sqrt(D)
    rows_of = [np.arange(qs[s], qs[s + 1]) for s in range(len(lens))]
    for k, opts in enumerate(chunk_options(rng, lens, nq, G * Hkv)):
        case = (case0[0], case0[1].copy(), case0[2].copy(), case0[3], case0[4])
        hide(case, opts, dtype, case[3], case[4], rows_of)
        ref, E, vmax = ref_chunk(case, qs, dtype, scale, opts)
        for out_dtype in {"f32", dtype}:
            got = call_chunk(torch, pa, case, qs, dtype, out_dtype, scale, opts, psize=[0, B, 4 * B][k % 3])
            assert_rows_close(got, ref, dtype, out_dtype, E, vmax)
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("nq,max_q", [(1, 1), (5, 5), (8, 16), (33, 33), (64, 64), (20, 64), (130, 130)])
def test_chunk_scored_row_blocks(gpu, nq, max_q):
    # one tile, two tiles, partly filled and missing second tiles, several items of a sequence
    torch, pa = gpu
    rng = synth.make_rng(7300 + nq)
    lens = [nq, nq + 1, 600, 1100, 64 + nq]
    case, qs = chunk_case(rng, "bf16", 8, 2, 128, 16, lens, [nq] * 5)
    docs = [pos - pos % 200 for n in lens for pos in range(n - nq, n)]
    for opts in (dict(cap=3.0, key_begin=docs), dict(window=90)):
        ref, E, vmax = ref_chunk(case, qs, "bf16", 0.1, opts)
        for out_dtype in ("bf16", "f32"):
            assert_rows_close(call_chunk(torch, pa, case, qs, "bf16", out_dtype, 0.1, opts, max_q=max_q), ref, "bf16",
                              out_dtype, E, vmax)
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_chunk_scored_many_items_of_mixed_tiles(gpu, dtype):
    # more work items than SMs, with full, partial and missing tiles and ranges that begin mid-step
    torch, pa = gpu
    rng = synth.make_rng(7350 + len(dtype))
    nq = [96, 64, 33, 80, 0, 70] * 10
    lens = [n + int(x) for n, x in zip(nq, rng.integers(1, 200, len(nq)))]
    case, qs = chunk_case(rng, dtype, 16, 4, 128, 16, lens, nq)
    lo = [int(rng.integers(0, pos + 1)) for n, m in zip(lens, nq) for pos in range(n - m, n)]
    opts = dict(cap=8.0, key_begin=lo)
    ref, E, vmax = ref_chunk(case, qs, dtype, 0.1, opts)
    assert_rows_close(call_chunk(torch, pa, case, qs, dtype, dtype, 0.1, opts), ref, dtype, dtype, E, vmax)
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("nq", [3, 80])
def test_chunk_scored_leaves_other_rows(gpu, nq):
    # rows outside every range, and those of a skipped sequence, stay as they were
    torch, pa = gpu
    rng = synth.make_rng(7400 + nq)
    (q, kc, vc, tables, lens), qs = chunk_case(rng, "bf16", 8, 2, 64, 16, [nq + 9, nq + 40, nq + 5], [nq] * 3)
    q = np.concatenate([q[:2], q, q[:5]])        # two rows before the first range, five behind the last
    case = (q, kc, vc, tables, lens)
    shifted = qs + 2
    ref, E, vmax = ref_chunk(case, shifted, "bf16", 0.1, dict(cap=4.0))
    got = call_chunk(torch, pa, case, shifted, "bf16", "bf16", 0.1, dict(cap=4.0))
    assert_rows_close(got[2:-5], ref[2:-5], "bf16", "bf16", E, vmax)
    assert (got[:2] == 7.0).all() and (got[-5:] == 7.0).all()
    assert pa.pa_device_errors(clear=True) == 0
    bad = lens.copy()
    bad[1] = nq - 1                              # fewer stored tokens than queries
    got = call_chunk(torch, pa, (q, kc, vc, tables, bad), shifted, "bf16", "bf16", 0.1, dict(cap=4.0))
    assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_BAD_LEN
    assert (got[2 + nq:2 + 2 * nq] == 7.0).all()
    assert_rows_close(got[2:2 + nq], ref[2:2 + nq], "bf16", "bf16", E, vmax)
    got = call_chunk(torch, pa, case, np.array([2, 2 + nq, nq, 2 + 3 * nq], np.int32), "bf16", "bf16", 0.1, {}, max_q=2 * nq + 2)
    assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_BAD_LEN
    assert (got == 7.0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decode_scored_bad_inputs_are_flagged(gpu, dtype):
    torch, pa = gpu
    rng = synth.make_rng(7500)
    q, K, V, kc, vc, tables, lens = random_case(rng, dtype, 3, 8, 2, 64, 16, [40, 300, 25])
    case = (q, kc, vc, tables, lens)
    ref, w, E, vmax = ref_decode(case, dtype, 0.125, {})
    # a sum row outside the array: that sequence's sums are dropped, outputs are not
    sums = torch.zeros(3, 2, tables.shape[1] * 16, device="cuda")
    got = call_decode(torch, pa, case, dtype, "f32", 0.125, {}, 0, sums, np.array([1, 3, 0]))
    assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_BAD_ROW
    assert_rows_close(got, ref, dtype, "f32", E, vmax)
    assert (sums[2] == 0).all()
    np.testing.assert_allclose(sums[1].cpu().numpy()[:, :40], w[0], rtol=3 * E + 2.0 ** -20)
    got = call_decode(torch, pa, case, dtype, "f32", 0.125, {}, 0, sums, np.array([1, -1, 0]))
    assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_BAD_ROW
    # a block outside the pool: its keys are skipped, and get no weight
    bad = tables.copy()
    bad[1, 5] = kc.shape[0] + 1
    sums.zero_()
    got = call_decode(torch, pa, (q, kc, vc, bad, lens), dtype, "f32", 0.125, {}, 0, sums)
    assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_BAD_BLOCK
    keep = np.r_[0:80, 96:300]
    K1, V1 = gather(kc, tables[1], 300, 16, dtype)[keep], gather(vc, tables[1], 300, 16, dtype)[keep]
    o, w1, _ = scored_rows(widen(q, dtype)[1:2], K1, V1, [283], [0], [284], 0.125)
    assert_rows_close(got[1], o[0], dtype, "f32", E, vmax)
    assert_rows_close(got[0], ref[0], dtype, "f32", E, vmax)
    have = sums[1].cpu().numpy()
    assert (have[:, 80:96] == 0).all()
    np.testing.assert_allclose(have[:, keep], w1[0].reshape(2, 4, 284).sum(1), rtol=3 * E + 2.0 ** -20)
    # lengths outside the table: clamped and flagged
    long = lens.copy()
    long[0], long[2] = -4, tables.shape[1] * 16 + 1
    full = tables.copy()
    full[full < 0] = 0
    got = call_decode(torch, pa, (q, np.nan_to_num(kc) if dtype == "f32" else kc, vc, full, long), dtype, "f32", 0.125, {})
    assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_BAD_LEN
    assert (got[0] == 0).all()
    assert_rows_close(got[1], ref[1], dtype, "f32", E, vmax)


def test_plain_score_is_pa_decode_and_pa_chunk(gpu):
    torch, pa = gpu
    rng = synth.make_rng(7600)
    from gpu_helpers import run_decode
    q, K, V, kc, vc, tables, lens = random_case(rng, "bf16", 4, 8, 2, 128, 16, [1, 90, 700, 33])
    case = (q, kc, vc, tables, lens)
    _, _, E, vmax = ref_decode(case, "bf16", 0.09, {})
    plain = run_decode(torch, pa, "bf16", q, kc, vc, tables, lens, 0.09)
    for score in (None, pa.make_score(), pa.make_score(window=2 ** 31 - 1)):
        got = call_decode(torch, pa, case, "bf16", "f32", 0.09, {}, score=score)
        assert_rows_close(got, plain, "bf16", "f32", 2 * E, vmax)


def test_decode_scored_scale_signs_and_equal_logits(gpu):
    # a scale of zero makes every key equal; a negative one turns the order round
    torch, pa = gpu
    rng = synth.make_rng(7650)
    q, K, V, kc, vc, tables, lens = random_case(rng, "f16", 3, 4, 2, 64, 16, [5, 100, 260])
    case = (q, kc, vc, tables, lens)
    for scale in (0.0, -0.2):
        for opts in ({}, dict(cap=2.0), dict(slopes=np.full(4, 0.1))):
            ref, _, E, vmax = ref_decode(case, "f16", scale, opts)
            assert_rows_close(call_decode(torch, pa, case, "f16", "f32", scale, opts), ref, "f16", "f32", E, vmax)
    nq = [4, 70]
    case, qs = chunk_case(rng, "f16", 4, 2, 64, 16, [80, 200], nq)
    for scale in (0.0, -0.2):
        for opts in ({}, dict(cap=2.0)):
            ref, E, vmax = ref_chunk(case, qs, "f16", scale, opts)
            assert_rows_close(call_chunk(torch, pa, case, qs, "f16", "f32", scale, opts), ref, "f16", "f32", E, vmax)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_scored_large_logits_and_caps(gpu, dtype):
    # logits far past the cap, on both sides, and without one over a dominant key
    torch, pa = gpu
    rng = synth.make_rng(7700)
    q, K, V, kc, vc, tables, lens = random_case(rng, dtype, 3, 8, 2, 128, 16, [300, 900, 17], std=3.0)
    case = (q, kc, vc, tables, lens)
    for opts in ({}, dict(cap=1.0), dict(cap=50.0), dict(cap=1e4), dict(cap=1e-3)):
        ref, _, E, vmax = ref_decode(case, dtype, 0.5, opts)
        assert_rows_close(call_decode(torch, pa, case, dtype, "f32", 0.5, opts), ref, dtype, "f32", E, vmax)
    for nq in ([5, 7, 3], [80, 70, 17]):
        case, qs = chunk_case(rng, dtype, 8, 2, 128, 16, [300, 500, 17], nq)
        for opts in ({}, dict(cap=1.0), dict(cap=20.0)):
            ref, E, vmax = ref_chunk(case, qs, dtype, 3.0, opts)
            assert_rows_close(call_chunk(torch, pa, case, qs, dtype, "f32", 3.0, opts), ref, dtype, "f32", E, vmax)


def test_scored_graph_replay_and_other_stream(gpu):
    # captured once, replayed on fresh inputs: the bits of an eager call, with a workspace of its own
    torch, pa = gpu
    rng = synth.make_rng(7800)
    S, Hq, Hkv, D, B = 5, 8, 2, 128, 16
    lens = [1, 400, 77, 900, 16]
    q, K, V, kc, vc, tables, lens = random_case(rng, "bf16", S, Hq, Hkv, D, B, lens)
    dims = pa.make_dims(S, Hq, Hkv, D, B, kc.shape[0], tables.shape[1], 64, "bf16")
    dq, dk, dv = (to_dev(torch, x, "bf16") for x in (q, kc, vc))
    dt, dl = i32(torch, tables), i32(torch, lens)
    score = pa.make_score(softcap=5.0, window=300)
    cols = tables.shape[1] * B
    outs = [torch.zeros(S, Hq, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    sums = [torch.zeros(S, Hkv, cols, device="cuda") for _ in range(2)]
    wss = [torch.empty(pa.pa_decode_scored_workspace_bytes(dims, True), dtype=torch.uint8, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pa.pa_decode_scored(dims, score, dq, dk, dv, dt, dl, 0.09, outs[0], wss[0], key_sums=sums[0], stream=side)
    for step in range(3):
        dq.copy_(to_dev(torch, values(rng, (S, Hq, D), 1.0, "bf16"), "bf16"))
        torch.cuda.synchronize()
        graph.replay()
        other = torch.cuda.Stream()
        call = pa.pa_decode_scored(dims, score, dq, dk, dv, dt, dl, 0.09, outs[1], wss[1], key_sums=sums[1], stream=other,
                                   prepare=True)
        call()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1])
        assert torch.equal(sums[0], sums[1])
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("S,hi,window", [(100, 4000, 0), (100, 12000, 0), (150, 9000, 3000), (1500, 60, 0)])
def test_decode_scored_wide_pieces_and_many_sequences(gpu, S, hi, window):
    # enough work for the plan to widen the pieces twofold and fourfold; more sequences than the plan has threads
    torch, pa = gpu
    rng = synth.make_rng(7900 + S + hi)
    Hq = Hkv = 8
    D, B = 64, 16
    lens = rng.integers(max(1, hi // 3), hi + 1, S).astype(np.int32)
    mb = -(-hi // B)
    N = int((-(-lens // B)).sum())
    tables = np.full((S, mb), -1, np.int32)
    perm, at = rng.permutation(N), 0
    for s, n in enumerate(lens):
        k = -(-int(n) // B)
        tables[s, :k] = perm[at:at + k]
        at += k
    gen = torch.Generator(device="cuda").manual_seed(S + hi)
    kc, vc = (torch.randn(N, Hkv, B, D, generator=gen, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(S, Hq, D, generator=gen, device="cuda").bfloat16()
    dims = pa.make_dims(S, Hq, Hkv, D, B, N, mb, 0, "bf16")
    out, sums = torch.empty(S, Hq, D, device="cuda"), torch.zeros(S, Hkv, mb * B, device="cuda")
    ws = torch.empty(pa.pa_decode_scored_workspace_bytes(dims, True), dtype=torch.uint8, device="cuda")
    score = pa.make_score(softcap=6.0, window=window)
    pa.pa_decode_scored(dims, score, q, kc, vc, i32(torch, tables), i32(torch, lens), 0.125, out, ws, key_sums=sums)
    plain = torch.empty_like(out)
    ws2 = torch.empty(pa.pa_decode_scored_workspace_bytes(dims, False), dtype=torch.uint8, device="cuda")
    pa.pa_decode_scored(dims, score, q, kc, vc, i32(torch, tables), i32(torch, lens), 0.125, plain, ws2)
    for s in range(S):
        n = int(lens[s])
        b = max(0, n - window) if window else 0
        blocks = torch.from_numpy(tables[s, :-(-n // B)].astype(np.int64)).cuda()
        K, V = (c[blocks].transpose(0, 1).reshape(Hkv, -1, D)[:, b:n].double() for c in (kc, vc))
        z = 6.0 * torch.tanh(0.125 * torch.einsum("hjd,hd->hj", K, q[s].double()) / 6.0)
        p = torch.softmax(z, -1)
        # logits of |z| <= 6 whose products sum to at most 64 * 0.125 * max|q| max|k|
        E = weight_error("bf16", 64 * 2.0 ** -23 * 0.125 * 64 * 25 + 6 * 2.0 ** -21 + 6 * 2.0 ** -22, n)
        ref = torch.einsum("hj,hjd->hd", p, V)
        for got in (out, plain):   # the sums' kernel joins partials in another order
            assert (got[s].double() - ref).abs().max() <= 2.5 * E * V.abs().max()
        assert ((sums[s, :, b:n].double() - p).abs() <= 3 * E * p + 1e-30).all()
        assert (sums[s, :, :b] == 0).all() and (sums[s, :, n:] == 0).all()
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("S,nq,hi", [(2100, 3, 40), (9, 1000, 1000), (700, 20, 60)])
def test_chunk_scored_plans_of_many_rows(gpu, S, nq, hi):
    # more sequences, blocks or rows than the plan keeps in shared memory or reads at once, with masks
    torch, pa = gpu
    rng = synth.make_rng(7950 + S)
    Hq, Hkv, D, B = 4, 1, 64, 16
    counts = rng.integers(0 if S > 9 else nq, nq + 1, S)
    lens = np.array([int(rng.integers(n, max(hi, n) + 1)) for n in counts], np.int32)
    mb = max(1, -(-int(lens.max()) // B))
    N = int((-(-lens // B)).sum()) + 1
    tables = np.full((S, mb), -1, np.int32)
    perm, at = rng.permutation(N), 0
    for s, n in enumerate(lens):
        k = -(-int(n) // B)
        tables[s, :k] = perm[at:at + k]
        at += k
    qs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    T = int(qs[-1])
    gen = torch.Generator(device="cuda").manual_seed(S)
    kc, vc = (torch.randn(N, Hkv, B, D, generator=gen, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(T, Hq, D, generator=gen, device="cuda").bfloat16()
    pos = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, counts)]).astype(np.int64)
    begin = np.where(rng.random(T) < 0.05, pos + 1, pos - pos % 37)   # documents, and some rows with nothing
    dims = pa.make_dims(S, Hq, Hkv, D, B, N, mb, 0, "bf16")
    out = torch.full((T, Hq, D), 7.0, device="cuda")
    ws = torch.empty(pa.pa_chunk_scored_workspace_bytes(dims, T, nq), dtype=torch.uint8, device="cuda")
    pa.pa_chunk_scored(dims, pa.make_score(key_begin=i32(torch, begin)), q, kc, vc, i32(torch, tables), i32(torch, lens),
                       i32(torch, qs), 0.125, out, nq, ws)
    for s in range(S):
        n, m = int(lens[s]), int(counts[s])
        if m == 0:
            continue
        blocks = torch.from_numpy(tables[s, :-(-n // B)].astype(np.int64)).cuda()
        K, V = (c[blocks].transpose(0, 1).reshape(-1, D)[:n].double() for c in (kc, vc))
        rows = slice(int(qs[s]), int(qs[s + 1]))
        z = 0.125 * torch.einsum("thd,jd->thj", q[rows].double(), K)
        j = torch.arange(n, device="cuda")
        b = torch.from_numpy(begin[rows]).cuda()[:, None]
        p0 = torch.from_numpy(pos[rows]).cuda()[:, None]
        seen = (j >= b) & (j <= p0)
        w = torch.softmax(z.masked_fill(~seen[:, None], -math.inf), -1).nan_to_num(0.0)
        ref = torch.einsum("thj,jd->thd", w, V)
        E = weight_error("bf16", 64 * 2.0 ** -23 * 0.125 * 64 * 25 + 2.0 ** -22 * 20, n)
        assert (out[rows].double() - ref).abs().max() <= 2.5 * E * V.abs().max()
        assert (out[rows][~seen.any(-1)] == 0).all()
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("nq", [2, 40, 130])
@pytest.mark.parametrize("opts", [dict(cap=6.0), dict(cap=6.0, slopes=0.25)])
def test_chunk_scored_bits_do_not_depend_on_masked_keys(gpu, opts, nq, dtype):
    # slots behind the last token, before every range, and in shared memory from another call
    torch, pa = gpu
    rng = synth.make_rng(7980 + nq + len(dtype))
    lens = [nq, nq + 41, 700]
    (q, kc, vc, tables, lens), qs = chunk_case(rng, dtype, 8, 2, 64, 16, lens, [nq] * 3)
    opts = dict(opts, key_begin=[max(0, p - 77) for n in lens for p in range(int(n) - nq, int(n))])
    if "slopes" in opts:
        opts["slopes"] = [opts["slopes"]] * 8
    first = [max(0, int(n) - nq - 77) for n in lens]
    gots = []
    for value in (0.0, 200.0, -90.0, 0.0):
        k1, v1 = kc.copy(), vc.copy()
        fill = synth.to_storage(np.full(1, value, np.float32), dtype)[0]
        for s, n in enumerate(lens):
            for j in list(range(first[s])) + list(range(int(n), -(-int(n) // 16) * 16)):
                k1[tables[s][j // 16], :, j % 16] = fill
                v1[tables[s][j // 16], :, j % 16] = fill
        gots.append(call_chunk(torch, pa, (q, k1, v1, tables, lens), qs, dtype, "f32", 0.05, opts))
    for got in gots[1:]:
        assert (got == gots[0]).all()
    assert pa.pa_device_errors(clear=True) == 0
