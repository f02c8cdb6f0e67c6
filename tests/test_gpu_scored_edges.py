"""GPU tests of scored attention at the edges of its contract."""
import numpy as np
import pytest

from gpu_helpers import require_gpu
from paged_helpers import random_case
from paged_kv_cache_127_gb300 import synth
from scored_helpers import assert_rows_close
from test_gpu_scored import call_chunk, call_decode, chunk_case, ref_chunk, ref_decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gpu():
    return require_gpu()


# Logits of std `scale * 8`, up to five times that: with these (scale, cap) a warp takes each form of the cap.
# Caps of more than 55 have a running maximum for bf16 too.
CAPS = [(0.1, 30.0), (0.1, 6.0), (0.1, 1.0), (1.0, 60.0), (1.0, 20.0), (-0.1, 5.0)]


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
