"""GPU tests of pa_evict: the tokens kept are compared index for index with a
plain selection, and the copied rows and sums bit for bit."""
import numpy as np
import pytest

from gpu_helpers import require_gpu, to_dev, to_host
from paged_kv_cache_127_gb300 import synth
from scored_helpers import kept_tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gpu():
    return require_gpu()


def run(torch, pa, dtype, Hkv, D, B, lens, keeps, recent, sums, rows=None, in_place=False, spare_cols=0):
    """Build, call, compare; returns the device error bits."""
    rng = synth.make_rng(9000 + Hkv + D + B + len(lens) + recent)
    S, cap = len(lens), sums.shape[2] - spare_cols
    mb = cap // B
    need = [-(-n // B) for n in lens]
    fresh = [-(-k // B) if 0 <= k < n else 0 for n, k in zip(lens, keeps)]
    N = sum(need) + sum(fresh) + 3
    perm = rng.permutation(N)
    tables, new = np.full((S, mb), -1, np.int32), np.full((S, mb), -1, np.int32)
    at = 0
    for s in range(S):
        tables[s, :need[s]] = perm[at:at + need[s]]
        at += need[s]
    for s in range(S):
        new[s, :fresh[s]] = perm[at:at + fresh[s]]
        at += fresh[s]
    kc, vc = (synth.normal(rng, (N, Hkv, B, D), 1.0, dtype) for _ in range(2))
    dk, dv = to_dev(torch, kc, dtype), to_dev(torch, vc, dtype)
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()
    dims = pa.make_dims(S, Hkv, Hkv, D, B, N, mb, 0, dtype)
    ds = torch.from_numpy(sums).cuda()
    out = ds if in_place else torch.full_like(ds, 5.0)
    new_lens = torch.full((S,), -9, dtype=torch.int32, device="cuda")
    ws = torch.full((max(pa.pa_evict_workspace_bytes(dims), 256),), 0xff, dtype=torch.uint8, device="cuda")
    pa.pa_evict(dims, dk, dv, i32(tables), i32(lens), i32(new), i32(keeps), recent, ds, out, new_lens, ws,
                sum_rows=None if rows is None else i32(rows))
    torch.cuda.synchronize()
    want_sums = sums.copy() if in_place else np.full_like(sums, 5.0)
    want_lens = []
    for s in range(S):
        n, keep = lens[s], keeps[s]
        r = s if rows is None else rows[s]
        evicts = 0 <= keep < n
        want_lens.append(keep if evicts else n)
        for h in range(Hkv):
            kept = kept_tokens(sums[r, h], n, keep, recent) if evicts else np.arange(n)
            want_sums[r, h] = 0.0
            want_sums[r, h, :len(kept)] = sums[r, h, kept]
            if not evicts:
                continue
            for i, j in enumerate(kept):
                src, dst = (tables[s, j // B], h, j % B), (new[s, i // B], h, i % B)
                kc[dst], vc[dst] = kc[src], vc[src]
    np.testing.assert_array_equal(new_lens.cpu().numpy(), want_lens)
    np.testing.assert_array_equal(out.cpu().numpy().view(np.uint32), want_sums.view(np.uint32))
    assert to_host(dk, dtype).tobytes() == kc.tobytes()
    assert to_host(dv, dtype).tobytes() == vc.tobytes()
    return pa.pa_device_errors(clear=True)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,B,Hkv", [(64, 16, 2), (128, 32, 3), (128, 16, 8), (40, 4, 1)])
def test_evict_sizes(gpu, dtype, D, B, Hkv):
    torch, pa = gpu
    rng = synth.make_rng(9100 + D + B)
    lens = [1, 17, 64, 100, 700, 2050, 0, 33]
    cap = -(-2050 // B) * B
    sums = rng.lognormal(0.0, 2.0, (8, Hkv, cap)).astype(np.float32)
    for recent, keeps in ((0, [0, 16, 64, 1, 350, 2049, 0, 40]), (5, [1, 5, 63, 3, 699, 1000, 4, 32]),
                          (300, [1, 2, 3, 99, 301, 300, 7, 0])):
        assert run(torch, pa, dtype, Hkv, D, B, lens, keeps, recent, sums) == 0


def test_evict_ties_zeros_and_special_values(gpu):
    # equal sums go by position; NaN is below -inf, -0 equals +0
    torch, pa = gpu
    rng = synth.make_rng(9200)
    L = 1500
    sums = np.zeros((6, 2, 1504), np.float32)
    sums[1] = 3.25
    sums[2] = rng.integers(0, 3, (2, 1504))
    sums[3] = rng.choice(np.array([0.0, -0.0, np.nan, -np.inf, np.inf, -1.5, 1e-42, -1e-42], np.float32), (2, 1504))
    sums[4] = np.nan
    sums[5] = -np.arange(1504) / 7
    for keep, recent in ((700, 0), (700, 100), (1, 0), (1499, 3), (1024, 1024)):
        assert run(torch, pa, "bf16", 2, 64, 16, [L] * 6, [keep] * 6, recent, sums) == 0


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_rows_in_place_and_long(gpu, in_place):
    # rows in another order, in a larger array, and a context longer than one CTA's shared memory could hold
    torch, pa = gpu
    rng = synth.make_rng(9300)
    lens, keeps = [61000, 3000, 50], [20000, 2999, 60]
    sums = rng.lognormal(0.0, 2.0, (5, 2, 61008)).astype(np.float32)
    assert run(torch, pa, "bf16", 2, 64, 16, lens, keeps, 64, sums, rows=[4, 0, 2], in_place=in_place, spare_cols=0) == 0
    sums = rng.lognormal(0.0, 2.0, (5, 2, 1000)).astype(np.float32)
    assert run(torch, pa, "f16", 2, 64, 16, [900, 30, 900], [128, 10, 901], 16, sums, rows=[4, 0, 2], in_place=in_place,
               spare_cols=40) == 0


def test_evict_bad_inputs_are_flagged(gpu):
    torch, pa = gpu
    rng = synth.make_rng(9400)
    sums = rng.random((3, 2, 64)).astype(np.float32)
    # a negative budget leaves the sequence as it is
    assert run(torch, pa, "bf16", 2, 64, 16, [60, 50], [-1, 20], 4, sums) == pa.PA_DEVERR_BAD_LEN
    # a sum row outside the array leaves the sequence as it is, and no sums are written
    dims = pa.make_dims(2, 2, 2, 64, 16, 20, 4, 0, "bf16")
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    kc, vc = (torch.randn(20, 2, 16, 64, device="cuda").bfloat16() for _ in range(2))
    tables = i32([[0, 1, 2, 3], [4, 5, 6, 7]])
    new = i32([[8, 9, -1, -1], [10, 25, -1, -1]])
    ds = torch.from_numpy(sums).cuda()
    out = torch.full_like(ds, 5.0)
    new_lens = i32([0, 0])
    ws = torch.empty(pa.pa_evict_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    k0 = kc.clone()
    pa.pa_evict(dims, kc, vc, tables, i32([60, 50]), new, i32([20, 60]), 4, ds, out, new_lens, ws, sum_rows=i32([3, 1]))
    assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_BAD_ROW
    assert new_lens.tolist() == [60, 50] and torch.equal(kc, k0) and (out[0] == 5).all() and (out[2] == 5).all()
    # a destination block outside the pool: its rows are skipped
    pa.pa_evict(dims, kc, vc, tables, i32([60, 50]), new, i32([20, 20]), 4, ds, out, new_lens, ws)
    assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_BAD_BLOCK
    kept = kept_tokens(sums[1, 0], 50, 20, 4)
    for i, j in enumerate(kept[:16]):
        assert torch.equal(kc[10, 0, i], k0[4 + j // 16, 0, j % 16])
    assert torch.equal(kc[11:], k0[11:])


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_many_pairs_take_small_blocks(gpu, in_place):
    # 320 (sequence, KV head) pairs, a CTA of 256 threads each; more kept than a tile of 1024 places
    torch, pa = gpu
    rng = synth.make_rng(9500)
    S, Hkv, B, cap = 40, 8, 16, 2048
    lens = [int(x) for x in rng.integers(1100, cap + 1, S)]
    lens[3], lens[7], lens[11] = 0, cap, 5
    keeps = [int(x) for x in rng.integers(1, 1900, S)]
    keeps[0], keeps[7] = 1025, cap - 1
    sums = rng.lognormal(0.0, 2.0, (S, Hkv, cap + 4)).astype(np.float32)
    sums[5] = rng.integers(0, 4, (Hkv, cap + 4))
    assert run(torch, pa, "bf16", Hkv, 8, B, lens, keeps, 77, sums, in_place=in_place, spare_cols=4) == 0


def test_evict_copies_several_tiles_a_block(gpu):
    # 512 pairs over tables of 1296 places: copy blocks of four tiles of 128 rows, counts that end inside each of them
    torch, pa = gpu
    rng = synth.make_rng(9510)
    S, Hkv, B, cap = 64, 8, 16, 1296
    lens = [int(x) for x in rng.integers(1000, cap + 1, S)]
    keeps = [int(x) for x in rng.integers(1, 900, S)]
    keeps[:6] = [128, 127, 129, 512, 513, 640]
    sums = rng.lognormal(0.0, 2.0, (S, Hkv, cap)).astype(np.float32)
    assert run(torch, pa, "bf16", Hkv, 64, B, lens, keeps, 30, sums) == 0


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n,keep", [(393400, 100001), (393500, 700), (61000, 50000)])
def test_evict_past_shared_memory_and_past_a_tile(gpu, n, keep, in_place):
    # tables of more than 393,152 places, whose keys a cluster's shared memory does not hold; more kept than a
    # tile of 32,768 places, with the sums moved in place
    torch, pa = gpu
    rng = synth.make_rng(9520 + keep)
    cap = -(-n // 32) * 32
    sums = rng.lognormal(0.0, 2.0, (1, 1, cap)).astype(np.float32)
    sums[0, 0, ::7] = 0.25
    assert run(torch, pa, "f16", 1, 64, 32, [n], [keep], 333, sums, in_place=in_place) == 0
