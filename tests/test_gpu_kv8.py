"""GPU tests of the 8-bit cache: the writes, the copy, decode and chunk attention."""
import math

import pytest

from gpu_helpers import require_gpu
from kv8_helpers import (assert_within, assert_written, attend_ref, codes_to, dtype_of, make_cache, rotate_ref, tables_for,
                         write_ref)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gpu():
    return require_gpu()


def generator(torch, seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ------------------------------------------------------------------ the writes
def write_case(torch, gen, dtype, D, B, Hq, Hkv, pairs, R, axes, strided=True):
    """Tokens of sequences (length, new tokens): q, k, v as column ranges of one projection, slots and positions."""
    dt = dtype_of(torch, dtype)
    tables, N = tables_for(torch, gen, [n for n, _ in pairs], B)
    slots = []
    for s, (n, m) in enumerate(pairs):
        row = tables[s].tolist()
        slots += [row[p // B] * B + p % B for p in range(n - m, n)]
    T = len(slots)
    pad = 8 if strided else 0
    fused = torch.randn(T, (Hq + 2 * Hkv) * D + pad, generator=gen, device="cuda").to(dt)
    q = fused[:, : Hq * D].unflatten(1, (Hq, D))
    k = fused[:, Hq * D: (Hq + Hkv) * D].unflatten(1, (Hkv, D))
    v = fused[:, (Hq + Hkv) * D: (Hq + 2 * Hkv) * D].unflatten(1, (Hkv, D))
    positions = torch.randint(-50, 70000, (axes, T), generator=gen, device="cuda", dtype=torch.int32)
    pair_axis = torch.randint(0, axes, (R // 2,), generator=gen, device="cuda", dtype=torch.int32)
    return q, k, v, torch.tensor(slots, dtype=torch.int64, device="cuda"), positions, pair_axis, N


def check_write(torch, pa, dtype, D, B, Hq, Hkv, q, k, v, slots, positions, pair_axis, N, R, interleaved, mscale, cache, in_place=False):
    """Runs the write over `cache` and holds q_out, codes and scales to the definition."""
    axes = positions.shape[0]
    f, _ = pa.pa_rope_freqs(R, 10000.0)
    freqs = torch.from_numpy(f[: R // 2].copy()).cuda()
    kr = rotate_ref(torch, k, positions, pair_axis, freqs, R, interleaved, mscale)
    qr = rotate_ref(torch, q, positions, pair_axis, freqs, R, interleaved, mscale)
    # the write overwrites its inputs when in place, the cache always: the references first
    refs = write_ref(torch, cache, slots, kr, v.double(), k, 316.0, max(1.0, abs(mscale)))
    q_out = q if in_place else torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    was = q_out.clone()
    dims = pa.make_dims(0, Hq, Hkv, D, B, N, 1, 0, dtype)
    c8 = pa.make_cache8(*cache)
    rope = pa.make_rope(R, freqs, interleaved, mscale)
    if axes == 1 and not bool(pair_axis.any()):
        pa.pa_rope_write_kv8(dims, rope, None, q, k, v, positions[0], slots, q_out, c8)
    else:
        pa.pa_rope_write_kv8(dims, rope, pa.make_axes(axes, pair_axis), q, k, v, positions, slots, q_out, c8)
    torch.cuda.synchronize()
    # a turned value: (cos, sin) off by 2^-22 of mscale each, three roundings of fp32
    slack = 2.0 ** -20
    assert_written(torch, cache[0], cache[2], refs[0], slack)
    assert_written(torch, cache[1], cache[3], refs[1], 0.0)
    live = (slots >= 0) & (slots < N * B)
    step = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype]
    ok = torch.isfinite(qr) & live[:, None, None]
    lim = step * qr.abs() + slack * max(1.0, abs(mscale)) * q_norm(qr) + 2.0 ** -25
    assert bool(((q_out.double() - qr).abs() <= lim)[ok].all())
    assert torch.equal(q_out[~live], was[~live])


def q_norm(x):
    return x.nan_to_num(0.0, 0.0, 0.0).abs().amax(-1, keepdim=True)


SHAPES = [("bf16", 128, 16, 32, 8), ("f16", 64, 32, 4, 4), ("bf16", 64, 16, 12, 6), ("f16", 128, 32, 8, 1), ("bf16", 128, 32, 11, 11)]
# (length with the new tokens, new tokens) of each sequence: one token; steps at every offset; ragged chunks
STEPS = [(1 + i, 1) for i in range(40)]
CHUNKS = [(70, 70), (37, 5), (16, 16), (33, 1), (200, 131), (17, 2), (64, 48), (1, 1), (31, 15)]


@pytest.mark.parametrize("dtype,D,B,Hq,Hkv", SHAPES)
@pytest.mark.parametrize("pairs", [[(23, 1)], STEPS, CHUNKS], ids=["one", "steps", "chunks"])
def test_write8_against_the_definition(gpu, dtype, D, B, Hq, Hkv, pairs):
    torch, pa = gpu
    for R, interleaved, axes, mscale in ((D, False, 1, 1.0), (D // 2, False, 3, 1.25), (D, True, 3, 1.0), (20, False, 2, 0.5), (22, True, 4, 1.0)):
        gen = generator(torch, 100 + R + axes)
        q, k, v, slots, positions, pair_axis, N = write_case(torch, gen, dtype, D, B, Hq, Hkv, pairs, R, axes)
        cache = make_cache(torch, gen, N, Hkv, B, D)
        check_write(torch, pa, dtype, D, B, Hq, Hkv, q, k, v, slots, positions, pair_axis, N, R, interleaved, mscale, cache,
                    in_place=R == 20 or axes == 1)
    assert pa.pa_device_errors(clear=True) == 0


def test_write8_many_tokens(gpu):
    """Tiles of 16 tokens: runs that cross them, blocks of 32 that cover two."""
    torch, pa = gpu
    for B, Hkv, pairs in ((16, 2, [(1500, 1490), (900, 893), (77, 70)]), (32, 4, [(2000, 1999), (700, 690), (5, 5)])):
        gen = generator(torch, B)
        q, k, v, slots, positions, pair_axis, N = write_case(torch, gen, "bf16", 64, B, Hkv, Hkv, pairs, 64, 1)
        cache = make_cache(torch, gen, N, Hkv, B, 64)
        check_write(torch, pa, "bf16", 64, B, Hkv, Hkv, q, k, v, slots, positions, pair_axis, N, 64, False, 1.0, cache)
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_write8_loud_quiet_and_not_finite(gpu, dtype):
    torch, pa = gpu
    gen = generator(torch, 5)
    D, B, Hq, Hkv = 64, 16, 4, 2
    q, k, v, slots, positions, pair_axis, N = write_case(torch, gen, dtype, D, B, Hq, Hkv, [(40, 25), (9, 4), (18, 3), (50, 1)], D, 1)
    big = 60000.0 if dtype == "f16" else 2.0 ** 100
    k[0] *= big / 8
    v[3, 1, 5] = big
    k[6, 0, 7] = math.inf
    k[6, 1, 9] = -math.inf
    v[8] = math.nan
    v[20, 0, 0] = -math.inf
    k[25:29] = 0.0
    v[25:29] = 0.0
    k[30] = 2.0 ** -24
    v[30, 1] = -0.0
    cache = make_cache(torch, gen, N, Hkv, B, D)
    check_write(torch, pa, dtype, D, B, Hq, Hkv, q, k, v, slots, positions, pair_axis, N, D, False, 1.0, cache)
    assert pa.pa_device_errors(clear=True) == 0


def test_write8_padding_and_bad_slots(gpu):
    torch, pa = gpu
    gen = generator(torch, 6)
    D, B, Hq, Hkv = 64, 16, 4, 2
    q, k, v, slots, positions, pair_axis, N = write_case(torch, gen, "bf16", D, B, Hq, Hkv, [(40, 30), (9, 4), (50, 17)], D, 2)
    slots[:3] = -1                     # padding before, between the sequences and behind them
    slots[30:34] = -5
    slots[-2:] = -1
    cache = make_cache(torch, gen, N, Hkv, B, D)
    check_write(torch, pa, "bf16", D, B, Hq, Hkv, q, k, v, slots, positions, pair_axis, N, D, False, 1.0, cache)
    assert pa.pa_device_errors(clear=True) == 0
    slots[10] = N * B
    slots[-5] = 1 << 40
    check_write(torch, pa, "bf16", D, B, Hq, Hkv, q, k, v, slots, positions, pair_axis, N, D, False, 1.0, cache)
    assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_BAD_SLOT
    pair_axis[3], pair_axis[30] = 2, -1
    f, _ = pa.pa_rope_freqs(D, 10000.0)
    dims = pa.make_dims(0, Hq, Hkv, D, B, N, 1, 0, "bf16")
    slots[10] = slots[-5] = -1
    q_out = torch.empty_like(q.contiguous())
    pa.pa_rope_write_kv8(dims, pa.make_rope(D, torch.from_numpy(f.copy()).cuda()), pa.make_axes(2, pair_axis), q, k, v, positions,
                         slots, q_out, pa.make_cache8(*cache))
    assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_BAD_AXIS
    live = slots >= 0
    for d in (3, 35, 30, 62):          # pairs of an axis that is none are not turned
        assert torch.equal(q_out[live][..., d], q[live][..., d])


def test_write8_step_by_step_is_the_write_at_once(gpu):
    """Tokens that get louder: each append rescales what was there, exactly but for subnormal codes."""
    torch, pa = gpu
    D, B, Hkv, n = 128, 16, 2, 40
    gen = generator(torch, 7)
    tables, N = tables_for(torch, gen, [n], B)
    slots = torch.tensor([int(tables[0, p // B]) * B + p % B for p in range(n)], device="cuda")
    k = (torch.randn(n, Hkv, D, generator=gen, device="cuda") * torch.exp2(torch.arange(n, device="cuda") / 6.0)[:, None, None]).to(torch.bfloat16)
    v = k.flip(2).contiguous()
    dims = pa.make_dims(0, Hkv, Hkv, D, B, N, 1, 0, "bf16")
    start = make_cache(torch, gen, N, Hkv, B, D)
    one, all_ = [x.clone() for x in start], [x.clone() for x in start]
    for t in range(n):
        pa.pa_write_kv8(dims, k[t:t + 1], v[t:t + 1], slots[t:t + 1], pa.make_cache8(*one))
    pa.pa_write_kv8(dims, k, v, slots, pa.make_cache8(*all_))
    for x, y in zip(one[2:], all_[2:]):
        assert torch.equal(x, y)
    for x, y in zip(one[:2], all_[:2]):
        x, y = codes_to(torch, x), codes_to(torch, y)
        assert bool(((x == y) | ((x - y).abs() <= 2.0 ** -9) & (y.abs() < 2.0 ** -5)).all())
    # and it is the definition: K's scale as V's, nothing turned
    refs = write_ref(torch, start, slots, k.double(), v.double(), k, 448.0, 1.0)
    assert_written(torch, all_[0], all_[2], refs[0], 0.0)
    assert_written(torch, all_[1], all_[3], refs[1], 0.0)
    assert pa.pa_device_errors(clear=True) == 0


def test_copy_blocks8(gpu):
    torch, pa = gpu
    for D, B, Hkv in ((64, 16, 1), (128, 32, 8), (64, 32, 300)):
        gen = generator(torch, D + Hkv)
        cache = make_cache(torch, gen, 12, Hkv, B, D)
        want = [x.clone().view(torch.uint8) if x.dtype != torch.float32 else x.clone() for x in cache]
        pairs = [(3, 5), (3, 7), (11, 0)]
        for s, d in pairs:
            for w in want:
                w[d] = w[s]
        dims = pa.make_dims(0, Hkv, Hkv, D, B, 12, 1, 0, "bf16")
        bad = pairs + [(12, 1), (2, -1)]
        pa.pa_copy_blocks8(dims, pa.make_cache8(*cache), torch.tensor(bad, device="cuda"))
        assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_BAD_PAIR
        for x, w in zip(cache, want):
            assert torch.equal(x.view(torch.uint8) if x.dtype != torch.float32 else x, w)


# ------------------------------------------------------------------ attention
def chunk_call(torch, pa, q, cache, tables, lens, counts, scale, dtype, out_dtype, window=0, sinks=0, most=None, decode=False):
    T, Hq, D = q.shape
    N, Hkv, B, _ = cache[0].shape
    dims = pa.make_dims(len(lens), Hq, Hkv, D, B, N, tables.shape[1], 0, dtype)
    out = torch.full((T, Hq, D), math.nan, dtype=dtype_of(torch, out_dtype), device="cuda")
    dl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    c8 = pa.make_cache8(*cache)
    if decode:
        ws = torch.full((pa.pa_decode8_workspace_bytes(dims),), 255, dtype=torch.uint8, device="cuda")
        pa.pa_decode8(dims, q, c8, tables, dl, scale, out, ws, window=window, sinks=sinks)
    else:
        qs = torch.tensor([sum(counts[:i]) for i in range(len(counts) + 1)], dtype=torch.int32, device="cuda")
        most = most or max(counts)
        ws = torch.full((max(pa.pa_chunk8_workspace_bytes(dims, T, most), 256),), 255, dtype=torch.uint8, device="cuda")
        pa.pa_chunk8(dims, q, c8, tables, dl, qs, scale, out, most, ws, window=window, sinks=sinks)
    torch.cuda.synchronize()
    return out


def poison(torch, cache, tables, lens, counts, window, sinks):
    """NaN codes in every slot that no row sees."""
    N, Hkv, B, D = cache[0].shape
    keep = torch.zeros(N * B, dtype=torch.bool, device="cuda")
    for s, (n, m) in enumerate(zip(lens, counts)):
        if n == 0 or m == 0:
            continue
        j = torch.arange(n, device="cuda")
        see = (j > n - m - window) | (j < sinks) if window else j >= 0
        slots = tables[s].long()[j // B] * B + j % B
        keep[slots[see]] = True
    for c in cache[:2]:
        x = c.view(torch.uint8).transpose(1, 2).reshape(N * B, Hkv, D).clone()
        x[~keep] = 0x7F
        c.view(torch.uint8).copy_(x.view(N, B, Hkv, D).transpose(1, 2))


DECODE_LENS = [0, 1, 15, 16, 17, 31, 32, 33, 100, 500, 1023, 1777, 64, 5]
HEADS = [("bf16", 128, 16, 32, 8), ("f16", 64, 32, 4, 4), ("bf16", 64, 16, 12, 6), ("f16", 128, 32, 8, 1), ("bf16", 128, 32, 64, 8)]


@pytest.mark.parametrize("dtype,D,B,Hq,Hkv", HEADS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (40, 4), (33, 33), (300, 100), (64, 0), (5000, 3)])
def test_decode8(gpu, dtype, D, B, Hq, Hkv, window, sinks):
    torch, pa = gpu
    gen = generator(torch, window + D)
    tables, N = tables_for(torch, gen, DECODE_LENS, B)
    cache = make_cache(torch, gen, N, Hkv, B, D, spread=1.0 + (window == 40), odd_scales=window == 64)
    counts = [1] * len(DECODE_LENS)
    poison(torch, cache, tables, DECODE_LENS, counts, window, sinks)
    q = (3 * torch.randn(len(DECODE_LENS), Hq, D, generator=gen, device="cuda")).to(dtype_of(torch, dtype))
    for scale in (0.09, -0.02):
        ref, bound = attend_ref(torch, q, cache, tables, DECODE_LENS, counts, scale, window, sinks)
        for out_dtype in ("f32", dtype):
            got = chunk_call(torch, pa, q, cache, tables, DECODE_LENS, counts, scale, dtype, out_dtype, window, sinks, decode=True)
            assert_within(got, ref, bound, out_dtype)
            assert bool((got[0] == 0).all())
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("S,lo,hi", [(1, 9000, 9000), (700, 1, 60), (3, 4000, 70000), (200, 300, 900)])
def test_decode8_splits(gpu, S, lo, hi):
    """One long sequence over many warps, many short ones in one warp, and what lies between."""
    torch, pa = gpu
    gen = generator(torch, S)
    lens = torch.randint(lo, hi + 1, (S,), generator=gen, device="cuda").tolist()
    tables, N = tables_for(torch, gen, lens, 16)
    cache = make_cache(torch, gen, N, 2, 16, 64)
    q = torch.randn(S, 8, 64, generator=gen, device="cuda").to(torch.bfloat16)
    for window, sinks in ((0, 0), (max(1, hi // 3), 7)):
        ref, bound = attend_ref(torch, q, cache, tables, lens, [1] * S, 0.125, window, sinks)
        got = chunk_call(torch, pa, q, cache, tables, lens, [1] * S, 0.125, "bf16", "f32", window, sinks, decode=True)
        assert_within(got, ref, bound, "f32")
        again = chunk_call(torch, pa, q, cache, tables, lens, [1] * S, 0.125, "bf16", "f32", window, sinks, decode=True)
        assert torch.equal(got, again)
    assert pa.pa_device_errors(clear=True) == 0


def chunk_lens(nq):
    """(length, rows): whole prompts, continued ones, one row, none, a length inside a block."""
    return [(nq, nq), (nq + 100, nq), (nq + 1, 1), (77, 0), (nq + 517, max(1, nq // 2)), (nq + 15, nq), (max(1, nq // 3), max(1, nq // 3))]


@pytest.mark.parametrize("dtype,D,B,Hq,Hkv", HEADS)
@pytest.mark.parametrize("nq", [1, 2, 5, 8, 15, 30, 64, 200])
def test_chunk8(gpu, dtype, D, B, Hq, Hkv, nq):
    torch, pa = gpu
    gen = generator(torch, nq + D)
    lens, counts = zip(*chunk_lens(nq))
    tables, N = tables_for(torch, gen, lens, B)
    q = (2 * torch.randn(sum(counts) + 3, Hq, D, generator=gen, device="cuda")).to(dtype_of(torch, dtype))
    for window, sinks in ((0, 0), (40, 4), (1, 0), (70, 130), (350, 33)):
        cache = make_cache(torch, gen, N, Hkv, B, D, spread=1.0 + (window == 40), odd_scales=window == 70)
        poison(torch, cache, tables, lens, counts, window, sinks)
        scale = -0.05 if window == 1 else 0.09
        ref, bound = attend_ref(torch, q[: sum(counts)], cache, tables, lens, counts, scale, window, sinks)
        for out_dtype in ("f32", dtype):
            got = chunk_call(torch, pa, q, cache, tables, lens, counts, scale, dtype, out_dtype, window, sinks)
            assert_within(got[: sum(counts)], ref, bound, out_dtype)
            assert bool(got[sum(counts):].isnan().all()), "rows behind the last sequence"
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("nq", [1, 6, 90])
def test_attend8_bad_blocks_lengths_and_order(gpu, nq):
    torch, pa = gpu
    gen = generator(torch, nq)
    dtype, D, B, Hq, Hkv = "bf16", 128, 16, 8, 2
    lens, counts = [nq + 100, nq + 40, nq + 300], [nq] * 3
    tables, N = tables_for(torch, gen, lens, B)
    cache = make_cache(torch, gen, N, Hkv, B, D)
    q = torch.randn(3 * nq, Hq, D, generator=gen, device="cuda").to(torch.bfloat16)
    bad = [(0, 2), (1, 0), (2, 5), (2, 6)]
    for i, (s, c) in enumerate(bad):
        tables[s, c] = [-1, N, 1 << 30, -(1 << 31)][i]
    ref, bound = attend_ref(torch, q, cache, tables, lens, counts, 0.1, bad=bad)
    for decode in ([True, False] if nq == 1 else [False]):
        got = chunk_call(torch, pa, q, cache, tables, lens, counts, 0.1, dtype, "f32", decode=decode)
        assert_within(got, ref, bound, "f32")
        assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_BAD_BLOCK
    if nq == 1:
        # every block gone: zeros
        none = torch.full_like(tables, -1)
        assert bool((chunk_call(torch, pa, q, cache, none, lens, counts, 0.1, dtype, "f32", decode=True) == 0).all())
        pa.pa_device_errors(clear=True)
        # lengths outside the table are clamped
        for n in (-3, 10 ** 6):
            got = chunk_call(torch, pa, q, cache, none, [n, 5, 5], counts, 0.1, dtype, "f32", decode=True)
            assert bool((got == 0).all())
            assert pa.pa_device_errors(clear=True) & pa.PA_DEVERR_BAD_LEN
        return
    # a sequence with more rows than keys, or than the bound, is left out
    tables, N = tables_for(torch, gen, lens, B)
    cache = make_cache(torch, gen, N, Hkv, B, D)
    short = [lens[0], nq - 1, lens[2]]
    ref, bound = attend_ref(torch, q, cache, tables, short, [nq, 0, nq], 0.1)
    got = chunk_call(torch, pa, q, cache, tables, short, counts, 0.1, dtype, "f32")
    assert bool(got[nq:2 * nq].isnan().all())
    ref2, bound2 = attend_ref(torch, q[2 * nq:], cache, tables[2:], short[2:], [nq], 0.1)
    assert_within(got[:nq], ref[:nq], bound[:nq], "f32")
    assert_within(got[2 * nq:], ref2, bound2, "f32")
    assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_BAD_LEN
    # query_start out of order: nothing is done
    dims = pa.make_dims(3, Hq, Hkv, D, B, N, tables.shape[1], 0, dtype)
    out = torch.full((3 * nq, Hq, D), math.nan, device="cuda")
    ws = torch.empty(pa.pa_chunk8_workspace_bytes(dims, 3 * nq, nq), dtype=torch.uint8, device="cuda")
    for starts in ([0, 2 * nq, nq, 3 * nq], [-1, nq, 2 * nq, 3 * nq], [0, nq, 2 * nq, 3 * nq + 1]):
        pa.pa_chunk8(dims, q, pa.make_cache8(*cache), tables, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                     torch.tensor(starts, dtype=torch.int32, device="cuda"), 0.1, out, nq, ws)
        assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_BAD_LEN
        assert bool(out.isnan().all())


@pytest.mark.parametrize("nq", [1, 7, 100])
def test_attend8_nan_key_and_query(gpu, nq):
    """A NaN that a row sees makes that row NaN; other sequences and heads are as they were."""
    torch, pa = gpu
    gen = generator(torch, 40 + nq)
    D, B, Hq, Hkv = 64, 16, 8, 2
    lens, counts = [nq + 60, nq + 20], [nq, nq]
    tables, N = tables_for(torch, gen, lens, B)
    cache = make_cache(torch, gen, N, Hkv, B, D)
    q = torch.randn(2 * nq, Hq, D, generator=gen, device="cuda").to(torch.float16)
    ref, bound = attend_ref(torch, q, cache, tables, lens, counts, 0.1)
    cache[0].view(torch.uint8)[int(tables[0, 1]), 0, 3, 5] = 0xFF
    q[nq, 6, 0] = math.nan
    got = chunk_call(torch, pa, q, cache, tables, lens, counts, 0.1, "f16", "f32", decode=nq == 1)
    assert bool(got[:nq, :4].isnan().all()) and bool(got[nq, 6].isnan().all())
    got[nq, 6], ref[nq, 6] = 0.0, 0.0
    assert_within(got[:nq, 4:], ref[:nq, 4:], bound[:nq, 4:], "f32")
    assert_within(got[nq:], ref[nq:], bound[nq:], "f32")


def test_attend8_scales_far_apart(gpu):
    """Blocks of very loud and very quiet values in one sequence, queries of any size."""
    torch, pa = gpu
    gen = generator(torch, 50)
    D, B, Hq, Hkv = 128, 16, 8, 2
    for nq in (1, 9, 70):
        lens = [nq + 400]
        tables, N = tables_for(torch, gen, lens, B)
        k, v, ks, vs = make_cache(torch, gen, N, Hkv, B, D)
        ks = torch.exp2(torch.randint(-40, -6, (N, Hkv), generator=gen, device="cuda").float())
        vs = torch.exp2(torch.randint(-30, 30, (N, Hkv), generator=gen, device="cuda").float())
        q = torch.randn(nq, Hq, D, generator=gen, device="cuda")
        q = (q * torch.exp2(torch.randint(-60, 8, (nq, Hq, 1), generator=gen, device="cuda").float())).to(torch.bfloat16)
        ref, bound = attend_ref(torch, q, (k, v, ks, vs), tables, lens, [nq], 0.1)
        got = chunk_call(torch, pa, q, (k, v, ks, vs), tables, lens, [nq], 0.1, "bf16", "f32", decode=nq == 1)
        assert_within(got, ref, bound, "f32")
