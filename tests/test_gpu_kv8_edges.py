"""GPU tests of the 8-bit cache's attention at the edges of its contract: blocks that no row sees, queries and scales far
from one, the bits of a decode's weights, many small items, steps behind each other without a wait."""
import math

import pytest

from gpu_helpers import require_gpu
from kv8_helpers import assert_within, attend_ref, dtype_of, make_cache, tables_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gpu():
    return require_gpu()


def generator(torch, seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def attend(torch, pa, q, cache, tables, lens, counts, scale, dtype, window=0, sinks=0, most=None, out_dtype="f32"):
    """A decode where every sequence has one row and `most` is none, else a chunk call."""
    T, Hq, D = q.shape
    N, Hkv, B, _ = cache[0].shape
    dims = pa.make_dims(len(lens), Hq, Hkv, D, B, N, tables.shape[1], 0, dtype)
    out = torch.full((T, Hq, D), math.nan, dtype=dtype_of(torch, out_dtype), device="cuda")
    dl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    c8 = pa.make_cache8(*cache)
    if most is None and all(c == 1 for c in counts):
        ws = torch.full((pa.pa_decode8_workspace_bytes(dims),), 255, dtype=torch.uint8, device="cuda")
        pa.pa_decode8(dims, q, c8, tables, dl, scale, out, ws, window=window, sinks=sinks)
    else:
        qs = torch.tensor([sum(counts[:i]) for i in range(len(counts) + 1)], dtype=torch.int32, device="cuda")
        most = most or max(counts)
        ws = torch.full((pa.pa_chunk8_workspace_bytes(dims, T, most),), 255, dtype=torch.uint8, device="cuda")
        pa.pa_chunk8(dims, q, c8, tables, dl, qs, scale, out, most, ws, window=window, sinks=sinks)
    torch.cuda.synchronize()
    return out


def unseen_blocks(n, m, B, window, sinks):
    """Columns of a sequence of n keys of which its last m tokens see no key."""
    begin = n - m - window + 1
    return [b for b in range(-(-n // B)) if (b + 1) * B <= begin and b * B >= sinks]


@pytest.mark.parametrize("dtype,D,B,Hq,Hkv", [("bf16", 128, 16, 32, 8), ("f16", 64, 32, 4, 4), ("bf16", 64, 16, 12, 6)])
@pytest.mark.parametrize("nq", [1, 3, 6, 20, 80])
@pytest.mark.parametrize("window,sinks", [(40, 4), (33, 0), (1, 0), (17, 20), (100, 33), (300, 1)])
def test_blocks_that_no_row_sees_need_not_be_there(gpu, dtype, D, B, Hq, Hkv, nq, window, sinks):
    """A server that frees what a window has left behind: such blocks' table entries may be anything, and so may the scales
    of the block that an entry names."""
    torch, pa = gpu
    gen = generator(torch, 7 * window + nq)
    lens = [nq + x for x in (0, 47, 48, 63, 64, 79, 95, 101, 500, 900)]
    counts = [nq] * len(lens)
    tables, N = tables_for(torch, gen, lens, B)
    cache = make_cache(torch, gen, N, Hkv, B, D)
    q = torch.randn(sum(counts), Hq, D, generator=gen, device="cuda").to(dtype_of(torch, dtype))
    ref, bound = attend_ref(torch, q, cache, tables, lens, counts, 0.09, window, sinks)
    gone = [(s, b) for s, n in enumerate(lens) for b in unseen_blocks(n, nq, B, window, sinks)]
    assert gone
    # the scales of the blocks: what an earlier user left
    for i, (s, b) in enumerate(gone):
        for scales in cache[2:]:
            scales[tables[s, b].long()] = (math.nan, 0.0, math.inf, -1.0)[i % 4]
    got = attend(torch, pa, q, cache, tables, lens, counts, 0.09, dtype, window, sinks)
    assert pa.pa_device_errors(clear=True) == 0
    assert_within(got, ref, bound, "f32")
    # the table entries: no block at all
    for i, (s, b) in enumerate(gone):
        tables[s, b] = (-1, N, -(2 ** 31), 2 ** 31 - 1)[i % 4]
    got = attend(torch, pa, q, cache, tables, lens, counts, 0.09, dtype, window, sinks)
    assert pa.pa_device_errors(clear=True) == 0
    assert_within(got, ref, bound, "f32")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("nq", [1, 5, 9, 70])
@pytest.mark.parametrize("q_exp,k_exp", [((-126, -110), (112, 118)), ((-100, -90), (90, 96)), ((90, 98), (-80, -76))])
def test_queries_and_scales_far_from_one(gpu, D, nq, q_exp, k_exp):
    """Tiny queries over loud keys and loud ones over quiet keys, with logits of order one: rows in bf16 down to its
    subnormal numbers."""
    torch, pa = gpu
    gen = generator(torch, 11 * nq + D)
    B, Hq, Hkv = 16, 8, 2
    lens = [nq + 200, nq + 31]
    tables, N = tables_for(torch, gen, lens, B)
    k, v, _, vs = make_cache(torch, gen, N, Hkv, B, D)
    ks = torch.exp2(torch.randint(k_exp[0], k_exp[1] + 1, (N, Hkv), generator=gen, device="cuda").float())
    q = torch.randn(2 * nq, Hq, D, generator=gen, device="cuda").double()
    q = (q * torch.exp2(torch.randint(q_exp[0], q_exp[1] + 1, (2 * nq, Hq, 1), generator=gen, device="cuda").double())).to(torch.bfloat16)
    q[0, 3] = 0.0
    scale = 2.0 ** -(sum(k_exp) / 2 + sum(q_exp) / 2 + 9)
    ref, bound = attend_ref(torch, q, (k, v, ks, vs), tables, lens, [nq, nq], scale)
    got = attend(torch, pa, q, (k, v, ks, vs), tables, lens, [nq, nq], scale, "bf16")
    assert_within(got, ref, bound, "f32")
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("dtype,D,B,Hq,Hkv,nq", [("bf16", 128, 16, 32, 8, 1), ("f16", 64, 32, 4, 4, 1), ("bf16", 64, 16, 12, 6, 8), ("f16", 128, 32, 8, 1, 2),
                                                 ("bf16", 128, 32, 4, 2, 3), ("f16", 64, 16, 8, 8, 16)])
def test_up_to_16_rows_weights_keep_22_bits(gpu, dtype, D, B, Hq, Hkv, nq):
    """Decodes, and chunks with at most 16 rows of a KV head: weights in two f16 terms.  attend_ref's bound has one term of
    2^-11 for them, once above and once below the fraction; two terms leave 2^-22.  With small logits and few keys
    one rounding to f16 would stand out (logits' own errors are 2^-23 D reach + 2^-20)."""
    torch, pa = gpu
    gen = generator(torch, D + nq)
    lens = [nq + x for x in (1, 2, 3, 5, 7, 11, 17, 40, 100)]
    counts = [nq] * len(lens)
    tables, N = tables_for(torch, gen, lens, B)
    k, v, ks, vs = make_cache(torch, gen, N, Hkv, B, D)
    q = torch.randn(sum(counts), Hq, D, generator=gen, device="cuda").to(dtype_of(torch, dtype))
    scale = 0.004
    ref, bound = attend_ref(torch, q, (k, v, ks, vs), tables, lens, counts, scale)
    weighted, _ = attend_ref(torch, q, (k, v.float().abs().to(v.dtype), ks, vs), tables, lens, counts, scale)   # sum p |V|
    got = attend(torch, pa, q, (k, v, ks, vs), tables, lens, counts, scale, dtype)
    assert_within(got, ref, bound - 2 * (2.0 ** -11 - 2.0 ** -22) * weighted, "f32")


@pytest.mark.parametrize("nq", [1, 4])
def test_windows_and_sinks_beyond_32_bits_are_refused(gpu, nq):
    torch, pa = gpu
    gen = generator(torch, nq)
    tables, N = tables_for(torch, gen, [60], 16)
    cache = make_cache(torch, gen, N, 2, 16, 64)
    q = torch.randn(nq, 4, 64, generator=gen, device="cuda").to(torch.float16)
    for window, sinks in ((2 ** 32, 0), (2 ** 32 + 5, 1), (8, 2 ** 32), (8, 2 ** 31), (2 ** 31, 0)):
        with pytest.raises(ValueError):
            attend(torch, pa, q, cache, tables, [60], [nq], 0.1, "f16", window, sinks)
    ref, bound = attend_ref(torch, q, cache, tables, [60], [nq], 0.1, 8, 2 ** 31 - 1)
    assert_within(attend(torch, pa, q, cache, tables, [60], [nq], 0.1, "f16", 8, 2 ** 31 - 1), ref, bound, "f32")


@pytest.mark.parametrize("dtype,D,B,nq,window", [("bf16", 64, 16, 33, 20), ("f16", 128, 32, 17, 0), ("bf16", 128, 16, 48, 16)])
def test_many_items_of_few_steps(gpu, dtype, D, B, nq, window):
    """Several hundred items of one to four steps, most with a last tile of few rows: slots of items change hands all the time."""
    torch, pa = gpu
    gen = generator(torch, nq)
    S, Hq, Hkv = 300, 8, 1
    counts = [1 + int(x) for x in torch.randint(0, nq, (S,), generator=gen, device="cuda")]
    lens = [c + int(x) for c, x in zip(counts, torch.randint(0, 90, (S,), generator=gen, device="cuda"))]
    tables, N = tables_for(torch, gen, lens, B)
    cache = make_cache(torch, gen, N, Hkv, B, D)
    q = torch.randn(sum(counts), Hq, D, generator=gen, device="cuda").to(dtype_of(torch, dtype))
    ref, bound = attend_ref(torch, q, cache, tables, lens, counts, 0.09, window, 3)
    first = None
    for _ in range(5):
        got = attend(torch, pa, q, cache, tables, lens, counts, 0.09, dtype, window, 3, most=nq)
        assert_within(got, ref, bound, "f32")
        first = got if first is None else first
        assert torch.equal(got, first)
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("nq", [1, 5, 20])
def test_steps_in_flight_are_the_steps_one_at_a_time(gpu, nq):
    """Writes and attention behind each other without a wait between them, scales growing at every step (neighbouring blocks'
    scales share cache lines): each launch sees what the one before it wrote."""
    torch, pa = gpu
    dtype, D, B, Hq, Hkv, S, steps = "bf16", 128, 16, 32, 8, 24, 60
    gen = generator(torch, nq)
    most = 20 + nq * steps
    tables, N = tables_for(torch, gen, [most] * S, B)
    start = make_cache(torch, gen, N, Hkv, B, D)
    start[2].fill_(2.0 ** -20)
    start[3].fill_(2.0 ** -20)
    freqs = torch.from_numpy(pa.pa_rope_freqs(D, 10000.0)[0].copy()).cuda()
    rope = pa.make_rope(D, freqs)
    dims = pa.make_dims(S, Hq, Hkv, D, B, N, tables.shape[1], 0, dtype)
    T = S * nq
    loud = torch.exp2(torch.arange(steps, device="cuda") / 4.0 - 6)[:, None, None, None]
    xs = (loud * torch.randn(steps, T, Hq + 2 * Hkv, D, generator=gen, device="cuda")).to(torch.bfloat16)
    at = [torch.arange(20 + i * nq, 20 + (i + 1) * nq, device="cuda") for i in range(steps)]
    slots = [(tables.long()[:, a // B] * B + a % B).reshape(-1).contiguous() for a in at]
    pos = [a.int().repeat(S).contiguous() for a in at]
    lens = [torch.full((S,), 20 + (i + 1) * nq, dtype=torch.int32, device="cuda") for i in range(steps)]
    starts = torch.arange(S + 1, dtype=torch.int32, device="cuda") * nq
    ws = torch.empty(pa.pa_decode8_workspace_bytes(dims) if nq == 1 else pa.pa_chunk8_workspace_bytes(dims, T, nq), dtype=torch.uint8, device="cuda")

    def run(wait):
        cache = tuple(c.clone() for c in start)
        c8 = pa.make_cache8(*cache)
        outs = [torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda") for _ in range(steps)]
        q = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        for i in range(steps):
            x = xs[i]
            pa.pa_rope_write_kv8(dims, rope, None, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], pos[i], slots[i], q, c8)
            if wait:
                torch.cuda.synchronize()
            if nq == 1:
                pa.pa_decode8(dims, q, c8, tables, lens[i], 0.01, outs[i], ws)
            else:
                pa.pa_chunk8(dims, q, c8, tables, lens[i], starts, 0.01, outs[i], nq, ws)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return outs, cache

    want, kept = run(True)
    for _ in range(3):
        got, cache = run(False)
        for i, (x, y) in enumerate(zip(got, want)):
            assert torch.equal(x, y), f"step {i}"
        for x, y in zip(cache, kept):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert pa.pa_device_errors(clear=True) == 0
