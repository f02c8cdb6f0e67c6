"""Host side of the scored attention, rotary and eviction calls, without a GPU:
refusals of the C ABI (no call here gets past its checks), the rotary
frequencies, and the allocator's eviction."""
import ctypes
import math

import numpy as np
import pytest

from paged_kv_cache_127_gb300 import build as pa_build
from paged_kv_cache_127_gb300 import synth


@pytest.fixture(scope="module")
def pa():
    pa_build.build()
    from paged_kv_cache_127_gb300 import binding
    return binding


def dims(pa, **kw):
    d = dict(num_seqs=2, num_q_heads=8, num_kv_heads=2, head_dim=64, block_size=16, num_blocks=10,
             max_blocks_per_seq=4, partition_size=0, kv_dtype="bf16")
    d.update(kw)
    return pa.make_dims(**d)


P = 1 << 20  # an aligned address that no call may follow


def decode(pa, d, score=None, sums=None, q=P, out=P, out_dtype=None, ws=P, ws_bytes=1 << 40):
    ref = lambda x: None if x is None else ctypes.byref(x)
    return pa.lib.pa_decode_scored(ctypes.byref(d), ref(score), q, P, P, P, P, 0.1, ref(sums), out,
                                   pa.PA_F32 if out_dtype is None else out_dtype, ws, ws_bytes, None)


def chunk(pa, d, score=None, T=9, max_q=5, out_dtype=0, ws_bytes=1 << 40, qs=P):
    ref = lambda x: None if x is None else ctypes.byref(x)
    return pa.lib.pa_chunk_scored(ctypes.byref(d), ref(score), P, P, P, P, P, qs, T, max_q, 0.1, P, out_dtype, P, ws_bytes, None)


def test_scored_refusals(pa):
    INV, UNS = pa.PA_ERR_INVALID, pa.PA_ERR_UNSUPPORTED
    nan, inf = float("nan"), float("inf")
    for call in (decode, chunk):
        for bad in (dict(softcap=-1.0), dict(softcap=nan), dict(softcap=inf), dict(window=-1), dict(slopes=P + 2),
                    dict(key_begin=P + 1), dict(key_end=P + 3)):
            sc = pa.pa_score(**{**dict(softcap=0.0, window=0), **bad})
            assert call(pa, dims(pa), sc) == INV, bad
        assert call(pa, dims(pa, head_dim=80)) == UNS
        assert call(pa, dims(pa, block_size=8)) == UNS
        assert call(pa, dims(pa, num_q_heads=6)) == UNS
        assert call(pa, dims(pa, num_q_heads=7)) == INV
        assert call(pa, dims(pa, partition_size=24)) == INV
        assert call(pa, dims(pa), out_dtype=pa.PA_F16) == INV
        assert call(pa, dims(pa), out_dtype=9) == INV
        assert call(pa, dims(pa), ws_bytes=64) == INV
        assert call(pa, dims(pa, num_seqs=0)) == pa.PA_OK
    assert decode(pa, dims(pa), q=P + 8) == INV
    assert decode(pa, dims(pa), out=None) == INV
    assert decode(pa, dims(pa), ws=P + 128) == INV
    assert chunk(pa, dims(pa), max_q=0) == INV
    assert chunk(pa, dims(pa), T=-1) == INV
    assert chunk(pa, dims(pa), qs=None) == INV
    assert chunk(pa, dims(pa), T=0) == pa.PA_OK
    for bad in (dict(sums=None), dict(sums=P + 4), dict(num_rows=-1), dict(cols=60), dict(cols=66), dict(rows=P + 2)):
        ks = pa.pa_key_sums(**{**dict(sums=P, rows=None, num_rows=2, cols=64), **bad})
        assert decode(pa, dims(pa), None, ks) == INV, bad
        assert evict(pa, dims(pa), ks) == INV, bad
    assert pa.pa_decode_scored_workspace_bytes(dims(pa, num_seqs=0)) == 0
    plain, with_sums = (pa.pa_decode_scored_workspace_bytes(dims(pa), x) for x in (False, True))
    assert with_sums >= plain + 2 * 8 * 64 * 4


def evict(pa, d, ks, **kw):
    a = dict(kc=P, vc=P, tables=P, lens=P, new=P, keep=P + 4096, recent=3, out=P + (1 << 30), new_lens=P + 8192, ws=P,
             ws_bytes=1 << 40)
    a.update(kw)
    return pa.lib.pa_evict(ctypes.byref(d), a["kc"], a["vc"], a["tables"], a["lens"], a["new"], a["keep"], a["recent"],
                           ctypes.byref(ks) if ks is not None else None, a["out"], a["new_lens"], a["ws"], a["ws_bytes"], None)


def test_evict_refusals(pa):
    INV = pa.PA_ERR_INVALID
    ks = pa.pa_key_sums(P, None, 2, 64)
    d = dims(pa)
    assert evict(pa, d, None) == INV
    for bad in (dict(recent=-1), dict(kc=None), dict(new=None), dict(ws=P + 16), dict(ws_bytes=100), dict(out=P + 16),
                dict(new_lens=P), dict(new_lens=P + 4), dict(new_lens=P + 4096), dict(out=P + (1 << 30) + 4), dict(tables=P + 1)):
        assert evict(pa, d, ks, **bad) == INV, bad
    assert evict(pa, dims(pa, head_dim=12), ks) == pa.PA_ERR_UNSUPPORTED
    assert evict(pa, dims(pa, num_seqs=40000, num_kv_heads=2), ks) == INV
    assert evict(pa, dims(pa, max_blocks_per_seq=(1 << 26) + 1), pa.pa_key_sums(P, None, 2, (1 << 30) + 16)) == INV
    assert pa.pa_evict_workspace_bytes(dims(pa, max_blocks_per_seq=(1 << 26) + 1)) == 0
    assert evict(pa, dims(pa, num_seqs=0), ks) == pa.PA_OK


def rope(pa, d, R=64, T=3, **kw):
    a = dict(q=P, qs=512, k=P, ks=128, v=P, vs=128, out=P + (1 << 24), os=512, freqs=P, mscale=1.0, inter=0)
    a.update(kw)
    r = pa.pa_rope(R, a["inter"], a["freqs"], a["mscale"])
    return pa.lib.pa_rope_write_kv(ctypes.byref(d), ctypes.byref(r), a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], P, P, T,
                                   a["out"], a["os"], P, P, None)


def test_rope_refusals(pa):
    INV = pa.PA_ERR_INVALID
    d = dims(pa)
    for bad in (dict(R=0), dict(R=3), dict(R=66), dict(R=-2), dict(mscale=float("nan")), dict(inter=2), dict(qs=511),
                dict(qs=504), dict(ks=127), dict(vs=0), dict(os=100), dict(qs=513), dict(q=P + 2), dict(freqs=None),
                dict(freqs=P + 4), dict(T=-1), dict(out=P + 512), dict(out=P, os=520), dict(k=None),
                # rows of 1024 bytes, 2048 apart: starts nearer than a row, from either side, a row later too
                dict(qs=1024, os=1024, out=P + 512), dict(qs=1024, os=1024, out=P + 1536),
                dict(qs=1024, os=1024, out=P + 2048), dict(qs=1024, os=1024, q=P + 512, out=P)):
        assert rope(pa, d, **bad) == INV, bad
    assert rope(pa, dims(pa, num_q_heads=7)) == INV
    assert rope(pa, dims(pa, num_q_heads=0)) == INV
    assert rope(pa, dims(pa, head_dim=12), R=4) == pa.PA_ERR_UNSUPPORTED
    assert rope(pa, d, T=0) == pa.PA_OK


def test_rope_freqs(pa):
    f, m = pa.pa_rope_freqs(8, 10000.0)
    np.testing.assert_allclose(f, [1, 0.1, 0.01, 0.001], rtol=1e-15)
    assert m == 1.0
    g, m = pa.pa_rope_freqs(8, 10000.0, "linear", 4.0)
    np.testing.assert_array_equal(g, f / 4)
    # the enlarged base: the fastest pair as it was, the slowest divided by the factor
    g, m = pa.pa_rope_freqs(64, 10000.0, "base", 4.0)
    f, _ = pa.pa_rope_freqs(64, 10000.0)
    assert g[0] == f[0] and m == 1.0
    np.testing.assert_allclose(g[-1], f[-1] / 4, rtol=1e-13)
    assert (np.diff(f / g) > 0).all()
    # the ramp and the bands by their own formulas, pair by pair
    R, theta, factor, L, fast, slow = 128, 500000.0, 8.0, 8192.0, 32.0, 1.0
    f, _ = pa.pa_rope_freqs(R, theta)
    g, m = pa.pa_rope_freqs(R, theta, "ramp", factor, L, fast, slow)
    at = lambda turns: R * math.log(L / (2 * math.pi * turns)) / (2 * math.log(theta))
    lo, hi = max(0, math.floor(at(fast))), min(R - 1, math.ceil(at(slow)))
    for i in range(R // 2):
        u = min(1.0, max(0.0, (i - lo) / (hi - lo)))
        assert abs(g[i] - (f[i] * (1 - u) + f[i] / factor * u)) <= 1e-15 * f[i]
    assert abs(m - (0.1 * math.log(factor) + 1)) < 1e-6
    assert g[0] == f[0] and abs(g[-1] * factor - f[-1]) < 1e-15
    g, m = pa.pa_rope_freqs(R, theta, "bands", factor, L, 4.0, 1.0)
    for i in range(R // 2):
        w = 2 * math.pi / f[i]
        u = (L / w - 1.0) / 3.0
        want = f[i] if w < L / 4 else f[i] / factor if w > L else (1 - u) * f[i] / factor + u * f[i]
        assert abs(g[i] - want) <= 1e-14 * f[i]
    assert m == 1.0
    # a context so short that no pair is fast, and one pair only
    g, _ = pa.pa_rope_freqs(2, 10000.0, "ramp", 2.0, 1.0, 32.0, 1.0)
    np.testing.assert_allclose(g, [1.0])
    for bad in (dict(rotary_dim=0), dict(rotary_dim=7), dict(theta=1.0), dict(theta=float("nan")), dict(scaling=9),
                dict(scaling="linear", factor=0.5), dict(scaling="base", factor=2.0, rotary_dim=2),
                dict(scaling="ramp", factor=2.0), dict(scaling="bands", factor=2.0, original_len=10.0, fast=1.0, slow=2.0),
                dict(scaling="ramp", factor=2.0, original_len=10.0, fast=4.0, slow=0.0)):
        with pytest.raises(pa.PaError):
            pa.pa_rope_freqs(**{**dict(rotary_dim=8), **bad})


def test_seq_evict(pa):
    with pa.Pool(12, 4) as pool:
        h = pool.handle
        a = pa.pa_seq_create(h)
        pa.pa_seq_append(h, a, 18)                       # blocks 0..4
        b = pa.pa_seq_fork(h, a)
        assert pa.pa_seq_evict(h, a, 18) is False        # within its budget
        assert pa.pa_seq_table(h, a).tolist() == [0, 1, 2, 3, 4]
        assert pa.pa_seq_evict(h, a, 9) is True
        assert pa.pa_seq_table(h, a).tolist() == [5, 6, 7] and pa.pa_seq_len(h, a) == 9
        # the fork keeps the old blocks, alone now
        assert pa.pa_seq_table(h, b).tolist() == [0, 1, 2, 3, 4]
        assert [pa.pa_block_refcount(h, i) for i in range(8)] == [1] * 8
        assert pa.pa_pool_num_free(h) == 4
        # too few free blocks: refused, nothing changed
        with pytest.raises(pa.PaError) as e:
            pa.pa_seq_evict(h, b, 17)
        assert e.value.status == pa.PA_ERR_OOM
        assert pa.pa_seq_table(h, b).tolist() == [0, 1, 2, 3, 4] and pa.pa_pool_num_free(h) == 4
        # its own blocks go to the back of the free list, in table order
        assert pa.pa_seq_evict(h, b, 5)
        assert pa.pa_seq_table(h, b).tolist() == [8, 9] and pa.pa_pool_num_free(h) == 7
        slots, pairs = pa.pa_seq_append(h, b, 4)         # three in block 9, one in the next free block
        assert slots.tolist() == [37, 38, 39, 40] and len(pairs) == 0
        assert pa.pa_seq_evict(h, b, 0) and pa.pa_seq_table(h, b).tolist() == [] and pa.pa_seq_len(h, b) == 0
        st = pa.pa_pool_get_stats(h)
        assert (st["tokens"], st["used_blocks"], st["shared_blocks"]) == (9, 3, 0)
        for bad, status in (((h, a, -1), pa.PA_ERR_INVALID), ((h, 99, 3), pa.PA_ERR_BAD_INDEX)):
            with pytest.raises(pa.PaError) as e:
                pa.pa_seq_evict(*bad)
            assert e.value.status == status
        pa.pa_pool_set_fail_after(h, 0)
        with pytest.raises(pa.PaError):
            pa.pa_seq_evict(h, a, 3)
        assert pa.pa_seq_len(h, a) == 9


def test_seq_evict_random_stream_keeps_the_counts(pa):
    rng = synth.make_rng(77)
    with pa.Pool(200, 16) as pool:
        h, live = pool.handle, []
        for _ in range(600):
            op = rng.integers(0, 5)
            try:
                if op == 0 or not live:
                    live.append(pa.pa_seq_create(h))
                elif op == 1:
                    pa.pa_seq_append(h, live[rng.integers(len(live))], int(rng.integers(1, 120)))
                elif op == 2:
                    live.append(pa.pa_seq_fork(h, live[rng.integers(len(live))]))
                elif op == 3:
                    s = live[rng.integers(len(live))]
                    keep, n, old = int(rng.integers(0, 150)), pa.pa_seq_len(h, s), set(pa.pa_seq_table(h, s).tolist())
                    changed = pa.pa_seq_evict(h, s, keep)
                    assert changed == (n > keep) and pa.pa_seq_len(h, s) == min(n, keep)
                    table = pa.pa_seq_table(h, s).tolist()
                    assert len(table) == -(-min(n, keep) // 16) and len(set(table)) == len(table)
                    if changed:
                        assert not old & set(table)
                        assert all(pa.pa_block_refcount(h, b) == 1 for b in table)
                else:
                    pa.pa_seq_free(h, live.pop(rng.integers(len(live))))
            except pa.PaError as e:
                assert e.status == pa.PA_ERR_OOM
            uses = np.zeros(200, int)
            for s in live:
                for b in pa.pa_seq_table(h, s):
                    uses[b] += 1
            assert [pa.pa_block_refcount(h, b) for b in range(200)] == uses.tolist()
            assert pa.pa_pool_num_free(h) == int((uses == 0).sum())


def test_seq_evict_batch_takes_no_block_that_the_batch_gave_up(pa):
    """Two evictions for one pa_evict call: the first one's old blocks are still to be copied from."""
    with pa.Pool(12, 16) as pool:
        h = pool.handle
        a, b = pa.pa_seq_create(h), pa.pa_seq_create(h)
        for s in (a, b):
            pa.pa_seq_append(h, s, 64)                   # blocks 0..3 and 4..7
        pa.pa_pool_export(h, [a, b], 4)
        assert pa.pa_seq_evict(h, a, 40)                 # 8, 9, 10; one block left that no eviction gave up
        assert pa.pa_seq_table(h, a).tolist() == [8, 9, 10] and pa.pa_pool_num_free(h) == 5
        with pytest.raises(pa.PaError) as e:
            pa.pa_seq_evict(h, b, 40)
        assert e.value.status == pa.PA_ERR_OOM
        assert pa.pa_seq_table(h, b).tolist() == [4, 5, 6, 7] and pa.pa_seq_len(h, b) == 64
        assert [pa.pa_block_refcount(h, i) for i in range(12)] == [0] * 4 + [1] * 7 + [0]
        assert pa.pa_seq_evict(h, b, 16)                 # what fits beside them is done
        assert pa.pa_seq_table(h, b).tolist() == [11]
        # the tables for pa_evict are out: the next batch may take the blocks that this one gave up
        pa.pa_pool_export(h, [a, b], 4)
        assert pa.pa_seq_evict(h, a, 33) and pa.pa_seq_table(h, a).tolist() == [0, 1, 2]


def test_seq_evict_batch_takes_given_up_blocks_neither_freed_nor_reused(pa):
    """A block given up in the batch stays out of it when a fork, an append or a free puts it through other hands first."""
    with pa.Pool(10, 16) as pool:
        h = pool.handle
        a = pa.pa_seq_create(h)
        pa.pa_seq_append(h, a, 48)                       # 0, 1, 2
        f = pa.pa_seq_fork(h, a)
        b = pa.pa_seq_create(h)
        pa.pa_seq_append(h, b, 64)                       # 3, 4, 5, 6
        assert pa.pa_seq_evict(h, a, 16)                 # 7; its old blocks live on in the fork
        pa.pa_seq_free(h, f)                             # 0, 1, 2 free now
        assert pa.pa_seq_evict(h, b, 32) and pa.pa_seq_table(h, b).tolist() == [8, 9]
        c = pa.pa_seq_create(h)
        pa.pa_seq_append(h, c, 32)                       # another call may take them: 0, 1
        assert pa.pa_seq_table(h, c).tolist() == [0, 1]
        pa.pa_seq_free(h, c)                             # free again, still to be copied from
        for keep in (16, 1):
            with pytest.raises(pa.PaError) as e:
                pa.pa_seq_evict(h, b, keep)
            assert e.value.status == pa.PA_ERR_OOM
        assert pa.pa_pool_num_free(h) == 7


def test_seq_evict_batches_stay_apart_in_a_random_stream(pa):
    rng = synth.make_rng(78)
    with pa.Pool(90, 16) as pool:
        h, live, given, refused = pool.handle, [], set(), 0
        for _ in range(3000):
            op = rng.integers(0, 9)
            try:
                if op == 0 or not live:
                    live.append(pa.pa_seq_create(h))
                elif op <= 2:
                    pa.pa_seq_append(h, live[rng.integers(len(live))], int(rng.integers(1, 200)))
                elif op == 3:
                    live.append(pa.pa_seq_fork(h, live[rng.integers(len(live))]))
                elif op <= 6:
                    s = live[rng.integers(len(live))]
                    keep, old = int(rng.integers(0, 150)), pa.pa_seq_table(h, s).tolist()
                    need, free = -(-keep // 16), {b for b in range(90) if pa.pa_block_refcount(h, b) == 0}
                    if pa.pa_seq_len(h, s) > keep:
                        try:
                            assert pa.pa_seq_evict(h, s, keep)
                        except pa.PaError:
                            assert need > len(free - given) and pa.pa_seq_table(h, s).tolist() == old
                            refused += need <= len(free)
                            continue
                        assert need <= len(free - given)
                        given |= set(old)
                        assert not given & set(pa.pa_seq_table(h, s).tolist())
                elif op == 7:
                    pa.pa_seq_free(h, live.pop(rng.integers(len(live))))
                else:
                    pa.pa_pool_export(h, live, 200)
                    given = set()
            except pa.PaError as e:
                assert e.status == pa.PA_ERR_OOM
        assert refused  # some for want of blocks that no eviction gave up


def test_prefix_cache_refuses_blocks_of_an_evicted_sequence(pa):
    """After an eviction a block's slots hold other tokens for each KV head: they are no prefix of anything."""
    with pa.Pool(40, 4) as pool, pa.Pool(20, 4) as host:
        h = pool.handle
        cache = pa.pa_prefix_cache_create(h)
        tokens = np.arange(100, 140, dtype=np.int32)
        insert = lambda s, n: pa.pa_prefix_insert(cache, tokens[:n], pa.pa_seq_table(h, s))

        def refused(s, n):
            before = [pa.pa_block_refcount(h, b) for b in range(40)], pa.pa_prefix_cached_blocks(cache)
            with pytest.raises(pa.PaError) as e:
                insert(s, n)
            assert e.value.status == pa.PA_ERR_INVALID
            assert before == ([pa.pa_block_refcount(h, b) for b in range(40)], pa.pa_prefix_cached_blocks(cache))

        a = pa.pa_seq_create(h)
        pa.pa_seq_append(h, a, 24)
        assert insert(a, 24) == 6                        # before the eviction, as ever
        assert pa.pa_seq_evict(h, a, 10)
        refused(a, 8)
        pa.pa_seq_append(h, a, 6)                        # new tokens behind the kept ones: the prefix before them is not theirs
        refused(a, 16)
        f = pa.pa_seq_fork(h, a)
        refused(f, 16)
        pa.pa_seq_append(h, f, 2)
        b = pa.pa_seq_create(h)
        pa.pa_seq_append(h, b, 9)
        assert pa.pa_seq_evict(h, b, 3)
        c = pa.pa_seq_fork(h, b)
        _, pairs = pa.pa_seq_append(h, c, 1)             # the shared partial block is copied, what it holds with it
        assert len(pairs) == 1
        refused(c, 4)
        out, _ = pa.pa_seq_swap_out(h, host.handle, c)
        back, _ = pa.pa_seq_swap_in(h, host.handle, out)
        refused(back, 4)
        # nothing kept, or the blocks in other hands: as new ones
        assert pa.pa_seq_evict(h, b, 0)
        pa.pa_seq_append(h, b, 8)
        tokens = tokens + 1000
        assert insert(b, 8) == 2
        for s in (a, f, back):
            pa.pa_seq_free(h, s)
        d = pa.pa_seq_create(h)
        pa.pa_seq_append(h, d, 4 * pa.pa_pool_num_free(h))
        tokens = np.arange(5000, 5200, dtype=np.int32)
        assert insert(d, 200) == len(pa.pa_seq_table(h, d))
        pa.pa_prefix_cache_destroy(cache)


def test_evict_refuses_rows_of_sums_that_its_loops_would_step_past(pa):
    # the kernel walks a row of sums in 32-bit steps of up to 8192
    far = P + (1 << 45)
    for cols in ((1 << 30) + 4, (1 << 31) - 4):
        assert evict(pa, dims(pa), pa.pa_key_sums(P, None, 2, cols), out=far) == pa.PA_ERR_INVALID
    assert evict(pa, dims(pa, num_seqs=0), pa.pa_key_sums(P, None, 2, 1 << 30), out=far) == pa.PA_OK


def test_rope_refuses_queries_written_over_keys_or_values(pa):
    INV, d = pa.PA_ERR_INVALID, dims(pa)
    far = P + (1 << 30)
    # q rows of 1024 bytes, k and v rows of 256
    for bad in (dict(k=far), dict(v=far), dict(k=far + 512), dict(k=far - 128), dict(v=far - 128, vs=512),
                # column ranges of one tensor, 2048 bytes a token: starting in the queries, ending in them, a token later
                dict(os=1024, k=far + 1008, ks=1024), dict(os=1024, v=far - 240, vs=1024),
                dict(os=1024, k=far + 2048 + 16, ks=1024), dict(os=1024, v=far - 2048 - 240, vs=1024)):
        assert rope(pa, d, out=far, **bad) == INV, bad


def test_rope_refuses_blocks_of_more_elements_than_32_bits_hold(pa):
    # the kernel steps from head to head of a block by block_size * head_dim elements, in 32 bits
    for B, D in ((1 << 25, 64), (1 << 24, 128), (1 << 30, 64)):
        assert rope(pa, dims(pa, block_size=B, head_dim=D, num_kv_heads=1, num_q_heads=1, num_blocks=1)) == pa.PA_ERR_INVALID
    assert rope(pa, dims(pa, block_size=(1 << 25) - 1), T=0) == pa.PA_OK
