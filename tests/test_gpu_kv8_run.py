"""GPU tests of the 8-bit cache's calls together, as a serving loop uses them with
the allocator, and of what single calls share: streams, graphs, workspaces, large
pools, every split of rows and heads, extreme windows and scales."""
import math

import numpy as np
import pytest

from gpu_helpers import require_gpu
from kv8_helpers import assert_within, attend_ref, codes_to, dtype_of, make_cache, rotate_ref, tables_for
from paged_kv_cache_127_gb300 import synth

pytestmark = pytest.mark.gpu
I32_MAX = 2 ** 31 - 1


@pytest.fixture(scope="module")
def gpu():
    return require_gpu()


def generator(torch, seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def ints(torch, x, dtype=None):
    return torch.tensor(x, dtype=dtype or torch.int32, device="cuda")


def starts_of(counts):
    return [sum(counts[:i]) for i in range(len(counts) + 1)]


def bits(torch, x):
    return x.contiguous().view(torch.uint8)


@pytest.mark.parametrize("dtype,D,B,Hq,Hkv,window,sinks", [("bf16", 64, 16, 8, 2, 0, 0), ("f16", 128, 32, 8, 4, 40, 4)])
def test_prompts_forks_decode_steps_and_drafts(gpu, dtype, D, B, Hq, Hkv, window, sinks):
    """Prompts of three axes, a fork inside a block, decode steps, drafted tokens, a freed sequence's blocks used again: every
    attention against 64 bits over the cache as it stands, and the cache against the keys and values that went in."""
    torch, pa = gpu
    dt, N, mb, R = dtype_of(torch, dtype), 80, 16, D // 2
    gen = generator(torch, D)
    scale = 1.0 / math.sqrt(D)
    # codes and scales as an earlier user left them
    cache = (torch.full((N, Hkv, B, D), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
             torch.full((N, Hkv, B, D), 0xFF, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
             torch.full((N, Hkv), math.nan, device="cuda"), torch.full((N, Hkv), 2.0 ** 100, device="cuda"))
    c8 = pa.make_cache8(*cache)
    freqs = torch.from_numpy(pa.pa_rope_freqs(R, 10000.0)[0][: R // 2].copy()).cuda()
    rope = pa.make_rope(R, freqs)
    pair_axis = torch.arange(R // 2, device="cuda", dtype=torch.int32) % 3
    axes = pa.make_axes(3, pair_axis)
    pool = pa.Pool(N, B, synth.free_order(synth.make_rng(5), N))
    h = pool.handle
    keys, vals = {}, {}     # per sequence, the (turned) keys and the values in 64 bits, [tokens, Hkv, D]

    def step(seqs, n, loud=1.0, decode=False):
        """n new tokens for each sequence: append, copy, turn and write, attend."""
        slots, pairs = pa.pa_seq_append_batch(h, seqs, n)
        lens = [pa.pa_seq_len(h, s) for s in seqs]
        T = len(seqs) * n
        dims = pa.make_dims(len(seqs), Hq, Hkv, D, B, N, mb, 0, dtype)
        if len(pairs):
            pa.pa_copy_pairs_check(pairs, N)
            pa.pa_copy_blocks8(dims, c8, torch.from_numpy(pairs).cuda())
        x = (loud * torch.randn(T, Hq + 2 * Hkv, D, generator=gen, device="cuda")).to(dt)
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        pos = torch.randint(0, 5000, (3, T), generator=gen, device="cuda", dtype=torch.int32)
        k64 = rotate_ref(torch, k, pos, pair_axis, freqs, R, False, 1.0)
        q_out = torch.empty(T, Hq, D, dtype=dt, device="cuda")
        pa.pa_rope_write_kv8(dims, rope, axes, q, k, v, pos, ints(torch, slots.reshape(-1).tolist(), torch.int64), q_out, c8)
        for i, s in enumerate(seqs):
            keys[s] = torch.cat([keys[s][: lens[i] - n], k64[i * n:(i + 1) * n]])
            vals[s] = torch.cat([vals[s][: lens[i] - n], v[i * n:(i + 1) * n].double()])
        tables = torch.full((len(seqs), mb), -1, dtype=torch.int32, device="cuda")
        for i, s in enumerate(seqs):
            t = pa.pa_seq_table(h, s)
            tables[i, : len(t)] = torch.from_numpy(np.array(t, dtype=np.int32)).cuda()
        out = torch.full((T, Hq, D), math.nan, dtype=dt, device="cuda")
        if decode:
            ws = torch.empty(pa.pa_decode8_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
            pa.pa_decode8(dims, q_out, c8, tables, ints(torch, lens), scale, out, ws, window=window, sinks=sinks)
        else:
            ws = torch.empty(pa.pa_chunk8_workspace_bytes(dims, T, n), dtype=torch.uint8, device="cuda")
            pa.pa_chunk8(dims, q_out, c8, tables, ints(torch, lens), ints(torch, starts_of([n] * len(seqs))), scale, out, n, ws,
                         window=window, sinks=sinks)
        ref, bound = attend_ref(torch, q_out, cache, tables, lens, [n] * len(seqs), scale, window, sinks)
        assert_within(out, ref, bound, dtype)
        # a stored value: rounded once (2^-4, or 2^-10 of the scale it was written at), and off by 2^-10 of each larger scale it
        # was brought to, powers of two that end at the block's: 2^-9 of that in all.  A turned key is within 2^-20 of its pair.
        for i, s in enumerate(seqs):
            blocks = tables[i, : -(-lens[i] // B)].long()
            for codes, sc, want in ((cache[0], cache[2], keys[s]), (cache[1], cache[3], vals[s])):
                have = (codes_to(torch, codes[blocks].view(torch.uint8)) * sc[blocks].double()[:, :, None, None]).transpose(1, 2).flatten(0, 1)[: lens[i]]
                unit = sc[blocks].double()[:, None].expand(-1, B, -1).flatten(0, 1)[: lens[i]][..., None]
                assert bool(((have - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -9 * unit + 2.0 ** -20 * 448 * unit).all())

    def new(fork=None):
        s = pa.pa_seq_create(h) if fork is None else pa.pa_seq_fork(h, fork)
        keys[s] = torch.zeros(0, Hkv, D, dtype=torch.float64, device="cuda") if fork is None else keys[fork]
        vals[s] = keys[s] if fork is None else vals[fork]
        return s

    a, b = new(), new()
    step([a], 85)
    step([b], 23)
    f = new(a)                                # shares its last, half-filled block with a
    for loud in (1.0, 0.01, 30.0, 1.0):       # the fork's copies and a's block part ways, scales grow
        step([f, a, b], 1, loud, decode=True)
    step([b, f], 5, 3.0)                      # drafted tokens
    pa.pa_seq_free(h, a)
    c = new()
    step([c], 70, 100.0)                      # over a's blocks
    for _ in range(3):
        step([c, f, b], 1, decode=True)
    step([f, c], 70)
    assert pa.pa_device_errors(clear=True) == 0
    pool.close()


def test_rejected_drafts_are_written_over(gpu):
    """An append that goes back: what lies behind the new tokens is void, what lies before them stays."""
    torch, pa = gpu
    gen = generator(torch, 3)
    D, B, Hkv, N = 64, 16, 2, 4
    cache = make_cache(torch, gen, N, Hkv, B, D)
    dims = pa.make_dims(1, 8, Hkv, D, B, N, 2, 0, "bf16")
    c8 = pa.make_cache8(*cache)
    x = torch.randn(20, Hkv, D, generator=gen, device="cuda").to(torch.bfloat16)
    slots = ints(torch, [16 + i for i in range(16)] + [48 + i for i in range(4)], torch.int64)   # blocks 1, 3
    pa.pa_write_kv8(dims, x, x, slots, c8)
    pa.pa_write_kv8(dims, 4 * x[:6], x[:6], slots[10:16], c8)                                     # again from token 10 on
    have = codes_to(torch, cache[1][1].view(torch.uint8)) * cache[3][1].double()[:, None, None]
    want = torch.cat([x[:10], x[:6]]).double().transpose(0, 1)
    unit = cache[3][1].double()[:, None, None]
    assert bool(((have - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -9 * unit).all())
    have = codes_to(torch, cache[0][1].view(torch.uint8)) * cache[2][1].double()[:, None, None]
    want = torch.cat([x[:10], 4 * x[:6]]).double().transpose(0, 1)
    unit = cache[2][1].double()[:, None, None]
    assert bool(((have - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -9 * unit).all())


def test_write8_one_slot_many_times(gpu):
    """A slot given many times voids its block, and nothing else."""
    torch, pa = gpu
    gen = generator(torch, 4)
    D, B, Hkv, N = 128, 32, 4, 9
    cache = make_cache(torch, gen, N, Hkv, B, D)
    was = [bits(torch, c).clone() for c in cache]
    x = torch.randn(200, Hkv, D, generator=gen, device="cuda").to(torch.float16)
    dims = pa.make_dims(1, 4, Hkv, D, B, N, 2, 0, "f16")
    pa.pa_write_kv8(dims, x, x, torch.full((200,), 5 * B + 7, dtype=torch.int64, device="cuda"), pa.make_cache8(*cache))
    torch.cuda.synchronize()
    for c, w in zip(cache, was):
        now = bits(torch, c)
        others = [i for i in range(N) if i != 5]
        assert torch.equal(now.view(N, -1)[others], w.view(N, -1)[others])
    assert pa.pa_device_errors(clear=True) == 0


class Bench:
    """A batch over one cache, its call and its reference."""

    def __init__(self, torch, pa, seed, nq, dtype="bf16", D=64, B=16, Hq=8, Hkv=2, S=4, window=0, sinks=0):
        gen = generator(torch, seed)
        self.torch, self.pa, self.nq, self.dtype, self.args = torch, pa, nq, dtype, (window, sinks)
        self.lens = [nq + int(x) for x in torch.randint(1, 700, (S,), generator=gen, device="cuda")]
        self.counts = [nq] * S
        self.tables, N = tables_for(torch, gen, self.lens, B)
        self.cache = make_cache(torch, gen, N, Hkv, B, D)
        self.c8 = pa.make_cache8(*self.cache)
        self.q = torch.randn(S * nq, Hq, D, generator=gen, device="cuda").to(dtype_of(torch, dtype))
        self.dims = pa.make_dims(S, Hq, Hkv, D, B, N, self.tables.shape[1], 0, dtype)
        self.dl, self.qs = ints(torch, self.lens), ints(torch, starts_of(self.counts))
        self.scale = 0.11
        self.out = torch.full((S * nq, Hq, D), math.nan, device="cuda")
        self.ws = self.workspace()

    def workspace(self):
        n = (self.pa.pa_decode8_workspace_bytes(self.dims) if self.nq == 1 else
             self.pa.pa_chunk8_workspace_bytes(self.dims, len(self.q), self.nq))
        return self.torch.full((n,), 255, dtype=self.torch.uint8, device="cuda")

    def call(self, out=None, ws=None, **kw):
        out, ws = self.out if out is None else out, self.ws if ws is None else ws
        w, s = self.args
        if self.nq == 1:
            return self.pa.pa_decode8(self.dims, self.q, self.c8, self.tables, self.dl, self.scale, out, ws, window=w, sinks=s, **kw)
        return self.pa.pa_chunk8(self.dims, self.q, self.c8, self.tables, self.dl, self.qs, self.scale, out, self.nq, ws,
                                 window=w, sinks=s, **kw)

    def check(self, out):
        ref, bound = attend_ref(self.torch, self.q, self.cache, self.tables, self.lens, self.counts, self.scale, *self.args)
        assert_within(out, ref, bound, "f32")


@pytest.mark.parametrize("nq", [1, 5, 90])
def test_attend8_on_two_streams_at_once(gpu, nq):
    torch, pa = gpu
    cases = [Bench(torch, pa, 70 + i, nq, S=20) for i in range(2)]
    want = []
    for c in cases:
        c.call()
        want.append(c.out.clone())
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = [[torch.full_like(c.out, math.nan) for _ in range(8)] for c in cases]
    torch.cuda.synchronize()
    for i in range(8):
        for c, o, st in zip(cases, outs, streams):
            c.call(o[i], stream=st)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(x, w) for x in o)
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("nq", [1, 5, 90])
def test_prepared_attend8_is_the_call(gpu, nq):
    torch, pa = gpu
    c = Bench(torch, pa, 80 + nq, nq, window=100, sinks=9)
    c.call()
    c.check(c.out)
    out = torch.full_like(c.out, math.nan)
    run = c.call(out, prepare=True)
    assert bool(out.isnan().all())
    for _ in range(3):
        run()
        torch.cuda.synchronize()
        assert torch.equal(out, c.out)
        out.fill_(math.nan)


@pytest.mark.parametrize("nq,dtype", [(1, "bf16"), (4, "f16"), (80, "bf16")])
def test_captured_step_is_the_eager_one(gpu, nq, dtype):
    """Copy, write and attention in one graph, replayed on inputs that change under it."""
    torch, pa = gpu
    D, B, Hq, Hkv, S = 128, 16, 8, 2, 3
    dt = dtype_of(torch, dtype)
    gen = generator(torch, 90 + nq)
    most = [400, 300, 200]
    tables, N = tables_for(torch, gen, most, B)
    start = make_cache(torch, gen, N, Hkv, B, D)
    T = S * nq
    freqs = torch.from_numpy(pa.pa_rope_freqs(D, 10000.0)[0].copy()).cuda()
    rope = pa.make_rope(D, freqs)

    class State:
        pass

    def state():
        s = State()
        s.cache = tuple(c.clone() for c in start)
        s.x = torch.zeros(T, Hq + 2 * Hkv, D, dtype=dt, device="cuda")
        s.pos, s.slots = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.full((T,), -1, dtype=torch.int64, device="cuda")
        s.lens, s.pairs = torch.full((S,), nq, dtype=torch.int32, device="cuda"), torch.zeros(1, 2, dtype=torch.int64, device="cuda")
        s.q, s.out = torch.zeros(T, Hq, D, dtype=dt, device="cuda"), torch.zeros(T, Hq, D, dtype=dt, device="cuda")
        s.dims = pa.make_dims(S, Hq, Hkv, D, B, N, tables.shape[1], 0, dtype)
        s.qs = ints(torch, starts_of([nq] * S))
        n = pa.pa_decode8_workspace_bytes(s.dims) if nq == 1 else pa.pa_chunk8_workspace_bytes(s.dims, T, nq)
        s.ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        return s

    def run(s):
        c8 = pa.make_cache8(*s.cache)
        pa.pa_copy_blocks8(s.dims, c8, s.pairs)
        pa.pa_rope_write_kv8(s.dims, rope, None, s.x[:, :Hq], s.x[:, Hq:Hq + Hkv], s.x[:, Hq + Hkv:], s.pos, s.slots, s.q, c8)
        if nq == 1:
            pa.pa_decode8(s.dims, s.q, c8, tables, s.lens, 0.1, s.out, s.ws, window=150, sinks=4)
        else:
            pa.pa_chunk8(s.dims, s.q, c8, tables, s.lens, s.qs, 0.1, s.out, nq, s.ws, window=150, sinks=4)

    eager, held = state(), state()
    run(held)                       # everything is loaded before the capture
    for c, w in zip(held.cache, start):
        c.copy_(w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run(held)
    torch.cuda.synchronize()
    for c, w in zip(held.cache, start):
        assert torch.equal(bits(torch, c), bits(torch, w)), "a captured call ran"
    length = [150, 17, 100]
    for turn in range(4):
        length = [n + nq if n + nq <= m else nq for n, m in zip(length, most)]
        slots = [int(tables[s, p // B]) * B + p % B for s in range(S) for p in range(length[s] - nq, length[s])]
        x = torch.randn(T, Hq + 2 * Hkv, D, generator=gen, device="cuda").to(dt)
        for s in (eager, held):
            s.x.copy_(x)
            s.slots.copy_(ints(torch, slots, torch.int64))
            s.pos.copy_(ints(torch, [p for s_ in range(S) for p in range(length[s_] - nq, length[s_])]))
            s.lens.copy_(ints(torch, length))
            s.pairs.copy_(ints(torch, [[int(tables[0, 0]), N - 1]], torch.int64))
        run(eager)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(torch, eager.out), bits(torch, held.out)), turn
        assert all(torch.equal(bits(torch, c), bits(torch, w)) for c, w in zip(eager.cache, held.cache)), turn
        ref, bound = attend_ref(torch, held.q, held.cache, tables, length, [nq] * S, 0.1, 150, 4)
        assert_within(held.out, ref, bound, dtype)
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("f16", 64), ("f16", 128)])
@pytest.mark.parametrize("Hkv", [3, 2, 4])
def test_every_split_of_rows_and_heads(gpu, dtype, D, Hkv):
    """Rows of a KV head in each of the kernel's shapes, KV heads in ones, twos and fours; a second group of heads."""
    torch, pa = gpu
    B = 16 if D == 64 else 32
    for Hkv_ in (Hkv, 2 * Hkv if Hkv != 2 else 6):
        for nq in (1, 7, 16, 24, 32, 45, 63, 64, 129):
            for window, sinks in ((0, 0), (50, 20)):
                c = Bench(torch, pa, nq + D, nq, dtype, D, B, Hkv_, Hkv_, 3, window, sinks)
                c.call()
                c.check(c.out)
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("nq", [1, 6, 70])
def test_windows_and_sinks_of_any_size(gpu, nq):
    torch, pa = gpu
    c = Bench(torch, pa, 120 + nq, nq)
    c.call()
    whole = c.out.clone()
    c.check(whole)
    for window, sinks in ((I32_MAX, 0), (I32_MAX, I32_MAX), (1, I32_MAX), (I32_MAX - 31, 5), (2 ** 20, 0)):
        c.args = (window, sinks)
        c.out.fill_(math.nan)
        c.call()
        c.args = (0, 0)
        c.check(c.out)
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("nq", [1, 9, 70])
@pytest.mark.parametrize("k_exp,v_exp,scale", [((-80, -75), (-80, -25), 0.1 * 2.0 ** 70), ((100, 104), (65, 119), 2.0 ** -108),
                                               ((-9, -6), (-30, 30), 0.1)])
def test_scales_at_the_ends_of_their_range(gpu, nq, k_exp, v_exp, scale):
    torch, pa = gpu
    gen = generator(torch, nq)
    D, B, Hq, Hkv = 128, 16, 8, 2
    lens = [nq + 400]
    tables, N = tables_for(torch, gen, lens, B)
    k, v, _, _ = make_cache(torch, gen, N, Hkv, B, D)
    ks = torch.exp2(torch.randint(k_exp[0], k_exp[1] + 1, (N, Hkv), generator=gen, device="cuda").float())
    vs = torch.exp2(torch.randint(v_exp[0], v_exp[1] + 1, (N, Hkv), generator=gen, device="cuda").float())
    q = torch.randn(nq, Hq, D, generator=gen, device="cuda").to(torch.bfloat16)
    dims = pa.make_dims(1, Hq, Hkv, D, B, N, tables.shape[1], 0, "bf16")
    out = torch.full((nq, Hq, D), math.nan, device="cuda")
    c8 = pa.make_cache8(k, v, ks, vs)
    if nq == 1:
        ws = torch.empty(pa.pa_decode8_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
        pa.pa_decode8(dims, q, c8, tables, ints(torch, lens), scale, out, ws)
    else:
        ws = torch.empty(pa.pa_chunk8_workspace_bytes(dims, nq, nq), dtype=torch.uint8, device="cuda")
        pa.pa_chunk8(dims, q, c8, tables, ints(torch, lens), ints(torch, [0, nq]), scale, out, nq, ws)
    ref, bound = attend_ref(torch, q, (k, v, ks, vs), tables, lens, [nq], scale)
    assert_within(out, ref, bound, "f32")


def test_pools_past_32_bits_of_codes(gpu):
    """More than 2^32 bytes of codes: the write, the copy and every attention at the pool's far end."""
    torch, pa = gpu
    gen = generator(torch, 8)
    D, B, Hq, Hkv = 128, 16, 16, 8
    N = 2 ** 32 // (Hkv * B * D) + 500
    codes = [torch.empty(N, Hkv, B, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.full((N, Hkv), math.nan, device="cuda") for _ in range(2)]
    c8 = pa.make_cache8(codes[0], codes[1], scales[0], scales[1])
    n = 300
    columns = -(-n // B)
    # the first and the last blocks, in turn; the very last block among them
    ids = [N - 1 - i // 2 if i % 2 == 0 else i for i in range(columns)]
    tables = ints(torch, [ids])
    x = torch.randn(n, Hq + 2 * Hkv, D, generator=gen, device="cuda").to(torch.bfloat16)
    slots = ints(torch, [ids[p // B] * B + p % B for p in range(n)], torch.int64)
    dims = pa.make_dims(1, Hq, Hkv, D, B, N, columns, 0, "bf16")
    freqs = torch.from_numpy(pa.pa_rope_freqs(D, 10000.0)[0].copy()).cuda()
    q = torch.empty(n, Hq, D, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    pa.pa_rope_write_kv8(dims, pa.make_rope(D, freqs), None, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], pos, slots, q, c8)
    small = [torch.cat([c.view(torch.uint8)[ids]]).view(torch.float8_e4m3fn) for c in codes] + [s[ids] for s in scales]
    near = ints(torch, [list(range(columns))])
    k64 = rotate_ref(torch, x[:, Hq:Hq + Hkv], pos[None], torch.zeros(D // 2, dtype=torch.int32, device="cuda"), freqs, D, False, 1.0)
    have = (codes_to(torch, small[0].view(torch.uint8)) * small[2].double()[:, :, None, None]).transpose(1, 2).flatten(0, 1)[:n]
    unit = small[2].double()[:, None].expand(-1, B, -1).flatten(0, 1)[:n][..., None]
    assert bool(((have - k64).abs() <= 2.0 ** -4 * k64.abs() + (2.0 ** -10 + 2.0 ** -20 * 448) * unit).all())
    for nq in (1, 6, 100):
        rows = q[n - nq:].contiguous()
        out = torch.full((nq, Hq, D), math.nan, device="cuda")
        if nq == 1:
            ws = torch.empty(pa.pa_decode8_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
            pa.pa_decode8(dims, rows, c8, tables, ints(torch, [n]), 0.09, out, ws)
        else:
            ws = torch.empty(pa.pa_chunk8_workspace_bytes(dims, nq, nq), dtype=torch.uint8, device="cuda")
            pa.pa_chunk8(dims, rows, c8, tables, ints(torch, [n]), ints(torch, [0, nq]), 0.09, out, nq, ws)
        ref, bound = attend_ref(torch, rows, small, near, [n], [nq], 0.09)
        assert_within(out, ref, bound, "f32")
    pa.pa_copy_blocks8(dims, c8, ints(torch, [[N - 1, N // 2], [ids[1], N - 400]], torch.int64))
    torch.cuda.synchronize()
    for c, s in zip(codes, scales):
        for src, dst in ((N - 1, N // 2), (ids[1], N - 400)):
            assert torch.equal(c.view(torch.uint8)[dst], c.view(torch.uint8)[src]) and torch.equal(s[dst], s[src])
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("dtype,D,B,Hq,Hkv", [("bf16", 128, 16, 32, 8), ("f16", 64, 32, 4, 4), ("bf16", 64, 16, 8, 1), ("f16", 128, 32, 2, 1)])
@pytest.mark.parametrize("lens,counts", [([5000], [160]), ([4100, 77, 2500], [70, 0, 200]), ([300, 64, 900], [150, 64, 129]),
                                         ([9000, 150], [64, 64]), ([12, 40], [12, 0])])
def test_chunks_whose_keys_are_shared_out(gpu, dtype, D, B, Hq, Hkv, lens, counts):
    """Few rows over many keys (or a table that could hold many): pieces of items, whole ones and their joins."""
    torch, pa = gpu
    gen = generator(torch, sum(lens) + D)
    tables, N = tables_for(torch, gen, lens, B, columns=400)
    T, most = sum(counts), max(max(counts), 64)
    q = (2 * torch.randn(T + 2, Hq, D, generator=gen, device="cuda")).to(dtype_of(torch, dtype))
    cache = make_cache(torch, gen, N, Hkv, B, D, odd_scales=True)
    dims = pa.make_dims(len(lens), Hq, Hkv, D, B, N, tables.shape[1], 0, dtype)
    c8 = pa.make_cache8(*cache)
    for window, sinks in ((0, 0), (3000, 100), (2000, 2500)):
        ref, bound = attend_ref(torch, q[:T], cache, tables, lens, counts, 0.09, window, sinks)
        for out_dtype in ("f32", dtype):
            outs = []
            for fill in (255, 0):
                out = torch.full((T + 2, Hq, D), math.nan, dtype=dtype_of(torch, out_dtype), device="cuda")
                ws = torch.full((pa.pa_chunk8_workspace_bytes(dims, T + 2, most),), fill, dtype=torch.uint8, device="cuda")
                pa.pa_chunk8(dims, q, c8, tables, ints(torch, lens), ints(torch, starts_of(counts)), 0.09, out, most, ws,
                             window=window, sinks=sinks)
                torch.cuda.synchronize()
                assert_within(out[:T], ref, bound, out_dtype)
                assert bool(out[T:].isnan().all()), "rows behind the last sequence"
                outs.append(out[:T])
            assert torch.equal(outs[0], outs[1]), "the same call gives the same bits"
    assert pa.pa_device_errors(clear=True) == 0
    # blocks that are not there, and an order that is none
    gone = [(0, 0)] + ([(0, 3), (0, 100)] if lens[0] > 101 * B else [])
    for s, c in gone:
        tables[s, c] = N + c
    ref, bound = attend_ref(torch, q[:T], cache, tables, lens, counts, 0.09, bad=gone)
    pa.pa_chunk8(dims, q, c8, tables, ints(torch, lens), ints(torch, starts_of(counts)), 0.09, out, most, ws)
    assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_BAD_BLOCK
    assert_within(out[:T], ref, bound, dtype)
    out.fill_(math.nan)
    pa.pa_chunk8(dims, q, c8, tables, ints(torch, lens), ints(torch, [1] + [0] * len(lens)), 0.09, out, most, ws)
    assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_BAD_LEN
    assert bool(out.isnan().all())


@pytest.mark.parametrize("nq", [1, 3, 80])
def test_binding_refuses_what_the_calls_cannot_take(gpu, nq):
    torch, pa = gpu
    c = Bench(torch, pa, 7, nq)
    good = {"q": c.q, "tables": c.tables, "dl": c.dl, "qs": c.qs, "c8": c.c8, "ws": c.ws, "out": c.out}
    k, v, ks, vs = c.cache
    two = lambda x: torch.cat([x, x], -1)[..., : x.shape[-1]]      # the right shape, other strides
    bad = [("q", c.q[:-1]), ("q", c.q.float()), ("q", c.q.cpu()), ("q", two(c.q)), ("tables", c.tables[:, :-1]),
           ("tables", c.tables.long()), ("tables", c.tables.cpu()), ("tables", two(c.tables)), ("dl", c.dl[:-1]), ("dl", c.dl.long()),
           ("dl", c.dl.cpu()), ("out", c.out[:-1]), ("out", c.out.double()), ("out", two(c.out)), ("out", c.out.cpu()),
           ("ws", None), ("ws", c.ws.cpu()), ("ws", c.ws[::2]), ("c8", pa.make_cache8(k[:-1], v, ks, vs)),
           ("c8", pa.make_cache8(k.view(torch.uint8), v, ks, vs)), ("c8", pa.make_cache8(k, v.cpu(), ks, vs)),
           ("c8", pa.make_cache8(k, v, ks.double(), vs)), ("c8", pa.make_cache8(k, v, ks, vs[:, :1])), ("c8", pa.make_cache8(k, v, ks, two(vs)))]
    if nq > 1:
        bad += [("qs", c.qs[:-1]), ("qs", c.qs.long()), ("qs", c.qs.cpu())]
    for name, x in bad:
        for key, value in good.items():
            setattr(c, key, value)
        setattr(c, name, x)
        if name == "ws" and x is None:
            with pytest.raises(ValueError):
                if nq == 1:
                    pa.pa_decode8(c.dims, c.q, c.c8, c.tables, c.dl, c.scale, c.out)
                else:
                    pa.pa_chunk8(c.dims, c.q, c.c8, c.tables, c.dl, c.qs, c.scale, c.out, nq)
        else:
            with pytest.raises(ValueError):
                c.call()
    for key, value in good.items():
        setattr(c, key, value)
    for ws in (c.ws[:256], c.ws[16:]):
        with pytest.raises(pa.PaError):
            c.call(ws=ws)
    c.call()
    c.check(c.out)
    x = torch.zeros(5, 2, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(5, 8, 64, dtype=torch.bfloat16, device="cuda")
    slots, pos = torch.arange(5, device="cuda"), torch.zeros(5, dtype=torch.int32, device="cuda")
    freqs = torch.zeros(32, dtype=torch.float64, device="cuda")
    rope, axes = pa.make_rope(64, freqs), pa.make_axes(2, torch.zeros(32, dtype=torch.int32, device="cuda"))
    for args in ((rope, None, q, x, x, pos[:-1], slots, q), (rope, None, q, x, x, pos.long(), slots, q), (rope, None, q, x, x, pos, slots.int(), q),
                 (rope, None, q, x, x, pos, slots[:, None], q), (rope, None, q, x, x, pos.cpu(), slots, q), (rope, axes, q, x, x, pos, slots, q),
                 (rope, None, q, x, q, pos, slots, q), (rope, None, q, x[:4], x, pos, slots, q), (rope, None, x, x, x, pos, slots, q),
                 (rope, None, q, x, x, pos, slots, q.float()), (pa.make_rope(64, freqs[:-1]), None, q, x, x, pos, slots, q),
                 (rope, pa.make_axes(1, axes.pair_axis[:-1]), q, x, x, pos[None], slots, q)):
        with pytest.raises(ValueError):
            pa.pa_rope_write_kv8(c.dims, *args, c.c8)
        with pytest.raises(ValueError):
            pa.pa_rope_axes_write_kv(c.dims, *args, torch.zeros(k.shape, dtype=torch.bfloat16, device="cuda"),
                                     torch.zeros(k.shape, dtype=torch.bfloat16, device="cuda"))
    for args in ((x, x, slots.int()), (x[:4], x, slots), (x, q, slots), (x, x.float(), slots)):
        with pytest.raises(ValueError):
            pa.pa_write_kv8(c.dims, *args, c.c8)
    for pairs in (slots, torch.zeros(2, 2, dtype=torch.int32, device="cuda"), torch.zeros(2, 3, dtype=torch.int64, device="cuda")):
        with pytest.raises(ValueError):
            pa.pa_copy_blocks8(c.dims, c.c8, pairs)


@pytest.mark.parametrize("nq", [1, 6, 90])
@pytest.mark.parametrize("B", [16, 32])
def test_every_id_that_is_no_block_is_flagged(gpu, nq, B):
    torch, pa = gpu
    c = Bench(torch, pa, 31 + nq, nq, B=B, S=2)
    for bad in (-1, -2, -3, len(c.cache[0]), 2 ** 31 - 1, -2 ** 31):
        for place in (0, (c.lens[1] - 1) // B):
            was = int(c.tables[1, place])
            c.tables[1, place] = bad
            c.call()
            assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_BAD_BLOCK, (bad, place)
            ref, bound = attend_ref(torch, c.q, c.cache, c.tables, c.lens, c.counts, c.scale, bad=[(1, place)])
            assert_within(c.out, ref, bound, "f32")
            c.tables[1, place] = was
    c.call()
    assert pa.pa_device_errors(clear=True) == 0
    c.check(c.out)
