"""GPU tests of the scored, rotary and eviction calls together, as a serving loop
uses them with the allocator, and of what single calls share: streams, graphs,
workspaces, large pools."""
import math

import numpy as np
import pytest

from gpu_helpers import require_gpu, to_dev, to_host
from paged_helpers import widen
from paged_kv_cache_127_gb300 import synth
from scored_helpers import assert_rows_close, kept_tokens, rotate, scored_rows, weight_error

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gpu():
    return require_gpu()


def test_prompt_decode_evict_decode_chunk(gpu):
    """A prompt, decode steps that collect sums, an eviction of one of three
    sequences (one forked), more steps, and a chunk of drafted tokens, each
    attention compared with fp64 over the tokens that should be there."""
    torch, pa = gpu
    rng = synth.make_rng(11000)
    dtype, Hq, Hkv, D, B, R, N, mb = "bf16", 8, 2, 64, 16, 32, 64, 12
    G, scale, cap, keep, recent = Hq // Hkv, 1 / math.sqrt(D), 8.0, 40, 12
    cols = mb * B
    pool = pa.Pool(N, B, synth.free_order(rng, N))
    h = pool.handle
    kc, vc = (torch.zeros(N, Hkv, B, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    freqs, mscale = pa.pa_rope_freqs(R, 10000.0, "ramp", 4.0, 64.0, 8.0, 1.0)
    rope = pa.make_rope(R, torch.from_numpy(freqs).cuda(), False, mscale)
    score = pa.make_score(softcap=cap)
    sums = torch.zeros(4, Hkv, cols, device="cuda")
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()
    # the model on the host: for each sequence and KV head the (key, value) rows and sums in order
    keys, vals, host_sums, position = {}, {}, {}, {}

    def write(seqs, n_each):
        """Append n_each tokens to each sequence: rotate, write, mirror.  Returns the rotated queries."""
        slots, pairs = pa.pa_seq_append_batch(h, seqs, n_each)
        T = len(seqs) * n_each
        x = synth.normal(rng, (T, Hq + 2 * Hkv, D), 1.0, dtype)
        pos = np.concatenate([np.arange(position[s], position[s] + n_each) for s in seqs])
        dims = pa.make_dims(len(seqs), Hq, Hkv, D, B, N, mb, 0, dtype)
        if len(pairs):
            pa.pa_copy_pairs_check(pairs, N)
            pa.pa_copy_blocks(dims, kc, vc, torch.from_numpy(pairs).cuda())
        dx = to_dev(torch, x, dtype)
        q = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
        pa.pa_rope_write_kv(dims, rope, dx[:, :Hq], dx[:, Hq:Hq + Hkv], dx[:, Hq + Hkv:], i32(pos),
                            torch.from_numpy(slots.reshape(-1).copy()).cuda(), q, kc, vc)
        k64, _ = rotate(widen(x[:, Hq:Hq + Hkv], dtype), pos, freqs, R, False, mscale)
        got = to_host(kc, dtype)
        for i, s in enumerate(seqs):
            for t in range(n_each):
                row = i * n_each + t
                b, o = divmod(int(slots[i, t]), B)
                stored = widen(got[b, :, o], dtype)      # the rounded keys are what attention reads
                assert np.abs(stored - k64[row]).max() <= 2.0 ** -8 * np.abs(k64[row]).max() + 1e-5
                for kh in range(Hkv):
                    keys[s][kh].append(stored[kh])
                    vals[s][kh].append(widen(x[row, Hq + Hkv + kh], dtype))
                    host_sums[s][kh].append(0.0)
            position[s] += n_each
        return q

    def new_seq(fork=None):
        s = pa.pa_seq_create(h) if fork is None else pa.pa_seq_fork(h, fork)
        for d in (keys, vals):
            d[s] = [[] for _ in range(Hkv)] if fork is None else [list(r) for r in d[fork]]
        host_sums[s] = [[0.0] * len(r) for r in keys[s]]
        position[s] = position[fork] if fork is not None else 0
        return s

    def reference(s, q_rows, causal):
        """q_rows [n, Hq, D] of the last n tokens of s, each KV head over its own tokens."""
        n = q_rows.shape[0]
        out, w, E, vmax = np.zeros((n, Hq, D)), [], 0.0, 0.0
        for kh in range(Hkv):
            K, V = np.array(keys[s][kh])[:, None], np.array(vals[s][kh])[:, None]
            L = K.shape[0]
            pos = np.arange(L - n, L)
            o, p, d = scored_rows(q_rows[:, kh * G:(kh + 1) * G], K, V, pos, np.zeros(n, int),
                                  pos + 1 if causal else np.full(n, L), scale, cap)
            out[:, kh * G:(kh + 1) * G] = o
            w.append(p[-1].sum(0))
            E, vmax = max(E, weight_error(dtype, d, L)), max(vmax, np.abs(V).max())
        return out, w, E, vmax

    rows = {}

    def decode(seqs):
        q = write(seqs, 1)
        tables, lens = pa.pa_pool_export(h, seqs, mb, -1)
        dims = pa.make_dims(len(seqs), Hq, Hkv, D, B, N, mb, 0, dtype)
        ws = torch.empty(pa.pa_decode_scored_workspace_bytes(dims, True), dtype=torch.uint8, device="cuda")
        out = torch.empty(len(seqs), Hq, D, device="cuda")
        pa.pa_decode_scored(dims, score, q, kc, vc, i32(tables), i32(lens), scale, out, ws, key_sums=sums,
                            sum_rows=i32([rows[s] for s in seqs]))
        q64, got = widen(to_host(q, dtype), dtype), out.cpu().numpy()
        for i, s in enumerate(seqs):
            ref, w, E, vmax = reference(s, q64[i:i + 1], False)
            assert_rows_close(got[i:i + 1], ref, dtype, "f32", E, vmax)
            for kh in range(Hkv):
                host_sums[s][kh] = [a + b for a, b in zip(host_sums[s][kh], w[kh])]
                have = sums[rows[s], kh].cpu().numpy()
                np.testing.assert_allclose(have[:len(w[kh])], host_sums[s][kh], rtol=1e-4, atol=1e-6)
                assert (have[len(w[kh]):] == 0).all()

    a = new_seq()
    write([a], 37)
    b = new_seq(fork=a)                      # shares three blocks with a, the last partial
    c = new_seq()
    write([c], 5)
    rows.update({a: 2, b: 0, c: 3})
    for _ in range(30):
        decode([a, b, c])                    # a and b: 67 tokens, c: 35
    for _ in range(3):
        decode([c, a])
    # evict a (70 tokens) down to 40; b keeps the blocks they share
    before = {s: to_host(kc, dtype)[pa.pa_seq_table(h, s)] for s in (b, c)}
    seqs = [c, a, b]
    old_tables, lens = pa.pa_pool_export(h, seqs, mb, -1)
    budget = [100, keep, 100]
    assert [pa.pa_seq_evict(h, s, k) for s, k in zip(seqs, budget)] == [False, True, False]
    new_tables, new_lens = pa.pa_pool_export(h, seqs, mb, -1)
    dims = pa.make_dims(3, Hq, Hkv, D, B, N, mb, 0, dtype)
    ws = torch.empty(pa.pa_evict_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    dev_lens = i32([0, 0, 0])
    used = sums.cpu().numpy()
    pa.pa_evict(dims, kc, vc, i32(old_tables), i32(lens), i32(new_tables), i32(budget), recent, sums, sums, dev_lens, ws,
                sum_rows=i32([rows[s] for s in seqs]))
    assert dev_lens.tolist() == new_lens.tolist() == [38, keep, 67]
    for kh in range(Hkv):
        kept = kept_tokens(used[rows[a], kh], 70, keep, recent)
        for d in (keys, vals, host_sums):
            d[a][kh] = [d[a][kh][j] for j in kept]
    for s in (b, c):
        assert (to_host(kc, dtype)[pa.pa_seq_table(h, s)] == before[s]).all()
    assert (sums[rows[a], :, keep:] == 0).all()
    for _ in range(4):
        decode([b, a, c])                    # over the kept tokens; each KV head of a has its own
    # five drafted tokens verified at once, a document border for c
    q = write([a, c], 5)
    tables, lens = pa.pa_pool_export(h, [a, c], mb, -1)
    dims = pa.make_dims(2, Hq, Hkv, D, B, N, mb, 0, dtype)
    ws = torch.empty(pa.pa_chunk_scored_workspace_bytes(dims, 10, 5), dtype=torch.uint8, device="cuda")
    out = torch.empty(10, Hq, D, device="cuda")
    pa.pa_chunk_scored(dims, score, q, kc, vc, i32(tables), i32(lens), i32([0, 5, 10]), scale, out, 5, ws)
    q64, got = widen(to_host(q, dtype), dtype), out.cpu().numpy()
    for i, s in enumerate((a, c)):
        ref, _, E, vmax = reference(s, q64[5 * i:5 * i + 5], True)
        assert_rows_close(got[5 * i:5 * i + 5], ref, dtype, "f32", E, vmax)
    assert pa.pa_device_errors(clear=True) == 0
    pool.close()


def test_offsets_past_32_bits(gpu):
    """Blocks at both ends of a pool of more than 2^32 elements: a rotary write, a
    decode with sums, a long chunk, and an eviction from one end to the other."""
    torch, pa = gpu
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    rng = synth.make_rng(11100)
    Hq, Hkv, D, B, L = 16, 8, 128, 32, 200
    N = (1 << 32) // (Hkv * B * D) + 64
    kc, vc = (torch.empty(N, Hkv, B, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    nb = -(-L // B)
    table = np.array([N - 1 - 3 * j if j % 2 else 2 * j for j in range(nb)], np.int32)
    fresh = np.array([N - 2 - 3 * j for j in range(nb)], np.int32)
    slots = np.array([int(table[i // B]) * B + i % B for i in range(L)], np.int64)
    x = synth.normal(rng, (L, Hq + 2 * Hkv, D), 1.0, "bf16")
    dx = to_dev(torch, x, "bf16")
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()
    dims = pa.make_dims(1, Hq, Hkv, D, B, N, nb, 0, "bf16")
    freqs, _ = pa.pa_rope_freqs(D)
    q = torch.empty(L, Hq, D, dtype=torch.bfloat16, device="cuda")
    pos = np.arange(L)
    pa.pa_rope_write_kv(dims, pa.make_rope(D, torch.from_numpy(freqs).cuda()), dx[:, :Hq], dx[:, Hq:Hq + Hkv], dx[:, Hq + Hkv:],
                        i32(pos), torch.from_numpy(slots).cuda(), q, kc, vc)
    at = torch.from_numpy(table.astype(np.int64)).cuda()
    rows = lambda c, t: widen(to_host(c[t].transpose(1, 2).reshape(-1, Hkv, D)[:L].contiguous(), "bf16"), "bf16")
    K, V, q64 = rows(kc, at), rows(vc, at), widen(to_host(q, "bf16"), "bf16")
    ref_k, _ = rotate(widen(x[:, Hq:Hq + Hkv], "bf16"), pos, freqs, D, False, 1.0)
    assert np.abs(K - ref_k).max() <= 2.0 ** -8 * np.abs(ref_k).max() + 1e-5
    np.testing.assert_array_equal(V, widen(x[:, Hq + Hkv:], "bf16"))
    scale = 1 / math.sqrt(D)
    sums = torch.zeros(1, Hkv, nb * B, device="cuda")
    out = torch.empty(1, Hq, D, device="cuda")
    ws = torch.empty(pa.pa_decode_scored_workspace_bytes(dims, True), dtype=torch.uint8, device="cuda")
    pa.pa_decode_scored(dims, None, q[-1:], kc, vc, i32(table[None]), i32([L]), scale, out, ws, key_sums=sums)
    ref, w, d = scored_rows(q64[-1:], K, V, [L - 1], [0], [L], scale)
    E = weight_error("bf16", d, L)
    assert_rows_close(out.cpu().numpy(), ref, "bf16", "f32", E, np.abs(V).max())
    out = torch.empty(L, Hq, D, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(pa.pa_chunk_scored_workspace_bytes(dims, L, L), dtype=torch.uint8, device="cuda")
    pa.pa_chunk_scored(dims, pa.make_score(softcap=20.0), q, kc, vc, i32(table[None]), i32([L]), i32([0, L]), scale, out, L, ws)
    ref, _, d = scored_rows(q64, K, V, pos, np.zeros(L, int), pos + 1, scale, 20.0)
    assert_rows_close(out.float().cpu().numpy(), ref, "bf16", "bf16", weight_error("bf16", d, L), np.abs(V).max())
    new_lens, ws = i32([0]), torch.empty(pa.pa_evict_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    used = sums.cpu().numpy()
    pa.pa_evict(dims, kc, vc, i32(table[None]), i32([L]), i32(fresh[None]), i32([70]), 16, sums, sums, new_lens, ws)
    moved = rows(kc, torch.from_numpy(fresh.astype(np.int64)).cuda())
    for kh in range(Hkv):
        kept = kept_tokens(used[0, kh], L, 70, 16)
        np.testing.assert_array_equal(moved[:70, kh], K[kept, kh])
    assert pa.pa_device_errors(clear=True) == 0


def test_two_streams_and_graphs_with_their_own_workspaces(gpu):
    """Chunk calls in flight at once on two streams, and two captured graphs (rotary
    write, decode, eviction) replayed in turn, give the bits of calls made alone."""
    torch, pa = gpu
    rng = synth.make_rng(11200)
    S, Hq, Hkv, D, B, L, n = 3, 16, 4, 128, 16, 300, 70
    mb = -(-L // B)
    N = 2 * S * mb + 4
    perm = rng.permutation(N)
    tables = perm[:S * mb].reshape(S, mb).astype(np.int32)
    fresh = perm[S * mb:2 * S * mb].reshape(S, mb).astype(np.int32)
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()
    normal = lambda *shape: to_dev(torch, synth.normal(rng, shape, 1.0, "bf16"), "bf16")
    dims = pa.make_dims(S, Hq, Hkv, D, B, N, mb, 0, "bf16")
    kc, vc = normal(N, Hkv, B, D), normal(N, Hkv, B, D)
    dt, dl, qs = i32(tables), i32([L, L - 9, n]), i32([0, n, 2 * n, 3 * n])
    score = pa.make_score(softcap=10.0, slopes=torch.rand(Hq, device="cuda"))
    qs_in = [normal(3 * n, Hq, D) for _ in range(2)]
    ws = [torch.empty(pa.pa_chunk_scored_workspace_bytes(dims, 3 * n, n), dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.empty(3 * n, Hq, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    alone = []
    for i in range(2):
        pa.pa_chunk_scored(dims, score, qs_in[i], kc, vc, dt, dl, qs, 0.09, outs[i], n, ws[i])
        alone.append(outs[i].clone())
        outs[i].zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(8):
        for i in range(2):
            pa.pa_chunk_scored(dims, score, qs_in[i], kc, vc, dt, dl, qs, 0.09, outs[i], n, ws[i], stream=streams[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], alone[0]) and torch.equal(outs[1], alone[1])

    freqs = torch.from_numpy(pa.pa_rope_freqs(D)[0]).cuda()
    rope = pa.make_rope(D, freqs, True)
    q, k, v = normal(S, Hq, D), normal(S, Hkv, D), normal(S, Hkv, D)
    slots = torch.tensor([int(tables[s, (ln - 1) // B]) * B + (ln - 1) % B for s, ln in enumerate([L, L - 9, n])], device="cuda")
    pos = i32([L - 1, L - 10, n - 1])
    budget = i32([64, 400, 16])

    def step(state, stream=None):
        pa.pa_rope_write_kv(dims, rope, q, k, v, pos, slots, state["q"], kc, vc, stream=stream)
        pa.pa_decode_scored(dims, score, state["q"], kc, vc, dt, dl, 0.09, state["out"], state["ws"], key_sums=state["sums"],
                            stream=stream)
        pa.pa_evict(dims, kc, vc, dt, dl, i32_fresh, budget, 8, state["sums"], state["kept"], state["lens"], state["wse"],
                    stream=stream)

    i32_fresh = i32(fresh)

    def state():
        return dict(q=torch.empty_like(q), out=torch.empty(S, Hq, D, device="cuda"), sums=torch.zeros(S, Hkv, mb * B, device="cuda"),
                    kept=torch.zeros(S, Hkv, mb * B, device="cuda"), lens=i32([0] * S),
                    ws=torch.empty(pa.pa_decode_scored_workspace_bytes(dims, True), dtype=torch.uint8, device="cuda"),
                    wse=torch.empty(pa.pa_evict_workspace_bytes(dims), dtype=torch.uint8, device="cuda"))

    eager, graphs = state(), []
    for _ in range(2):
        st = state()
        g = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=side):
            step(st, side)
        graphs.append((g, st))
    for turn in range(3):
        step(eager)
        torch.cuda.synchronize()
        want_k = kc.clone()
        for g, st in graphs:
            g.replay()
            torch.cuda.synchronize()
            for name in ("q", "out", "sums", "kept", "lens"):
                assert torch.equal(st[name], eager[name]), name
            assert torch.equal(kc, want_k)
    assert pa.pa_device_errors(clear=True) == 0


def test_results_do_not_depend_on_the_run(gpu):
    """The same call twice gives the same bits (no atomics in any sum)."""
    torch, pa = gpu
    rng = synth.make_rng(11300)
    S, Hq, Hkv, D, B = 40, 8, 2, 64, 16
    lens = rng.integers(1, 900, S)
    mb = -(-900 // B)
    N = S * mb
    tables = rng.permutation(N).reshape(S, mb).astype(np.int32)
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()
    normal = lambda *shape: to_dev(torch, synth.normal(rng, shape, 1.0, "f16"), "f16")
    dims = pa.make_dims(S, Hq, Hkv, D, B, N, mb, 64, "f16")
    kc, vc, q = normal(N, Hkv, B, D), normal(N, Hkv, B, D), normal(S, Hq, D)
    got = []
    for _ in range(4):
        sums, out = torch.zeros(S, Hkv, mb * B, device="cuda"), torch.empty(S, Hq, D, device="cuda")
        ws = torch.empty(pa.pa_decode_scored_workspace_bytes(dims, True), dtype=torch.uint8, device="cuda")
        pa.pa_decode_scored(dims, pa.make_score(softcap=3.0), q, kc, vc, i32(tables), i32(lens), 0.125, out, ws, key_sums=sums)
        got.append((out, sums))
    for out, sums in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(sums, got[0][1])


def test_large_values_under_a_fixed_maximum(gpu):
    """Capped bf16 chunks use a constant for the softmax maximum: logits saturated on
    both sides of the cap, with values up to 2^50, stay finite and right."""
    torch, pa = gpu
    rng = synth.make_rng(11400)
    Hq, Hkv, D, B, L = 4, 1, 64, 16, 320
    N = L // B
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()
    dims = pa.make_dims(1, Hq, Hkv, D, B, N, N, 0, "bf16")
    for sign in (1.0, -1.0):
        k = np.ones((L, Hkv, D)) * sign
        q = synth.normal(rng, (L, Hq, D), 1.0, "bf16")
        q64 = np.abs(widen(q, "bf16")) * 8 + 4      # every logit far past the cap, on one side
        dq = torch.from_numpy(q64).cuda().bfloat16()
        v64 = widen(synth.normal(rng, (L, Hkv, D), 1.0, "bf16"), "bf16") * 2.0 ** 50
        kc = torch.from_numpy(k.reshape(N, B, Hkv, D)).cuda().bfloat16().transpose(1, 2).contiguous()
        vc = torch.from_numpy(v64.reshape(N, B, Hkv, D)).cuda().bfloat16().transpose(1, 2).contiguous()
        out = torch.empty(L, Hq, D, device="cuda")
        ws = torch.empty(pa.pa_chunk_scored_workspace_bytes(dims, L, L), dtype=torch.uint8, device="cuda")
        for cap in (50.0, 55.0, 30.0):
            pa.pa_chunk_scored(dims, pa.make_score(softcap=cap), dq, kc, vc, i32(np.arange(N)[None]), i32([L]), i32([0, L]), 1.0,
                               out, L, ws)
            pos = np.arange(L)
            ref, _, d = scored_rows(dq.double().cpu().numpy(), k, v64, pos, np.zeros(L, int), pos + 1, 1.0, cap)
            assert_rows_close(out.cpu().numpy(), ref, "bf16", "f32", weight_error("bf16", d, L), np.abs(v64).max())
