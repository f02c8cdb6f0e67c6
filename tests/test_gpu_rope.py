"""GPU tests of pa_rope_write_kv against a plain reference in extended precision.

Tolerance: the turn's fraction as fp32 and sincospif give (cos, sin) to 2^-21
absolute; two products and a sum in fp32 add 2^-23 of |a| + |b|; the result is
rounded once (half a step of its type)."""
import numpy as np
import pytest

from gpu_helpers import require_gpu, to_dev, to_host
from paged_helpers import widen
from paged_kv_cache_127_gb300 import synth
from scored_helpers import HALF_STEP, rotate

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gpu():
    return require_gpu()


def check(got, x, pos, freqs, R, interleaved, mscale, dtype):
    ref, mag = rotate(widen(x, dtype), pos, freqs, R, interleaved, mscale)
    tol = mag * (2.0 ** -21 + 2.0 ** -22) + HALF_STEP[dtype] * np.abs(ref) * (mag > 0) + 2.0 ** -24 * (dtype == "f16") * (mag > 0)
    bad = np.abs(widen(got, dtype) - ref) > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} outside"


def run(torch, pa, dtype, T, Hq, Hkv, D, B, R, interleaved, pos, slots, N, rng, fused=True, mscale=1.0, in_place=False):
    freqs, _ = pa.pa_rope_freqs(R, 10000.0)
    heads = Hq + 2 * Hkv
    x = synth.normal(rng, (T, heads, D), 1.0, dtype)
    kc, vc = (synth.normal(rng, (N, Hkv, B, D), 1.0, dtype) for _ in range(2))
    all_ = to_dev(torch, x, dtype)
    q, k, v = all_[:, :Hq], all_[:, Hq:Hq + Hkv], all_[:, Hq + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    out = q if in_place else torch.full_like(all_[:, :Hq].contiguous(), 7.0)
    dk, dv = to_dev(torch, kc, dtype), to_dev(torch, vc, dtype)
    dims = pa.make_dims(0, Hq, Hkv, D, B, N, 1, 0, dtype)
    pa.pa_rope_write_kv(dims, pa.make_rope(R, torch.from_numpy(freqs).cuda(), interleaved, mscale), q, k, v,
                        torch.from_numpy(np.asarray(pos, np.int32)).cuda(), torch.from_numpy(np.asarray(slots, np.int64)).cuda(),
                        out, dk, dv)
    torch.cuda.synchronize()
    ok = (np.asarray(slots) >= 0) & (np.asarray(slots) < N * B)
    got_q = to_host(out.contiguous(), dtype)
    check(got_q[ok], x[ok, :Hq], np.asarray(pos)[ok], freqs, R, interleaved, mscale, dtype)
    # padding and skipped tokens: nothing written
    want = x[:, :Hq] if in_place else np.broadcast_to(to_host(torch.full((1,), 7.0).to(all_.dtype), dtype), got_q.shape)
    np.testing.assert_array_equal(got_q[~ok], want[~ok])
    k2, v2 = to_host(dk, dtype), to_host(dv, dtype)
    for t in np.nonzero(ok)[0]:
        b, o = divmod(int(slots[t]), B)
        check(k2[b, :, o][None], x[t:t + 1, Hq:Hq + Hkv], [pos[t]], freqs, R, interleaved, mscale, dtype)
        np.testing.assert_array_equal(v2[b, :, o], x[t, Hq + Hkv:])
        kc[b, :, o], vc[b, :, o] = k2[b, :, o], v2[b, :, o]
    np.testing.assert_array_equal(k2, kc)     # every other slot holds what it held
    np.testing.assert_array_equal(v2, vc)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,R", [(128, 128), (128, 64), (64, 64), (64, 20), (128, 2), (96, 90), (80, 48), (8, 8), (128, 74),
                                 (256, 30), (72, 72), (64, 62), (2560, 1500)])
def test_rope_layouts_and_sizes(gpu, dtype, D, R, interleaved):
    torch, pa = gpu
    rng = synth.make_rng(8000 + D + R + interleaved)
    for T, Hq, Hkv, B in ((1, 4, 1, 16), (37, 6, 3, 32), (5, 8, 8, 16)):
        N = 9
        slots = rng.permutation(N * B)[:T]
        pos = rng.integers(0, 5000, T)
        run(torch, pa, dtype, T, Hq, Hkv, D, B, R, interleaved, pos, slots, N, rng, fused=T != 5)
    assert pa.pa_device_errors(clear=True) == 0


def test_rope_far_and_negative_positions_padding_and_bad_slots(gpu):
    torch, pa = gpu
    rng = synth.make_rng(8100)
    pos = np.array([0, 1, 2 ** 20 + 3, 2 ** 31 - 1, -7, -2 ** 31, 131071, 12])
    slots = np.array([5, 40, 0, 159, 12, 13, -1, 160])
    for dtype in ("f32", "bf16"):
        run(torch, pa, dtype, 8, 4, 2, 128, 16, 128, False, pos, slots, 10, rng)
        assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_BAD_SLOT


def test_rope_in_place_and_mscale(gpu):
    torch, pa = gpu
    rng = synth.make_rng(8200)
    for dtype, fused in (("bf16", True), ("f32", False), ("f16", True)):
        slots = np.where(np.arange(50) % 7 == 3, -1, rng.permutation(64)[:50])
        run(torch, pa, dtype, 50, 8, 2, 64, 16, 32, True, rng.integers(0, 99999, 50), slots, 4, rng, fused, 1.2079, True)
    assert pa.pa_device_errors(clear=True) == 0


def test_rope_matches_the_separate_write(gpu):
    # at position 0 with mscale 1 the call is pa_write_kv, bit for bit
    torch, pa = gpu
    rng = synth.make_rng(8300)
    T, Hq, Hkv, D, B, N = 40, 4, 2, 64, 16, 6
    k, v = (to_dev(torch, synth.normal(rng, (T, Hkv, D), 1.0, "bf16"), "bf16") for _ in range(2))
    q = to_dev(torch, synth.normal(rng, (T, Hq, D), 1.0, "bf16"), "bf16")
    slots = torch.from_numpy(rng.permutation(N * B)[:T]).cuda()
    dims = pa.make_dims(0, Hq, Hkv, D, B, N, 1, 0, "bf16")
    a = [torch.zeros(N, Hkv, B, D, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    pa.pa_write_kv(dims, k, v, slots, a[0], a[1])
    freqs = torch.from_numpy(pa.pa_rope_freqs(D)[0]).cuda()
    out = torch.empty_like(q)
    pa.pa_rope_write_kv(dims, pa.make_rope(D, freqs), q, k, v, torch.zeros(T, dtype=torch.int32, device="cuda"), slots, out,
                        a[2], a[3])
    assert torch.equal(a[0], a[2]) and torch.equal(a[1], a[3]) and torch.equal(out, q)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_output_beside_its_input(gpu, interleaved):
    # q_out as another column range of the tensor that holds q
    torch, pa = gpu
    rng = synth.make_rng(8400)
    T, Hq, Hkv, D, B, N = 50, 4, 2, 64, 16, 6
    x = synth.normal(rng, (T, Hq, D), 1.0, "bf16")
    both = torch.zeros(T, 2 * Hq, D, dtype=torch.bfloat16, device="cuda")
    both[:, Hq:] = to_dev(torch, x, "bf16")
    k, v = (to_dev(torch, synth.normal(rng, (T, Hkv, D), 1.0, "bf16"), "bf16") for _ in range(2))
    kc, vc = (torch.zeros(N, Hkv, B, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pos = rng.integers(0, 3000, T)
    freqs = pa.pa_rope_freqs(D)[0]
    pa.pa_rope_write_kv(pa.make_dims(0, Hq, Hkv, D, B, N, 1, 0, "bf16"),
                        pa.make_rope(D, torch.from_numpy(freqs).cuda(), interleaved), both[:, Hq:], k, v,
                        torch.from_numpy(pos.astype(np.int32)).cuda(), torch.arange(T, device="cuda"), both[:, :Hq], kc, vc)
    check(to_host(both[:, :Hq].contiguous(), "bf16"), x, pos, freqs, D, interleaved, 1.0, "bf16")
    np.testing.assert_array_equal(to_host(both[:, Hq:].contiguous(), "bf16"), x)
    with pytest.raises(pa.PaError):
        pa.pa_rope_write_kv(pa.make_dims(0, Hq, Hkv, D, B, N, 1, 0, "bf16"),
                            pa.make_rope(D, torch.from_numpy(freqs).cuda(), interleaved), both[:, Hq:], k, v,
                            torch.from_numpy(pos.astype(np.int32)).cuda(), torch.arange(T, device="cuda"),
                            both[:, Hq - 1:2 * Hq - 1], kc, vc)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,Hq,Hkv,D,R", [(3, 40, 8, 128, 20), (700, 12, 4, 64, 38), (40, 5, 1, 80, 6)])
def test_rope_in_place_where_pairs_lie_across_units(gpu, dtype, T, Hq, Hkv, D, R, interleaved):
    # heads in several rounds of a block, tokens in several blocks, the output over its input
    torch, pa = gpu
    rng = synth.make_rng(8500 + T + R)
    N = -(-T // 16) + 1
    slots = np.where(np.arange(T) % 11 == 5, -1, rng.permutation(N * 16)[:T])
    run(torch, pa, dtype, T, Hq, Hkv, D, 16, R, interleaved, rng.integers(0, 9999, T), slots, N, rng, True, 0.87, True)
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_rope_copies_the_elements_behind_the_rotary_dim_bit_for_bit(gpu, dtype, interleaved):
    # NaN of any payload, infinities and zeros of both signs there stay as they are
    torch, pa = gpu
    D, B, N, T = 64, 16, 2, 9
    odd = {"f32": np.uint32([0x7f800001, 0xffc12345, 0x7f800000, 0x80000000]), "f16": np.uint16([0x7c01, 0xfe12, 0xfc00, 0x8000]),
           "bf16": np.uint16([0x7f81, 0xffc5, 0xff80, 0x8000])}[dtype]
    raw = torch.from_numpy(np.resize(odd.view(np.int32 if dtype == "f32" else np.int16), (T, 3, D)).copy()).cuda()
    x = raw.view({"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dtype])
    for R in (2, 6, 16, 20, 50, 62):
        y = x.clone()
        y[:, :, :R] = 1.0
        kc, vc = (torch.zeros(N, 1, B, D, dtype=x.dtype, device="cuda") for _ in range(2))
        out = torch.zeros(T, 1, D, dtype=x.dtype, device="cuda")
        freqs = torch.from_numpy(pa.pa_rope_freqs(R)[0]).cuda()
        pa.pa_rope_write_kv(pa.make_dims(0, 1, 1, D, B, N, 1, 0, dtype), pa.make_rope(R, freqs, interleaved), y[:, :1], y[:, 1:2],
                            y[:, 2:], torch.arange(T, dtype=torch.int32, device="cuda"), torch.arange(T, device="cuda"), out, kc, vc)
        bits = lambda z: z.contiguous().view(raw.dtype)
        assert torch.equal(bits(out[:, 0, R:]), raw[:, 0, R:])
        assert torch.equal(bits(kc.view(-1, D)[:T, R:]), raw[:, 1, R:])
        assert torch.equal(bits(vc.view(-1, D)[:T]), bits(y[:, 2]))
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,R", [(2433, 4, 2, 64, 64), (2432, 8, 1, 128, 32), (2501, 2, 2, 40, 16)])
def test_rope_two_tokens_a_block(gpu, T, Hq, Hkv, D, R, interleaved):
    # many tokens: two a block, the last block's second one missing, padding and bad slots in either place
    torch, pa = gpu
    rng = synth.make_rng(10500 + T + R)
    N, B = T // 16 + 4, 16
    pos = rng.integers(-5, 200000, T)
    slots = rng.permutation(N * B)[:T]
    slots[rng.integers(0, T, 60)] = -1
    slots[[0, 1, 7, 100, T - 1]] = [-1, N * B, N * B + 5, -7, slots[T - 1]]
    run(torch, pa, "bf16", T, Hq, Hkv, D, B, R, interleaved, pos, slots, N, rng, mscale=1.25)
    assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_BAD_SLOT
