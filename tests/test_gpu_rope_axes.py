"""GPU tests of rotary positions with several axes over 16- and 32-bit caches."""
import pytest

from gpu_helpers import require_gpu
from kv8_helpers import HALF_STEP, dtype_of, rotate_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gpu():
    return require_gpu()


@pytest.mark.parametrize("dtype,D,R,interleaved", [
    ("bf16", 128, 128, False), ("f16", 64, 64, True), ("f32", 64, 20, False), ("bf16", 128, 74, False), ("f16", 128, 22, True),
    ("f32", 128, 64, True), ("bf16", 64, 2, False), ("bf16", 2304, 2048, False)])
@pytest.mark.parametrize("T,axes", [(1, 3), (37, 1), (2500, 2), (300, 16)])
def test_rope_axes_against_the_formula(gpu, dtype, D, R, interleaved, T, axes):
    torch, pa = gpu
    if D > 128 and T > 300:
        T = 40
    gen = torch.Generator(device="cuda").manual_seed(T + R)
    Hq, Hkv, B = 4, 2, 16
    dt = dtype_of(torch, dtype)
    N = -(-T // B) + 2
    q, k, v = (torch.randn(T, h, D, generator=gen, device="cuda").to(dt) for h in (Hq, Hkv, Hkv))
    positions = torch.randint(-100000, 100000, (axes, T), generator=gen, device="cuda", dtype=torch.int32)
    pair_axis = torch.randint(0, axes, (R // 2,), generator=gen, device="cuda", dtype=torch.int32)
    slots = torch.randperm(N * B, generator=gen, device="cuda")[:T].contiguous()
    slots[T // 2] = -1
    f, _ = pa.pa_rope_freqs(R, 10000.0)
    freqs = torch.from_numpy(f[: R // 2].copy()).cuda()
    mscale = 1.0 if axes != 2 else 1.3
    kc, vc = torch.zeros(N, Hkv, B, D, dtype=dt, device="cuda"), torch.zeros(N, Hkv, B, D, dtype=dt, device="cuda")
    q_out = torch.zeros_like(q)
    dims = pa.make_dims(0, Hq, Hkv, D, B, N, 1, 0, dtype)
    rope = pa.make_rope(R, freqs, interleaved, mscale)
    pa.pa_rope_axes_write_kv(dims, rope, pa.make_axes(axes, pair_axis), q, k, v, positions, slots, q_out, kc, vc)
    qr = rotate_ref(torch, q, positions, pair_axis, freqs, R, interleaved, mscale)
    kr = rotate_ref(torch, k, positions, pair_axis, freqs, R, interleaved, mscale)
    live = slots >= 0
    blk, off = slots[live] // B, slots[live] % B
    # (cos, sin) off by 2^-22 of mscale, three roundings of fp32, one of the type
    for got, want in ((q_out[live], qr[live]), (kc[blk, :, off], kr[live])):
        lim = HALF_STEP[dtype] * want.abs() + 2.0 ** -20 * mscale * want.abs().amax(-1, keepdim=True) + 2.0 ** -25
        assert bool(((got.double() - want).abs() <= lim).all())
    assert torch.equal(vc[blk, :, off], v[live])
    assert bool((q_out[~live] == 0).all())
    untouched = torch.ones(N * B, dtype=torch.bool, device="cuda")
    untouched[slots[live]] = False
    assert bool((kc.transpose(1, 2).reshape(N * B, -1)[untouched] == 0).all())
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("R,interleaved", [(128, False), (64, True), (20, False)])
def test_rope_axes_alike_are_the_plain_rotation(gpu, R, interleaved):
    """Text: the same position on every axis gives pa_rope_write_kv's bits, and so does one axis."""
    torch, pa = gpu
    gen = torch.Generator(device="cuda").manual_seed(R)
    T, Hq, Hkv, D, B, N = 70, 8, 2, 128, 16, 6
    q, k, v = (torch.randn(T, h, D, generator=gen, device="cuda").to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    positions = torch.randint(0, 90000, (T,), generator=gen, device="cuda", dtype=torch.int32)
    slots = torch.randperm(N * B, generator=gen, device="cuda")[:T].contiguous()
    freqs = torch.from_numpy(pa.pa_rope_freqs(R, 500000.0)[0][: R // 2].copy()).cuda()
    rope, dims = pa.make_rope(R, freqs, interleaved), pa.make_dims(0, Hq, Hkv, D, B, N, 1, 0, "bf16")
    results = []
    for mode in range(3):
        out, kc, vc = torch.zeros_like(q), *(torch.zeros(N, Hkv, B, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        if mode == 0:
            pa.pa_rope_write_kv(dims, rope, q, k, v, positions, slots, out, kc, vc)
        elif mode == 1:
            pa.pa_rope_axes_write_kv(dims, rope, None, q, k, v, positions, slots, out, kc, vc)
        else:
            axis = (torch.arange(R // 2, device="cuda") % 3).int()
            pa.pa_rope_axes_write_kv(dims, rope, pa.make_axes(3, axis), q, k, v, positions.expand(3, T).contiguous(), slots, out, kc, vc)
        results.append((out, kc, vc))
    for r in results[1:]:
        for x, y in zip(results[0], r):
            assert torch.equal(x, y)


def test_rope_axes_of_no_axis_are_flagged(gpu):
    torch, pa = gpu
    for D, R, interleaved in ((128, 128, False), (64, 20, False), (2304, 64, True)):
        T, Hq, Hkv, B, N = 3, 2, 1, 16, 2
        q, k, v = (torch.randn(T, h, D, device="cuda").to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
        axis = torch.zeros(R // 2, dtype=torch.int32, device="cuda")
        axis[4], axis[5] = 2, -9
        freqs = torch.ones(R // 2, dtype=torch.float64, device="cuda")
        kc, vc = (torch.zeros(N, Hkv, B, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        out = torch.zeros_like(q)
        pa.pa_rope_axes_write_kv(pa.make_dims(0, Hq, Hkv, D, B, N, 1, 0, "bf16"), pa.make_rope(R, freqs, interleaved),
                                 pa.make_axes(2, axis), q, k, v, torch.full((2, T), 5, dtype=torch.int32, device="cuda"),
                                 torch.arange(T, device="cuda"), out, kc, vc)
        assert pa.pa_device_errors(clear=True) == pa.PA_DEVERR_BAD_AXIS
        for p in (4, 5):
            for d in ((2 * p, 2 * p + 1) if interleaved else (p, p + R // 2)):
                assert torch.equal(out[..., d], q[..., d])
