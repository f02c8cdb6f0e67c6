"""GPU test: the rotary write gives the same bits whichever kernel takes a layout."""
import pytest

from gpu_helpers import require_gpu
from kv8_helpers import dtype_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gpu():
    return require_gpu()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("R", [64, 80, 96, 128])
@pytest.mark.parametrize("T", [3, 700, 2500])
def test_a_head_turned_whole_has_the_bits_of_a_part_of_a_larger_one(gpu, dtype, R, T):
    """The first R elements of a head of 2 R, and the same elements as a head of their own."""
    torch, pa = gpu
    gen = torch.Generator(device="cuda").manual_seed(T + R)
    dt = dtype_of(torch, dtype)
    Hq, Hkv, B = 4, 2, 16
    N = -(-T // B) + 1
    wide = [torch.randn(T, h, 2 * R, generator=gen, device="cuda").to(dt) for h in (Hq, Hkv, Hkv)]
    positions = torch.randint(0, 100000, (T,), generator=gen, device="cuda", dtype=torch.int32)
    slots = torch.randperm(N * B, generator=gen, device="cuda")[:T].contiguous()
    freqs = torch.from_numpy(pa.pa_rope_freqs(R, 10000.0)[0][: R // 2].copy()).cuda()
    rope = pa.make_rope(R, freqs, False, 1.3)
    got = []
    for D in (2 * R, R):
        q, k, v = (x[..., :D].contiguous() for x in wide)
        out = torch.zeros_like(q)
        kc, vc = (torch.zeros(N, Hkv, B, D, dtype=dt, device="cuda") for _ in range(2))
        pa.pa_rope_write_kv(pa.make_dims(0, Hq, Hkv, D, B, N, 1, 0, dtype), rope, q, k, v, positions, slots, out, kc, vc)
        got.append((out[..., :R], kc[..., :R], vc[..., :R]))
    for part, whole in zip(*got):
        assert torch.equal(part, whole)
    assert pa.pa_device_errors(clear=True) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,R,interleaved", [(128, 128, False), (64, 64, False), (128, 64, False), (128, 128, True), (64, 22, True), (128, 72, False),
                                             (64, 20, False)])
@pytest.mark.parametrize("T", [1, 37, 2600])
def test_the_writes_into_either_cache_turn_queries_alike(gpu, dtype, D, R, interleaved, T):
    torch, pa = gpu
    gen = torch.Generator(device="cuda").manual_seed(T + R)
    dt = dtype_of(torch, dtype)
    Hq, Hkv, B = 8, 4, 16
    N = -(-T // B) + 1
    q, k, v = (torch.randn(T, h, D, generator=gen, device="cuda").to(dt) for h in (Hq, Hkv, Hkv))
    positions = torch.randint(0, 100000, (2, T), generator=gen, device="cuda", dtype=torch.int32)
    axes = pa.make_axes(2, torch.randint(0, 2, (R // 2,), generator=gen, device="cuda", dtype=torch.int32))
    slots = torch.arange(T, device="cuda")
    freqs = torch.from_numpy(pa.pa_rope_freqs(R, 10000.0)[0][: R // 2].copy()).cuda()
    rope, dims = pa.make_rope(R, freqs, interleaved, 0.7), pa.make_dims(0, Hq, Hkv, D, B, N, 1, 0, dtype)
    one, two = torch.zeros_like(q), torch.zeros_like(q)
    kc, vc = (torch.zeros(N, Hkv, B, D, dtype=dt, device="cuda") for _ in range(2))
    pa.pa_rope_axes_write_kv(dims, rope, axes, q, k, v, positions, slots, one, kc, vc)
    codes = [torch.zeros(N, Hkv, B, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.zeros(N, Hkv, device="cuda") for _ in range(2)]
    pa.pa_rope_write_kv8(dims, rope, axes, q, k, v, positions, slots, two, pa.make_cache8(*codes, *scales))
    assert torch.equal(one, two)
    assert pa.pa_device_errors(clear=True) == 0
