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
