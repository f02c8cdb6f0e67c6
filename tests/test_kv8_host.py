"""Host side of the 8-bit cache's calls and of rotary axes, without a GPU: refusals of
the C ABI (no call here gets past its checks) and workspace sizes."""
import ctypes

import pytest

from paged_kv_cache_127_gb300 import build as pa_build


@pytest.fixture(scope="module")
def pa():
    pa_build.build()
    from paged_kv_cache_127_gb300 import binding
    return binding


P = 1 << 20  # an aligned address that no call may follow


def dims(pa, **kw):
    d = dict(num_seqs=2, num_q_heads=8, num_kv_heads=2, head_dim=64, block_size=16, num_blocks=10, max_blocks_per_seq=4,
             partition_size=0, kv_dtype="bf16")
    d.update(kw)
    return pa.make_dims(**d)


def ref(x):
    return None if x is None else ctypes.byref(x)


def cache8(pa, **kw):
    c = dict(k=P, v=P, k_scales=P, v_scales=P)
    c.update(kw)
    return pa.pa_cache8(**c)


def decode(pa, d, win=None, cache=True, q=P, out=P, out_dtype=0, ws=P, ws_bytes=1 << 40, tables=P, lens=P):
    c = cache8(pa) if cache is True else cache
    return pa.lib.pa_decode8(ref(d), ref(win), q, ref(c), tables, lens, 0.1, out, out_dtype, ws, ws_bytes, None)


def chunk(pa, d, win=None, cache=True, q=P, out=P, out_dtype=0, ws=P, ws_bytes=1 << 40, tables=P, lens=P, T=9, max_q=5, qs=P):
    c = cache8(pa) if cache is True else cache
    return pa.lib.pa_chunk8(ref(d), ref(win), q, ref(c), tables, lens, qs, T, max_q, 0.1, out, out_dtype, ws, ws_bytes, None)


def rope(pa, **kw):
    r = dict(rotary_dim=64, interleaved=0, freqs=P, mscale=1.0)
    r.update(kw)
    return pa.pa_rope(**r)


def write8(pa, d, rp=True, axes=None, cache=True, q=P, qs=512, k=2 * P, ks=128, v=3 * P, vs=128, pos=P, slots=P, T=3, q_out=4 * P, qos=512):
    rp = rope(pa) if rp is True else rp
    c = cache8(pa) if cache is True else cache
    return pa.lib.pa_rope_write_kv8(ref(d), ref(rp), ref(axes), q, qs, k, ks, v, vs, pos, slots, T, q_out, qos, ref(c), None)


def axes_write(pa, d, rp=True, axes=None, q=P, qs=512, k=2 * P, ks=128, v=3 * P, vs=128, pos=P, slots=P, T=3, q_out=4 * P, qos=512, kc=5 * P, vc=6 * P):
    rp = rope(pa) if rp is True else rp
    return pa.lib.pa_rope_axes_write_kv(ref(d), ref(rp), ref(axes), q, qs, k, ks, v, vs, pos, slots, T, q_out, qos, kc, vc, None)


def plain_write8(pa, d, cache=True, k=2 * P, ks=128, v=3 * P, vs=128, slots=P, T=3):
    c = cache8(pa) if cache is True else cache
    return pa.lib.pa_write_kv8(ref(d), k, ks, v, vs, slots, T, ref(c), None)


def copy8(pa, d, cache=True, pairs=P, n=2):
    c = cache8(pa) if cache is True else cache
    return pa.lib.pa_copy_blocks8(ref(d), ref(c), pairs, n, None)


def test_shapes_that_all_calls_refuse(pa):
    INV, UNS = pa.PA_ERR_INVALID, pa.PA_ERR_UNSUPPORTED
    for call in (decode, chunk, write8, plain_write8, copy8):
        assert call(pa, None) == INV
        for bad in (dict(head_dim=80), dict(head_dim=256), dict(block_size=8), dict(block_size=64), dict(kv_dtype="f32")):
            assert call(pa, dims(pa, **bad)) == UNS, bad
        for bad in (dict(num_kv_heads=0), dict(num_blocks=0), dict(kv_dtype=7), dict(head_dim=-64),
                    dict(num_blocks=1 << 30, num_kv_heads=2)):
            assert call(pa, dims(pa, **bad)) == INV, bad
        assert call(pa, dims(pa), cache=None) == INV
        for bad in (dict(k=None), dict(v=None), dict(k_scales=None), dict(v_scales=None), dict(k=P + 8), dict(v=P + 1),
                    dict(k_scales=P + 2), dict(v_scales=P + 1)):
            assert call(pa, dims(pa), cache=cache8(pa, **bad)) == INV, bad


def test_attention_refusals(pa):
    INV, UNS = pa.PA_ERR_INVALID, pa.PA_ERR_UNSUPPORTED
    for call in (decode, chunk):
        assert call(pa, dims(pa, num_q_heads=6)) == UNS
        assert call(pa, dims(pa, num_q_heads=32)) == UNS
        assert call(pa, dims(pa, num_q_heads=7)) == INV
        assert call(pa, dims(pa, num_seqs=-1)) == INV
        assert call(pa, dims(pa, max_blocks_per_seq=0)) == INV
        assert call(pa, dims(pa, max_blocks_per_seq=1 << 27)) == INV
        for bad in (dict(window=-1, sinks=0), dict(window=4, sinks=-1), dict(window=0, sinks=-2)):
            assert call(pa, dims(pa), pa.pa_window(**bad)) == INV, bad
        assert call(pa, dims(pa), out_dtype=pa.PA_F16) == INV
        assert call(pa, dims(pa), out_dtype=9) == INV
        assert call(pa, dims(pa), ws_bytes=64) == INV
        assert call(pa, dims(pa), ws=None) == INV
        assert call(pa, dims(pa), ws=P + 128) == INV
        for bad in (dict(q=None), dict(out=None), dict(tables=None), dict(lens=None), dict(q=P + 8), dict(out=P + 4),
                    dict(tables=P + 2), dict(lens=P + 1)):
            assert call(pa, dims(pa), **bad) == INV, bad
        assert call(pa, dims(pa, num_seqs=0)) == pa.PA_OK
    for bad in (dict(max_q=0), dict(max_q=(1 << 20) + 1), dict(T=-1), dict(qs=None), dict(qs=P + 2)):
        assert chunk(pa, dims(pa), **bad) == INV, bad
    assert chunk(pa, dims(pa, num_seqs=65536)) == INV
    assert chunk(pa, dims(pa), T=1 << 29) == INV
    assert chunk(pa, dims(pa), T=0) == pa.PA_OK


def test_write_refusals(pa):
    INV = pa.PA_ERR_INVALID
    for call in (write8, axes_write):
        for bad in (dict(rotary_dim=0), dict(rotary_dim=63), dict(rotary_dim=66), dict(interleaved=2), dict(mscale=float("nan")),
                    dict(mscale=float("inf")), dict(freqs=None), dict(freqs=P + 4)):
            assert call(pa, dims(pa), rope(pa, **bad)) == INV, bad
        assert call(pa, dims(pa), rp=None) == INV
        for bad in (dict(num_axes=0, pair_axis=P), dict(num_axes=17, pair_axis=P), dict(num_axes=3, pair_axis=None),
                    dict(num_axes=3, pair_axis=P + 2)):
            assert call(pa, dims(pa), axes=pa.pa_axes(**bad)) == INV, bad
        for bad in (dict(T=-1), dict(q=None), dict(k=None), dict(v=None), dict(pos=None), dict(slots=None), dict(q_out=None),
                    dict(qs=504), dict(ks=120), dict(vs=64), dict(qos=256), dict(qs=516), dict(ks=132), dict(q=P + 8),
                    dict(slots=P + 4), dict(pos=P + 2), dict(q_out=P, qos=1024), dict(q_out=P + 1024), dict(q_out=2 * P), dict(q_out=3 * P + 256)):
            assert call(pa, dims(pa), **bad) == INV, bad
        assert call(pa, dims(pa, num_q_heads=7)) == INV
        assert call(pa, dims(pa), T=0) == pa.PA_OK
    for bad in (dict(T=-1), dict(k=None), dict(v=None), dict(slots=None), dict(ks=120), dict(vs=132), dict(k=P + 8), dict(slots=P + 4)):
        assert plain_write8(pa, dims(pa), **bad) == INV, bad
    assert plain_write8(pa, dims(pa), T=0) == pa.PA_OK
    assert axes_write(pa, dims(pa), kc=None) == INV and axes_write(pa, dims(pa), vc=6 * P + 8) == INV
    for bad in (dict(n=-1), dict(pairs=None), dict(pairs=P + 4)):
        assert copy8(pa, dims(pa), **bad) == INV, bad
    assert copy8(pa, dims(pa), n=0) == pa.PA_OK


def test_workspaces(pa):
    d = dims(pa)
    assert pa.pa_decode8_workspace_bytes(dims(pa, num_seqs=0)) == 0
    assert pa.pa_decode8_workspace_bytes(dims(pa, head_dim=96)) == 0
    assert pa.pa_chunk8_workspace_bytes(d, 9, 0) == 0
    assert 0 < pa.pa_decode8_workspace_bytes(d) < pa.pa_decode8_workspace_bytes(dims(pa, num_seqs=200, max_blocks_per_seq=100))
    # no more than the warps of the card can fill, whatever the tables hold
    most = pa.pa_decode8_workspace_bytes(dims(pa, num_seqs=4000, max_blocks_per_seq=10000, head_dim=128))
    assert most < 12 << 20


def test_writes_of_too_many_tokens_are_refused(pa):
    assert plain_write8(pa, dims(pa), T=2 ** 31 - 1) == pa.PA_ERR_INVALID
    assert plain_write8(pa, dims(pa), T=2 ** 31 - 20) == pa.PA_ERR_INVALID
    assert write8(pa, dims(pa), T=2 ** 31 - 1) == pa.PA_ERR_INVALID
