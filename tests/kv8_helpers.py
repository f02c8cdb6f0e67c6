"""Plain 64-bit forms of the 8-bit cache's calls, and the bounds their results are held to."""
from __future__ import annotations

import math

HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}   # of a rounding, relative to the value
CODE_HALF, CODE_SUB = 2.0 ** -4, 2.0 ** -10                            # of an e4m3 code: normal (relative), subnormal


def dtype_of(torch, name):
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def codes_to(torch, codes):
    """e4m3 codes as float64 values."""
    return codes.view(torch.float8_e4m3fn).float().double()


def make_cache(torch, gen, N, Hkv, B, D, spread=1.0, odd_scales=False):
    """A random cache of codes and scales: (k, v, k_scales, v_scales)."""
    def one():
        x = torch.randn(N, Hkv, B, D, generator=gen, device="cuda")
        codes = (x * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
        e = torch.randint(-9, -5, (N, Hkv), generator=gen, device="cuda").float() * spread
        s = torch.exp2(torch.round(e))
        if odd_scales:
            s = s * (1 + torch.rand(N, Hkv, generator=gen, device="cuda"))
        return codes, s
    k, ks = one()
    v, vs = one()
    return k, v, ks, vs


def tables_for(torch, gen, lens, B, extra=3, columns=0):
    need = [-(-n // B) for n in lens]
    N = sum(need) + extra
    place = torch.randperm(N, generator=gen, device="cuda").to(torch.int32)
    columns = max(columns, max(need + [1]))
    t = torch.full((len(lens), columns), -7, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(need):
        t[s, :n] = place[at:at + n]
        at += n
    return t, N


def seen_mask(torch, pos, length, window, sinks):
    """[rows, length]: the keys that each row sees."""
    j = torch.arange(length, device=pos.device)[None]
    m = j <= pos[:, None]
    if window:
        m &= (j > pos[:, None] - window) | (j < sinks)
    return m


def attend_ref(torch, q, cache, tables, lens, counts, scale, window=0, sinks=0, bad=()):
    """(out, bound) in 64 bits for rows q [T, Hq, D] of a chunk call (a decode: counts of 1); `bad` holds the
    (sequence, column) of table entries that are not there.

    The bound of |result - out| apart from the output's own rounding, from these terms: a logit's products are
    exact in fp32 and their sum of D terms is off by D 2^-23 sum |q k| (the tensor cores may truncate);
    its scaling, the scale's logarithm and the exponential are off by 2^-20 (1 + |z|) in the exponent; a weight is
    rounded to f16 (2^-11; a decode keeps 22 bits, which this covers); sums of n terms by n 2^-23; each
    enters once above and once below the fraction, hence twice.  Weights under f16's range lose 2^-31 of the
    largest each.
    """
    k8, v8, ks, vs = cache
    B, D, Hkv = k8.shape[2], k8.shape[3], k8.shape[1]
    Hq = q.shape[1]
    G = Hq // Hkv
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    bound = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    first = 0
    for s, (n, m) in enumerate(zip(lens, counts)):
        if n == 0 or m == 0:
            first += m
            continue
        blocks = tables[s, : -(-n // B)].long().clone()
        gone = torch.zeros(len(blocks) * B, dtype=torch.bool, device=q.device)
        for (bs, col) in bad:
            if bs == s and col < len(blocks):
                gone[col * B:(col + 1) * B] = True
                blocks[col] = 0
        K = (codes_to(torch, k8[blocks].view(torch.uint8)) * ks[blocks].double()[:, :, None, None]).transpose(0, 1).flatten(1, 2)[:, :n]
        V = (codes_to(torch, v8[blocks].view(torch.uint8)) * vs[blocks].double()[:, :, None, None]).transpose(0, 1).flatten(1, 2)[:, :n]
        pos = torch.arange(n - m, n, device=q.device)
        see = seen_mask(torch, pos, n, window, sinks) & ~gone[:n][None]
        any_row = see.any(0)
        K = torch.where(any_row[None, :, None], K, 0.0)
        V = torch.where(any_row[None, :, None], V, 0.0)
        for h in range(Hq):
            x = q[first:first + m, h].double()
            z = (scale * (x @ K[h // G].t())).masked_fill(~see, -math.inf)
            p = torch.softmax(z, -1).nan_to_num(0.0)
            o = p @ V[h // G]
            reach = abs(scale) * (x.abs() @ K[h // G].abs().t()).masked_fill(~see, 0.0).amax(-1)
            e = D * 2.0 ** -23 * reach + 2.0 ** -20 * (1 + reach) + 2.0 ** -11 + n * 2.0 ** -23
            out[first:first + m, h] = o
            bound[first:first + m, h] = 2 * e[:, None] * (p @ V[h // G].abs()) + n * 2.0 ** -31 * V[h // G].abs().max()
        first += m
    return out, bound


def assert_within(got, ref, bound, dtype):
    d = (got.double() - ref).abs()
    lim = bound + HALF_STEP[dtype] * (ref.abs() + bound) + 2.0 ** -140
    if dtype == "f16":
        lim = lim + 2.0 ** -25
    assert bool((d <= lim).all()), f"off by up to {float((d / lim).nan_to_num(1e9).max())} of the bound"


def rotate_ref(torch, x, positions, pair_axis, freqs, R, interleaved, mscale):
    """x [T, heads, D] (any type) with its first R elements turned, in float64; positions [axes, T]."""
    y = x.double().clone()
    half = R // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        t = positions[int(pair_axis[i])].double() * float(freqs[i])
        c, s = (torch.cos(t) * mscale)[:, None], (torch.sin(t) * mscale)[:, None]
        u, w = x[..., a].double(), x[..., b].double()
        y[..., a] = u * c - w * s
        y[..., b] = w * c + u * s
    return y


def power_at_least(x, most):
    """The smallest power of two >= 2^-40 whose `most`-fold holds x (a Python float)."""
    e = -40
    while x > most * 2.0 ** e:
        e += 1
    return 2.0 ** e


def write_ref(torch, cache, slots, k, v, raw_k, k_most, grow):
    """What the write makes of a cache (k8, v8, ks, vs): for K and V (values float64 [N, Hkv, B, D] that the codes should
    be nearest to in units of the scale, or exact old codes; scales; mask of the slots written).  k, v: the
    values to store (float64); raw_k: the keys before their rotation; grow: max(1, |mscale|)."""
    k8, v8, ks, vs = cache
    N, Hkv, B, D = k8.shape
    result = []
    for codes, scales, x, raw, most, f in ((k8, ks, k, raw_k, k_most, grow), (v8, vs, v, v, 448.0, 1.0)):
        now, sc = codes_to(torch, codes).cpu(), scales.double().cpu().clone()
        written = torch.zeros(N, B, dtype=torch.bool)
        sl, x, raw = slots.cpu().tolist(), x.cpu(), raw.double().cpu()
        by_block = {}
        for t, slot in enumerate(sl):
            if 0 <= slot < N * B:
                by_block.setdefault(slot // B, []).append((slot % B, t))
        for blk, toks in by_block.items():
            off = min(o for o, _ in toks)
            for h in range(Hkv):
                vals = torch.cat([raw[t, h] for _, t in toks]).abs()
                vals = vals[torch.isfinite(vals)]
                top = float(vals.max()) if len(vals) else 0.0
                # the library multiplies in fp32
                top = float(torch.tensor(top, dtype=torch.float32) * torch.tensor(f, dtype=torch.float32))
                need = power_at_least(top, most)
                old = float(sc[blk, h])
                new = need if off == 0 else max(need, old)
                if off > 0 and new > old:
                    now[blk, h, :off] = (now[blk, h, :off] * (old / new)).float().to(torch.float8_e4m3fn).double()
                sc[blk, h] = new
                for o, t in toks:
                    now[blk, h, o] = x[t, h] / new
                    written[blk, o] = True
        result.append((now, sc, written))
    return result


def assert_written(torch, codes, scales, ref, slack):
    """Codes against write_ref's: old slots exactly, written ones to half a step of a code plus `slack` (what the values
    themselves may be off by, relative to the largest of their pair, here to the scale's bound of 448)."""
    want, sc, written = ref
    assert torch.equal(scales.cpu().double(), sc), "scales"
    have = codes_to(torch, codes.view(torch.uint8)).cpu()
    w = written[:, None, :, None].expand_as(have)
    same = (have == want) | (have.isnan() & want.isnan())
    assert bool(same[~w].all()), "slots that the call does not write"
    bad = ~torch.isfinite(want)
    assert bool(have[w & bad].isnan().all()), "what is not finite is stored as NaN"
    ok = w & ~bad
    lim = torch.clamp(CODE_HALF * want.abs(), min=CODE_SUB) + slack * 448
    d = (have - want).abs()
    assert bool((d[ok] <= lim[ok]).all()), f"a code is off by {float((d[ok] / lim[ok]).max())} of the bound"
