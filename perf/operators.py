"""Cases of four operators around the paged KV cache, each in a plain form
(elementary torch operations in fp32, no fused call) and as the library's call:

  rope    rotary positions of new queries and keys, and the write of keys and
          values into their cache slots (pa_rope_write_kv);
  decode  one query per sequence over its paged context, with scores capped by
          a tanh, biased by distance or masked to a range of keys, and the
          attention weight of every key added to a running sum
          (pa_decode_scored);
  chunk   the same scores for several new tokens per sequence
          (pa_chunk_scored);
  evict   the keys with the largest sums and the most recent ones copied to
          fresh blocks, for each KV head on its own (pa_evict).

A case is a dict of plain values.  Sequence lengths, chunk lengths and document
borders follow from the case; values and block placement from the seed.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ------------------------------------------------------------------ cases
def _rope(name, **kw):
    c = {"name": name, "op": "rope", "T": 1, "Hq": 32, "Hkv": 8, "D": 128, "B": 16, "dtype": "bf16", "R": 128,
         "interleaved": False, "theta": 10000.0, "scaling": "plain", "factor": 1.0, "far": 4096}
    c.update(kw)
    return c


def _decode(name, **kw):
    c = {"name": name, "op": "decode", "S": 1, "Hq": 32, "Hkv": 8, "D": 128, "B": 16, "dtype": "bf16", "out": "bf16",
         "lens": "uniform", "lo": 1, "hi": 4096, "cap": 0.0, "window": 0, "slopes": False, "docs": 0, "sums": False}
    c.update(kw)
    return c


def _chunk(name, **kw):
    c = {"name": name, "op": "chunk", "S": 1, "Hq": 32, "Hkv": 8, "D": 128, "B": 16, "dtype": "bf16", "out": "bf16",
         "lens": "uniform", "lo": 0, "hi": 4096, "nlo": 1, "nhi": 1, "cap": 0.0, "window": 0, "slopes": False,
         "docs": 0, "prefix": 0}
    c.update(kw)
    return c


def _evict(name, **kw):
    c = {"name": name, "op": "evict", "S": 1, "Hkv": 8, "D": 128, "B": 16, "dtype": "bf16", "lens": "uniform",
         "lo": 4096, "hi": 4096, "keep": 2048, "recent": 256}
    c.update(kw)
    return c


def listed():
    return [
        # one new token of one sequence: only latency counts
        _rope("rope_one", T=1),
        # a decode step of 256 sequences at far positions, frequencies stretched for a long context
        _rope("rope_step", T=256, Hq=64, Hkv=8, B=32, scaling="ramp", factor=8.0, far=65536),
        # a prompt pass of 16 x 512 tokens, neighbouring pairs, half of each head rotated
        _rope("rope_prompt", T=8192, Hq=32, Hkv=32, dtype="f16", R=64, interleaved=True),
        # a few short fp32 sequences, biased by distance (the smallest call)
        _decode("decode_few", S=3, Hq=4, Hkv=4, D=64, dtype="f32", out="f32", lo=12, hi=47, slopes=True),
        # the 8B-shaped decode batch with capped scores and the sums that eviction reads
        _decode("decode_cap_sums", S=256, lens="lognormal", lo=1, hi=4096, cap=30.0, sums=True),
        # multi-head, biased by distance, only the current document of each packed sequence
        _decode("decode_bias_docs", S=64, Hq=32, Hkv=32, dtype="f16", out="f16", lo=1, hi=2048, slopes=True, docs=1500),
        # long sequences of which each layer sees a window
        _decode("decode_window", S=32, Hq=64, Hkv=8, B=32, lo=8192, hi=32768, window=4096, sums=True),
        # five drafted tokens of 256 sequences verified at once, capped scores
        _chunk("chunk_verify", S=256, lens="lognormal", lo=1, hi=4096, nlo=5, nhi=5, cap=30.0),
        # 512-token prompt chunks over packed documents, capped scores
        _chunk("chunk_docs", S=16, lo=0, hi=3584, nlo=512, nhi=512, cap=50.0, docs=4000),
        # ragged prompts whose first tokens all see each other, biased by distance
        _chunk("chunk_prefix", S=5, D=64, dtype="f16", out="f16", lo=0, hi=1500, nlo=200, nhi=777, slopes=True, prefix=300),
        # 64 sequences that outgrew their budget
        _evict("evict_batch", S=64, lens="uniform", lo=2500, hi=4096, keep=2048, recent=256),
        # one long sequence cut to a quarter
        _evict("evict_long", S=1, D=64, dtype="f16", lo=32768, hi=32768, keep=8192, recent=1000),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "decode", "decode", "chunk", "chunk", "evict"])
    Hq, Hkv = rng.choice([(32, 8), (64, 8), (32, 32), (8, 1), (12, 6), (16, 2), (4, 4)])
    D, B = rng.choice([64, 128]), rng.choice([16, 32])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "rope":
        scaling = rng.choice(["plain", "linear", "ramp"])
        c = _rope("", T=_log_int(rng, 1, 8192), Hq=Hq, Hkv=Hkv, D=D, B=B, dtype=rng.choice(["f32", "bf16", "f16"]),
                  R=rng.choice([D, D, D // 2, 32, 20, 2 * rng.randint(1, D // 2)]), interleaved=rng.random() < 0.5,
                  theta=rng.choice([10000.0, 500000.0]), scaling=scaling,
                  factor=1.0 if scaling == "plain" else rng.choice([2.0, 4.0, 8.0]), far=_log_int(rng, 16, 131072))
        if c["T"] * (c["Hq"] + c["Hkv"]) * BYTES[c["dtype"]] * D > 8192 * 96 * 256:
            c["T"] = c["T"] // 4
    elif op == "decode":
        S = _log_int(rng, 1, 256)
        hi = _log_int(rng, 1, min(32768, 700000 // S))
        c = _decode("", S=S, Hq=Hq, Hkv=Hkv, D=D, B=B, dtype=dtype, out=dtype, lo=rng.choice([1, max(1, hi // 2)]), hi=hi,
                    cap=rng.choice([0.0, 20.0, 30.0, 50.0]), window=rng.choice([0, 0, _log_int(rng, 1, hi)]),
                    slopes=rng.random() < 0.4, docs=rng.choice([0, 0, _log_int(rng, 1, hi)]), sums=rng.random() < 0.5)
        if rng.random() < 0.15:
            c.update(dtype="f32", out="f32", S=min(S, 32), hi=min(hi, 4096), lo=1)
    elif op == "chunk":
        n = _log_int(rng, 1, 800)
        S = _log_int(rng, 1, max(1, min(256, 8192 // n)))
        hi = _log_int(rng, 1, min(4096, 600000 // S))
        c = _chunk("", S=S, Hq=Hq, Hkv=Hkv, D=D, B=B, dtype=dtype, out=dtype, lo=0, hi=hi,
                   nlo=max(1, n - rng.choice([0, 0, n // 2])), nhi=n, cap=rng.choice([0.0, 30.0, 50.0]),
                   window=rng.choice([0, 0, _log_int(rng, 1, hi)]), slopes=rng.random() < 0.4,
                   docs=rng.choice([0, 0, _log_int(rng, 1, hi)]), prefix=rng.choice([0, 0, _log_int(rng, 1, hi)]))
        if c["Hq"] == 64 and c["S"] * n > 4096:
            c["S"] = max(1, c["S"] // 2)
    else:
        S = _log_int(rng, 1, 64)
        hi = _log_int(rng, 64, min(32768, 250000 // S))
        keep = rng.randint(1, hi)
        c = _evict("", S=S, Hkv=rng.choice([1, 2, 6, 8]), D=D, B=B, dtype=rng.choice([dtype, dtype, "f32"]), lo=max(1, hi // 2), hi=hi, keep=keep,
                   recent=rng.randint(0, keep))
    del c["name"]
    return c


# ------------------------------------------------------------------ what follows from the case alone
def _shape_rng(case):
    return random.Random("%s %s %s %s" % (case["op"], case.get("S", case.get("T")), case.get("hi"), case["D"]))


def _lengths(case):
    """Stored tokens of each sequence (chunk: before its new tokens)."""
    r = _shape_rng(case)
    if case["lens"] == "lognormal":  # median 600, as in the repository's 8B-shaped batch
        return [min(case["hi"], max(case["lo"], int(round(600.0 * math.exp(0.8 * r.gauss(0.0, 1.0)))))) for _ in range(case["S"])]
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["S"])]


def _chunks(case):
    """(context length with the new tokens, new tokens) of each sequence."""
    r = random.Random(_shape_rng(case).random())
    return [(n + m, m) for n, m in ((n, r.randint(case["nlo"], case["nhi"])) for n in _lengths(case))]


def _borders(case, length, s):
    """First positions of the documents packed into sequence s, ragged around case["docs"] tokens each."""
    r = random.Random(1000003 * s + length)
    at, got = 0, []
    while at < length:
        got.append(at)
        at += max(1, int(case["docs"] * r.uniform(0.4, 1.6)))
    return got


def _ranges(case):
    """Per query: (sequence, position, first key, one past the last key)."""
    rows = []
    pairs = [(n, 1) for n in _lengths(case)] if case["op"] == "decode" else _chunks(case)
    for s, (length, n) in enumerate(pairs):
        starts = _borders(case, length, s) if case["docs"] else [0]
        k = 0
        for pos in range(length - n, length):
            while k + 1 < len(starts) and starts[k + 1] <= pos:
                k += 1
            begin, end = starts[k], pos + 1
            if case.get("prefix"):
                end = min(length, max(end, case["prefix"]))
            if case["window"]:
                begin = max(begin, pos - case["window"] + 1)
            rows.append((s, pos, begin, end))
    return rows


def work(case):
    b, D = BYTES[case["dtype"]], case["D"]
    if case["op"] == "rope":
        T, heads = case["T"], case["Hq"] + case["Hkv"]
        return {"bytes": T * (2 * heads * D + 2 * case["Hkv"] * D) * b + T * 12, "flops": 3 * T * heads * case["R"]}
    if case["op"] == "evict":
        lens = _lengths(case)
        kept = sum(min(n, case["keep"]) for n in lens if n > case["keep"])
        sums = sum(n + min(n, case["keep"]) for n in lens)
        return {"bytes": 4 * kept * case["Hkv"] * D * b + 4 * sums * case["Hkv"], "flops": 0}
    rows = _ranges(case)
    seen = {}
    for s, pos, begin, end in rows:  # the distinct keys that some query of a sequence sees
        if begin < end:
            lo, hi = seen.get(s, (begin, end))
            seen[s] = (min(lo, begin), max(hi, end))
    keys = sum(hi - lo for lo, hi in seen.values())
    pairs = sum(max(0, end - begin) for s, pos, begin, end in rows)
    io = len(rows) * case["Hq"] * D * (b + BYTES[case["out"]])
    if case.get("sums"):
        io += 8 * keys * case["Hkv"]
    return {"bytes": 2 * keys * case["Hkv"] * D * b + io, "flops": 4 * D * case["Hq"] * pairs}


# ------------------------------------------------------------------ inputs
def _frequencies(case):
    """Radians per position of each rotated pair, and the factor on cos and sin."""
    R, theta, factor = case["R"], case["theta"], case["factor"]
    f = torch.tensor([theta ** (-2.0 * i / R) for i in range(R // 2)], dtype=torch.float64)
    if case["scaling"] == "linear":
        return f / factor, 1.0
    if case["scaling"] == "ramp":  # fast pairs as they were, slow ones stretched, a ramp between
        dim = lambda turns: R * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
        low, high = math.floor(dim(32.0)), math.ceil(dim(1.0))
        ramp = ((torch.arange(R // 2, dtype=torch.float64) - low) / max(high - low, 1e-3)).clamp(0, 1)
        return f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _tables(lens, B, extra, gen, columns=0):
    """Block tables over a shuffled pool with a few blocks to spare: [S, columns], padded with -1."""
    need = [-(-n // B) for n in lens]
    N = sum(need) + extra
    columns = columns or max(1, max(need))
    place = torch.randperm(N, generator=gen, device="cuda").to(torch.int32)
    count = torch.tensor(need, device="cuda")
    j = torch.arange(columns, device="cuda")
    at = (count.cumsum(0) - count)[:, None] + j[None, :]
    tables = torch.where(j[None, :] < count[:, None], place[at.clamp(max=N - 1)], torch.full_like(place[:1], -1))
    return tables.contiguous(), N, place[sum(need):]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * std).to(dt)

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    D, B, Hkv = case["D"], case["B"], case["Hkv"]
    st = dict(case)
    if case["op"] == "rope":
        T, Hq = case["T"], case["Hq"]
        N = -(-T // B) + 4
        freqs, mscale = _frequencies(case)
        # queries, keys and values as one projection leaves them: column ranges of one row per token
        fused = normal(T, (Hq + 2 * Hkv) * D)
        q, k, v = fused.split([Hq * D, Hkv * D, Hkv * D], dim=1)
        st.update(q=q.view(T, Hq, D), k=k.view(T, Hkv, D), v=v.view(T, Hkv, D), freqs=freqs.cuda(), mscale=mscale,
                  positions=torch.randint(0, case["far"], (T,), generator=gen, device="cuda", dtype=torch.int32),
                  slots=torch.randperm(N * B, generator=gen, device="cuda")[:T].contiguous(),
                  q_out=torch.zeros(T, Hq, D, dtype=dt, device="cuda"), k_cache=normal(N, Hkv, B, D),
                  v_cache=normal(N, Hkv, B, D))
        return st
    if case["op"] == "evict":
        lens = _lengths(case)
        cols = -(-case["hi"] // B) * B
        tables, N, spare = _tables(lens, B, 4 + sum(-(-case["keep"] // B) for n in lens if n > case["keep"]), gen, cols // B)
        per = -(-case["keep"] // B)
        fresh = torch.full((len(lens), cols // B), -1, dtype=torch.int32, device="cuda")
        gone = torch.tensor([s for s, n in enumerate(lens) if n > case["keep"]], device="cuda", dtype=torch.int64)
        fresh[gone, :per] = spare[: per * gone.numel()].view(-1, per)
        # weights of many decode steps: a heavy tail, and keys that nothing looked at
        sums = torch.exp(2.0 * torch.randn(len(lens), Hkv, cols, generator=gen, device="cuda"))
        sums = torch.where(torch.rand(sums.shape, generator=gen, device="cuda") < 0.05, 0.0, sums)
        st.update(tables=tables, new_tables=fresh, lens=i32(lens), keep_lens=i32([case["keep"]] * len(lens)), sums=sums,
                  k_cache=normal(N, Hkv, B, D), v_cache=normal(N, Hkv, B, D), sums_out=torch.zeros_like(sums),
                  new_lens=torch.zeros(len(lens), dtype=torch.int32, device="cuda"))
        return st
    Hq = case["Hq"]
    if case["op"] == "decode":
        lens = _lengths(case)
        T, most = len(lens), 1
    else:
        lens, counts = zip(*_chunks(case))
        T, most = sum(counts), max(counts)
        st["query_start"] = i32([sum(counts[:s]) for s in range(len(counts) + 1)])
    tables, N, _ = _tables(lens, B, 4, gen)
    # logits of a spread that the cap bends; with none they are those of unit queries
    std = 4.0 if case["cap"] else 1.0
    st.update(q=normal(T, Hq, D, std=std), k_cache=normal(N, Hkv, B, D), v_cache=normal(N, Hkv, B, D), tables=tables,
              lens=i32(list(lens)), scale=1.0 / math.sqrt(D), most=most, key_begin=None, key_end=None, slope=None,
              sum=None, result=torch.zeros(T, Hq, D, dtype=DTYPES[case["out"]], device="cuda"))
    rows = _ranges(dict(case, window=0))
    if case["docs"]:
        st["key_begin"] = i32([r[2] for r in rows])
    if case.get("prefix"):
        st["key_end"] = i32([r[3] for r in rows])
    if case["slopes"]:
        st["slope"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], device="cuda")
    if case.get("sums"):
        # the sums of a few earlier steps
        st["sum"] = 0.02 * torch.rand(len(lens), Hkv, tables.shape[1] * B, generator=gen, device="cuda")
    return st


# ------------------------------------------------------------------ the operators
def run(state):
    return (_own if own else _plain)[state["op"]](state)


def _plain_rope(st):
    R, D = st["R"], st["D"]
    turns = st["positions"].double()[:, None] * st["freqs"][None, :]
    cos = (torch.cos(turns) * st["mscale"]).float()[:, None, :]
    sin = (torch.sin(turns) * st["mscale"]).float()[:, None, :]

    def rotate(x):
        x = x.float()
        r, rest = x[..., :R], x[..., R:]
        a, b = (r[..., 0::2], r[..., 1::2]) if st["interleaved"] else (r[..., : R // 2], r[..., R // 2:])
        y = (a * cos - b * sin, b * cos + a * sin)
        return torch.cat([torch.stack(y, -1).flatten(-2) if st["interleaved"] else torch.cat(y, -1), rest], -1)

    block, offset = st["slots"] // st["B"], st["slots"] % st["B"]
    st["q_out"].copy_(rotate(st["q"]))
    st["k_cache"][block, :, offset] = rotate(st["k"]).to(st["k_cache"].dtype)
    st["v_cache"][block, :, offset] = st["v"]
    return {"q": st["q_out"], "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _context(cache, tables):
    """[S, Hkv, columns * B, D] in fp32 of each sequence, through its table."""
    S, columns = tables.shape
    _, Hkv, B, D = cache.shape
    return cache[tables.clamp(min=0).long()].permute(0, 2, 1, 3, 4).reshape(S, Hkv, columns * B, D).float()


def _plain_scored(st, q, pos, begin, end, slope_rows):
    """q [S, Hkv, n, G, D] fp32 with its position and key range [S, n]: weights [S, Hkv, n, G, L] and outputs."""
    S, Hkv, n, G, D = q.shape
    k, v = _context(st["k_cache"], st["tables"]), _context(st["v_cache"], st["tables"])
    at = torch.arange(k.shape[2], device="cuda")
    x = torch.matmul(q.reshape(S, Hkv, n * G, D), k.transpose(-1, -2)).view(S, Hkv, n, G, -1) * st["scale"]
    if st["cap"]:
        x = torch.tanh(x / st["cap"]) * st["cap"]
    if slope_rows is not None:
        x = x - slope_rows * (pos[:, :, None] - at).abs().float()[:, None, :, None, :]
    seen = (at >= begin[:, :, None]) & (at < end[:, :, None])
    if st["window"]:
        seen = seen & (at > pos[:, :, None] - st["window"])
    x = torch.where(seen[:, None, :, None, :], x, -math.inf)
    most = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(most == -math.inf, 0.0, most))
    total = x.sum(-1, keepdim=True)
    x = x / torch.where(total == 0, 1.0, total)
    return x, torch.matmul(x.view(S, Hkv, n * G, -1), v).view(S, Hkv, n, G, D)


def _slope_rows(st, G):
    return None if st["slope"] is None else st["slope"].view(1, st["Hkv"], 1, G, 1)


def _plain_decode(st):
    S, Hq, D = st["q"].shape
    Hkv = st["Hkv"]
    lens = st["lens"][:, None]
    begin = torch.zeros_like(lens) if st["key_begin"] is None else st["key_begin"][:, None]
    w, o = _plain_scored(st, st["q"].float().view(S, Hkv, 1, Hq // Hkv, D), lens - 1, begin, lens, _slope_rows(st, Hq // Hkv))
    st["result"].copy_(o.reshape(S, Hq, D))
    if st["sum"] is None:
        return {"out": st["result"]}
    st["sum"] += w.sum((2, 3))
    return {"out": st["result"], "sums": st["sum"]}


def _plain_chunk(st):
    T, Hq, D = st["q"].shape
    S, n, Hkv = st["lens"].shape[0], st["most"], st["Hkv"]
    G = Hq // Hkv
    start = st["query_start"].long()
    i = torch.arange(T, device="cuda")
    s = torch.searchsorted(start, i, right=True) - 1
    t = i - start[s]

    def padded(rows, fill):
        to = torch.full((S, n) + rows.shape[1:], fill, dtype=rows.dtype, device="cuda")
        to[s, t] = rows
        return to

    pos = st["lens"].long()[s] - (start[s + 1] - start[s]) + t
    begin = torch.zeros_like(pos) if st["key_begin"] is None else st["key_begin"].long()
    end = pos + 1 if st["key_end"] is None else st["key_end"].long()
    q = padded(st["q"].float(), 0.0).view(S, n, Hkv, G, D).transpose(1, 2)
    _, o = _plain_scored(st, q, padded(pos, 0), padded(begin, 0), padded(end, 0), _slope_rows(st, G))
    st["result"].copy_(o.transpose(1, 2).reshape(S, n, Hq, D)[s, t])
    return {"out": st["result"]}


def _plain_evict(st):
    S, Hkv, cols = st["sums"].shape
    keep, recent, B = st["keep"], st["recent"], st["B"]
    at = torch.arange(cols, device="cuda")
    lens = st["lens"].long()[:, None, None]
    cut = lens > keep
    old = (at < lens - recent).expand(S, Hkv, cols)
    # the first keep - recent of the older keys by falling sum, equal sums by rising index
    order = torch.sort(torch.where(old, st["sums"], -math.inf), dim=-1, descending=True, stable=True).indices
    chosen = torch.zeros(S, Hkv, cols, dtype=torch.bool, device="cuda")
    chosen.scatter_(2, order[..., : keep - recent], True)
    chosen = ((chosen & old) | (at >= lens - recent)) & (at < lens)
    # the kept keys in their order: their indices first, then the others
    first = torch.sort(torch.where(chosen, at, at + cols), dim=-1).indices[..., :keep]
    new = torch.minimum(lens, torch.full_like(lens, keep))
    s, h = torch.arange(S, device="cuda")[:, None, None], torch.arange(Hkv, device="cuda")[None, :, None]
    to = torch.arange(first.shape[-1], device="cuda")
    # sequences within their budget keep their blocks: here they copy their first row to itself
    row = torch.where(cut, first, 0)
    source = st["tables"].long()[s, row // B]
    target = torch.where(cut, st["new_tables"].long()[s, to // B], source)
    slot = torch.where(cut, to % B, 0)
    for cache in (st["k_cache"], st["v_cache"]):
        cache[target, h, slot] = cache[source, h, row % B]
    moved = torch.zeros_like(st["sums"])
    moved[..., : first.shape[-1]] = torch.gather(st["sums"], 2, first)
    st["sums_out"].copy_(torch.where(at < new, torch.where(cut, moved, st["sums"]), 0.0))
    st["new_lens"].copy_(new.view(-1))
    return {"k_cache": st["k_cache"], "v_cache": st["v_cache"], "sums": st["sums_out"], "lens": st["new_lens"]}


_plain = {"rope": _plain_rope, "decode": _plain_decode, "chunk": _plain_chunk, "evict": _plain_evict}


def _dims(pa, st, seqs, columns):
    N, Hkv, B, D = st["k_cache"].shape
    return pa.make_dims(seqs, st.get("Hq", Hkv), Hkv, D, B, N, columns, 0, st["dtype"])


def _scratch(st, nbytes):
    """The workspace that a program keeps for its calls of one shape."""
    if "workspace" not in st:
        st["workspace"] = torch.empty(max(nbytes, 256), dtype=torch.uint8, device="cuda")
    return st["workspace"]


def _own_rope(st):
    from paged_kv_cache_127_gb300 import binding as pa
    pa.pa_rope_write_kv(_dims(pa, st, 0, 1), pa.make_rope(st["R"], st["freqs"], st["interleaved"], st["mscale"]),
                        st["q"], st["k"], st["v"], st["positions"], st["slots"], st["q_out"], st["k_cache"], st["v_cache"])
    return {"q": st["q_out"], "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _own_decode(st):
    from paged_kv_cache_127_gb300 import binding as pa
    dims = _dims(pa, st, *st["tables"].shape)
    score = pa.make_score(softcap=st["cap"], window=st["window"], slopes=st["slope"], key_begin=st["key_begin"])
    ws = _scratch(st, pa.pa_decode_scored_workspace_bytes(dims, st["sum"] is not None))
    pa.pa_decode_scored(dims, score, st["q"], st["k_cache"], st["v_cache"], st["tables"], st["lens"], st["scale"],
                        st["result"], ws, key_sums=st["sum"])
    return {"out": st["result"]} if st["sum"] is None else {"out": st["result"], "sums": st["sum"]}


def _own_chunk(st):
    from paged_kv_cache_127_gb300 import binding as pa
    dims = _dims(pa, st, *st["tables"].shape)
    score = pa.make_score(softcap=st["cap"], window=st["window"], slopes=st["slope"], key_begin=st["key_begin"],
                          key_end=st["key_end"])
    ws = _scratch(st, pa.pa_chunk_scored_workspace_bytes(dims, st["q"].shape[0], st["most"]))
    pa.pa_chunk_scored(dims, score, st["q"], st["k_cache"], st["v_cache"], st["tables"], st["lens"], st["query_start"],
                       st["scale"], st["result"], st["most"], ws)
    return {"out": st["result"]}


def _own_evict(st):
    from paged_kv_cache_127_gb300 import binding as pa
    dims = _dims(pa, st, *st["tables"].shape)
    ws = _scratch(st, pa.pa_evict_workspace_bytes(dims))
    pa.pa_evict(dims, st["k_cache"], st["v_cache"], st["tables"], st["lens"], st["new_tables"], st["keep_lens"], st["recent"],
                st["sums"], st["sums_out"], st["new_lens"], ws)
    return {"k_cache": st["k_cache"], "v_cache": st["v_cache"], "sums": st["sums_out"], "lens": st["new_lens"]}


_own = {"rope": _own_rope, "decode": _own_decode, "chunk": _own_chunk, "evict": _own_evict}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(st)
    if case["op"] == "evict":
        return _exact_evict(case, st)
    rows = _ranges(case)
    if sum(r[3] - r[2] for r in rows if r[3] > r[2]) * case["Hq"] * case["D"] > 6e11:
        return None
    Hq, Hkv, B = case["Hq"], case["Hkv"], case["B"]
    G = Hq // Hkv
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    sums = None if st["sum"] is None else st["sum"].double()
    lens, table_rows = st["lens"].tolist(), st["tables"].tolist()
    begins = torch.tensor([r[2] for r in rows], device="cuda")
    ends = torch.tensor([r[3] for r in rows], device="cuda")
    first = 0
    for s, length in enumerate(lens):
        n = 0
        while first + n < len(rows) and rows[first + n][0] == s:
            n += 1
        blocks = torch.tensor(table_rows[s][: -(-length // B)], device="cuda")
        keys = st["k_cache"][blocks].transpose(0, 1).flatten(1, 2)[:, :length].double()
        values = st["v_cache"][blocks].transpose(0, 1).flatten(1, 2)[:, :length].double()
        j = torch.arange(length, device="cuda")
        mine = slice(first, first + n)
        position = torch.arange(length - n, length, device="cuda")
        hidden = (j[None] < begins[mine, None]) | (j[None] >= ends[mine, None])
        for h in range(Hq):
            z = st["scale"] * (st["q"][mine, h].double() @ keys[h // G].t())
            if case["cap"]:
                z = case["cap"] * torch.tanh(z / case["cap"])
            if st["slope"] is not None:
                z -= float(st["slope"][h].double()) * (j[None] - position[:, None]).abs()
            p = torch.softmax(z.masked_fill(hidden, -math.inf), -1).nan_to_num(0.0)
            out[mine, h] = p @ values[h // G]
            if sums is not None:
                sums[s, h // G, :length] += p.sum(0)
        first += n
    return {"out": out} if sums is None else {"out": out, "sums": sums}


def _exact_rope(st):
    R, B = st["R"], st["B"]
    angle = torch.outer(st["positions"].double(), st["freqs"])
    turn = torch.polar(torch.full_like(angle, st["mscale"]), angle)[:, None, :]
    pair = torch.arange(R // 2, device="cuda")
    re, im = (2 * pair, 2 * pair + 1) if st["interleaved"] else (pair, pair + R // 2)

    def spin(x):
        y = x.double().clone()
        z = torch.complex(y[..., re], y[..., im]) * turn
        y[..., re], y[..., im] = z.real, z.imag
        return y

    kc, vc = st["k_cache"].double(), st["v_cache"].double()
    kc[st["slots"].div(B, rounding_mode="floor"), :, st["slots"].remainder(B)] = spin(st["k"])
    vc[st["slots"].div(B, rounding_mode="floor"), :, st["slots"].remainder(B)] = st["v"].double()
    return {"q": spin(st["q"]), "k_cache": kc, "v_cache": vc}


def _exact_evict(case, st):
    kc, vc = st["k_cache"].double(), st["v_cache"].double()
    sums, out = st["sums"].double().cpu(), torch.zeros(st["sums"].shape, dtype=torch.float64)
    lens, keep, recent, B = st["lens"].tolist(), case["keep"], case["recent"], case["B"]
    for s, n in enumerate(lens):
        if n <= keep:
            out[s, :, :n] = sums[s, :, :n]
            continue
        to = torch.arange(keep, device="cuda")
        dst = st["new_tables"][s].long()[to // B]
        for h in range(case["Hkv"]):
            w = sums[s, h, : n - recent].numpy()
            best = (-w).argsort(kind="stable")[: keep - recent]
            best.sort()
            kept = torch.cat([torch.from_numpy(best), torch.arange(n - recent, n)])
            out[s, h, :keep] = sums[s, h, kept]
            kept = kept.cuda()
            src = st["tables"][s].long()[kept // B]
            kc[dst, h, to % B] = st["k_cache"][src, h, kept % B].double()
            vc[dst, h, to % B] = st["v_cache"][src, h, kept % B].double()
    return {"k_cache": kc, "v_cache": vc, "sums": out, "lens": None}
