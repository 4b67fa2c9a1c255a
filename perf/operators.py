"""Timed cases of the cache operators: rotary positions with the store into a paged KV cache,
attention of single or tree-drafted tokens over that cache, the accumulated attention weight of
its blocks, and the eviction of the blocks that gathered least.

With ``own`` false every operator runs in its plain form (elementary torch operations in 32 bits,
angles in 64); with ``own`` true ``run`` makes the library's calls.  Head counts, head sizes, page
sizes and context lengths are those of the workloads in ``rank_kv_block_amd/workloads.py`` (the
4-head tiny shape, the 32/8-head and the 64/8-head shapes of 128 values a head).
"""

import functools
import math

import torch

own = False

DEV = "cuda"
FP8 = torch.float8_e4m3fn
FP8_MAX = 448.0


def listed():
    return [
        # one decode step of one sequence of the tiny shape: a launch's latency
        dict(name="rotate_step", op="store", Hq=4, Hk=1, D=64, B=16, tokens=1, rot=64, interleaved=False,
             scaling="none", far=1000, fp8=False, fused=True),
        # a prefill chunk on a long context: rotated queries out, keys and values into an FP8 cache,
        # half of each head rotated, neighbours paired
        dict(name="rotate_chunk_fp8", op="store", Hq=32, Hk=8, D=128, B=16, tokens=2048, rot=64, interleaved=True,
             scaling="llama3", far=131072, fp8=True, fused=True),
        # gradient of the rotated queries of two sequences in training at a stretched context
        dict(name="rotate_gradient", op="rotate", Hq=64, Hk=8, D=128, tokens=8190, rot=128, interleaved=False,
             scaling="yarn", far=1000000, backward=True),
        # one decode step of the tiny shape: latency
        dict(name="attend_tiny", op="attend", Hq=4, Hk=1, D=64, B=16, seqs=1, rows=1, blocks=64, fp8=False,
             tree=False, ragged=False, weights=False),
        # one long sequence (131k tokens), one token, with the blocks' weights for eviction
        dict(name="attend_long", op="attend", Hq=32, Hk=8, D=128, B=16, seqs=1, rows=1, blocks=8192, fp8=False,
             tree=False, ragged=False, weights=True),
        # batched decode of 64 sequences up to 32k tokens each, FP8 cache
        dict(name="attend_batch_fp8", op="attend", Hq=32, Hk=8, D=128, B=16, seqs=64, rows=1, blocks=2048, fp8=True,
             tree=False, ragged=True, weights=False),
        # small draft trees verified for a few sequences of the 64-head shape, 32-token pages
        dict(name="attend_tree_13", op="attend", Hq=64, Hk=8, D=128, B=32, seqs=8, rows=13, blocks=257, fp8=False,
             tree=True, ragged=True, weights=False),
        # the largest draft trees over a batch, with the blocks' weights
        dict(name="attend_tree_64", op="attend", Hq=64, Hk=8, D=128, B=16, seqs=16, rows=64, blocks=1024, fp8=False,
             tree=True, ragged=True, weights=True),
        # weights of one decode step of the long sequence
        dict(name="weight_long", op="weight", Hq=32, Hk=8, D=128, B=16, seqs=1, rows=1, blocks=8192),
        # weights of the accepted tokens of a batch's draft trees
        dict(name="weight_trees", op="weight", Hq=32, Hk=8, D=128, B=16, seqs=64, rows=16, blocks=2048),
        # a batch trimmed to its budget of blocks
        dict(name="evict_batch", op="evict", Hq=32, Hk=8, D=128, B=16, seqs=64, blocks=2048, budget=1920, first=1,
             last=8),
        # the long sequence of the 64-head shape trimmed
        dict(name="evict_long", op="evict", Hq=64, Hk=8, D=128, B=32, seqs=1, blocks=32768, budget=30001, first=4,
             last=64),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["store", "store", "rotate", "attend", "attend", "attend", "attend", "weight", "evict"])
    Hk = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 4, 5, 8])
    D = rng.choice([64, 128, 128])
    c = dict(op=op, Hq=Hk * g, Hk=Hk, D=D)
    if op in ("store", "rotate"):
        c.update(tokens=_log_int(rng, 1, 4096), rot=rng.choice([D, D // 2, D // 4]), interleaved=rng.random() < 0.5,
                 scaling=rng.choice(["none", "linear", "ntk", "llama3", "yarn"]), far=_log_int(rng, 100, 1000000))
        if op == "store":
            c.update(B=rng.choice([8, 16, 32]), fp8=rng.random() < 0.5, fused=rng.random() < 0.7)
        else:
            c["backward"] = rng.random() < 0.7
        return c
    c["B"] = rng.choice([8, 16, 16, 32])
    if op == "evict":
        c["seqs"] = _log_int(rng, 1, 64)
        c["blocks"] = _log_int(rng, 20, 131072 // c["seqs"])
        c.update(budget=max(1, int(c["blocks"] * rng.uniform(0.3, 0.99))), first=rng.randrange(5),
                 last=rng.randrange(1, 17))
        return c
    c["rows"] = 1 if rng.random() < 0.4 else _log_int(rng, 2, 64)
    c["seqs"] = _log_int(rng, 1, 64)
    if op == "weight":
        c["blocks"] = _log_int(rng, 2, max(2, 60000000 // (c["seqs"] * c["rows"] * c["Hq"]) // 2))
        c["blocks"] = min(c["blocks"], 16384)
        return c
    # tokens of all sequences: at most a sixteenth of a million for trees of many rows, half a million else
    most = 500000 if c["rows"] * g <= 32 else 120000
    c["blocks"] = max(1 + c["rows"] // c["B"], _log_int(rng, 4, max(5, most // c["seqs"] // c["B"])))
    c.update(fp8=rng.random() < 0.5, tree=c["rows"] > 1 and rng.random() < 0.7, ragged=rng.random() < 0.7,
             weights=rng.random() < 0.4)
    return c


# ------------------------------------------------------------------ rotary frequencies

THETA = 500000.0
ORIGINAL = 8192.0


def _scaling(kind):
    """(factor, low, high) of a scaled rotation: the factors of long-context models in use."""
    return {"none": (1.0, 0.0, 0.0), "linear": (4.0, 0.0, 0.0), "ntk": (8.0, 0.0, 0.0), "llama3": (8.0, 1.0, 4.0),
            "yarn": (16.0, 1.0, 32.0)}[kind]


def _frequencies(rot, kind):
    """Radians a position for each rotated pair, float64, and the factor on cosine and sine."""
    factor, low, high = _scaling(kind)
    i = torch.arange(rot // 2, dtype=torch.float64)
    theta = THETA * factor ** (rot / (rot - 2)) if kind == "ntk" else THETA
    f = theta ** (-2.0 * i / rot)
    if kind == "linear":
        return f / factor, 1.0
    if kind == "llama3":
        wave = 2 * math.pi / f
        mid = (ORIGINAL / wave - low) / (high - low)
        return torch.where(wave < ORIGINAL / high, f, torch.where(wave > ORIGINAL / low, f / factor,
                                                                  (1 - mid) * f / factor + mid * f)), 1.0
    if kind == "yarn":
        at = [rot * math.log(ORIGINAL / (n * 2 * math.pi)) / (2 * math.log(THETA)) for n in (high, low)]
        first, last = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        ramp = ((i - first) / max(last - first, 0.001)).clamp(0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _turn(x, positions, freq, mscale, interleaved, backward, wide):
    """x [n, H, D] with its first 2 * len(freq) values of each head rotated; in float64 if wide, else float32."""
    kind = torch.float64 if wide else torch.float32
    half = freq.numel()
    angle = positions.double()[:, None] * freq[None]
    c, s = (mscale * angle.cos()).to(kind)[:, None], (mscale * angle.sin()).to(kind)[:, None]
    s = -s if backward else s
    x = x.to(kind)
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack((a * c - b * s, a * s + b * c), -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat((a * c - b * s, a * s + b * c), -1)
    return torch.cat((turned, x[..., 2 * half:]), -1)


# ------------------------------------------------------------------ inputs

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)


def _prepare_rotation(c, gen):
    n, Hq, Hk, D = c["tokens"], c["Hq"], c["Hk"], c["D"]
    freq, mscale = _frequencies(c["rot"], c["scaling"])
    s = dict(freq=freq.to(DEV), mscale=mscale)
    start = int(torch.randint(0, c["far"], (1,), generator=gen, device=DEV))
    s["positions"] = (start + torch.arange(n, device=DEV)).to(torch.int32)
    if c["op"] == "rotate":
        s["x"] = _normal(gen, n, Hq, D).bfloat16()
        s["out"] = torch.empty_like(s["x"])
        return s
    if c["fused"]:      # one buffer holds each token's queries, keys and values side by side
        qkv = _normal(gen, n, Hq + 2 * Hk, D).bfloat16()
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    else:
        s["q"], s["k"], s["v"] = (_normal(gen, n, h, D).bfloat16() for h in (Hq, Hk, Hk))
    B = c["B"]
    N = n // B + 3
    pages = torch.randperm(N, generator=gen, device=DEV)
    first = int(torch.randint(0, B, (1,), generator=gen, device=DEV))
    at = first + torch.arange(n, device=DEV)
    s["slots"] = pages[at // B] * B + at % B
    if n > 8:
        s["slots"][n // 3] = -1     # a padding token
    kind = FP8 if c["fp8"] else torch.bfloat16
    s["k_cache"], s["v_cache"] = (torch.zeros((N, B, Hk, D), device=DEV).to(kind) for _ in range(2))
    s["k_scale"], s["v_scale"] = (0.03125, 0.0234375) if c["fp8"] else (1.0, 1.0)
    s["q_out"] = torch.empty((n, Hq, D), device=DEV, dtype=torch.bfloat16)
    s["blocks"] = N
    return s


def _lengths(c, gen):
    S, most = c["seqs"], c["blocks"] * c["B"]
    if not c.get("ragged", True):
        return torch.full((S,), most - 1 if most > c.get("rows", 1) else most, dtype=torch.int32, device=DEV)
    u = torch.rand((S,), generator=gen, device=DEV)
    low = max(most // 4, min(most, c.get("rows", 1)))
    n = (low + u * (most - low)).to(torch.int32)
    n[0] = most
    return n


def _trees(c, gen):
    """Each row's ancestors and itself as a word of bits: row j hangs on a random earlier row or on the context."""
    S, M = c["seqs"], c["rows"]
    u = torch.rand((S, M), generator=gen, device=DEV).cpu()
    words = torch.zeros((S, M), dtype=torch.int64)
    for j in range(M):
        parent = (u[:, j] * (j + 1)).long() - 1
        above = torch.where(parent >= 0, words.gather(1, parent.clamp(min=0)[:, None])[:, 0], torch.zeros((), dtype=torch.int64))
        words[:, j] = above | (1 << j if j < 63 else -(1 << 63))
    return words.to(DEV)


def _prepare_attend(c, gen):
    S, M, Hq, Hk, D, B, n = (c[x] for x in ("seqs", "rows", "Hq", "Hk", "D", "B", "blocks"))
    N = S * n + 5
    s = dict(blocks=N, kv_len=_lengths(c, gen))
    s["tables"] = torch.randperm(N, generator=gen, device=DEV)[:S * n].view(S, n).to(torch.int32)
    s["draft"] = None
    if M > 1:
        s["draft"] = (1 + torch.rand((S,), generator=gen, device=DEV) * M).to(torch.int32).clamp(max=M)
        s["draft"][0] = M
    s["tree"] = _trees(c, gen) if c["tree"] else None
    kind = FP8 if c["fp8"] else torch.bfloat16
    for x in ("k_cache", "v_cache"):
        s[x] = torch.empty((N, B, Hk, D), device=DEV, dtype=kind)
        for at in range(0, N, 16384):       # 16384 pages at a time: the float32 draws stay small
            part = s[x][at:at + 16384]
            part.copy_(_normal(gen, *part.shape).mul_(16 if c["fp8"] else 1).to(kind))
    s["k_scale"], s["v_scale"] = (0.0625, 0.0625) if c["fp8"] else (1.0, 1.0)
    s["q"] = (2 * _normal(gen, S, M, Hq, D)).bfloat16()
    s["scale"] = 1 / math.sqrt(D)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((S, M, Hq), device=DEV, dtype=torch.float32)
    s["block_lse"] = torch.full((S, n, M, Hq), -math.inf, device=DEV) if c["weights"] else None
    return s


def _prepare_weight(c, gen):
    S, M, Hq, B, n = (c[x] for x in ("seqs", "rows", "Hq", "B", "blocks"))
    s = dict(kv_len=_lengths(c, gen), blocks=16)
    used = (s["kv_len"].long() + B - 1) // B
    live = torch.arange(n, device=DEV)[None] < used[:, None]
    x = _normal(gen, S, n, M, Hq).mul_(1.5)
    x[:, 0] += 6        # the first block gathers much of the weight
    x.masked_fill_(~live[:, :, None, None], -math.inf)
    s["block_lse"], s["lse"] = x, torch.logsumexp(x, 1)
    s["accepted"] = None
    if M > 1:           # the accepted path: a few of the rows
        bits = torch.rand((S, M), generator=gen, device=DEV) < 0.3
        bits[:, 0] = True
        word = torch.tensor([1 << j if j < 63 else -(1 << 63) for j in range(M)], device=DEV)
        s["accepted"] = (bits * word).sum(1)
    s["mass"] = _normal(gen, S, n).mul_(2).exp_()
    s["mass_out"] = s["mass"].clone()
    s["decay"] = 0.98
    return s


def _prepare_evict(c, gen):
    S, n = c["seqs"], c["blocks"]
    s = dict(kv_len=_lengths(c, gen), blocks=16)
    s["tables"] = torch.randperm(S * n, generator=gen, device=DEV).view(S, n).to(torch.int32)
    mass = _normal(gen, S, n).mul_(2).exp_()
    mass[torch.rand((S, n), generator=gen, device=DEV) < 0.1] = 0       # blocks no query looked at: ties
    s["mass"] = mass
    s["tables_out"], s["mass_out"] = s["tables"].clone(), mass.clone()
    s["kv_len_out"], s["evicted"] = (torch.empty((S,), device=DEV, dtype=torch.int32) for _ in range(2))
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    make = dict(store=_prepare_rotation, rotate=_prepare_rotation, attend=_prepare_attend, weight=_prepare_weight,
                evict=_prepare_evict)[case["op"]]
    return dict(make(case, gen), case=case)


# ------------------------------------------------------------------ plain forms

def _stored(x, kind, scale):
    """Values as a cache of type `kind` holds them, in its bit patterns."""
    if kind == FP8:
        return (x.float() / scale).clamp(-FP8_MAX, FP8_MAX).to(FP8).view(torch.uint8)
    return x.to(torch.bfloat16).view(torch.int16)


def _plain_rotate(s):
    c = s["case"]
    return _turn(s["x"], s["positions"], s["freq"], s["mscale"], c["interleaved"], c["backward"], False).bfloat16()


def _plain_store(s):
    c = s["case"]
    q, k = (_turn(s[x], s["positions"], s["freq"], s["mscale"], c["interleaved"], False, False) for x in "qk")
    real = (s["slots"] >= 0).nonzero()[:, 0]
    at = s["slots"][real]
    for x, cache, scale in ((k, s["k_cache"], s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])):
        bits = cache.view(torch.uint8 if cache.dtype == FP8 else torch.int16)
        bits.view(-1, *bits.shape[2:])[at] = _stored(x[real], cache.dtype, scale)
    return q.bfloat16(), s["k_cache"], s["v_cache"]


def _gathered(cache, tables):
    """A cache's values through the block tables, float32 [S, Hk, tokens, D]."""
    S, n = tables.shape
    bits = cache.view(torch.uint8 if cache.dtype == FP8 else torch.int16)[tables.long()]
    x = bits.view(cache.dtype).view(S, n * cache.shape[1], *cache.shape[2:])
    return x.transpose(1, 2).float().contiguous()


def _visible(s):
    """Whether drafted row i of a sequence sees its token t, [S, M, tokens]."""
    c = s["case"]
    M, T = c["rows"], c["blocks"] * c["B"]
    t = torch.arange(T, device=DEV)
    i = torch.arange(M, device=DEV)
    n = s["kv_len"].long()
    drafted = n.clamp(max=M) if s["draft"] is None else s["draft"].long()
    j = t[None] - (n - drafted)[:, None]                        # a token's place in the draft; below 0 in the context
    if s["tree"] is None:
        seen = j[:, None] <= i[None, :, None]
    else:
        seen = (j < 0)[:, None] | ((s["tree"][:, :, None] >> j.clamp(0, 63)[:, None]) & 1).bool()
    return seen & (t[None] < n[:, None])[:, None] & (i[None] < drafted[:, None])[:, :, None]


def _log_sum(x):
    """log(sum(exp)) over the last dimension, -inf where it has nothing."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    return (x - m).exp().sum(-1).log() + m[..., 0]


def _plain_attend(s):
    c = s["case"]
    S, M, Hq, Hk, D, B, n = (c[x] for x in ("seqs", "rows", "Hq", "Hk", "D", "B", "blocks"))
    g = Hq // Hk
    q = s["q"].float().view(S, M, Hk, g, D).transpose(1, 2).reshape(S, Hk, M * g, D)
    x = torch.matmul(q, _gathered(s["k_cache"], s["tables"]).transpose(2, 3)) * (s["scale"] * s["k_scale"])
    x = x.view(S, Hk, M, g, n * B).masked_fill(~_visible(s)[:, None, :, None], -math.inf)
    lse = _log_sum(x)
    top = torch.where(lse == -math.inf, torch.zeros_like(lse), lse)
    p = (x - top[..., None]).exp().view(S, Hk, M * g, n * B)
    out = torch.matmul(p, _gathered(s["v_cache"], s["tables"])) * s["v_scale"]
    out = out.view(S, Hk, M, g, D).transpose(1, 2).reshape(S, M, Hq, D).bfloat16()
    found = [out, lse.transpose(1, 2).reshape(S, M, Hq)]
    if c["weights"]:
        found.append(_log_sum(x.view(S, Hk, M, g, n, B)).permute(0, 4, 2, 1, 3).reshape(S, n, M, Hq))
    return found


def _share(s, wide):
    """Each block's share of the accepted rows' attention, summed over rows and heads, [S, blocks]."""
    c = s["case"]
    kind = torch.float64 if wide else torch.float32
    x = (s["block_lse"].to(kind) - s["lse"].to(kind)[:, None]).exp()
    if s["accepted"] is not None:
        bits = (s["accepted"][:, None] >> torch.arange(c["rows"], device=DEV)) & 1
        x = x * bits[:, None, :, None]
    return x.sum((2, 3))


def _plain_weight(s):
    c = s["case"]
    used = (s["kv_len"].long() + c["B"] - 1) // c["B"]
    live = torch.arange(c["blocks"], device=DEV)[None] < used[:, None]
    return torch.where(live, s["decay"] * s["mass"] + _share(s, False), s["mass"])


def _plain_evict(s):
    c = s["case"]
    B, n = c["B"], c["blocks"]
    used = (s["kv_len"].long() + B - 1) // B
    b = torch.arange(n, device=DEV)[None]
    free = (b >= c["first"]) & (b < (used - c["last"])[:, None])
    count = torch.minimum((used - c["budget"]).clamp(min=0), free.sum(1))
    order = torch.where(free, s["mass"], torch.full_like(s["mass"], math.inf)).argsort(dim=1, stable=True)
    place = torch.empty_like(order).scatter_(1, order, b.expand_as(order))
    gone = free & (place < count[:, None])
    # kept blocks in their order, evicted ones behind them, entries past the sequence where they were
    group = gone.long() + 2 * (b >= used[:, None]).long()
    to = group.argsort(dim=1, stable=True)
    tables = s["tables"].gather(1, to)
    mass = s["mass"].gather(1, to).masked_fill(group.gather(1, to) == 1, 0)
    return tables, mass, (s["kv_len"] - count * B).to(torch.int32), count.to(torch.int32)


# ------------------------------------------------------------------ the library's calls

@functools.lru_cache(maxsize=None)
def _handle(Hq, Hk, D, B, blocks):
    import rank_kv_block_amd as rk
    return rk.pred_create(rk.dims(1, Hq, Hk, D, 8, B, blocks), 1)


@functools.lru_cache(maxsize=None)
def _rope(rot, kind, interleaved, backward):
    """The rotation a program keeps: its frequencies on the device."""
    import rank_kv_block_amd as rk
    factor, low, high = _scaling(kind)
    turns, mscale = rk.pred_rope_turns(rot, THETA, kind, factor, low, high, ORIGINAL)
    return rk.Rope(torch.from_numpy(turns.view("int64")).to(DEV), rot, interleaved, mscale, backward)


def _kept(s, name, make):
    """What a program makes once beside its cache and keeps: the cache's description, a workspace."""
    if name not in s:
        s[name] = make()
    return s[name]


def _own(s):
    import rank_kv_block_amd as rk
    c = s["case"]
    if c["op"] == "rotate":
        rk.pred_rotate(_handle(c["Hq"], c["Hk"], c["D"], 16, 16),
                       _rope(c["rot"], c["scaling"], c["interleaved"], c["backward"]), s["x"], s["positions"], s["out"])
        return s["out"]
    h = _handle(c["Hq"], c["Hk"], c["D"], c["B"], s["blocks"])
    if c["op"] in ("store", "attend"):
        cache = _kept(s, "cache", lambda: rk.KVCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]))
    if c["op"] == "store":
        rk.pred_rotate_store(h, _rope(c["rot"], c["scaling"], c["interleaved"], False), s["q"], s["k"], s["v"],
                             s["positions"], s["slots"], cache, s["q_out"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    if c["op"] == "attend":
        ws = _kept(s, "workspace", lambda: torch.empty(
            rk.pred_attend_workspace_bytes(h, c["seqs"], c["rows"], c["blocks"]), dtype=torch.uint8, device=DEV))
        rk.pred_attend(h, cache, s["q"], s["tree"], s["tables"], s["kv_len"], s["draft"], s["scale"], s["out"],
                       s["lse"], s["block_lse"], ws)
        return [s["out"], s["lse"]] + ([s["block_lse"]] if c["weights"] else [])
    if c["op"] == "weight":
        rk.pred_accumulate_weight(h, s["lse"], s["block_lse"], s["accepted"], s["kv_len"], s["decay"], s["mass"],
                                  s["mass_out"])
        return s["mass_out"]
    ws = _kept(s, "workspace", lambda: torch.empty(
        rk.pred_evict_workspace_bytes(c["blocks"], c["seqs"]), dtype=torch.uint8, device=DEV))
    rk.pred_evict_blocks(h, s["tables"], s["mass"], s["kv_len"], c["budget"], c["first"], c["last"], s["tables_out"],
                         s["mass_out"], s["kv_len_out"], s["evicted"], ws)
    return s["tables_out"], s["mass_out"], s["kv_len_out"], s["evicted"]


def run(state):
    if own:
        return _own(state)
    return dict(store=_plain_store, rotate=_plain_rotate, attend=_plain_attend, weight=_plain_weight,
                evict=_plain_evict)[state["case"]["op"]](state)


# ------------------------------------------------------------------ work

def work(case):
    c = case
    Hq, Hk, D = c["Hq"], c["Hk"], c["D"]
    if c["op"] == "rotate":
        return dict(bytes=c["tokens"] * (4 * Hq * D + 4), flops=c["tokens"] * Hq * c["rot"] * 3)
    if c["op"] == "store":
        item = 1 if c["fp8"] else 2
        return dict(bytes=c["tokens"] * (4 * Hq * D + 2 * Hk * D * (2 + item) + 12),
                    flops=c["tokens"] * (Hq + Hk) * c["rot"] * 3)
    S, n = c["seqs"], c["blocks"]
    if c["op"] == "evict":
        return dict(bytes=S * n * 16, flops=0)
    # sequences of uneven length hold five eighths of their table on average
    tokens = S * n * c["B"] * (0.625 if c.get("ragged", True) and S > 1 else 1.0)
    M = c["rows"]
    if c["op"] == "weight":
        rows = M if M == 1 else 0.3 * M
        return dict(bytes=tokens / c["B"] * (rows * Hq * 4 + 8), flops=tokens / c["B"] * rows * Hq * 3)
    item = 1 if c["fp8"] else 2
    moved = tokens * Hk * D * 2 * item + S * M * Hq * (D * 4 + 4) + S * n * 4
    if c["weights"]:
        moved += tokens / c["B"] * M * Hq * 4
    rows = M if M == 1 else 0.5 * M         # drafts of uneven length: half of the rows on average
    return dict(bytes=moved, flops=tokens * rows * Hq * D * 4)


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_rotation(c, s):
    """Each pair as a complex number times mscale * exp(+-i * position * frequency)."""
    freq, pos = s["freq"], s["positions"].double()
    half = freq.numel()

    def turned(x, sign):
        x = x.double()
        head = x[..., :2 * half]
        pair = head.unflatten(-1, (half, 2)) if c["interleaved"] else head.unflatten(-1, (2, half)).transpose(-1, -2)
        z = torch.complex(pair[..., 0].contiguous(), pair[..., 1].contiguous())
        z = z * torch.polar(torch.full_like(pos[:, None] * freq, s["mscale"]), sign * pos[:, None] * freq)[:, None]
        pair = torch.view_as_real(z)
        head = pair.flatten(-2) if c["interleaved"] else pair.transpose(-1, -2).flatten(-2)
        return torch.cat((head, x[..., 2 * half:]), -1)

    if c["op"] == "rotate":
        return turned(s["x"], -1.0 if c["backward"] else 1.0)
    rows = s["slots"].tolist()
    keep = [i for i, slot in enumerate(rows) if slot >= 0]
    at = [rows[i] for i in keep]
    found = [turned(s["q"], 1.0)]
    for x, cache, scale in ((turned(s["k"], 1.0), s["k_cache"], s["k_scale"]),
                            (s["v"].double(), s["v_cache"], s["v_scale"])):
        whole = torch.zeros(cache.shape, dtype=torch.float64, device=DEV)
        whole.view(-1, *cache.shape[2:])[at] = x[keep] / scale
        found.append(whole)
    return tuple(found)


def _exact_attend(c, s):
    """One sequence and kv head at a time, the softmax by its definition over the tokens a row sees."""
    S, M, Hq, Hk, D, B, n = (c[x] for x in ("seqs", "rows", "Hq", "Hk", "D", "B", "blocks"))
    g = Hq // Hk
    out = torch.zeros((S, M, Hq, D), dtype=torch.float64, device=DEV)
    lse = torch.full((S, M, Hq), -math.inf, dtype=torch.float64, device=DEV)
    block = torch.full((S, n, M, Hq), -math.inf, dtype=torch.float64, device=DEV) if c["weights"] else None
    item = torch.uint8 if c["fp8"] else torch.int16
    for q in range(S):
        length = int(s["kv_len"][q])
        rows = min(M, length) if s["draft"] is None else int(s["draft"][q])
        used = (length + B - 1) // B
        pages = s["tables"][q, :used].long()
        k, v = (s[x].view(item)[pages].view(s[x].dtype).flatten(0, 1)[:length].double() for x in ("k_cache", "v_cache"))
        see = torch.ones((rows, length), dtype=torch.bool, device=DEV)
        for i in range(rows):
            word = int(s["tree"][q, i]) if s["tree"] is not None else (1 << (i + 1)) - 1
            seen = [bool(word >> j & 1) for j in range(rows)]
            see[i, length - rows:] = torch.tensor(seen, device=DEV)
        for h in range(Hk):
            head = slice(h * g, h * g + g)
            x = s["q"][q, :rows, head].double().flatten(0, 1) @ k[:, h].t() * (s["scale"] * s["k_scale"])
            x = x.view(rows, g, length).masked_fill(~see[:, None], -math.inf)
            lse[q, :rows, head] = torch.logsumexp(x, -1)
            out[q, :rows, head] = (torch.softmax(x, -1).nan_to_num(0.0).flatten(0, 1) @ v[:, h]).view(rows, g, D) * s["v_scale"]
            if block is not None:
                x = torch.nn.functional.pad(x, (0, used * B - length), value=-math.inf)
                block[q, :used, :rows, head] = torch.logsumexp(x.view(rows, g, used, B), -1).permute(2, 0, 1)
    return [out, lse] + ([block] if block is not None else [])


def _exact_weight(c, s):
    mass = s["mass"].double()
    words = [None] * c["seqs"] if s["accepted"] is None else s["accepted"].tolist()
    for q in range(c["seqs"]):
        used = -(-int(s["kv_len"][q]) // c["B"])
        rows = [i for i in range(c["rows"]) if words[q] is None or words[q] >> i & 1]
        share = torch.exp(s["block_lse"][q, :used][:, rows].double() - s["lse"][q, rows].double())
        mass[q, :used] = s["decay"] * mass[q, :used] + share.flatten(1).sum(1)
    return mass


def _exact_evict(c, s):
    tables, mass, lengths = s["tables"].tolist(), s["mass"].double().tolist(), s["kv_len"].tolist()
    gone_of = []
    for q in range(c["seqs"]):
        used = -(-lengths[q] // c["B"])
        free = range(c["first"], max(c["first"], used - c["last"]))
        gone = sorted(free, key=lambda b: (mass[q][b], b))[:max(0, used - c["budget"])]
        out = set(gone)
        order = [b for b in range(used) if b not in out] + sorted(gone) + list(range(used, c["blocks"]))
        tables[q] = [tables[q][b] for b in order]
        mass[q] = [0.0 if b in out else mass[q][b] for b in order]
        lengths[q] -= len(gone) * c["B"]
        gone_of.append(len(gone))
    whole = functools.partial(torch.tensor, dtype=torch.int32, device=DEV)
    return whole(tables), torch.tensor(mass, dtype=torch.float64, device=DEV), whole(lengths), whole(gone_of)


def exact(case, seed):
    s = prepare(case, seed)
    return dict(store=_exact_rotation, rotate=_exact_rotation, attend=_exact_attend, weight=_exact_weight,
                evict=_exact_evict)[case["op"]](case, s)
