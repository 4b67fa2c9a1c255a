"""The paged KV cache operators, written from their definitions in float64 (test infrastructure only).

Rotary positions (every scaling of the frequencies), the store into a paged cache in bf16 or e4m3, attention of
single or tree-drafted tokens, accumulated attention weight and eviction.  Pins: ``tests/test_oracle_cache.py``
(hand-worked rotations and evictions, an exhaustive e4m3 round trip, a brute-force softmax)."""

import math

import numpy as np


# ---------------------------------------------------------------- rotary positions

def frequencies(rot, theta, kind="none", factor=1.0, low=0.0, high=0.0, original=0.0):
    """Radians a position of each pair [rot / 2], float64, and the factor on cosines and sines."""
    if kind == "ntk":
        theta = theta * factor ** (rot / (rot - 2))
    f = [theta ** (-2.0 * i / rot) for i in range(rot // 2)]
    mscale = 1.0
    if kind == "linear":
        f = [x / factor for x in f]
    elif kind == "llama3":
        out = []
        for x in f:
            wavelength = 2 * math.pi / x
            if wavelength < original / high:
                out.append(x)
            elif wavelength > original / low:
                out.append(x / factor)
            else:
                m = (original / wavelength - low) / (high - low)
                out.append((1 - m) * x / factor + m * x)
        f = out
    elif kind == "yarn":
        def dim_of(turns):
            return rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(theta))
        a, b = max(math.floor(dim_of(high)), 0), min(math.ceil(dim_of(low)), rot - 1)
        ramp = [min(max((i - a) / max(b - a, 0.001), 0.0), 1.0) for i in range(rot // 2)]
        f = [x / factor * r + x * (1 - r) for x, r in zip(f, ramp)]
        mscale = 0.1 * math.log(factor) + 1
    return np.array(f), mscale


def rotate(x, positions, freq, mscale=1.0, interleaved=False, backward=False):
    """x [n, H, D] float64 -> rotated float64."""
    out = np.array(x, dtype=np.float64)
    half = len(freq)
    for t, pos in enumerate(positions):
        angle = float(pos) * freq
        c, s = mscale * np.cos(angle), mscale * np.sin(angle)
        if backward:
            s = -s
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            out[t, :, a] = x[t, :, a] * c[i] - x[t, :, b] * s[i]
            out[t, :, b] = x[t, :, a] * s[i] + x[t, :, b] * c[i]
    return out


def e4m3_values():
    """The value of each of the 256 e4m3 patterns (NaN for 0x7F and 0xFF)."""
    v = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if e == 15 and m == 7:
            x = np.nan
        v[b] = -x if b & 128 else x
    return v


# ---------------------------------------------------------------- attention

def attend_one(q, k, v, seen, scale):
    """One sequence and kv head: q [rows, D], k, v [tokens, D] float64, seen [rows, tokens] bool ->
    (out [rows, D], lse [rows], scores [rows, tokens] with -inf where unseen, absolute [rows, D] =
    sum of softmax weight times |v|)."""
    rows, tokens = seen.shape
    x = np.full((rows, tokens), -np.inf)
    out, lse, absolute = np.zeros(q.shape), np.full(rows, -np.inf), np.zeros(q.shape)
    for i in range(rows):
        at = np.nonzero(seen[i])[0]
        if len(at) == 0:
            continue
        x[i, at] = scale * (k[at] @ q[i])
        m = x[i, at].max()
        p = np.exp(x[i, at] - m)
        lse[i] = m + math.log(p.sum())
        out[i] = (p / p.sum()) @ v[at]
        absolute[i] = (p / p.sum()) @ np.abs(v[at])
    return out, lse, x, absolute


def seen_by(rows, length, drafted, tree_words):
    """[rows, length] bool: what each drafted row sees (rows at or past `drafted`: nothing)."""
    see = np.zeros((rows, length), bool)
    for i in range(min(rows, drafted)):
        see[i, :length - drafted] = True
        for j in range(drafted):
            bit = j <= i if tree_words is None else bool(int(tree_words[i]) >> j & 1)
            see[i, length - drafted + j] = bit
    return see


def block_lse_one(x, block):
    """x [rows, tokens] scores -> [blocks, rows]: the log-sum-exp of each block's tokens."""
    rows, tokens = x.shape
    n = -(-tokens // block)
    out = np.full((n, rows), -np.inf)
    for b in range(n):
        part = x[:, b * block:(b + 1) * block]
        m = part.max(1)
        ok = m > -np.inf
        out[b, ok] = m[ok] + np.log(np.exp(part[ok] - m[ok, None]).sum(1))
    return out


# ---------------------------------------------------------------- weight and eviction

def accumulate(mass, lse, block_lse, used, decay, rows):
    """One sequence: mass [n], lse [M, H], block_lse [n, M, H] -> the new mass; `rows` count."""
    out = np.array(mass, np.float64)
    for b in range(used):
        total = 0.0
        for i in rows:
            ok = lse[i] > -np.inf
            total += np.exp(block_lse[b, i, ok].astype(np.float64) - lse[i, ok].astype(np.float64)).sum()
        out[b] = decay * out[b] + total
    return out


def evict(table, mass, length, block, budget, first, last):
    """One sequence -> (table, mass, length, evicted)."""
    n = -(-length // block)
    candidates = list(range(min(first, n), max(n - last, min(first, n))))
    count = min(max(0, n - budget), len(candidates))
    key = [(float("-inf"), 0) if math.isnan(mass[b]) else (float(mass[b]) + 0.0, 1) for b in range(n)]
    key = [(-1 if k[1] == 0 else 0, 0.0 if k[1] == 0 else k[0]) for k in key]      # NaN before every number
    gone = set(sorted(candidates, key=lambda b: (key[b], b))[:count])
    order = [b for b in range(n) if b not in gone] + [b for b in range(n) if b in gone]
    new_table, new_mass = list(table), list(mass)
    for at, b in enumerate(order):
        new_table[at] = table[b]
        new_mass[at] = 0.0 if b in gone else mass[b]
    return new_table, new_mass, length - count * block, count
