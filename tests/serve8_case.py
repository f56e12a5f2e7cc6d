"""Plain 64-bit forms of the 8-bit cache rows, of beam selection and of beam reordering.

A row of an 8-bit cache: 512 e4m3 values, 64 rotary values in 16 bits, 16 exponents (biased by 127) of the
scales of 32 latent values each.  The scale is the least power of two 2^k that brings the group's largest value
to 448, the largest e4m3, or below; k is no less than -110 (bf16) or -15 (f16), and at its greatest, 120 or 8, values
end at 240 times it.

Bounds.  e4m3 has three fraction bits: a value is off by half a step, 2^(e - 4) for |value| in [2^e, 2^(e + 1)) with e
no less than -6, in units of the scale.  The value that is rounded is computed in fp32: a mean of squares by
fourteen additions of positive terms, each off by 2^-24 (half of it behind the square root), a square root, a
quotient and two products: 7 + 4 units of 2^-24, DELTA with some room."""
import numpy as np
import torch

LATENT, ROPE = 512, 64
ROW = LATENT + ROPE
GROUP = 32
ROW8 = LATENT + 2 * ROPE + LATENT // GROUP
LEAST, MOST = {"bf16": -110, "f16": -15}, {"bf16": 120, "f16": 8}
LARGEST = {"bf16": (2.0 - 2.0 ** -8) * 2.0 ** 127, "f16": 65520.0 - 2.0 ** -20}   # below these a value rounds to a finite one
TYPE = {"bf16": torch.bfloat16, "f16": torch.float16}
DELTA = 16 * 2.0 ** -24


def e4m3():
    """The value of each of the 256 bytes."""
    byte = np.arange(256)
    e, m = (byte >> 3) & 15, byte & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v[(byte & 127) == 127] = np.nan
    return np.where(byte >= 128, -v, v)


VALUES = e4m3()


def exponents(most, dtype):
    """k of groups whose largest values are `most`."""
    k = np.full(most.shape, LEAST[dtype], int)
    some = most > 0
    k[some] = np.maximum(np.ceil(np.log2(most[some] / 448.0)).astype(int), LEAST[dtype])
    while True:                                               # the logarithm may be off by a rounding
        low = most > 448.0 * 2.0 ** k.astype(float)
        high = (k > LEAST[dtype]) & (most <= 448.0 * 2.0 ** (k.astype(float) - 1))
        if not (low.any() or high.any()):
            return np.minimum(k, MOST[dtype])
        k = k + low - high


def half_step(x):
    """Half of e4m3's step at |x|."""
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -30)))
    return 2.0 ** (np.maximum(e, -6) - 4)


def codes(x):
    """The bytes of the e4m3 values nearest to x, ties to even."""
    step = 2 * half_step(x)
    q = np.clip(np.round(x / step) * step, -448, 448)
    at = np.searchsorted(VALUES[:127], np.abs(q))
    assert np.array_equal(VALUES[at], np.abs(q))
    return (at + 128 * np.signbit(x)).astype(np.uint8)


def pack(latent, rope, dtype):
    """Rows of bytes of latent [..., 512] (64-bit) and rope [..., 64] (a 16-bit tensor)."""
    y = latent.reshape(*latent.shape[:-1], LATENT // GROUP, GROUP)
    k = exponents(np.abs(y).max(-1), dtype)
    q = codes(y / 2.0 ** k[..., None].astype(float)).reshape(latent.shape)
    return torch.cat([torch.from_numpy(q), rope.contiguous().view(torch.uint8), torch.from_numpy((k + 127).astype(np.uint8))], -1)


def unpack(rows, dtype):
    """The values of rows of bytes, in 64 bits."""
    rows = rows.cpu()
    q = VALUES[rows[..., :LATENT].numpy()]
    k = rows[..., LATENT + 2 * ROPE:].numpy().astype(float) - 127
    rope = rows[..., LATENT:LATENT + 2 * ROPE].contiguous().view(TYPE[dtype]).double().numpy()
    return np.concatenate([q * np.repeat(2.0 ** k, GROUP, -1), rope], -1)


def check_rows(rows, latent, dtype):
    """Bytes of rows whose exact latent values are `latent`: the scales' rule, and half a step at each value."""
    rows = rows.cpu()
    got = unpack(rows, dtype)[..., :LATENT]
    k = rows[..., LATENT + 2 * ROPE:].numpy().astype(int) - 127
    lost = ~(np.abs(latent) < LARGEST[dtype])
    assert np.array_equal(np.isnan(got), lost)
    y = np.where(lost, 0.0, latent)
    most = np.abs(y).reshape(*y.shape[:-1], -1, GROUP).max(-1)
    low, high = exponents(most * (1 - DELTA), dtype), exponents(most * (1 + DELTA), dtype)
    assert np.all((k >= low) & (k <= high))
    scale = np.repeat(2.0 ** k.astype(float), GROUP, -1)
    x = y / scale
    bound = half_step(x * (1 + DELTA)) + DELTA * np.abs(x)
    bound = np.where((scale == 2.0 ** MOST[dtype]) & (np.abs(x) > 240), np.abs(x) - 240 + 1e-9 * np.abs(x), bound)
    off = np.abs(np.where(lost, 0.0, got) / scale - x)
    assert np.all(off <= bound), np.max(off - bound)


def select(logits, scores, keep):
    """logits [g, b, v], scores [g, b] -> scores, parents, tokens [g, keep] in 64 bits."""
    g, b, v = logits.shape
    out = np.full((g, keep), -np.inf), np.full((g, keep), -1), np.full((g, keep), -1)
    for i in range(g):
        found = []
        for j in range(b):
            z = np.where(np.isnan(logits[i, j]), -np.inf, logits[i, j])
            top = z.max()
            if not np.isfinite(scores[i, j]) or not np.isfinite(top):
                continue
            total = scores[i, j] + (z - (top + np.log(np.exp(z - top).sum())))
            order = np.lexsort((np.arange(v), -z))[:keep]
            found += [(-total[t], j, t) for t in order if np.isfinite(z[t])]
        for r, (s, j, t) in enumerate(sorted(found)[:keep]):
            out[0][i, r], out[1][i, r], out[2][i, r] = -s, j, t
    return out


def reorder(cache, table, lens, parents, page):
    """cache [layers, pages, page, ...], table [g * b, cols], lens [g], parents [g, b] -> cache, table."""
    cache, old, new = cache.clone(), cache, table.clone()
    g, b = parents.shape
    for i in range(g):
        mine = [int(p) if 0 <= p < b else -1 for p in parents[i]]
        left = [p for p in range(b) if p not in mine]
        whole, part = lens[i] // page, lens[i] % page
        for j, p in enumerate(mine):
            if p < 0 or p in mine[:j]:
                donor = left.pop(0)
                p = donor if p < 0 else p
            else:
                donor = p
            new[i * b + j, :whole] = table[i * b + p, :whole]
            new[i * b + j, whole:] = table[i * b + donor, whole:]
            if donor != p and part:
                cache[:, table[i * b + donor, whole], :part] = old[:, table[i * b + p, whole], :part]
    return cache, new
