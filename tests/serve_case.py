"""Plain 64-bit forms of the serving operators, and the error that one 16-bit
evaluation may have against them.

Bounds.  With u the unit roundoff of the 16-bit type (2^-8 bf16, 2^-11 f16: eight and eleven significant bits), w
that of fp32 (2^-24): a score is a sum of n products of 16-bit values in fp32,
off by at most n w sum|q k| scale; its exponential inherits that as a relative
error (with a few w of its own), the weight is rounded to 16 bits (u, and in f16
2^-25 of the largest weight where it is subnormal), weights and values are
summed in fp32 and the result is rounded once (u).  Relative errors of weights
count twice, once through the normaliser."""
import numpy as np

LATENT, ROPE = 512, 64
ROW = LATENT + ROPE
UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
W = 2.0 ** -24


def attend(q, k, v, see, scale, dtype):
    """One head: q [n, d], k [m, d], v [m, e], see [n, m] -> out, lse and their
    bounds.  Rows that see nothing are 0 and -inf; hidden keys have no part."""
    n, m = see.shape
    out, lse = np.zeros((n, v.shape[1])), np.full(n, -np.inf)
    bo, bl = np.zeros((n, v.shape[1])), np.zeros(n)
    u = UNIT[dtype]
    for i in range(n):
        j = np.flatnonzero(see[i])
        if not len(j):
            continue
        s = (k[j] @ q[i]) * scale
        top = s.max()
        p = np.exp(s - top)
        lse[i] = top + np.log(p.sum())
        p /= p.sum()
        out[i] = p @ v[j]
        es = (q.shape[1] + 4) * W * scale * (np.abs(k[j]) @ np.abs(q[i])).max() + 8 * W * (1 + np.abs(s).max())
        spread = p @ np.abs(v[j])
        bo[i] = (2 * es + u + len(j) * W) * spread + u * np.abs(out[i])
        if dtype == "f16":
            bo[i] += len(j) * 2.0 ** -24 * np.abs(v[j]).max() + 2.0 ** -25
        bl[i] = 2 * es + 8 * W * (1 + abs(lse[i])) + len(j) * W
    return out, lse, bo, bl


def visible(n, length, mask=None):
    """What n tokens, the last of `length` positions, see of them: a chain, or
    the context and the nodes of each token's set."""
    ctx = length - n
    see = np.zeros((n, max(length, 0)), bool)
    for i in range(n):
        for pos in range(length):
            d = pos - ctx
            see[i, pos] = d < 0 or ((d <= i) if mask is None else d in mask[i])
    return see


def words_of(sets, words):
    """The sets of visible nodes as rows of 64-bit words (nodes past them are lost)."""
    m = np.zeros((len(sets), words), np.uint64)
    for i, nodes in enumerate(sets):
        for d in nodes:
            if d < 64 * words:
                m[i, d // 64] |= np.uint64(1) << np.uint64(d % 64)
    return m.view(np.int64)


def ancestors(parents):
    sets = []
    for j, p in enumerate(parents):
        sets.append({j} | (sets[p] if p >= 0 else set()))
    return sets


def norm_rows(c, weight, eps, cos, sin, interleaved):
    """Cache rows of c [T, 576] and the largest error of one rounding's worth."""
    lat = c[:, :LATENT] / np.sqrt((c[:, :LATENT] ** 2).mean(1, keepdims=True) + eps) * weight
    return np.concatenate([lat, rotate(c[:, LATENT:], cos, sin, interleaved)], 1)


def rotate(x, cos, sin, interleaved):
    y = np.empty_like(x)
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :ROPE // 2], x[..., ROPE // 2:])
    if interleaved:
        y[..., 0::2], y[..., 1::2] = a * cos - b * sin, a * sin + b * cos
    else:
        y[..., :ROPE // 2], y[..., ROPE // 2:] = a * cos - b * sin, a * sin + b * cos
    return y


def verify(p, q, tokens, parents, u, race, cap):
    """One sequence.  Returns path, next tokens and the smallest relative margin
    of any decision (a test's inputs are sound where it is far above fp32)."""
    p = np.where(p > 0, p, 0.0)
    n, cur, path, margin = len(tokens), 0, [0], np.inf
    out = []
    while True:
        over, left, refused, taken = 0.0, 1.0, [], None
        gone = set()
        for c in range(cur + 1, n):
            if parents[c] != cur or len(path) >= cap:
                continue
            x = tokens[c]
            if q is not None:
                if refused:
                    left = np.maximum(p[cur] - over * q[cur], 0).sum()
                a, b = u[c] * q[cur, x] * left, max(p[cur, x] - over * q[cur, x], 0.0)
            else:
                a, b = u[c] * left, (0.0 if x in gone else p[cur, x])
            if max(a, b) > 0:
                margin = min(margin, abs(a - b) / max(a, b))
            if a < b:
                taken = c
                break
            refused.append(c)
            if q is not None:
                over += left
            else:
                left -= 0.0 if x in gone else p[cur, x]
                gone.add(x)
        if taken is None:
            break
        cur = taken
        path.append(cur)
        out.append(tokens[cur])
    r = p[cur].copy()
    if refused:
        if q is not None:
            r = np.maximum(r - over * q[cur], 0)
        else:
            r[list(gone)] = 0
        if not (r > 0).any():
            r = p[cur]
    score = r * race
    best = int(np.argmax(score))
    rest = np.delete(score, best)
    if len(rest) and score[best] > 0:
        margin = min(margin, (score[best] - rest.max()) / score[best])
    return path, out + [best], margin
