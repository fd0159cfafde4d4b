"""Plain 64-bit definitions of the language-model operators (test infrastructure only).

numpy, one rounding rule or formula at a time, no code shared with the library: microscaled 4-bit
encoding and decoding, log probabilities with entropy and the largest entries, and the
distillation loss from a teacher's top log probabilities with its gradient.
"""
import numpy as np

from oracle import oracle

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)
NEAREST, STOCHASTIC = 0, 1


# ----------------------------------------------------------------------------- 4-bit blocks
def pitch(cols):
    return -(-cols // 256) * 8


def draws(rows, cols, seed, worker=0, index_base=0):
    """r = fp32(hash) * 2^-32 of every element of a matrix, as the gradient quantisers draw it."""
    h = oracle.hash_fill(oracle.worker_key(seed, worker), index_base, rows * cols)
    return (np.asarray(h, np.uint32).astype(np.float32).astype(np.float64) * 2.0 ** -32).reshape(rows, cols)


def encode_block(x, rounding, r=None):
    """(scale byte, codes) of one block of values."""
    x = np.asarray(x, np.float64)
    codes = np.zeros(x.size, np.uint8)
    if not np.all(np.isfinite(x)):
        return 255, codes
    a = np.abs(x).max() if x.size else 0.0
    if a == 0:
        e = -127
    elif rounding == NEAREST:
        e = int(np.frexp(a)[1]) - 1 - 2                      # floor(log2 a) - 2
    else:
        e = int(np.frexp(a)[1]) - 4                          # below any scale that covers a
        while a > 6.0 * 2.0 ** e:
            e += 1
    e = max(e, -127)
    v = np.abs(x) / 2.0 ** e
    for i, t in enumerate(v):
        if rounding == NEAREST:
            dist = np.abs(GRID - t)
            best = np.flatnonzero(dist == dist.min())
            c = best[0] if best.size == 1 or best[0] % 2 == 0 else best[1]
        else:
            c = int(np.flatnonzero(GRID <= t)[-1])
            if c < 7 and r[i] < (t - GRID[c]) / (GRID[c + 1] - GRID[c]):
                c += 1
        codes[i] = c | (8 if np.signbit(x[i]) else 0)
    return e + 127, codes


def quantize(x, rounding, r=None):
    """Packed (codes, scales) of the rows of x."""
    rows, cols = x.shape
    p = pitch(cols)
    nib = np.zeros((rows, p * 32), np.uint8)
    scales = np.zeros((rows, p), np.uint8)
    for i in range(rows):
        for b in range(-(-cols // 32)):
            at = slice(b * 32, min(cols, b * 32 + 32))
            s, c = encode_block(x[i, at], rounding, None if r is None else r[i, at])
            scales[i, b] = s
            nib[i, at] = c
    return nib[:, 0::2] | (nib[:, 1::2] << 4), scales


def decode(codes, scales, cols):
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)
    v = GRID[nib & 7] * np.where(nib & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (v * np.repeat(s, 32, 1))[:, :cols]


# ----------------------------------------------------------------------------- rows of logits
def log_softmax(z, temperature):
    """Row by row; a row of nothing but -inf has log probabilities -inf."""
    u = np.asarray(z, np.float64) / temperature
    m = u.max(1, keepdims=True)
    with np.errstate(all="ignore"):
        d = u - np.where(np.isfinite(m), m, np.where(np.isnan(m) | (m > 0), np.nan, 0.0))
        return d - np.log(np.exp(d).sum(1, keepdims=True)) if np.all(np.isfinite(m)) else \
            np.where(np.isneginf(m), -np.inf, d - np.log(np.exp(d).sum(1, keepdims=True)))


def logprobs(z, tokens, top, temperature=1.0):
    lp = log_softmax(z, temperature)
    rows, vocab = lp.shape
    logprob = np.array([lp[i, t] if 0 <= t < vocab else 0.0 for i, t in enumerate(tokens)])
    with np.errstate(all="ignore"):
        p = np.exp(lp)
        entropy = -np.where(p == 0, 0.0, p * np.where(p == 0, 0.0, lp)).sum(1)
    zz = np.asarray(z, np.float64)
    # descending, NaN first, equal ones in the order of their index
    ids = np.array([sorted(range(vocab), key=lambda j: (not np.isnan(row[j]), -row[j] if not np.isnan(row[j]) else 0, j))[:top]
                    for row in zz]) if top else np.zeros((rows, 0), int)
    return logprob, entropy, ids, np.take_along_axis(lp, ids, 1) if top else np.zeros((rows, 0))


def taught_entries(ids, vocab):
    """Places of a row's ids that count: inside the vocabulary, each id once."""
    seen, keep = set(), []
    for j, i in enumerate(ids):
        if 0 <= i < vocab and i not in seen:
            seen.add(int(i))
            keep.append(j)
    return keep


def distill(z, ids, lps, temperature=1.0, tail=False, weight=None):
    """(loss, gradient of sum(weight * loss), (p_R, q_R) of each row)."""
    z = np.asarray(z, np.float64)
    rows, vocab = z.shape
    lq = log_softmax(z, temperature)
    loss, grad, rest = np.zeros(rows), np.zeros_like(z), np.zeros((rows, 2))
    for i in range(rows):
        keep = taught_entries(ids[i], vocab)
        if not keep:
            continue
        at = np.asarray(ids[i])[keep].astype(int)
        lp = np.asarray(lps[i], np.float64)[keep]
        if not tail and lp.max() > -np.inf:
            lp = lp - lp.max()                       # only proportions count
        p = np.exp(lp)
        outside = np.ones(vocab, bool)
        outside[at] = False
        q = np.exp(lq[i])
        q_r = q[outside].sum()
        # the rest's logarithm and each entry's share of it, also where q_r is below 64 bits' range
        log_qr, share = -np.inf, np.zeros(vocab)
        if outside.any() and not np.isneginf(lq[i][outside].max()):
            top = lq[i][outside].max()
            share[outside] = np.exp(lq[i][outside] - top)
            log_qr = top + np.log(share.sum())
            share /= share.sum()
        p_r = 0.0
        if tail:
            p_r = max(0.0, 1.0 - p.sum()) if outside.any() else 0.0
            if q_r == 0 and p_r < 2.0 ** -16:
                p_r = 0.0
        elif p.sum() == 0:
            continue
        else:
            p = p / p.sum()
        rest[i] = p_r, q_r
        with np.errstate(all="ignore"):
            loss[i] = temperature ** 2 * (p[p > 0] * (np.log(p[p > 0]) - lq[i, at][p > 0])).sum()
            if p_r > 0:
                loss[i] += temperature ** 2 * p_r * (np.log(p_r) - log_qr)
            g = (p.sum() + p_r) * q - p_r * share    # q (P - p_R / q_R)
        g[at] = (p.sum() + p_r) * q[at] - p
        grad[i] = g * temperature * (1.0 if weight is None else weight[i])
    return loss, grad, rest
