"""Plain 64-bit definitions of the operators around a language model's layers (test infrastructure
only): 8-bit matrices with a scale for each row and their product, token embeddings with their
gradient, and the orthogonalised update.  numpy, no code shared with the library.
"""
import numpy as np

NEAREST, STOCHASTIC = 0, 1
QUINTIC = (3.4445, -4.7750, 2.0315)


# ----------------------------------------------------------------------------- 8-bit rows
def pitch(cols):
    return -(-cols // 128) * 128


def quantize(x, rounding, r=None):
    """Packed (codes, scales) of the rows of x (fp32 or wider values that fp32 holds)."""
    x = np.asarray(x, np.float32)
    rows, cols = x.shape
    codes, scales = np.zeros((rows, pitch(cols)), np.int8), np.zeros(rows, np.float32)
    for i in range(rows):
        if not np.all(np.isfinite(x[i])):
            scales[i] = np.nan
            continue
        t = np.abs(x[i]).max()
        with np.errstate(all="ignore"):
            inv = np.float32(127) / t
        if not np.isfinite(inv):
            continue
        scales[i] = t / np.float32(127)
        if rounding == NEAREST:
            codes[i, :cols] = np.rint(x[i].astype(np.float64) * np.float64(inv))
        else:
            u = np.minimum(np.abs(x[i]) * inv, np.float32(127)).astype(np.float64)
            low = np.floor(u)
            codes[i, :cols] = (low + (r[i] < u - low)) * np.where(np.signbit(x[i]), -1, 1)
    return codes, scales


def matmul(a, a_scales, b, b_scales, bias=None):
    """(result, the exact product's magnitude) from codes and scales, in 64 bits."""
    sums = a.astype(np.int64) @ b.astype(np.int64).T
    v = sums.astype(np.float64) * a_scales.astype(np.float64)[:, None] * b_scales.astype(np.float64)
    return (v if bias is None else v + np.asarray(bias, np.float64)), np.abs(v)


# ----------------------------------------------------------------------------- embeddings
def embedding(table, ids, scale):
    table = np.asarray(table, np.float64)
    out = np.zeros((len(ids), table.shape[1]))
    for t, i in enumerate(ids):
        if 0 <= i < len(table):
            out[t] = table[i] * np.float64(np.float32(scale))
    return out


def embedding_grad(dout, ids, vocab, scale):
    """(gradient, sums of magnitudes, tokens of each id)."""
    dout = np.asarray(dout, np.float64)
    grad, mass, count = np.zeros((vocab, dout.shape[1])), np.zeros((vocab, dout.shape[1])), np.zeros(vocab, int)
    for t, i in enumerate(ids):
        if 0 <= i < vocab:
            grad[i] += dout[t]
            mass[i] += np.abs(dout[t])
            count[i] += 1
    s = np.float64(np.float32(scale))
    return grad * s, mass * abs(s), count


# ----------------------------------------------------------------------------- updates
def orthogonalise(g, steps=5, coefficients=QUINTIC):
    a, b, c = coefficients
    x = np.asarray(g, np.float64)
    flip = x.shape[0] > x.shape[1]
    x = x.T if flip else x
    norm = np.sqrt((x * x).sum())
    x = x / norm if norm > 0 else x
    for _ in range(steps):
        p = x @ x.T
        x = a * x + (b * p + c * (p @ p)) @ x
    return x.T if flip else x


def half(x, scale):
    return (x * scale).astype(np.float16).astype(np.float64) / scale


def bf16(x):
    """fp32 values rounded to bf16, to nearest, ties to even."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32).astype(np.float64)


def orthogonalise_rounded(g, steps=5, coefficients=QUINTIC):
    """The same with products of halves, diagonals apart in every step, X in fp32, the result in bf16.  How
    far it is from orthogonalise() is how far those roundings alone take it.  (The library's differ in
    the steps before the last two, see orthogonalise_in_halves: on a broad spectrum by a few percent.)"""
    a, b, c = coefficients
    x = np.asarray(g, np.float64)
    flip = x.shape[0] > x.shape[1]
    x = x.T if flip else x
    norm = np.sqrt((x * x).sum())
    x = (x / norm if norm > 0 else x).astype(np.float32).astype(np.float64)
    for _ in range(steps):
        h = half(x, 256.0)
        p = (h @ h.T).astype(np.float32).astype(np.float64)
        d = np.diag(p).copy()
        f = half(p - np.diag(d), 1024.0)
        sq = f @ f
        q = b * f + c * ((d[:, None] + d) * f + sq)
        diag = b * d + c * (d * d + np.diag(sq))
        np.fill_diagonal(q, 0.0)
        x = ((a + diag)[:, None] * x + half(q, 1024.0) @ h).astype(np.float32).astype(np.float64)
    x = bf16(x)
    return x.T if flip else x


def orthogonalise_in_halves(g, steps=5, coefficients=QUINTIC):
    """The same, with what keeps roundings out of directions that X does not have.  X's halves h differ
    from X by noise in every direction, and the diagonal's part, which acts on rows apart, would leave
    it there, to grow a-fold a step.  Before the last two steps therefore: sides to 64 x 512 multiply X as
    two halves an element; else the diagonal multiplies h too, so that b A + c A^2 acts as a whole."""
    a, b, c = coefficients
    x = np.asarray(g, np.float64)
    flip = x.shape[0] > x.shape[1]
    x = x.T if flip else x
    small = x.shape[0] <= 64 and x.shape[1] <= 512
    norm = np.sqrt((x * x).sum())
    x = (x / norm if norm > 0 else x).astype(np.float32).astype(np.float64)
    for step in range(steps):
        h = half(x, 256.0)
        p = (h @ h.T).astype(np.float32).astype(np.float64)
        d = np.diag(p).copy()
        f = half(p - np.diag(d), 1024.0)
        sq = f @ f
        q = b * f + c * ((d[:, None] + d) * f + sq)
        diag = b * d + c * (d * d + np.diag(sq))
        np.fill_diagonal(q, 0.0)
        taken = h + half(x - h, 256.0) if small and step < steps - 2 else h
        own = h if not small and step < steps - 2 else x
        x = (a * x + diag[:, None] * own + half(q, 1024.0) @ taken).astype(np.float32).astype(np.float64)
    x = bf16(x)
    return x.T if flip else x


def low_rank(rows, cols, kind, seed):
    """Matrices of few directions, as the gradients of few tokens or of few live channels are."""
    rng = np.random.default_rng(seed)

    def few(n, k):
        v = np.zeros(n)
        v[rng.choice(n, min(n, k), replace=False)] = rng.standard_normal(min(n, k))
        return v

    if kind.startswith("rank"):
        r = int(kind[4:])
        x = rng.standard_normal((rows, r)) @ rng.standard_normal((r, cols))
    elif kind == "rows":        # one direction in two to four rows
        x = np.outer(few(rows, rng.integers(2, 5)), rng.standard_normal(cols))
    elif kind == "columns":
        x = np.outer(rng.standard_normal(rows), few(cols, rng.integers(2, 5)))
    elif kind == "both":
        x = np.outer(few(rows, 4), few(cols, 4))
    elif kind == "live":        # eight tokens, half of the channels of each alive
        x = np.maximum(rng.standard_normal((rows, 8)), 0) @ np.maximum(rng.standard_normal((8, cols)), 0)
    else:
        raise ValueError(kind)
    return (x * 1e-3).astype(np.float32)


LOW_RANK = ("rank1", "rank2", "rank8", "rows", "columns", "both", "live")
