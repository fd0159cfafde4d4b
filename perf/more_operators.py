"""Cases, plain forms and 64-bit values of the operators around a language model's layers.

Three operators and their counterparts, as one training path uses them: the token embedding
("embed") and its gradient ("embed_grad"), the product of 8-bit integers with a scale for each
token and channel ("i8", and "i8_backward": the two products of a linear layer's backward pass
with the quantisation of the incoming gradient), and the orthogonalised update ("ortho").

Where `own` is false, run() computes the operators with elementary torch operations; where it is
true, it calls the library's entry points as a user's program does.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)        # a x + b x^3 + c x^5, the usual quintic


# ----------------------------------------------------------------------------- the cases
def listed():
    return [
        # a small decoding batch's tokens on their way into a model: the latency of a call
        dict(name="embed token", op="embed", tokens=8, vocab=50257, dim=768, dtype="bf16",
             scale=1.0),
        # a training batch of sequences, a large vocabulary, a scale of sqrt(dim)
        dict(name="embed batch", op="embed", tokens=16383, vocab=131071, dim=4096, dtype="bf16",
             scale=64.0),
        # the gradient of a 50257 x 768 table from one batch, written whole for the exchange
        dict(name="embed grad", op="embed_grad", tokens=8191, vocab=50257, dim=768, dtype="bf16",
             scale=1.0),
        # the gradient of a large table, fp32 for the exchange
        dict(name="embed grad large", op="embed_grad", tokens=16384, vocab=131071, dim=4096,
             dtype="bf16", scale=64.0),
        # serving, one token through a 4096 -> 11008 layer: the weights' bytes
        dict(name="i8 token", op="i8", m=1, n=11008, k=4096, a="bf16", out="bf16"),
        # serving, a ragged batch through a vocabulary head 768 -> 50257
        dict(name="i8 head", op="i8", m=333, n=50257, k=768, a="bf16", out="bf16"),
        # a teacher's forward product on a batch of sequences
        dict(name="i8 large", op="i8", m=8192, n=11008, k=4096, a="bf16", out="bf16"),
        # training, both products of a layer's backward pass, the gradient quantised on the way
        dict(name="i8 backward", op="i8_backward", m=4095, n=4096, k=11008),
        # the smallest update: a stem convolution's 64 filters of 3 x 7 x 7
        dict(name="ortho filters", op="ortho", batch=1, rows=64, cols=147, dtype="f32"),
        # twelve layers' equal matrices in one call
        dict(name="ortho layers", op="ortho", batch=12, rows=768, cols=2304, dtype="f32"),
        # a square matrix of a large layer
        dict(name="ortho square", op="ortho", batch=1, rows=4096, cols=4096, dtype="f32"),
        # a large layer's tall matrix
        dict(name="ortho large", op="ortho", batch=1, rows=11008, cols=4096, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("embed", "embed_grad", "embed_grad", "i8", "i8", "i8_backward", "ortho",
                     "ortho"))
    if op in ("embed", "embed_grad"):
        dim = _log_int(rng, 32, 8192)
        vocab = _log_int(rng, 512, min(262144, (1 << 28) // dim))
        return dict(op=op, tokens=_log_int(rng, 1, min(65536, (1 << 26) // dim)), vocab=vocab,
                    dim=dim, dtype=rng.choice(("f32", "bf16")), scale=rng.choice((1.0, dim ** 0.5)))
    if op == "i8":
        return dict(op=op, m=_log_int(rng, 1, 8192), n=_log_int(rng, 256, 11008),
                    k=_log_int(rng, 64, 4096), a=rng.choice(("bf16", "f32")),
                    out=rng.choice(("bf16", "f32")))
    if op == "i8_backward":
        return dict(op=op, m=_log_int(rng, 16, 4095), n=_log_int(rng, 256, 4096),
                    k=_log_int(rng, 256, 8192))
    rows, cols = _log_int(rng, 16, 4096), _log_int(rng, 16, 8192)
    if rng.random() < 0.5:
        rows, cols = cols, rows
    small = min(rows, cols)
    most = max(1, min(24, (1 << 33) // (small * rows * cols)))
    return dict(op=op, batch=_log_int(rng, 1, most), rows=rows, cols=cols,
                dtype=rng.choice(("f32", "bf16")))


def work(case):
    op = case["op"]
    if op in ("embed", "embed_grad"):
        t, v, d = case["tokens"], case["vocab"], case["dim"]
        size = DTYPES[case["dtype"]].itemsize
        if op == "embed":                               # a row that comes again is read again
            return {"bytes": 2 * t * d * size + 8 * t, "flops": t * d}
        return {"bytes": t * d * size + 8 * t + v * d * 4, "flops": t * d}
    if op in ("i8", "i8_backward"):
        m, n, k = case["m"], case["n"], case["k"]
        if op == "i8":
            return {"bytes": m * k * DTYPES[case["a"]].itemsize + n * k + 4 * n
                    + m * n * DTYPES[case["out"]].itemsize, "flops": 2 * m * n * k}
        return {"bytes": 2 * m * n + n * k + m * k + 2 * m * k + 4 * n * k, "flops": 4 * m * n * k}
    n, m = sorted((case["rows"], case["cols"]))
    # two symmetric products, half of each, and a whole one, five times
    return {"bytes": case["batch"] * n * m * (DTYPES[case["dtype"]].itemsize + 2),
            "flops": case["batch"] * 5 * (n * n * m + n * n * n + 2 * n * n * m)}


# ----------------------------------------------------------------------------- the inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _token_ids(tokens, vocab, g):
    """Ids of a text: their frequency falls with their rank; one in 32 is padding (no id)."""
    u = torch.rand(tokens, device="cuda", generator=g, dtype=torch.float64)
    rank = (torch.exp(u * math.log(vocab + 1.0)) - 1.0).long().clamp(max=vocab - 1)
    ids = (rank * 7919 + 13) % vocab if math.gcd(7919, vocab) == 1 else rank
    return torch.where(torch.rand(tokens, device="cuda", generator=g) < 1 / 32, -1, ids)


def _activations(rows, cols, g):
    """Normal entries; one channel in 64 is ten times as large, as in a trained network."""
    x = torch.randn(rows, cols, device="cuda", generator=g)
    big = torch.rand(cols, device="cuda", generator=g) < 1 / 64
    return x * torch.where(big, 10.0, 1.0)


def _gradient(rows, cols, g):
    """Heavy-tailed entries of size 1e-4, one row in 16 all zero (padding tokens)."""
    x = torch.randn(rows, cols, device="cuda", generator=g)
    x = x * x.abs() * 1e-4
    return x * (torch.rand(rows, 1, device="cuda", generator=g) >= 1 / 16)


def _update(batch, rows, cols, g):
    """A momentum's matrices: a few strong directions over a broad floor."""
    x = torch.randn(batch, rows, cols, device="cuda", generator=g)
    r = min(8, rows, cols)
    u = torch.randn(batch, rows, r, device="cuda", generator=g)
    v = torch.randn(batch, r, cols, device="cuda", generator=g)
    return (x + torch.matmul(u, v)) * 1e-3


def _weights(rows, cols, g):
    return torch.randn(rows, cols, device="cuda", generator=g) * 0.02


def prepare(case, seed):
    g, op, s = _generator(seed), case["op"], dict(case, seed=seed)
    if op == "embed":
        s["table"] = _weights(case["vocab"], case["dim"], g).to(DTYPES[case["dtype"]])
        s["ids"] = _token_ids(case["tokens"], case["vocab"], g)
    elif op == "embed_grad":
        s["dout"] = _gradient(case["tokens"], case["dim"], g).to(DTYPES[case["dtype"]])
        s["ids"] = _token_ids(case["tokens"], case["vocab"], g)
    elif op == "i8":
        s["A"] = _activations(case["m"], case["k"], g).to(DTYPES[case["a"]])
        s["W"] = _pack(_weights(case["n"], case["k"], g))
        s["bias"] = torch.randn(case["n"], device="cuda", generator=g) * 0.1
    elif op == "i8_backward":
        s["dY"] = _gradient(case["m"], case["n"], g).to(torch.bfloat16)
        s["Wt"] = _pack(_weights(case["k"], case["n"], g))      # the weights by columns
        s["Xt"] = _pack(_activations(case["k"], case["m"], g))  # the activations by columns
    else:
        s["G"] = _update(case["batch"], case["rows"], case["cols"], g).to(DTYPES[case["dtype"]])
    return s


# ----------------------------------------------------------------------------- plain forms
def _key(seed, worker):
    """Low 32 bits of SplitMix64's output number worker + 1 from the state `seed`."""
    m = (1 << 64) - 1
    z = (seed + (worker + 1) * 0x9E3779B97F4A7C15) & m
    z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & m
    z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & m
    return (z ^ (z >> 31)) & 0xFFFFFFFF


def _uniform(shape, seed):
    """The draw of every element of a matrix: its place hashed with the key, in [0, 1]."""
    h = torch.arange(shape[0] * shape[1], device="cuda") ^ _key(seed, 0)
    h = ((h ^ (h >> 16)) * 0x85EBCA6B) & 0xFFFFFFFF
    h = ((h ^ (h >> 13)) * 0xC2B2AE35) & 0xFFFFFFFF
    return ((h ^ (h >> 16)).float() * 2.0 ** -32).view(shape)


def _codes(x, r=None):
    """Codes in [-127, 127] and the scale of each row of fp32 rows: to nearest (the products in 64
    bits, where a rounded one next to a border could cross it), or by the draws r.  Both quotients
    are rounded once to fp32."""
    top = x.abs().amax(1, keepdim=True)
    inv = (127.0 / top.double()).float()
    fine = torch.isfinite(inv)
    scale = torch.where(fine, (top.double() / 127.0).float(), 0.0)
    inv = torch.where(fine, inv, 0.0)
    if r is None:
        return torch.round(x.double() * inv.double()).float(), scale
    u = (x.abs() * inv).clamp(max=127.0)
    low = torch.floor(u)
    return torch.copysign(low + (r < u - low), x), scale


def _pack(x):
    """Rows of 8-bit codes, to nearest, padded with zeros to a multiple of 128, with their scales
    and the row's length."""
    c, scale = _codes(x)
    c = torch.nn.functional.pad(c.to(torch.int8), (0, -x.shape[1] % 128))
    return c.contiguous(), scale.view(-1).contiguous(), x.shape[1]


def _product(a, sa, packed):
    """The products of codes and the scales of their rows."""
    codes, scales, cols = packed
    return torch.matmul(a, codes[:, :cols].float().T) * sa * scales


def _plain_embed(s):
    ids, there = s["ids"].clamp(min=0), s["ids"] >= 0
    out = s["table"][ids].float() * s["scale"]
    return torch.where(there[:, None], out, 0.0).to(s["table"].dtype)


def _plain_embed_grad(s):
    there = s["ids"] >= 0
    d = torch.where(there[:, None], s["dout"].float(), 0.0)
    out = torch.zeros(s["vocab"], s["dim"], device="cuda")
    return out.index_add_(0, s["ids"].clamp(min=0), d).mul_(s["scale"])


def _plain_i8(s):
    a, sa = _codes(s["A"].float())
    return (_product(a, sa, s["W"]) + s["bias"]).to(DTYPES[s["out"]])


def _plain_i8_backward(s):
    dy = s["dY"].float()
    r = _uniform(dy.shape, s["seed"])
    dx = _product(*_codes(dy, r), s["Wt"])
    dw = _product(*_codes(dy.T, r.T), s["Xt"])
    return {"dX": dx.to(torch.bfloat16), "dW": dw}


def _plain_ortho(s):
    a, b, c = COEFFICIENTS
    x = s["G"].float()
    if s["rows"] > s["cols"]:
        x = x.transpose(1, 2).contiguous()
    x = x / x.square().sum((1, 2), keepdim=True).sqrt()
    for _ in range(5):
        gram = torch.matmul(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.matmul(b * gram + c * torch.matmul(gram, gram), x)
    if s["rows"] > s["cols"]:
        x = x.transpose(1, 2)
    return x.to(torch.bfloat16).contiguous()


PLAIN = {"embed": _plain_embed, "embed_grad": _plain_embed_grad, "i8": _plain_i8,
         "i8_backward": _plain_i8_backward, "ortho": _plain_ortho}


# ----------------------------------------------------------------------------- the library's calls
def _own_embed(s, gq):
    return gq.embedding(s["table"], s["ids"], scale=s["scale"])


def _own_embed_grad(s, gq):
    return gq.embedding_grad(s["dout"], s["ids"], s["vocab"], scale=s["scale"], out_dtype=gq.F32)


def _own_i8(s, gq):
    return gq.int_matmul(s["A"], gq.IntTensor(*s["W"]), bias=s["bias"],
                        out_dtype=gq.BF16 if s["out"] == "bf16" else gq.F32)


def _own_i8_backward(s, gq):
    q, qt = gq.int_quantize(s["dY"], rounding=gq.INT_STOCHASTIC, seed=s["seed"], by_cols=True)
    return {"dX": gq.int_matmul(q, gq.IntTensor(*s["Wt"]), out_dtype=gq.BF16),
            "dW": gq.int_matmul(qt, gq.IntTensor(*s["Xt"]), out_dtype=gq.F32)}


def _own_ortho(s, gq):
    return gq.orthogonalise(s["G"], steps=5, coefficients=COEFFICIENTS)


OWN = {"embed": _own_embed, "embed_grad": _own_embed_grad, "i8": _own_i8,
       "i8_backward": _own_i8_backward, "ortho": _own_ortho}


def run(state):
    if own:
        from allreduce_compatible_gradient_amd import gq
        return OWN[state["op"]](state, gq)
    return PLAIN[state["op"]](state)


# ----------------------------------------------------------------------------- 64-bit values
def _exact_draws(shape, seed):
    """The draws in unsigned 32-bit arithmetic on the host."""
    h = np.arange(shape[0] * shape[1], dtype=np.uint32) ^ np.uint32(_key(seed, 0))
    h ^= h >> np.uint32(16)
    h *= np.uint32(0x85EBCA6B)
    h ^= h >> np.uint32(13)
    h *= np.uint32(0xC2B2AE35)
    h ^= h >> np.uint32(16)
    r = h.astype(np.float32).astype(np.float64) / 2.0 ** 32
    return torch.from_numpy(r.reshape(shape)).cuda()


def _exact_quantised(x, r=None):
    """Rows as code times scale.  The factor 127 / top and the scale are fp32 numbers by
    definition, and the drawn codes' fraction is taken of the fp32 product."""
    top = x.abs().max(1, keepdim=True).values
    factor = (127 / top.double()).float().double()
    scale = (top.double() / 127).float().double()
    none = ~(factor < 3.5e38)
    v = x.double() * factor.masked_fill(none, 0)
    if r is None:
        code = torch.round(v)
    else:
        v = v.abs().float().double().clamp(max=127)
        code = torch.sign(x).double() * (v.floor() + (r < v.frac()).double())
    return code * scale.masked_fill(none, 0)


def _exact_packed(packed):
    codes, scales, cols = packed
    return codes.double()[:, :cols] * scales.double()[:, None]


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "embed":
        rows = s["table"].double() * case["scale"]
        return torch.cat([rows, torch.zeros_like(rows[:1])])[s["ids"]]      # -1: the last row
    if op == "embed_grad":
        order = torch.argsort(s["ids"], stable=True)
        ids, d = s["ids"][order], s["dout"].double()[order]
        ends = torch.cumsum(d, 0)                       # differences of running sums, in 64 bits
        ends = torch.cat([torch.zeros_like(ends[:1]), ends])
        v = torch.arange(case["vocab"], device="cuda")
        first = torch.searchsorted(ids, v)
        last = torch.searchsorted(ids, v, right=True)
        del d
        return (ends[last] - ends[first]) * case["scale"]
    if op == "i8":
        return _exact_quantised(s["A"].float()) @ _exact_packed(s["W"]).T + s["bias"].double()
    if op == "i8_backward":
        dy, r = s["dY"].float(), _exact_draws(s["dY"].shape, seed)
        return {"dX": _exact_quantised(dy, r) @ _exact_packed(s["Wt"]).T,
                "dW": _exact_quantised(dy.T, r.T) @ _exact_packed(s["Xt"]).T}
    a, b, c = COEFFICIENTS
    out = []
    for g in s["G"].double():
        flip = g.shape[0] > g.shape[1]
        x = (g.T if flip else g) / torch.linalg.matrix_norm(g)
        for _ in range(5):
            p = x @ x.T
            bx = p @ x
            x = a * x + b * bx + c * (p @ bx)           # a X + b (X X^T) X + c (X X^T)^2 X
        out.append(x.T if flip else x)
    return torch.stack(out)
