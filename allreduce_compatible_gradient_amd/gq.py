"""Thin Python binding of libgq.so (the C ABI in include/gq.h).

Argument marshalling only: every step of the path runs in the library's HIP kernels.  PyTorch
supplies device memory and the current stream; outputs that the caller does not pass are
allocated with ``torch.empty`` on the inputs' device.  If libgq.so is missing this module
raises at import: there is no CPU fallback.
"""
from __future__ import annotations

import ctypes as C
import os
import threading
from typing import List, Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgq.so")

OK, EINVAL, EOVERFLOW, EALIGN, ELAUNCH, ENONFINITE, ENOMEM = range(7)
F32, BF16 = 0, 1
UNIFORM, EXP = 0, 1
NORM_L2, NORM_MAX = 0, 1
MX = 2                                   # element type of packed microscaled matrices
MX_NEAREST, MX_STOCHASTIC = 0, 1

if not os.path.exists(LIB_PATH):
    raise ImportError("libgq.so is not built (%s); run `python -m "
                      "allreduce_compatible_gradient_amd.build`" % LIB_PATH)

_lib = C.CDLL(LIB_PATH)
_p, _i32, _i64, _u32, _u64, _d, _f = (C.c_void_p, C.c_int32, C.c_int64, C.c_uint32, C.c_uint64,
                                       C.c_double, C.c_float)
_SIGS = {
    "gq_create": (_i32, [C.POINTER(C.c_void_p)]),
    "gq_destroy": (None, [_p]),
    "gq_last_error": (C.c_char_p, [_p]),
    "gq_version": (C.c_char_p, []),
    "gq_read_status": (_i32, [_p, _p]),
    "gq_global_norm": (_i32, [_p, _p, _i32, _i32, _i64, _p, _i32, _p, _p, _p]),
    "gq_quantize_pack": (_i32, [_p, _p, _i32, _i64, _p, _i32, _p, _i32, _i32, _i32, _u64, _u32,
                                _u32, _p, _p]),
    "gq_accumulate_codes": (_i32, [_p, _p, _i32, _i64, _i32, _i32, _i32, _i32, _p, _p]),
    "gq_dequantize": (_i32, [_p, _p, _i32, _i64, _p, _i32, _p, _i32, _i32, _i32, _i32, _p, _p]),
    "gq_fused_mean": (_i32, [_p, _p, _i32, _i32, _i64, _p, _i32, _p, _i32, _i32, _i32, _u64, _u32,
                             _i32, _p, _p, _i32, _p, _p]),
    "gq_worker_scales": (_i32, [_p, _p, _i32, _i32, _i64, _p, _i32, _i32, _p, _p]),
    "gq_worker_mean": (_i32, [_p, _p, _i32, _i32, _i64, _p, _i32, _p, _i32, _i32, _u64, _u32,
                              _i32, _p, _p]),
    "gq_decode_workers": (_i32, [_p, _p, _i32, _i64, _p, _i32, _p, _i32, _i32, _i32, _i32, _p,
                                 _p]),
    "gq_logquant": (_i32, [_p, _p, _i64, _i32, _d, _i32, _p, _p, _p, _p]),
    "gq_wire_lane_bytes": (_i32, [_i32, _i32, _i32]),
    "gq_quantize_wire": (_i32, [_p, _p, _i32, _i64, _p, _i32, _p, _i32, _i32, _u64, _u32, _u32,
                                _i32, _p, _p]),
    "gq_dequantize_wire": (_i32, [_p, _p, _i64, _p, _i32, _p, _i32, _i32, _i32, _i32, _p, _p]),
    "gq_powersgd_logquant": (_i32, [_p, _p, _p, _p, _i64, _i64, _i32, _d, _i32, _i32, _p, _p,
                                    _p, _p, _p, _p, _p, _p]),
    "gq_lq_step_workers": (_i32, [_p, _p, _p, _p, _i32, _i64, _i64, _i32, _d, _i32, _i32, _p,
                                  _p, _p, _p, _p, _p, _p, _p]),
    "gq_trim": (_i32, [_p]),
    "gq_mx_pitch": (_i64, [_i64]),
    "gq_mx_quantize": (_i32, [_p, _p, _i32, _i64, _i64, _i64, _i32, _u64, _u32, _u32, _p, _p, _p,
                              _p, _p]),
    "gq_mx_dequantize": (_i32, [_p, _p, _p, _i64, _i64, _i32, _p, _i64, _p]),
    "gq_mx_matmul": (_i32, [_p, _p, _i32, _p, _i64, _p, _p, _i64, _i64, _i64, _p, _i32, _i32, _p,
                            _i64, _p]),
    "gq_token_logprobs": (_i32, [_p, _p, _i32, _i64, _i64, _i64, _p, _f, _i32, _p, _p, _p, _p,
                                 _p]),
    "gq_distill_loss": (_i32, [_p, _p, _i32, _i64, _i64, _i64, _p, _p, _i32, _f, _i32, _p, _p, _p,
                               _p, _i64, _p]),
    "gq_distill_grad": (_i32, [_p, _p, _i32, _i64, _i64, _i64, _p, _p, _i32, _f, _i32, _p, _p, _p,
                               _i64, _p]),
    "gq_global_norm_noalloc": (_i32, [_p, _p, _i32, _i32, _i64, _p, _i32, _p, _p, _p]),
}
for _name, (_res, _args) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args


class GQError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__("gq error %d: %s" % (code, msg))
        self.code = code


class Context:
    """A gq_ctx on the current device.  Not thread-safe; one per stream."""

    def __init__(self):
        h = C.c_void_p()
        st = _lib.gq_create(C.byref(h))
        if st != OK:
            raise GQError(st, "gq_create failed")
        self.handle = h

    def close(self):
        if self.handle:
            _lib.gq_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def check(self, st: int):
        if st != OK:
            raise GQError(st, _lib.gq_last_error(self.handle).decode())


_tls = threading.local()


def context() -> Context:
    """The default context of this thread for the current device.  It is shared by every
    stream, which keeps the usual pattern working -- warm up eagerly, then capture the same
    calls into a graph on another stream without allocating during capture; work issued on
    two streams at the same time needs a Context for each (ctx=...), since a context's
    scratch must not be used by two streams at once."""
    dev = torch.cuda.current_device()
    ctxs = getattr(_tls, "ctxs", None)
    if ctxs is None:
        ctxs = _tls.ctxs = {}
    if dev not in ctxs:
        ctxs[dev] = Context()
    return ctxs[dev]


def version() -> str:
    return _lib.gq_version().decode()


# ----------------------------------------------------------------------------- marshalling
_raw_stream = torch._C._cuda_getCurrentRawStream  # 0.1 us; a torch.cuda.Stream object takes 3


def _stream():
    return _raw_stream(torch.cuda.current_device())


def _dev(t: torch.Tensor, name: str, dtype=None) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    return t.data_ptr()


def _elt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError("gradients must be float32 or bfloat16, got %s" % t.dtype)


def _torch_dtype(code: int):
    return torch.float32 if code == F32 else torch.bfloat16


def _ptr_array(ptrs: Sequence[int]):
    return (C.c_void_p * len(ptrs))(*ptrs)


def _offsets(offsets, n):
    if offsets is None:
        return None, 1, None
    import numpy as np
    arr = np.ascontiguousarray(offsets, dtype=np.int64)
    return arr.ctypes.data_as(C.c_void_p), int(arr.size - 1), arr


def code_bytes(n: int, bits: int) -> int:
    return n if bits == 8 else (n + 1) // 2


# ----------------------------------------------------------------------------- Global-QSGD
def global_norm(grads: Sequence[torch.Tensor], offsets=None, scale_out=None, norms_out=None,
                ctx: Optional[Context] = None):
    """S_g = fp32(max_k ||x_k restricted to segment g||_2).  Returns (scale, norms)."""
    ctx = ctx or context()
    n = grads[0].numel()
    dt = _elt(grads[0])
    ptrs = [_dev(g, "grads[%d]" % k, grads[0].dtype) for k, g in enumerate(grads)]
    off, nseg, keep = _offsets(offsets, n)
    dev = grads[0].device
    if scale_out is None:
        scale_out = torch.empty(nseg, dtype=torch.float32, device=dev)
    ctx.check(_lib.gq_global_norm(ctx.handle, _ptr_array(ptrs), len(grads), dt, n, off, nseg,
                                  _dev(scale_out, "scale_out", torch.float32),
                                  None if norms_out is None else
                                  _dev(norms_out, "norms_out", torch.float64), _stream()))
    return scale_out, norms_out


def global_norm_noalloc(grads: Sequence[torch.Tensor], offsets, scale_out, norms_out=None,
                        ctx: Optional[Context] = None):
    """gq_global_norm_noalloc: global_norm with its temporaries in the library's fixed buffer;
    the caller passes scale_out (nseg fp32) and optionally norms_out (K*nseg fp64)."""
    ctx = ctx or context()
    n = grads[0].numel()
    dt = _elt(grads[0])
    ptrs = [_dev(g, "grads[%d]" % k, grads[0].dtype) for k, g in enumerate(grads)]
    off, nseg, keep = _offsets(offsets, n)
    ctx.check(_lib.gq_global_norm_noalloc(ctx.handle, _ptr_array(ptrs), len(grads), dt, n, off,
                                          nseg, _dev(scale_out, "scale_out", torch.float32),
                                          None if norms_out is None else
                                          _dev(norms_out, "norms_out", torch.float64),
                                          _stream()))
    return scale_out, norms_out


def quantize_pack(grad, scale, grid, levels, bits, seed, worker, index_base=0, offsets=None,
                  codes=None, ctx: Optional[Context] = None):
    ctx = ctx or context()
    n = grad.numel()
    off, nseg, keep = _offsets(offsets, n)
    if codes is None:
        codes = torch.empty(code_bytes(n, bits), dtype=torch.uint8, device=grad.device)
    ctx.check(_lib.gq_quantize_pack(ctx.handle, _dev(grad, "grad"), _elt(grad), n, off, nseg,
                                    _dev(scale, "scale", torch.float32), grid, levels, bits,
                                    seed, worker, index_base, _dev(codes, "codes", torch.uint8),
                                    _stream()))
    return codes


def accumulate_codes(codes: Sequence[torch.Tensor], n, grid, levels, bits, acc_bits, sums=None,
                     ctx: Optional[Context] = None):
    ctx = ctx or context()
    ptrs = [_dev(c, "codes[%d]" % k, torch.uint8) for k, c in enumerate(codes)]
    if sums is None:
        sums = torch.empty(n, dtype=torch.int16 if acc_bits == 16 else torch.int32,
                           device=codes[0].device)
    ctx.check(_lib.gq_accumulate_codes(ctx.handle, _ptr_array(ptrs), len(codes), n, grid, levels,
                                       bits, acc_bits, _dev(sums, "sums"), _stream()))
    return sums


def dequantize(sums, scale, grid, levels, K, out_dtype=F32, offsets=None, out=None,
               ctx: Optional[Context] = None):
    ctx = ctx or context()
    n = sums.numel()
    acc_bits = 16 if sums.dtype == torch.int16 else 32
    off, nseg, keep = _offsets(offsets, n)
    if out is None:
        out = torch.empty(n, dtype=_torch_dtype(out_dtype), device=sums.device)
    ctx.check(_lib.gq_dequantize(ctx.handle, _dev(sums, "sums", (torch.int16, torch.int32)),
                                 acc_bits, n, off, nseg, _dev(scale, "scale", torch.float32),
                                 grid, levels, K, out_dtype, _dev(out, "out"), _stream()))
    return out


def wire_lane_bytes(grid, levels, world) -> int:
    """Bytes per element of the summable wire payload for `world` workers (0: none fits)."""
    return int(_lib.gq_wire_lane_bytes(grid, levels, world))


def wire_bytes(n: int, grid, levels, world) -> int:
    return (n * wire_lane_bytes(grid, levels, world) + 3) // 4 * 4


def quantize_wire(grad, scale, grid, levels, seed, worker, world, index_base=0, offsets=None,
                  payload=None, ctx: Optional[Context] = None):
    """One worker's quantisation as a summable payload (uint8 tensor, a multiple of 4 bytes)."""
    ctx = ctx or context()
    n = grad.numel()
    off, nseg, keep = _offsets(offsets, n)
    if payload is None:
        payload = torch.empty(max(wire_bytes(n, grid, levels, world), 4), dtype=torch.uint8,
                              device=grad.device)
    ctx.check(_lib.gq_quantize_wire(ctx.handle, _dev(grad, "grad"), _elt(grad), n, off, nseg,
                                    _dev(scale, "scale", torch.float32), grid, levels, seed,
                                    worker, index_base, world,
                                    _dev(payload, "payload", torch.uint8), _stream()))
    return payload


def dequantize_wire(payload, n, scale, grid, levels, world, out_dtype=F32, offsets=None,
                    out=None, ctx: Optional[Context] = None):
    """The mean from the word-wise sum of `world` payloads."""
    ctx = ctx or context()
    off, nseg, keep = _offsets(offsets, n)
    if out is None:
        out = torch.empty(n, dtype=_torch_dtype(out_dtype), device=payload.device)
    ctx.check(_lib.gq_dequantize_wire(ctx.handle, _dev(payload, "payload", torch.uint8), n, off,
                                      nseg, _dev(scale, "scale", torch.float32), grid, levels,
                                      world, out_dtype, _dev(out, "out"), _stream()))
    return out


def fused_mean(grads, scale, grid, levels, bits, seed, acc_bits, out_dtype=F32, index_base=0,
               offsets=None, codes=None, sums=None, out=None, ctx: Optional[Context] = None):
    """Quantise every worker, sum the codes and decode the mean in one pass.  ``codes`` (list
    of K uint8 tensors) and ``sums`` are written only when given."""
    ctx = ctx or context()
    n = grads[0].numel()
    ptrs = [_dev(g, "grads[%d]" % k, grads[0].dtype) for k, g in enumerate(grads)]
    off, nseg, keep = _offsets(offsets, n)
    if out is None:
        out = torch.empty(n, dtype=_torch_dtype(out_dtype), device=grads[0].device)
    cptr = None
    if codes is not None:
        cptr = _ptr_array([_dev(c, "codes[%d]" % k, torch.uint8) for k, c in enumerate(codes)])
    ctx.check(_lib.gq_fused_mean(ctx.handle, _ptr_array(ptrs), len(grads), _elt(grads[0]), n, off,
                                 nseg, _dev(scale, "scale", torch.float32), grid, levels, bits,
                                 seed, index_base, acc_bits, cptr,
                                 None if sums is None else _dev(sums, "sums"), out_dtype,
                                 _dev(out, "out"), _stream()))
    return out


# ----------------------------------------------------------------------------- baselines
def worker_scales(grads, norm=NORM_L2, offsets=None, out=None, ctx: Optional[Context] = None):
    """Each worker's own scale per segment (K x nseg fp32): L2 norm, or largest magnitude for
    NORM_MAX (QSGD / QSGDinf)."""
    ctx = ctx or context()
    n = grads[0].numel()
    ptrs = [_dev(g, "grads[%d]" % k, grads[0].dtype) for k, g in enumerate(grads)]
    off, nseg, keep = _offsets(offsets, n)
    if out is None:
        out = torch.empty(len(grads), nseg, dtype=torch.float32, device=grads[0].device)
    ctx.check(_lib.gq_worker_scales(ctx.handle, _ptr_array(ptrs), len(grads), _elt(grads[0]), n,
                                    off, nseg, norm, _dev(out, "out", torch.float32), _stream()))
    return out


def worker_mean(grads, scales, grid, levels, seed, out_dtype=F32, index_base=0, offsets=None,
                out=None, ctx: Optional[Context] = None):
    """Mean of the workers' decoded values, each quantised and decoded with its own scale
    (scales: K x nseg fp32, e.g. from worker_scales)."""
    ctx = ctx or context()
    n = grads[0].numel()
    ptrs = [_dev(g, "grads[%d]" % k, grads[0].dtype) for k, g in enumerate(grads)]
    off, nseg, keep = _offsets(offsets, n)
    if scales.numel() != len(grads) * nseg:
        raise ValueError("scales must hold K * nseg values")
    if out is None:
        out = torch.empty(n, dtype=_torch_dtype(out_dtype), device=grads[0].device)
    ctx.check(_lib.gq_worker_mean(ctx.handle, _ptr_array(ptrs), len(grads), _elt(grads[0]), n,
                                  off, nseg, _dev(scales, "scales", torch.float32), grid, levels,
                                  seed, index_base, out_dtype, _dev(out, "out"), _stream()))
    return out


def decode_workers(codes, n, scales, grid, levels, bits, out_dtype=F32, offsets=None, out=None,
                   ctx: Optional[Context] = None):
    """Receiver's mean of K workers' packed codes (list of uint8 tensors), each decoded with
    its own scale (scales: K x nseg fp32)."""
    ctx = ctx or context()
    off, nseg, keep = _offsets(offsets, n)
    if scales.numel() != len(codes) * nseg:
        raise ValueError("scales must hold K * nseg values")
    if out is None:
        out = torch.empty(n, dtype=_torch_dtype(out_dtype), device=codes[0].device)
    cptr = _ptr_array([_dev(c, "codes[%d]" % k, torch.uint8) for k, c in enumerate(codes)])
    ctx.check(_lib.gq_decode_workers(ctx.handle, cptr, len(codes), n, off, nseg,
                                     _dev(scales, "scales", torch.float32), grid, levels, bits,
                                     out_dtype, _dev(out, "out"), _stream()))
    return out


def read_status(ctx: Optional[Context] = None) -> int:
    """Synchronises the current stream; returns ENONFINITE if a norm was not finite."""
    ctx = ctx or context()
    return _lib.gq_read_status(ctx.handle, _stream())


# ----------------------------------------------------------------------------- LQ-SGD
def logquant(F, alpha, bits, codes=None, colmax=None, F_hat=None, want_hat=True,
             ctx: Optional[Context] = None):
    ctx = ctx or context()
    rows, r = F.shape
    dev = F.device
    if codes is None:
        codes = torch.empty(rows, r, dtype=torch.int8, device=dev)
    if colmax is None:
        colmax = torch.empty(r, dtype=torch.float32, device=dev)
    if F_hat is None and want_hat:
        F_hat = torch.empty(rows, r, dtype=torch.float32, device=dev)
    ctx.check(_lib.gq_logquant(ctx.handle, _dev(F, "F", torch.float32), rows, r, alpha, bits,
                               _dev(codes, "codes", torch.int8),
                               _dev(colmax, "colmax", torch.float32),
                               None if F_hat is None else _dev(F_hat, "F_hat", torch.float32),
                               _stream()))
    return codes, colmax, F_hat


def powersgd_logquant(G, E, Q, alpha, bits, out=None, want_hat=True, want_pre=False,
                      bits_q=None, ctx: Optional[Context] = None):
    """One LQ-SGD compressor step; E and Q are updated in place.  ``bits`` is the code width of
    P, ``bits_q`` that of Q' (default: the same).  Returns a dict of outputs."""
    ctx = ctx or context()
    n, m = G.shape
    r = Q.shape[1]
    dev = G.device
    o = dict(out or {})
    o.setdefault("p_codes", torch.empty(n, r, dtype=torch.int8, device=dev))
    o.setdefault("p_colmax", torch.empty(r, dtype=torch.float32, device=dev))
    o.setdefault("q_codes", torch.empty(m, r, dtype=torch.int8, device=dev))
    o.setdefault("q_colmax", torch.empty(r, dtype=torch.float32, device=dev))
    if want_hat:
        o.setdefault("p_hat", torch.empty(n, r, dtype=torch.float32, device=dev))
    if want_pre:
        o.setdefault("p_pre", torch.empty(n, r, dtype=torch.float32, device=dev))
        o.setdefault("q_pre", torch.empty(m, r, dtype=torch.float32, device=dev))

    def opt(k):
        return None if o.get(k) is None else _dev(o[k], k, torch.float32)

    ctx.check(_lib.gq_powersgd_logquant(
        ctx.handle, _dev(G, "G", torch.float32), _dev(E, "E", torch.float32),
        _dev(Q, "Q", torch.float32), n, m, r, alpha, bits, bits if bits_q is None else bits_q,
        _dev(o["p_codes"], "p_codes", torch.int8), _dev(o["p_colmax"], "p_colmax", torch.float32),
        _dev(o["q_codes"], "q_codes", torch.int8), _dev(o["q_colmax"], "q_colmax", torch.float32),
        opt("p_hat"), opt("p_pre"), opt("q_pre"), _stream()))
    return o


def lq_step_workers(Gs, Es, Qs, alpha, bits, bits_q=None, out=None, want_pre=False,
                    ctx: Optional[Context] = None):
    """One LQ-SGD step of K workers (lists of n x m gradients, n x m errors and m x r warm
    starts; E's and Q's are updated in place).  Returns a dict with every worker's message
    stacked by worker (p_codes K x n x r, p_colmax K x r, q_codes K x m x r, q_colmax K x r)
    and G_hat (n x m), the mean of the decoded messages; with want_pre also every worker's
    factors before quantisation (p_pre K x n x r, q_pre K x m x r)."""
    ctx = ctx or context()
    K = len(Gs)
    if not (len(Es) == K and len(Qs) == K):
        raise ValueError("Gs, Es and Qs must have one entry per worker")
    n, m = Gs[0].shape
    r = Qs[0].shape[1]
    for k in range(K):
        if tuple(Gs[k].shape) != (n, m) or tuple(Es[k].shape) != (n, m):
            raise ValueError("worker %d: G and E must be %d x %d" % (k, n, m))
        if tuple(Qs[k].shape) != (m, r):
            raise ValueError("worker %d: Q must be %d x %d" % (k, m, r))
    dev = Gs[0].device
    o = dict(out or {})
    o.setdefault("p_codes", torch.empty(K, n, r, dtype=torch.int8, device=dev))
    o.setdefault("p_colmax", torch.empty(K, r, dtype=torch.float32, device=dev))
    o.setdefault("q_codes", torch.empty(K, m, r, dtype=torch.int8, device=dev))
    o.setdefault("q_colmax", torch.empty(K, r, dtype=torch.float32, device=dev))
    o.setdefault("G_hat", torch.empty(n, m, dtype=torch.float32, device=dev))
    if want_pre:
        o.setdefault("p_pre", torch.empty(K, n, r, dtype=torch.float32, device=dev))
        o.setdefault("q_pre", torch.empty(K, m, r, dtype=torch.float32, device=dev))

    def opt(k):
        return None if o.get(k) is None else _dev(o[k], k, torch.float32)

    gp = _ptr_array([_dev(G, "G[k]", torch.float32) for G in Gs])
    ep = _ptr_array([_dev(E, "E[k]", torch.float32) for E in Es])
    qp = _ptr_array([_dev(Q, "Q[k]", torch.float32) for Q in Qs])
    ctx.check(_lib.gq_lq_step_workers(
        ctx.handle, gp, ep, qp, K, n, m, r, alpha, bits, bits if bits_q is None else bits_q,
        _dev(o["p_codes"], "p_codes", torch.int8), _dev(o["p_colmax"], "p_colmax", torch.float32),
        _dev(o["q_codes"], "q_codes", torch.int8), _dev(o["q_colmax"], "q_colmax", torch.float32),
        _dev(o["G_hat"], "G_hat", torch.float32), opt("p_pre"), opt("q_pre"), _stream()))
    return o


# ----------------------------------------------------------------------------- 4-bit matrices
class MXTensor:
    """A packed microscaled 4-bit matrix of rows x cols: ``codes`` rows x 16 * mx_pitch(cols)
    and ``scales`` rows x mx_pitch(cols) bytes, padded with zeros as gq.h describes."""
    __slots__ = ("codes", "scales", "rows", "cols")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, cols: int):
        pitch = mx_pitch(cols)
        if (codes.dim() != 2 or tuple(scales.shape) != (codes.shape[0], pitch)
                or codes.shape[1] != 16 * pitch):
            raise ValueError("a packed matrix of %d columns has rows of %d code and %d scale bytes"
                             % (cols, 16 * pitch, pitch))
        self.codes, self.scales, self.rows, self.cols = codes, scales, codes.shape[0], cols

    @staticmethod
    def empty(rows: int, cols: int, device) -> "MXTensor":
        pitch = mx_pitch(cols)
        t = MXTensor.__new__(MXTensor)
        t.codes = torch.empty(rows, 16 * pitch, dtype=torch.uint8, device=device)
        t.scales = torch.empty(rows, pitch, dtype=torch.uint8, device=device)
        t.rows, t.cols = rows, cols
        return t


def mx_pitch(cols: int) -> int:
    """Blocks of 32 in a packed row of ``cols`` elements, padding included."""
    return (cols + 255) // 256 * 8


def _rows(t: torch.Tensor, name: str, dtype=None):
    """(address, row stride) of a matrix whose rows are contiguous."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.dim() != 2:
        raise ValueError("%s must be a matrix" % name)
    rows, cols = t.shape
    ld, inner = t.stride()
    if inner != 1 and cols > 1 and rows > 0:
        raise ValueError("%s must be a matrix with contiguous rows" % name)
    return t.data_ptr(), (ld if rows > 1 else max(ld, cols))


def mx_quantize(x, rounding=MX_NEAREST, seed=0, worker=0, index_base=0, by_rows=True,
                by_cols=False, out: Optional[MXTensor] = None, out_t: Optional[MXTensor] = None,
                ctx: Optional[Context] = None):
    """Quantise a matrix to microscaled 4-bit floating point.  Returns (packed rows, packed
    columns), an MXTensor of x and one of its transpose; None for one that is not asked for."""
    ctx = ctx or context()
    p, ld = _rows(x, "x")
    rows, cols = x.shape
    q = (out or MXTensor.empty(rows, cols, x.device)) if by_rows else None
    qt = (out_t or MXTensor.empty(cols, rows, x.device)) if by_cols else None
    if q is not None and (q.rows != rows or q.cols != cols):
        raise ValueError("out must be a packed %d x %d matrix" % (rows, cols))
    if qt is not None and (qt.rows != cols or qt.cols != rows):
        raise ValueError("out_t must be a packed %d x %d matrix" % (cols, rows))
    ctx.check(_lib.gq_mx_quantize(
        ctx.handle, p, _elt(x), rows, cols, ld, rounding, seed, worker, index_base,
        None if q is None else _dev(q.codes, "out.codes", torch.uint8),
        None if q is None else _dev(q.scales, "out.scales", torch.uint8),
        None if qt is None else _dev(qt.codes, "out_t.codes", torch.uint8),
        None if qt is None else _dev(qt.scales, "out_t.scales", torch.uint8), _stream()))
    return q, qt


def mx_dequantize(q: MXTensor, out_dtype=BF16, out=None, ctx: Optional[Context] = None):
    """The values of a packed matrix (rows x cols, bf16 or fp32)."""
    ctx = ctx or context()
    if out is None:
        out = torch.empty(q.rows, q.cols, dtype=_torch_dtype(out_dtype), device=q.codes.device)
    p, ld = _rows(out, "out", _torch_dtype(out_dtype))
    if tuple(out.shape) != (q.rows, q.cols):
        raise ValueError("out must be %d x %d" % (q.rows, q.cols))
    ctx.check(_lib.gq_mx_dequantize(ctx.handle, _dev(q.codes, "codes", torch.uint8),
                                    _dev(q.scales, "scales", torch.uint8), q.rows, q.cols,
                                    out_dtype, p, ld, _stream()))
    return out


def mx_matmul(a, b: MXTensor, bias=None, out_dtype=BF16, out=None, accumulate=False,
              ctx: Optional[Context] = None):
    """a @ b.T (+ bias) (+ out): ``b`` packed N x K; ``a`` packed M x K, or an fp32 / bf16 matrix
    that the call quantises to nearest.  Returns M x N of out_dtype."""
    ctx = ctx or context()
    if isinstance(a, MXTensor):
        m, k = a.rows, a.cols
        pa, ta, sa, lda = (_dev(a.codes, "a.codes", torch.uint8), MX,
                           _dev(a.scales, "a.scales", torch.uint8), 0)
    else:
        pa, lda = _rows(a, "a")
        (m, k), ta, sa = a.shape, _elt(a), None
    if k != b.cols:
        raise ValueError("a has %d columns, b has %d" % (k, b.cols))
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = torch.empty(m, b.rows, dtype=_torch_dtype(out_dtype), device=b.codes.device)
    po, ldo = _rows(out, "out", _torch_dtype(out_dtype))
    if tuple(out.shape) != (m, b.rows):
        raise ValueError("out must be %d x %d" % (m, b.rows))
    if bias is not None and bias.numel() != b.rows:
        raise ValueError("bias must hold %d values" % b.rows)
    ctx.check(_lib.gq_mx_matmul(ctx.handle, pa, ta, sa, lda, _dev(b.codes, "b.codes", torch.uint8),
                                _dev(b.scales, "b.scales", torch.uint8), m, b.rows, k,
                                None if bias is None else _dev(bias, "bias", torch.float32),
                                1 if accumulate else 0, out_dtype, po, ldo, _stream()))
    return out


# ----------------------------------------------------------------------------- rows of logits
def token_logprobs(logits, tokens, top=0, temperature=1.0, out=None,
                   ctx: Optional[Context] = None):
    """(logprob, entropy, top_ids, top_logprobs) of each row: the given token's log probability,
    the row's entropy and its ``top`` largest entries (None where top = 0).  ``out``: those
    tensors, to be written in place of new ones."""
    ctx = ctx or context()
    p, ld = _rows(logits, "logits")
    rows, vocab = logits.shape
    if tokens.numel() != rows:
        raise ValueError("tokens must hold one entry a row")
    if out is None:
        dev = logits.device
        out = (torch.empty(rows, dtype=torch.float32, device=dev),
               torch.empty(rows, dtype=torch.float32, device=dev),
               torch.empty(rows, top, dtype=torch.int32, device=dev) if top > 0 else None,
               torch.empty(rows, top, dtype=torch.float32, device=dev) if top > 0 else None)
    elif out[0].numel() != rows or out[1].numel() != rows or (
            top > 0 and (tuple(out[2].shape) != (rows, top) or tuple(out[3].shape) != (rows, top))):
        raise ValueError("out must be (rows, rows, rows x top, rows x top)")
    ctx.check(_lib.gq_token_logprobs(
        ctx.handle, p, _elt(logits), rows, vocab, ld, _dev(tokens, "tokens", torch.int64),
        temperature, top, _dev(out[0], "out[0]", torch.float32),
        _dev(out[1], "out[1]", torch.float32),
        _dev(out[2], "out[2]", torch.int32) if top > 0 else None,
        _dev(out[3], "out[3]", torch.float32) if top > 0 else None, _stream()))
    return out


def _teacher(logits, top_ids, top_logprobs):
    if top_ids.dim() != 2 or top_ids.shape[0] != logits.shape[0] \
            or top_logprobs.shape != top_ids.shape:
        raise ValueError("top_ids and top_logprobs must be rows x top")
    return (_dev(top_ids, "top_ids", torch.int32),
            _dev(top_logprobs, "top_logprobs", torch.float32), top_ids.shape[1])


def _row_weight(w, rows):
    if w is None:
        return None
    if w.numel() != rows:
        raise ValueError("row_weight must hold one entry a row")
    return _dev(w, "row_weight", torch.float32)


def distill_loss(logits, top_ids, top_logprobs, temperature=1.0, tail=False, row_weight=None,
                 dlogits=None, ctx: Optional[Context] = None):
    """Each row's distillation loss from a teacher's top log probabilities.  Without row_weight
    and dlogits: (loss, stats), the stats for distill_grad.  With either: (loss, dlogits), the
    gradient of sum(row_weight * loss) from the same call; ``dlogits`` may be ``logits``."""
    ctx = ctx or context()
    p, ld = _rows(logits, "logits")
    rows, vocab = logits.shape
    ids, lps, top = _teacher(logits, top_ids, top_logprobs)
    loss = torch.empty(rows, dtype=torch.float32, device=logits.device)
    stats, pd, ldd = None, None, 0
    if row_weight is None and dlogits is None:
        stats = torch.empty(rows, 4, dtype=torch.float32, device=logits.device)
    else:
        if dlogits is None:
            dlogits = torch.empty_like(logits, memory_format=torch.contiguous_format)
        pd, ldd = _rows(dlogits, "dlogits", logits.dtype)
        if dlogits.shape != logits.shape:
            raise ValueError("dlogits must be %d x %d" % (rows, vocab))
    ctx.check(_lib.gq_distill_loss(
        ctx.handle, p, _elt(logits), rows, vocab, ld, ids, lps, top, temperature,
        1 if tail else 0, _row_weight(row_weight, rows), _dev(loss, "loss"),
        None if stats is None else _dev(stats, "stats"), pd, ldd, _stream()))
    return loss, (dlogits if stats is None else stats)


def distill_grad(logits, top_ids, top_logprobs, temperature, tail, stats, row_weight=None,
                 dlogits=None, ctx: Optional[Context] = None):
    """The gradient of sum(row_weight * loss) from distill_loss' stats."""
    ctx = ctx or context()
    p, ld = _rows(logits, "logits")
    rows, vocab = logits.shape
    ids, lps, top = _teacher(logits, top_ids, top_logprobs)
    if dlogits is None:
        dlogits = torch.empty_like(logits, memory_format=torch.contiguous_format)
    pd, ldd = _rows(dlogits, "dlogits", logits.dtype)
    if dlogits.shape != logits.shape or stats.numel() != 4 * rows:
        raise ValueError("dlogits must be %d x %d and stats %d x 4" % (rows, vocab, rows))
    ctx.check(_lib.gq_distill_grad(
        ctx.handle, p, _elt(logits), rows, vocab, ld, ids, lps, top, temperature,
        1 if tail else 0, _dev(stats, "stats", torch.float32), _row_weight(row_weight, rows), pd,
        ldd, _stream()))
    return dlogits


def trim(ctx: Optional[Context] = None) -> None:
    """Wait for the device and free the buffers the context has retired (see gq_trim)."""
    ctx = ctx or context()
    ctx.check(_lib.gq_trim(ctx.handle))
