"""Products of a few tokens with 4-bit weights that have group scales.

    y = int4_matvec(x, w, scales, group)

x [T, K] bf16 or fp16 (up to 64 tokens; built for 1 to 16), w uint8 [K, N / 2] in the layer's int4 layout
(`workloads.pack_int4`), scales [ceil(K / group), N] fp32, bf16 or fp16, group
a multiple of 32:

    y[t, n] = sum_k x[t, k] q[k, n] scales[k // group, n]

in fp32, rounded once to x's type.  NaN stands for what could not be computed:
a row of x that is not finite, and columns whose copies inside the kernel did
not come within a second.  An inference product: it records no
gradient, and refuses an x that asks for one.
"""
from __future__ import annotations

import torch

from .binding import ELEMS, MAX_INT, check_op, load_library, op_stream

MAX_TOKENS = 64
MAX_SIDE = 1 << 30  # of K and N
_X_TYPES = (torch.bfloat16, torch.float16)


def _refuse(x, w, scales, group, out):
    """Name what is wrong with a call that `_shapes` did not accept."""
    if x.dim() != 2 or w.dim() != 2 or scales.dim() != 2:
        raise ValueError("l4moe: x [T, K], w [K, N / 2] and scales [ceil(K / group), N] are matrices")
    T, K = x.shape
    N = 2 * w.shape[1]
    if x.dtype not in _X_TYPES:
        raise ValueError(f"l4moe: x has dtype {x.dtype}, expected bfloat16 or float16")
    if w.dtype != torch.uint8:
        raise ValueError(f"l4moe: w has dtype {w.dtype}, expected uint8")
    if scales.dtype not in ELEMS:
        raise ValueError(f"l4moe: scales have dtype {scales.dtype}, expected float32, bfloat16 or float16")
    if group < 32 or group % 32 or group > MAX_INT:
        raise ValueError(f"l4moe: group = {group}, expected a multiple of 32 below 2^31")
    if K > MAX_SIDE or N > MAX_SIDE:
        raise ValueError(f"l4moe: K = {K}, N = {N}, expected at most {MAX_SIDE}")
    if T > MAX_TOKENS:
        raise ValueError(f"l4moe: {T} tokens, expected at most {MAX_TOKENS}")
    if K < 1 or N < 2 or w.shape[0] != K:
        raise ValueError(f"l4moe: w has shape {tuple(w.shape)}, expected ({K}, N / 2)")
    if tuple(scales.shape) != (-(-K // group), N):
        raise ValueError(f"l4moe: scales have shape {tuple(scales.shape)}, expected {(-(-K // group), N)}")
    if out is not None and (tuple(out.shape) != (T, N) or out.dtype != x.dtype):
        raise ValueError(f"l4moe: out must be {x.dtype} of shape {(T, N)}")
    for t, name in ((x, "x"), (w, "w"), (scales, "scales"), (out, "out")):
        if t is None:
            continue
        if not t.is_contiguous():
            raise ValueError(f"l4moe: {name} must be contiguous (row-major)")
        if not t.is_cuda:
            raise ValueError(f"l4moe: {name} must be a CUDA tensor")
        if t.device != x.device:
            raise ValueError(f"l4moe: {name} is on {t.device}, x on {x.device}")
    if torch.is_grad_enabled() and (x.requires_grad or scales.requires_grad):
        raise ValueError("l4moe: int4_matvec has no gradient; call it under torch.no_grad() or detach x and scales")


def _accepts(x, w, scales, group, out, T, K, N):
    """The conditions of `_refuse` in one pass (a call of a few microseconds
    pays for every look at a tensor)."""
    dev = x.get_device()
    return (x.dtype in _X_TYPES and w.dtype is torch.uint8 and scales.dtype in ELEMS and 32 <= group <= MAX_INT
            and group % 32 == 0 and T <= MAX_TOKENS and 1 <= K <= MAX_SIDE and 2 <= N <= MAX_SIDE and w.shape == (K, N // 2)
            and scales.shape == (-(-K // group), N) and dev >= 0 and w.get_device() == dev
            and scales.get_device() == dev and x.is_contiguous() and w.is_contiguous() and scales.is_contiguous()
            and (out is None or (out.shape == (T, N) and out.dtype is x.dtype and out.get_device() == dev
                                 and out.is_contiguous()))
            and not ((x.requires_grad or scales.requires_grad) and torch.is_grad_enabled()))


def int4_matvec(x: torch.Tensor, w: torch.Tensor, scales: torch.Tensor, group: int, out: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """x [T, K] times the 4-bit weight w with group scales: [T, N] in x's type."""
    group = int(group)
    if x.dim() != 2 or w.dim() != 2 or scales.dim() != 2:
        _refuse(x, w, scales, group, out)
    (T, K), N = x.shape, 2 * w.shape[1]
    if not _accepts(x, w, scales, group, out, T, K, N):
        _refuse(x, w, scales, group, out)
        raise ValueError("l4moe: int4_matvec does not take these arguments")
    with op_stream(x, stream, x, w, scales, out) as st:
        if out is None:
            out = x.new_empty((T, N))
        check_op(_call()(T, K, N, group, x.data_ptr(), ELEMS[x.dtype], w.data_ptr(), scales.data_ptr(),
                         ELEMS[scales.dtype], out.data_ptr(), st))
    return out


_function = None


def _call():
    global _function
    if _function is None:
        _function = load_library().l4moe_int4_matvec
    return _function
