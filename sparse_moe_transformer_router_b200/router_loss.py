"""The losses that train a router, and the per-expert counts of its choices.

    r = router_loss(logits, k, balance=1e-2, z=1e-3, mask=mask)
    r.loss, r.balance, r.z    fp32 scalars on the device
    r.counts                  int32 [E]: entries that chose each expert
    r.rows                    fp32 scalar: the counted rows
    r.grad(upstream)          the gradient of the logits

For the n counted rows (kept by the mask, and with a logit other than -inf),
f_e = counts_e / (k n) and share_te = softmax_e(logits_t) (score="softmax") or
sigmoid(logits_te) / sum_j sigmoid(logits_tj) (score="sigmoid"):

    balance = E sum_e f_e mean_t(share_te)
    z       = mean_t(logsumexp(logits_t)^2)
    loss    = balance_weight balance + z_weight z

A NaN or +inf in a counted row makes z and loss NaN, and balance too, except
that a +inf under score="sigmoid" is a sigmoid of 1 there.

Each row chooses its k largest logits as the layer's router does (the lower
index first among equal ones), or idx [T, k] holds the choices: those of a
layer that has run (`layer.routing()["idx"]`), of a router with its bias, or
with dropped entries (any index outside [0, E)).

Where the logits take part in autograd (a leaf or the output of the router's
product), `r.loss` has their gradient: `(task_loss + r.loss).backward()`.
The other values carry none.  With `stream`, everything the call computes is
that stream's work: wait for it before using the values on another one.  The
backward pass of `r.loss` runs there too, and autograd makes the streams wait
for one another around it.  Before a backward pass is captured into a CUDA
graph, let go of eager losses of the same leaves, as for any torch function.
One pass reads the logits for the values, one
more for the gradient; everything runs in the library's CUDA kernels on the
caller's stream, with no host synchronisation.
"""
from __future__ import annotations

import functools

import torch

from .binding import ELEMS, MAX_INT, check_op, load_library, op_stream

SCORES = {"softmax": 0, "sigmoid": 1}
MAX_EXPERTS = 256
MAX_K = 4


def _accepts(logits, k, score, mask, idx):
    """The conditions of `_refuse` in one pass (a call of a few microseconds
    pays for every look at a tensor)."""
    if logits.dim() != 2:
        return False
    T, E = logits.shape
    dev = logits.get_device()
    return (logits.dtype in ELEMS and 1 <= E <= MAX_EXPERTS and 1 <= k <= MAX_K and k <= E and T * k <= MAX_INT and score in SCORES
            and dev >= 0 and logits.is_contiguous()
            and (mask is None or (mask.shape == (T,) and mask.dtype is torch.bool and mask.get_device() == dev
                                  and mask.is_contiguous()))
            and (idx is None or (idx.shape == (T, k) and idx.dtype is torch.int32 and idx.get_device() == dev
                                 and idx.is_contiguous())))


def _refuse(logits, k, score, mask, idx):
    """Name what is wrong with a call (the rarer good ones pass: row strides,
    a flat idx)."""
    if logits.dim() != 2:
        raise ValueError(f"l4moe: logits must be [T, E], got shape {tuple(logits.shape)}")
    T, E = logits.shape
    if logits.dtype not in ELEMS:
        raise ValueError(f"l4moe: logits have dtype {logits.dtype}, expected float32, bfloat16 or float16")
    if not 1 <= E <= MAX_EXPERTS:
        raise ValueError(f"l4moe: {E} experts, expected 1 to {MAX_EXPERTS}")
    if not 1 <= k <= min(MAX_K, E):
        raise ValueError(f"l4moe: k = {k}, expected 1 to {min(MAX_K, E)}")
    if T * k > MAX_INT:  # (the counts are 32-bit)
        raise ValueError(f"l4moe: {T} rows of {k} choices, expected fewer than 2^31 in all")
    if score not in SCORES:
        raise ValueError(f"l4moe: unknown score {score!r}")
    _rows(logits, "logits")
    for t, name, shape, dtype in ((mask, "mask", (T,), torch.bool), (idx, "idx", (T, k), torch.int32)):
        if t is None:
            continue
        if tuple(t.shape) != shape and not (name == "idx" and tuple(t.shape) == (T * k,)):
            raise ValueError(f"l4moe: {name} has shape {tuple(t.shape)}, expected {shape}")
        if t.dtype != dtype:
            raise ValueError(f"l4moe: {name} has dtype {t.dtype}, expected {dtype}")
        if not t.is_contiguous():
            raise ValueError(f"l4moe: {name} must be contiguous")
        if t.device != logits.device:
            raise ValueError(f"l4moe: {name} is on {t.device}, logits on {logits.device}")
    if not logits.is_cuda:
        raise ValueError("l4moe: logits must be a CUDA tensor")


def _rows(t, name):
    """Rows of neighbouring elements, any distance of at least a row apart."""
    T, E = t.shape
    if (E > 1 and t.stride(1) != 1) or (T > 1 and t.stride(0) < E):
        raise ValueError(f"l4moe: {name}' rows must be contiguous and must not overlap")


def _stride(t):
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


class RouterLoss:
    """The values of one `router_loss` call (views of one device buffer)."""

    def __init__(self, logits, mask, score, result, home):
        self._logits, self._mask, self._score, self._result = logits, mask, score, result
        self._home = home  # the stream (raw handle) that the result's memory belongs to
        self.loss, self.balance, self.z, self.rows = result[:4].unbind()

    @property
    def counts(self) -> torch.Tensor:
        return self._result.view(torch.int32)[4:4 + self._logits.shape[1]]

    def grad(self, upstream: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """The gradient of the logits, times `upstream` (an fp32 device
        scalar; None: 1), in the logits' type.  `out`: where to write it (not
        over the logits).  The logits (and the mask) must still hold what the
        call read, and the stream must have waited for the call's."""
        logits = self._logits
        T, E = logits.shape
        if upstream is not None:
            if upstream.dtype is not torch.float32 or upstream.numel() != 1 or \
                    upstream.get_device() != logits.get_device():
                raise ValueError("l4moe: upstream must be one float32 on the logits' device")
        if out is not None:
            if out.shape != logits.shape or out.dtype != logits.dtype or out.device != logits.device:
                raise ValueError("l4moe: out must have the logits' shape, dtype and device")
            _rows(out, "out")
        with op_stream(logits, stream, logits, self._mask, upstream, out) as st:
            if st != self._home:
                self._result.record_stream(torch.cuda.current_stream(logits.device))
            if out is None:
                out = logits.new_empty((T, E))
            check_op(load_library().l4moe_router_loss_grad(
                T, E, logits.data_ptr(), ELEMS[logits.dtype], _stride(logits),
                None if self._mask is None else self._mask.data_ptr(), self._score, self._result.data_ptr(),
                None if upstream is None else upstream.data_ptr(), out.data_ptr(), _stride(out), st))
        return out


@functools.lru_cache(maxsize=256)
def _workspace(T, E, device) -> int:
    """l4moe_router_loss_workspace on the current device (`device`)."""
    return load_library().l4moe_router_loss_workspace(T, E)


def _forward(logits, k, balance, z, score, mask, idx, stream=None) -> RouterLoss:
    lib = load_library()
    T, E = logits.shape
    with op_stream(logits, stream, logits, mask, idx) as st:
        n = _workspace(T, E, logits.get_device())
        words = 4 + 2 * E + 1
        # one buffer: the result, then the workspace
        buf = logits.new_empty(words + n // 4, dtype=torch.float32)
        at = buf.data_ptr()
        check_op(lib.l4moe_router_loss(
            T, E, k, logits.data_ptr(), ELEMS[logits.dtype], _stride(logits), None if mask is None else mask.data_ptr(),
            None if idx is None else idx.data_ptr(), SCORES[score], balance, z, at, at + 4 * words, n, st))
    return RouterLoss(logits, mask, SCORES[score], buf, st)


class _Loss(torch.autograd.Function):
    """The loss as a function of the logits."""

    @staticmethod
    def forward(ctx, logits, mask, args, box):
        r = _forward(logits.detach(), *args)
        box.append(r)
        ctx.save_for_backward(logits, r._result, mask)
        ctx.score, ctx.home = r._score, r._home
        return r.loss.clone()

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, upstream):
        logits, result, mask = ctx.saved_tensors
        r = RouterLoss(logits.detach(), mask, ctx.score, result, ctx.home)
        return r.grad(upstream.contiguous()), None, None, None


def router_loss(logits: torch.Tensor, k: int = 1, *, balance: float = 1e-2, z: float = 1e-3, score: str = "softmax",
                mask: torch.Tensor | None = None, idx: torch.Tensor | None = None, stream=None) -> RouterLoss:
    """Balance loss, z loss and per-expert counts of a router's logits.

    logits [T, E] fp32, bf16 or fp16 (rows of neighbouring elements; row
    strides are taken as they are), 1 <= E <= 256, 1 <= k <= min(4, E);
    mask bool [T]: the rows that count (None: all); idx int32 [T, k]: the
    choices (None: each row's k largest logits).  balance and z are the
    weights of the two losses in `loss`."""
    k = int(k)
    if not _accepts(logits, k, score, mask, idx):
        _refuse(logits, k, score, mask, idx)
    args = (k, float(balance), float(z), score, mask, idx)
    if not (logits.requires_grad and torch.is_grad_enabled()):
        return _forward(logits, *args, stream)
    box = []
    with op_stream(logits, stream, logits, mask, idx):  # the loss's copy and its backward pass are that stream's too
        loss = _Loss.apply(logits, mask, args, box)
    r = box[0]
    r.loss = loss
    return r
