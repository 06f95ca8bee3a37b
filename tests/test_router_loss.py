"""router_loss: balance loss, z loss, counts and the gradient of the logits
against the definition in 64 bits.

Tolerances.  A share is exp(l - max) / sum: the fast exp of 16-bit logits is
off by 2 + 1.173 |x| ulp of 2^-23 (CUDA's documented bound for __expf), 49 ulp
= 5.9e-6 at the |x| <= 40 that these inputs reach; the accurate one by 2 ulp.
The row's sum, its reciprocal and the product add a few ulp, a lane's and a
block's fp32 sums of up to 100 rows at most 100 * 2^-24 = 6e-6.  REL = 2e-5
covers these together, relative to the sums of magnitudes; lse is off by REL
(1 + |max|).  The gradient then is rounded once to the logits' type: half a
step, finfo(t).eps / 2 of its value (and half of f16's smallest step 2^-24).
Counts are exact."""
import math

import pytest
import torch

from sparse_moe_transformer_router_b200 import binding
from sparse_moe_transformer_router_b200.router_loss import router_loss

REL = 2e-5
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def reference(logits, k, wb, wz, score="softmax", mask=None, idx=None):
    """The definition in 64 bits on the CPU: loss, balance, z, rows, counts,
    gradient, and the magnitude its terms are summed from."""
    l = logits.detach().double().cpu()
    T, E = l.shape
    keep = ~torch.isneginf(l).all(1)
    if mask is not None:
        keep &= mask.cpu()
    rows = int(keep.sum())
    n = max(rows, 1)
    lk = l[keep]
    if idx is None:
        key = torch.where(torch.isnan(lk), torch.full_like(lk, -math.inf), lk)
        nan = torch.isnan(lk).long()
        chosen = torch.empty((rows, k), dtype=torch.long)
        for t in range(rows):  # numbers by value then index, then NaN by index
            chosen[t] = torch.tensor(sorted(range(E), key=lambda e: (int(nan[t, e]), -float(key[t, e]), e))[:k])
    else:
        chosen = idx.cpu().long().view(T, k)[keep]
    counts = torch.zeros(E, dtype=torch.int64)
    for e in chosen.flatten().tolist():
        if 0 <= e < E:
            counts[e] += 1
    f = counts.double() / (k * n)
    lse = torch.logsumexp(lk, 1)
    soft = torch.softmax(lk, 1)
    if score == "sigmoid":
        p = torch.softmax(-torch.nn.functional.softplus(-lk), 1)
        slope = torch.sigmoid(-lk)
    else:
        p, slope = soft, torch.ones_like(soft)
    P = p.sum(0) / n
    balance, z = E * (f * P).sum(), (lse ** 2).sum() / n
    a, zc = wb * E * f / n, 2 * wz / n
    dot = (p * a).sum(1, keepdim=True)
    grad, mag = torch.zeros(T, E, dtype=torch.float64), torch.zeros(T, E, dtype=torch.float64)
    grad[keep] = p * slope * (a - dot) + zc * lse[:, None] * soft
    top = lk.abs().amax(1, keepdim=True) if rows else torch.zeros(0, 1, dtype=torch.float64)
    mag[keep] = p * slope * (a + dot) + zc * (lse.abs()[:, None] + 1 + top) * soft
    return {"loss": wb * balance + wz * z, "balance": balance, "z": z, "rows": rows, "counts": counts,
            "grad": grad, "mag": mag, "lse": lse, "top": top}


def check(r, ref, logits, wb, wz, up=1.0, grad=None):
    assert r.rows.item() == ref["rows"]
    assert torch.equal(r.counts.cpu().long(), ref["counts"])
    n = max(ref["rows"], 1)
    tb = REL * abs(float(ref["balance"]))
    tz = REL * float(((ref["lse"].abs() + 1 + ref["top"].flatten()) * 2 * ref["lse"].abs()).sum() / n) + \
        REL * float(ref["z"])
    assert abs(r.balance.item() - float(ref["balance"])) <= tb
    assert abs(r.z.item() - float(ref["z"])) <= tz
    assert abs(r.loss.item() - float(ref["loss"])) <= abs(wb) * tb + abs(wz) * tz + 2e-7 * abs(float(ref["loss"]))
    g = (r.grad(None if up == 1.0 else torch.tensor(up, device=logits.device)) if grad is None else grad)
    assert g.dtype == logits.dtype and g.shape == logits.shape
    want, mag = ref["grad"] * up, ref["mag"] * abs(up)
    tol = REL * mag + (torch.finfo(g.dtype).eps / 2 * 1.01) * want.abs() + torch.finfo(g.dtype).smallest_normal * \
        torch.finfo(g.dtype).eps / 2 * 1.01
    err = (g.double().cpu() - want).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


def make(T, E, dtype, seed=0, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    return ((torch.randn(T, E, generator=g) * spread) + torch.randn(E, generator=g)).to(TYPES[dtype]).cuda()


# ------------------------------------------------------------------ refusals
def test_refusals_of_the_binding():
    x = torch.zeros(4, 8)
    for bad, kw, text in (
            (torch.zeros(4), {}, r"\[T, E\]"),
            (torch.zeros(4, 8, dtype=torch.float64), {}, "dtype"),
            (torch.zeros(4, 257), {}, "experts"),
            (torch.zeros(4, 0), {}, "experts"),
            (x, {"k": 0}, "k = 0"),
            (x, {"k": 5}, "k = 5"),
            (torch.zeros(4, 2), {"k": 3}, "k = 3"),
            (x, {"score": "tanh"}, "score"),
            (x, {"mask": torch.zeros(5, dtype=torch.bool)}, "mask has shape"),
            (x, {"mask": torch.zeros(4)}, "mask has dtype"),
            (x, {"idx": torch.zeros(4, 2, dtype=torch.int32)}, "idx has shape"),
            (x, {"idx": torch.zeros(4, 1, dtype=torch.int64)}, "idx has dtype"),
            (x, {"mask": torch.zeros(8, dtype=torch.bool)[::2]}, "contiguous"),
            (torch.zeros(8, 4).t(), {}, "rows"),
            (torch.zeros(1, 8).expand(4, 8), {}, "rows"),
            (x, {}, "CUDA tensor")):
        with pytest.raises(ValueError, match=text):
            router_loss(bad, **kw)


def test_batches_past_32_bit_counts_are_refused():
    for T, k in ((2 ** 31, 1), (2 ** 32 + 4, 1), (2 ** 30, 2)):
        with pytest.raises(ValueError, match="choices"):
            router_loss(torch.empty((T, 2), dtype=torch.bfloat16, device="meta"), k)
    lib = binding.load_library()
    assert lib.l4moe_router_loss(2 ** 30, 8, 2, 256, 0, 8, None, None, 0, 1.0, 1.0, 256, 256, 0, None) == binding.ERR_ARG


def test_a_gradient_over_its_logits_is_refused():
    lib = binding.load_library()

    def grad(dl, ld=8, ldd=8, T=4):
        return lib.l4moe_router_loss_grad(T, 8, 1 << 20, 0, ld, None, 0, 256, None, dl, ldd, None)

    A = 1 << 20
    for kw in ({"dl": A}, {"dl": A + 32}, {"dl": A - 96}, {"dl": A + 12, "ld": 20, "ldd": 20},
               {"dl": A + 32, "ld": 16, "ldd": 8}, {"dl": A + 52, "ld": 16, "ldd": 16}):
        assert grad(**kw) == binding.ERR_ARG, kw
        assert b"overlaps" in lib.l4moe_last_error(None)
    if not torch.cuda.is_available():  # columns side by side, and rows that follow: as far as the missing device
        for kw in ({"dl": A + 32, "ld": 16, "ldd": 16}, {"dl": A - 32, "ld": 16, "ldd": 16}, {"dl": A + 128}):
            assert grad(**kw) == binding.ERR_CUDA, kw


def test_the_loss_of_another_stream_is_copied_on_that_stream(monkeypatch):
    """Without a GPU: stand-ins for the stream scope and the library note where
    the values, the loss's copy for autograd and its gradient are enqueued."""
    from torch.utils._python_dispatch import TorchDispatchMode

    from sparse_moe_transformer_router_b200 import router_loss as module
    current, seen = ["own"], []

    class Scope:
        def __init__(self, tensor, stream, *used):
            self.stream = current[-1] if stream is None else stream

        def __enter__(self):
            current.append(self.stream)
            return self.stream

        def __exit__(self, *exc):
            current.pop()

    class Library:
        def l4moe_router_loss(self, *args):
            seen.append(("values", args[-1]))
            return 0

    class Copies(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            if func.overloadpacket is torch.ops.aten.clone:
                seen.append(("copy", current[-1]))
            return func(*args, **(kwargs or {}))

    monkeypatch.setattr(module, "op_stream", Scope)
    monkeypatch.setattr(module, "load_library", Library)
    monkeypatch.setattr(module, "_accepts", lambda *args: True)
    monkeypatch.setattr(module, "_workspace", lambda *args: 0)
    for stream in ("side", None):
        seen.clear()
        with Copies():
            r = module.router_loss(torch.zeros(4, 8).requires_grad_(), 1, stream=stream)
        where = stream or "own"
        assert r.loss.requires_grad and seen == [("values", where), ("copy", where)]


def test_refusals_of_the_library():
    lib = binding.load_library()
    A = 256  # a pointer value that no refused call follows

    def loss(T=4, E=8, k=1, logits=A, type=0, ld=8, mask=None, idx=None, score=0, result=A, ws=A, n=1 << 20):
        return lib.l4moe_router_loss(T, E, k, logits, type, ld, mask, idx, score, 1.0, 1.0, result, ws, n, None)

    def grad(T=4, E=8, logits=A, type=0, ld=8, score=0, result=A, up=None, dl=A, ldd=8):
        return lib.l4moe_router_loss_grad(T, E, logits, type, ld, None, score, result, up, dl, ldd, None)

    for kw in ({"T": -1}, {"E": 0}, {"E": 257, "ld": 257}, {"k": 0}, {"k": 5}, {"E": 2, "k": 3}, {"logits": None},
               {"ld": 7}, {"score": 2}, {"result": None}, {"ws": None}):
        assert loss(**kw) == binding.ERR_ARG, kw
    for kw in ({"T": -1}, {"E": 0}, {"logits": None}, {"ld": 7}, {"ldd": 7}, {"score": 2}, {"result": None},
               {"dl": None}):
        assert grad(**kw) == binding.ERR_ARG, kw
    assert loss(type=3) == binding.ERR_DTYPE and grad(type=-1) == binding.ERR_DTYPE
    for kw in ({"logits": A + 2}, {"result": A + 2}, {"ws": A + 1}, {"idx": A + 2}):
        assert loss(**kw) == binding.ERR_ALIGN, kw
    for kw in ({"logits": A + 2}, {"result": A + 1}, {"up": A + 2}, {"dl": A + 2}):
        assert grad(**kw) == binding.ERR_ALIGN, kw
    assert b"router_loss" in lib.l4moe_last_error(None)
    assert lib.l4moe_router_loss_workspace(-1, 8) == 0 and lib.l4moe_router_loss_workspace(4, 257) == 0


def test_the_references_gradient_is_that_of_its_loss():
    """The formula's gradient against autograd of the 64-bit loss (counts held) and central differences."""
    torch.manual_seed(3)
    l = torch.randn(5, 6, dtype=torch.float64)
    mask = torch.tensor([True, True, False, True, True])
    for score in ("softmax", "sigmoid"):
        ref = reference(l, 2, 0.7, 0.3, score, mask)
        f = ref["counts"].double() / (2 * 4)

        def loss(v):
            p = torch.softmax(v, 1) if score == "softmax" else torch.sigmoid(v) / torch.sigmoid(v).sum(1, keepdim=True)
            return (0.7 * 6 * (f * p[mask].mean(0)).sum() + 0.3 * (torch.logsumexp(v[mask], 1) ** 2).mean())

        v = l.clone().requires_grad_()
        loss(v).backward()
        assert torch.allclose(v.grad, ref["grad"], rtol=1e-12, atol=1e-14)
        for t, e in ((0, 0), (2, 3), (4, 5)):
            d = torch.zeros_like(l)
            d[t, e] = 1e-6
            num = (loss(l + d) - loss(l - d)) / 2e-6
            assert abs(float(num - ref["grad"][t, e])) < 1e-8


# ---------------------------------------------------------------------- values
SHAPES = [(1, 1), (1, 2), (3, 4), (64, 4), (33, 7), (257, 8), (100, 9), (1000, 16), (77, 17), (130, 32), (65, 33),
          (500, 64), (90, 100), (1025, 128), (300, 129), (2100, 256), (64, 255)]


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,E", SHAPES)
def test_values_and_gradient(T, E, dtype, score):
    logits = make(T, E, dtype, seed=T + E)
    k = min(4, E, 1 + T % 4)
    g = torch.Generator().manual_seed(5)
    mask = (torch.rand(T, generator=g) < 0.8).cuda() if T % 2 else None
    up = 4096.0 if dtype == "f16" else 1.0
    r = router_loss(logits, k, balance=0.5, z=0.25, score=score, mask=mask)
    check(r, reference(logits, k, 0.5, 0.25, score, mask), logits, 0.5, 0.25, up)


@pytest.mark.gpu
@pytest.mark.parametrize("k", [1, 2, 3, 4])
def test_ties_and_signed_zeros_take_the_lower_index(k):
    g = torch.Generator().manual_seed(k)
    logits = torch.randint(-1, 2, (400, 24), generator=g).float()
    logits[::3] *= -1.0  # -0 among the zeros
    logits = logits.cuda()
    check(router_loss(logits, k, balance=1.0, z=0.1), reference(logits, k, 1.0, 0.1), logits, 1.0, 0.1)


@pytest.mark.gpu
@pytest.mark.parametrize("E,k", [(5, 1), (16, 2), (128, 4)])
def test_given_choices(E, k):
    T = 700
    logits = make(T, E, "bf16", seed=9)
    g = torch.Generator().manual_seed(1)
    idx = torch.randint(-2, E + 3, (T, k), generator=g, dtype=torch.int32)  # some outside [0, E)
    idx[5] = 0  # the same expert k times
    idx[6] = torch.iinfo(torch.int32).max
    idx[7] = torch.iinfo(torch.int32).min
    idx = idx.cuda()
    mask = (torch.arange(T) % 5 != 0).cuda()
    for given in (idx, idx.view(-1)):
        r = router_loss(logits, k, balance=0.3, z=0.2, mask=mask, idx=given)
        check(r, reference(logits, k, 0.3, 0.2, mask=mask, idx=idx), logits, 0.3, 0.2)


@pytest.mark.gpu
def test_long_batch_over_many_blocks():
    """More row groups than blocks; sizes whose last group is ragged."""
    logits = make(20011, 128, "f32", seed=4)
    r = router_loss(logits, 1, balance=0.01, z=0.001)
    check(r, reference(logits, 1, 0.01, 0.001), logits, 0.01, 0.001)
    again = router_loss(logits, 1, balance=0.01, z=0.001)
    assert torch.equal(again.loss, r.loss) and torch.equal(again.balance, r.balance) and torch.equal(again.z, r.z)
    assert torch.equal(again.grad(), r.grad())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
def test_row_strides_and_offsets(dtype):
    """Rows inside a wider matrix, at offsets that no 16-byte load can take."""
    wide = make(90, 75, dtype, seed=2)
    for c0, E in ((0, 64), (3, 64), (11, 40), (8, 16)):
        part = wide[:, c0:c0 + E]
        r = router_loss(part, 2, balance=1.0, z=0.5, score="sigmoid")
        ref = reference(part, 2, 1.0, 0.5, "sigmoid")
        check(r, ref, part, 1.0, 0.5)
        out = torch.full((90, 80), 7.0, dtype=wide.dtype, device="cuda")
        g = r.grad(out=out[:, 5:5 + E])
        assert g.data_ptr() == out[:, 5:].data_ptr()
        check(r, ref, part, 1.0, 0.5, grad=g)
        assert bool((out[:, :5] == 7).all()) and bool((out[:, 5 + E:] == 7).all())


# ------------------------------------------------------------ masks and odd rows
@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [0, 1, 9, 3000])
def test_no_counted_row(T, score):
    logits = make(T, 16, "f32")
    r = router_loss(logits, 2, score=score, mask=torch.zeros(T, dtype=torch.bool, device="cuda"))
    for v in (r.loss, r.balance, r.z, r.rows):
        assert v.item() == 0.0
    assert bool((r.counts == 0).all()) and bool((r.grad() == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [4, 16, 100, 256])
def test_rows_left_out_may_hold_anything(E, score):
    T = 300
    logits = make(T, E, "f32", seed=E)
    mask = torch.ones(T, dtype=torch.bool)
    for t, v in ((0, math.nan), (7, math.inf), (8, -math.inf), (299, 3e38)):
        logits[t] = v
        mask[t] = False
    logits[20] = -math.inf                      # kept by the mask, but nothing to choose from
    logits[21, 1:] = -math.inf                  # one expert left
    logits[22, : E // 2] = -math.inf            # some experts masked
    mask = mask.cuda()
    r = router_loss(logits, 2, balance=0.5, z=0.25, score=score, mask=mask)
    ref = reference(logits, 2, 0.5, 0.25, score, mask)
    g = r.grad()
    assert bool((g[[0, 7, 8, 20, 299]] == 0).all())
    # rows with -inf: |max| of the reference's bound is infinite there, take the finite entries'
    finite = torch.where(torch.isinf(logits) & ~mask[:, None].logical_not(), torch.full_like(logits, -60.0), logits)
    top = torch.where(torch.isfinite(finite), finite, torch.zeros_like(finite)).abs().amax(1).double().cpu()
    ref["top"] = top[mask.cpu() & ~torch.isneginf(logits.cpu()).all(1)][:, None]
    keep = (mask.cpu() & ~torch.isneginf(logits.cpu()).all(1))
    soft = torch.softmax(logits.double().cpu()[keep], 1)
    zc = 2 * 0.25 / ref["rows"]
    a = 0.5 * E * ref["counts"].double() / (2 * ref["rows"]) / ref["rows"]
    lk = logits.double().cpu()[keep]
    p = soft if score == "softmax" else torch.softmax(-torch.nn.functional.softplus(-lk), 1)
    ref["mag"][keep] = p * (a + (p * a).sum(1, keepdim=True)) + zc * (ref["lse"].abs()[:, None] + 1 + ref["top"]) * soft
    check(r, ref, logits, 0.5, 0.25, grad=g)


@pytest.mark.gpu
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_nan_in_a_counted_row_reaches_the_loss(value):
    """It must not be hidden; its row's gradient is NaN, the other rows' is
    not; NaN is chosen only when nothing else is left."""
    logits = make(50, 8, "f32")
    logits[3, 2] = value
    r = router_loss(logits, 1)
    assert all(math.isnan(v.item()) for v in (r.loss, r.balance, r.z))
    want = reference(logits, 1, 1.0, 1.0)
    assert torch.equal(r.counts.cpu().long(), want["counts"])
    g = r.grad()
    assert bool(torch.isnan(g[3]).any()) and bool(torch.isfinite(g[:3]).all()) and bool(torch.isfinite(g[4:]).all())
    logits[3] = math.nan
    r = router_loss(logits, 2)
    assert math.isnan(r.loss.item())
    assert torch.equal(r.counts.cpu().long(), reference(logits, 2, 1.0, 1.0)["counts"])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
def test_an_infinite_logit_is_a_sigmoid_of_one(dtype):
    """balance keeps a value, z and the loss do not."""
    logits = make(50, 8, dtype)
    logits[3, 2] = math.inf
    r = router_loss(logits, 2, balance=0.5, z=0.25, score="sigmoid")
    ref = reference(logits, 2, 0.5, 0.25, "sigmoid")
    assert torch.equal(r.counts.cpu().long(), ref["counts"])
    assert abs(r.balance.item() - float(ref["balance"])) <= REL * float(ref["balance"])
    assert math.isnan(r.z.item()) and math.isnan(r.loss.item())
    g = r.grad()
    assert bool(torch.isnan(g[3]).any()) and bool(torch.isfinite(g[:3]).all()) and bool(torch.isfinite(g[4:]).all())


@pytest.mark.gpu
def test_sigmoid_scores_of_very_low_and_very_high_logits():
    """Sigmas that underflow in 32 bits (their shares do not), and that are 1."""
    base = torch.randn(40, 12, generator=torch.Generator().manual_seed(0))
    for shift in (-200.0, -95.0, -31.0, -29.0, 25.0, 120.0):
        logits = (base + shift).cuda()
        check(router_loss(logits, 2, balance=1.0, z=0.0, score="sigmoid"),
              reference(logits, 2, 1.0, 0.0, "sigmoid"), logits, 1.0, 0.0)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,up", [(2, 65536.0), (3000, 1.0)])
def test_rows_of_large_and_small_logits(T, up, dtype, score):
    """exp of these is far from 1 and still inside fp32's range; a gradient's
    factors times its reciprocal, or its sums, need not be."""
    base = torch.randn(T, 16, generator=torch.Generator().manual_seed(5))
    for shift in (-60.0, -26.0, 30.0, 45.0, 60.0, 80.0):
        logits = (base + shift).to(TYPES[dtype]).cuda()
        # (the long batch's choices, the same ones, are given: the reference's own take long)
        idx = None if T == 2 else torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :2].int().contiguous()
        for wb, wz in ((1e-2, 0.0), (0.5, 1e-3)):
            check(router_loss(logits, 2, balance=wb, z=wz, score=score, idx=idx),
                  reference(logits, 2, wb, wz, score, idx=idx), logits, wb, wz, up=up)


# --------------------------------------------------------------------- the calls
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
def test_autograd(dtype):
    torch.manual_seed(0)
    W = (torch.randn(32, 16, device="cuda") * 0.3).requires_grad_()
    x = torch.randn(64, 32, device="cuda")
    logits = (x @ W).to(TYPES[dtype])
    r = router_loss(logits, 2, balance=0.5, z=0.25)
    assert r.loss.requires_grad and not r.balance.requires_grad
    (3.0 * r.loss).backward()
    ref = reference(logits, 2, 0.5, 0.25)
    want = x.double().cpu().t() @ (3 * ref["grad"])
    # the rounding of dlogits, through the product: half a step of each value and fp32's own
    tol = x.double().abs().cpu().t() @ (3 * (REL * ref["mag"] + torch.finfo(logits.dtype).eps * ref["grad"].abs() + 1e-7))
    assert bool(((W.grad.double().cpu() - want).abs() <= tol).all())
    # without autograd nothing is recorded, and the values are the same bits
    with torch.no_grad():
        q = router_loss(logits, 2, balance=0.5, z=0.25)
    assert not q.loss.requires_grad and torch.equal(q.loss, r.loss.detach())
    with pytest.raises(RuntimeError, match="does not require grad|twice"):
        g, = torch.autograd.grad(router_loss(logits, 2).loss, logits, create_graph=True)
        g.sum().backward()


@pytest.mark.gpu
def test_gradient_matches_differences_of_the_loss():
    """The library's own loss, moved along random directions (fp32: the
    difference of two losses near 4 is off by 4 * 2^-24 * 4 / (2 h))."""
    logits = make(16, 8, "f32", seed=11, spread=1.0)
    idx = torch.randint(0, 8, (16, 2), dtype=torch.int32, device="cuda")
    r = router_loss(logits, 2, balance=1.0, z=0.5, idx=idx)
    g, h = r.grad().double(), 1e-2
    for seed in range(4):
        d = torch.randn(16, 8, generator=torch.Generator().manual_seed(seed)).cuda()
        up = router_loss(logits + h * d, 2, balance=1.0, z=0.5, idx=idx).loss.double()
        dn = router_loss(logits - h * d, 2, balance=1.0, z=0.5, idx=idx).loss.double()
        num = float((up - dn) / (2 * h))
        # third-order term: h^2 / 6 times a third derivative below 10 for unit directions of 128 values
        assert abs(num - float((g * d.double()).sum())) < 4 * 2 ** -22 / h + h * h / 6 * 10


@pytest.mark.gpu
def test_streams_and_two_calls_at_once():
    a, b = make(4000, 64, "bf16", seed=1), make(4000, 64, "bf16", seed=2)
    want = [(r.loss.clone(), r.grad()) for r in (router_loss(a, 2), router_loss(b, 2))]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        r1, r2 = router_loss(a, 2, stream=s1), router_loss(b, 2, stream=s2.cuda_stream)
        got.append((r1, r1.grad(stream=s1), r2, r2.grad(stream=s2.cuda_stream)))
    torch.cuda.synchronize()
    for r1, g1, r2, g2 in got:
        assert torch.equal(r1.loss, want[0][0]) and torch.equal(g1, want[0][1])
        assert torch.equal(r2.loss, want[1][0]) and torch.equal(g2, want[1][1])


@pytest.mark.gpu
@pytest.mark.parametrize("raw", [False, True])
def test_autograd_of_a_call_on_another_stream(raw):
    """The loss and its gradient, with a side stream that is busy when the
    values are asked for and again before the backward pass."""
    x, own = make(3000, 24, "f32", seed=4), torch.cuda.current_stream()
    ref = reference(x, 2, 0.5, 0.25)
    side = torch.cuda.Stream()
    for busy in range(2):
        leaf = x.clone().requires_grad_()
        side.wait_stream(own)
        with torch.cuda.stream(side):
            # (the memory that the result will be given, with other values)
            other = router_loss(torch.zeros_like(x), 2)
            del other
            torch.cuda._sleep(20_000_000)  # about 10 ms
        r = router_loss(leaf * 1.0 if busy else leaf, 2, balance=0.5, z=0.25,
                        stream=side.cuda_stream if raw else side)
        own.wait_stream(side)
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        (3.0 * r.loss).backward()
        g = leaf.grad.clone()
        torch.cuda.synchronize()
        check(r, ref, x, 0.5, 0.25, up=3.0, grad=g)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [40, 3000])
def test_capture_and_replay(T):
    logits = make(T, 32, "bf16", seed=6)
    router_loss(logits, 2).grad()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = router_loss(logits, 2, balance=0.5, z=0.25)
        g = r.grad()
    for seed in (7, 8):
        logits.copy_(make(T, 32, "bf16", seed=seed))
        graph.replay()
        torch.cuda.synchronize()
        check(r, reference(logits, 2, 0.5, 0.25), logits, 0.5, 0.25, grad=g)


@pytest.mark.gpu
def test_capture_of_the_gradient_through_autograd():
    logits = make(200, 24, "f32", seed=3).requires_grad_()
    torch.autograd.grad(router_loss(logits, 2, balance=0.5, z=0.25).loss, logits)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = router_loss(logits, 2, balance=0.5, z=0.25)
        g, = torch.autograd.grad(2.0 * r.loss, logits)
    with torch.no_grad():
        logits.copy_(make(200, 24, "f32", seed=4))
    graph.replay()
    torch.cuda.synchronize()
    check(router_loss(logits.detach(), 2, balance=0.5, z=0.25), reference(logits, 2, 0.5, 0.25), logits.detach(), 0.5,
          0.25, up=2.0, grad=g)


@pytest.mark.gpu
def test_logits_changed_after_the_call_are_noticed_by_autograd():
    leaf = make(20, 8, "f32").requires_grad_()
    logits = leaf * 1.0
    r = router_loss(logits, 1)
    logits.add_(1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        r.loss.backward()


@pytest.mark.gpu
def test_a_mask_changed_after_the_call_is_noticed_by_autograd():
    logits = make(20, 8, "f32").requires_grad_()
    mask = torch.ones(20, dtype=torch.bool, device="cuda")
    r = router_loss(logits, 1, mask=mask)
    mask[3] = False
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        r.loss.backward()


@pytest.mark.gpu
def test_tensors_released_while_another_stream_still_uses_them():
    x = make(4000, 64, "bf16")
    first = router_loss(x, 2)
    want, grad = first.loss.clone(), first.grad()
    side = torch.cuda.Stream()
    mine = x.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # about 10 ms: the calls below wait behind it
    r = router_loss(mine, 2, stream=side)
    del mine
    r._logits = x  # (the result holds its logits)
    held = [torch.full_like(x, float("nan")) for _ in range(4)]  # would be given mine's memory
    torch.cuda.synchronize()
    assert torch.equal(r.loss, want) and len(held) == 4
    # the result's own memory, read by a gradient on another stream
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    r = router_loss(x, 2)
    side.wait_stream(torch.cuda.current_stream())
    words = r._result.numel()
    g = r.grad(stream=side)
    del r
    held = [torch.full((words,), float("nan"), device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(g, grad) and len(held) == 4


@pytest.mark.gpu
@pytest.mark.parametrize("T", [700, 40000])
def test_one_expert_and_padded_batches(T):
    """E = 1, and a batch whose second half is padding (any size of launch)."""
    one = make(T, 1, "f32")
    check(router_loss(one, 1, balance=1.0, z=0.1), reference(one, 1, 1.0, 0.1), one, 1.0, 0.1)
    logits = make(T, 20, "bf16", seed=1)
    mask = torch.arange(T, device="cuda") < T // 2
    logits[T // 2:] = math.nan
    r = router_loss(logits, 2, balance=1.0, z=0.1, mask=mask)
    half = router_loss(logits[:T // 2], 2, balance=1.0, z=0.1)
    ref = reference(logits[:T // 2], 2, 1.0, 0.1)
    check(half, ref, logits[:T // 2], 1.0, 0.1)
    g = r.grad()
    assert bool((g[T // 2:] == 0).all()) and torch.equal(r.counts, half.counts)
    check(r, ref, logits[:T // 2], 1.0, 0.1, grad=g[:T // 2])


@pytest.mark.gpu
def test_counts_of_a_layers_routing():
    """The layer's own routing, read back and given: the counts are the layer's."""
    from sparse_moe_transformer_router_b200.binding import L4MoE
    from sparse_moe_transformer_router_b200.workloads import LayerConfig, generate
    cfg = LayerConfig("loss", 200, 128, 8, 128, 128, "bf16", wr_std=0.1)
    inp = generate(cfg, seed=0, device="cuda")
    layer = L4MoE(cfg.d_model, cfg.expert_ffn, cfg.shared_ffn, cfg.num_experts, cfg.dtype)
    layer.set_top_k(2)
    layer.forward(inp.x, inp.W_router, inp.W_gate_up, inp.W_down, inp.Ws_gate_up, inp.Ws_down)
    routing = layer.routing()
    logits = inp.x.float() @ inp.W_router.float()
    r = router_loss(logits, 2, balance=1.0, z=0.5, idx=routing["idx"])
    assert torch.equal(r.counts, routing["counts"])
    idx = routing["idx"].clone()
    check(r, reference(logits, 2, 1.0, 0.5, idx=idx.view(-1, 2)), logits, 1.0, 0.5)
