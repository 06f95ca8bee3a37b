"""4-bit weights with group scales: int4_matvec and the layer that runs such
experts, against the definition in 64 bits.

Tolerances of the product.  Per 32-row block the tensor core adds, in two
steps of 16 products and a start value, terms of magnitude |x| (q + 8) and 8
|x| to an fp32 sum; each step may lose 17 units of 2^-23 of its terms'
magnitudes (aligned to the largest and cut), so a block is off by at most 34
* 2^-23 * sum |x| (|q| + 16); the blocks' fp32 sums and scales add (blocks +
8) * 2^-24 of sum |x q s|.  bf16 rows are f16 divided by a power of two:
half a step 2^-39 of the largest magnitude.  Then one rounding: half a step,
finfo(t).eps / 2 of the value and half of the smallest subnormal.  Where all
sums are small integers times one power of two nothing is lost, and the
result must be the correctly rounded one bit for bit."""
import ctypes

import pytest
import torch

from sparse_moe_transformer_router_b200 import binding
from sparse_moe_transformer_router_b200.binding import L4MoE, L4MoEError
from sparse_moe_transformer_router_b200.int4 import MAX_TOKENS, int4_matvec
from sparse_moe_transformer_router_b200.workloads import pack_int4, quantize_int4_groups

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def unpack(w):
    """Packed [K, N / 2] -> codes [K, N] in 64 bits (CPU)."""
    w = w.cpu().to(torch.int64)
    q = torch.stack((w & 15, w >> 4), dim=-1).flatten(-2)
    return torch.where(q > 7, q - 16, q).double()


def each_row(s, group, K):
    return s.double().cpu().repeat_interleave(group, dim=0)[:K]


def product_bound(x, q, s, blocks):
    """What an fp32 sum of the kernel's terms may be off by (see above)."""
    ax = x.abs()
    loose = 34 * 2.0 ** -23 * (ax @ ((q.abs() + 16) * s.abs()))
    fma = (blocks + 8) * 2.0 ** -24 * (ax @ (q * s).abs())
    cut = 2.0 ** -39 * ax.amax(1, keepdim=True) * ((q.abs() + 16) * s.abs()).sum(0)
    return loose + fma + cut


def half_step(want, dtype):
    f = torch.finfo(dtype)
    return f.eps / 2 * want.abs() + f.smallest_normal * f.eps / 2


def check(y, x, w, s, group):
    K, dtype = x.shape[1], y.dtype
    xd, q, sd = x.double().cpu(), unpack(w), each_row(s, group, K)
    want = xd @ (q * sd)
    tol = product_bound(xd, q, sd, -(-K // 32))
    tol = tol + half_step(want.abs() + tol, dtype)
    err = (y.double().cpu() - want).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


def make(T, K, N, group, xt, st, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, K, generator=g).to(TYPES[xt]).cuda()
    q = torch.randint(-8, 8, (K, N), generator=g, dtype=torch.int8)
    s = ((torch.rand(-(-K // group), N, generator=g) + 0.5) * 0.01).to(TYPES[st]).cuda()
    return x, pack_int4(q).cuda(), s


# ------------------------------------------------------------------- refusals
def test_refusals_of_the_binding():
    x, w, s = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(64, 16, dtype=torch.uint8), torch.zeros(2, 32)
    for args, text in (
            ((x[0], w, s, 32), "matrices"),
            ((x.float(), w, s, 32), "x has dtype"),
            ((x, w.to(torch.int8), s, 32), "w has dtype"),
            ((x, w, s.double(), 32), "scales have dtype"),
            ((x, w, s, 0), "group"), ((x, w, s, 16), "group"), ((x, w, s, 40), "group"), ((x, w, s, -32), "group"),
            ((torch.zeros(MAX_TOKENS + 1, 64, dtype=torch.bfloat16), w, s, 32), "tokens"),
            ((x, w[:32], s, 32), "w has shape"),
            ((x, w, s, 64), "scales have shape"), ((x, w, s[:, :16], 32), "scales have shape"),
            ((x, w, s, 32, torch.zeros(2, 32)), "out must be"),
            ((x, w, s, 32, torch.zeros(3, 32, dtype=torch.bfloat16)), "out must be"),
            ((x.t().contiguous().t(), w, s, 32), "x must be contiguous"),
            ((x, w, s, 32), "CUDA tensor")):
        with pytest.raises(ValueError, match=text):
            int4_matvec(*args)


def test_sizes_past_the_librarys_integers_are_refused():
    x, w, s = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(64, 16, dtype=torch.uint8), torch.zeros(1, 32)
    for group in (2 ** 31, 2 ** 32 + 32):  # the second would reach the library as 32
        with pytest.raises(ValueError, match="group"):
            int4_matvec(x, w, s, group)
    N = 2 ** 32 + 32
    wide = torch.empty((1, N // 2), dtype=torch.uint8, device="meta")
    with pytest.raises(ValueError, match="at most"):
        int4_matvec(torch.empty((1, 1), dtype=torch.bfloat16, device="meta"), wide,
                    torch.empty((1, N), device="meta"), 32)
    layer = object.__new__(L4MoE)
    layer.dtype = "int4"
    with pytest.raises(ValueError, match="group"):
        layer.set_weight_scales([], [], None, None, group=2 ** 32 + 32)


def test_refusals_of_the_library():
    lib = binding.load_library()
    A = 256

    def call(T=1, K=64, N=32, group=32, x=A, xt=1, w=A, s=A, st=0, y=A):
        return lib.l4moe_int4_matvec(T, K, N, group, x, xt, w, s, st, y, None)

    for kw in ({"T": -1}, {"T": MAX_TOKENS + 1}, {"K": 0}, {"N": 0}, {"N": 31}, {"group": 0}, {"group": 48},
               {"group": -32}, {"x": None}, {"w": None}, {"s": None}, {"y": None}, {"K": 2 ** 31 - 1},
               {"N": 2 ** 31 - 2}):
        assert call(**kw) == binding.ERR_ARG, kw
    for kw in ({"xt": 0}, {"xt": 3}, {"st": 5}):
        assert call(**kw) == binding.ERR_DTYPE, kw
    for kw in ({"x": A + 2}, {"w": A + 8}, {"s": A + 4}, {"y": A + 2}):
        assert call(**kw) == binding.ERR_ALIGN, kw
    assert b"int4_matvec" in lib.l4moe_last_error(None)
    assert call(T=0, x=None) == binding.OK
    assert lib.l4moe_set_group_scales(None, 32, 0, None, None, None, None) == binding.ERR_ARG


def test_outputs_over_inputs_are_refused():
    lib = binding.load_library()
    at = {"x": 1 << 20, "w": 2 << 20, "s": 3 << 20}  # never followed
    for over in at.values():
        for y in (over, over + 16, over - 16):  # y: 2 x 64 bf16, 256 bytes
            assert lib.l4moe_int4_matvec(2, 64, 64, 32, at["x"], 1, at["w"], at["s"], 0, y, None) == binding.ERR_ARG


def test_refusals_of_group_scales():
    layer = object.__new__(L4MoE)  # no library call: only the host-side checks
    layer.d_model, layer.expert_ffn, layer.shared_ffn, layer.num_experts, layer.dtype = 64, 128, 192, 2, "int4"
    layer.device = torch.device("cuda", 0)
    gu, dn = [torch.zeros(2, 256) for _ in range(2)], [torch.zeros(4, 64) for _ in range(2)]
    sgu, sdn = torch.zeros(2, 384), torch.zeros(6, 64)
    for args, group, text in (
            ((gu, dn, sgu, sdn), 48, "group"), ((gu, dn, sgu, sdn), 16, "group"),
            ((gu[:1], dn, sgu, sdn), 32, "2 experts"),
            ((gu, dn, None, sdn), 32, "required"), ((gu, dn, sgu.double(), sdn), 32, "required"),
            (([gu[0], gu[1].half()], dn, sgu, sdn), 32, r"s_gate_up\[1\] has dtype"),
            ((gu, [dn[0], torch.zeros(2, 64)], sgu, sdn), 32, r"s_down\[1\] has shape"),
            ((gu, dn, sgu, torch.zeros(4, 64)), 32, "ss_down has shape"),
            ((gu, dn, sgu, sdn), 32, "CUDA tensor")):
        with pytest.raises(ValueError, match=text):
            layer.set_weight_scales(*args, group=group)
    layer.dtype = "int8"
    with pytest.raises(ValueError, match="int4"):
        layer.set_weight_scales(gu, dn, sgu, sdn, group=32)


@pytest.mark.parametrize("K,group", [(64, 32), (70, 32), (96, 128)])
def test_group_quantiser(K, group):
    w = torch.randn(K, 10, generator=torch.Generator().manual_seed(K))
    w[:32, 3] = 0
    packed, s = quantize_int4_groups(w, group)
    q = unpack(packed)
    assert s.shape == (-(-K // group), 10) and q.abs().max() <= 7
    err = (q * each_row(s, group, K) - w.double()).abs()
    assert bool((err <= each_row(s, group, K) * 0.5000001).all())  # half a step of its group
    assert bool((quantize_int4_groups(w, group, torch.float16)[1] == s.half()).all())


# ------------------------------------------------------------------ the product
SHAPES = [(1, 32, 16, 32), (1, 1, 2, 32), (3, 33, 18, 32), (1, 64, 256, 64), (8, 64, 272, 32), (9, 96, 130, 64),
          (16, 100, 512, 32), (5, 1001, 1234, 32), (2, 2048, 64, 128), (1, 2080, 48, 128), (16, 2049, 34, 96),
          (1, 5120, 1024, 128), (7, 4128, 640, 4128), (13, 300, 66, 1024), (17, 128, 256, 32), (64, 160, 80, 64),
          (1, 17000, 32, 128), (12, 16416, 16, 32)]


@pytest.mark.gpu
@pytest.mark.parametrize("xt", ["bf16", "f16"])
@pytest.mark.parametrize("st", list(TYPES))
@pytest.mark.parametrize("T,K,N,group", SHAPES)
def test_matvec(T, K, N, group, xt, st):
    x, w, s = make(T, K, N, group, xt, st, seed=T + K)
    check(int4_matvec(x, w, s, group), x, w, s, group)


@pytest.mark.gpu
@pytest.mark.parametrize("xt", ["bf16", "f16"])
@pytest.mark.parametrize("T,K,N", [(1, 256, 512), (4, 224, 34), (16, 700, 160), (33, 64, 64)])
def test_exact_sums_are_rounded_once(T, K, N, xt):
    """Small integers and power-of-two scales: the sums are exact in fp32, so
    the output is the correctly rounded one; every code and column is seen."""
    g = torch.Generator().manual_seed(K)
    x = torch.randint(-4, 5, (T, K), generator=g).to(TYPES[xt]).cuda()
    q = torch.randint(-8, 8, (K, N), generator=g, dtype=torch.int8)
    q[:16, 0] = torch.arange(-8, 8)
    s = torch.exp2(torch.randint(-2, 3, (-(-K // 64), N), generator=g).float()).cuda()
    w = pack_int4(q).cuda()
    want = x.double().cpu() @ (unpack(w) * each_row(s, 64, K))
    assert torch.equal(int4_matvec(x, w, s, 64).cpu(), want.to(TYPES[xt]))


@pytest.mark.gpu
def test_one_row_of_the_weight_at_a_time():
    """A unit vector in each place of K reads that row of the weight: q s, exact in fp16."""
    K, N, group = 192, 48, 64
    _, w, _ = make(1, K, N, group, "f16", "f32")
    s = torch.exp2(torch.arange(3 * N).float().view(3, N) % 5 - 2).cuda()
    want = unpack(w) * each_row(s, group, K)
    eye = torch.eye(K, dtype=torch.float16, device="cuda")
    for r in range(0, K, 64):
        assert torch.equal(int4_matvec(eye[r:r + 64], w, s, group).double().cpu(), want[r:r + 64])
    y = int4_matvec(eye[5:6].to(torch.bfloat16), w, s, group)
    assert torch.equal(y.double().cpu(), want[5:6])


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [2.0 ** -140, 2.0 ** -126, 1e-30, 1.0, 1e30, 3e38])
def test_bf16_rows_of_any_magnitude(scale):
    """bf16 has fp32's range: rows far from f16's are brought into it."""
    g = torch.Generator().manual_seed(1)
    x = (torch.randn(6, 320, generator=g).clamp(-1, 1) * scale).to(torch.bfloat16).cuda()
    x[2] *= 1e-3
    x[3, 5:] = 0
    x[4] = 0
    _, w, s = make(1, 320, 64, 64, "bf16", "f32")
    s = s * (1e-3 if scale > 1e20 else 1.0)
    check(int4_matvec(x, w, s, 64), x, w, s, 64)


@pytest.mark.gpu
def test_f16_extremes():
    g = torch.Generator().manual_seed(2)
    x = torch.randn(4, 128, generator=g).half()
    x[0] = 65504.0
    x[1] *= 2.0 ** -22  # subnormals
    x[2] = 0
    x = x.cuda()
    _, w, s = make(1, 128, 64, 64, "f16", "f16")
    s = s * 0.01
    check(int4_matvec(x, w, s, 64), x, w, s, 64)
    big = int4_matvec(x, w, torch.ones(2, 64, device="cuda"), 64)  # sums past f16's range: infinity
    want = x[0].double().cpu() @ unpack(w)
    assert bool((torch.isinf(big[0].cpu()) == (want.abs() >= 65520)).all())


@pytest.mark.gpu
@pytest.mark.parametrize("xt", ["bf16", "f16"])
@pytest.mark.parametrize("T", [4, 12])
def test_a_row_that_is_not_finite_is_nan_alone(T, xt):
    x, w, s = make(T, 200, 96, 32, xt, "f32")
    clean = int4_matvec(x, w, s, 32)
    x[1, 7], x[2, 199], x[3, 0] = float("inf"), float("-inf"), float("nan")
    y = int4_matvec(x, w, s, 32)
    assert bool(torch.isnan(y[1:4]).all())
    keep = [0] + list(range(4, T))
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.gpu
def test_not_finite_scales_stay_in_their_column():
    x, w, s = make(3, 128, 64, 64, "bf16", "f32")
    clean = int4_matvec(x, w, s, 64)
    s[1, 9] = float("nan")
    y = int4_matvec(x, w, s, 64)
    assert bool(torch.isnan(y[:, 9]).all())
    keep = [c for c in range(64) if c != 9]
    assert torch.equal(y[:, keep], clean[:, keep])


@pytest.mark.gpu
def test_empty_batch_and_out():
    x, w, s = make(2, 64, 32, 32, "bf16", "f32")
    assert int4_matvec(x[:0], w, s, 32).shape == (0, 32)
    out = torch.full((4, 32), 3.0, dtype=torch.bfloat16, device="cuda")
    y = int4_matvec(x, w, s, 32, out=out[1:3])
    assert y.data_ptr() == out[1].data_ptr() and bool((out[0] == 3).all()) and bool((out[3] == 3).all())
    check(out[1:3], x, w, s, 32)
    with pytest.raises(ValueError, match="no gradient"):
        int4_matvec(x.requires_grad_(), w, s, 32)
    with torch.no_grad():
        int4_matvec(x, w, s, 32)


@pytest.mark.gpu
def test_streams_capture_and_repeats():
    x, w, s = make(5, 4096, 2048, 128, "bf16", "f16")
    want = int4_matvec(x, w, s, 128)
    check(want, x, w, s, 128)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [int4_matvec(x, w, s, 128, stream=st) for _ in range(20) for st in (s1, s2.cuda_stream)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = int4_matvec(x, w, s, 128)
    x.copy_(make(5, 4096, 2048, 128, "bf16", "f16", seed=3)[0])
    graph.replay()
    torch.cuda.synchronize()
    check(y, x, w, s, 128)


@pytest.mark.gpu
def test_inputs_released_while_another_stream_still_uses_them():
    x, w, s = make(5, 4096, 2048, 128, "bf16", "f16")
    want = int4_matvec(x, w, s, 128)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        mine = x.clone()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)  # about 10 ms: the call below waits behind it
        y = int4_matvec(mine, w, s, 128, stream=stream)
        del mine
        held = [torch.full_like(x, float("nan")) for _ in range(4)]  # would be given mine's memory
        torch.cuda.synchronize()
        assert torch.equal(y, want) and len(held) == 4


@pytest.mark.gpu
def test_weights_past_two_gigabytes():
    """Byte offsets past 2^31 (rows of 40000 columns, 110000 of them)."""
    K, N, group = 110000, 40000, 128
    w = torch.randint(0, 256, (K, N // 2), dtype=torch.uint8, device="cuda")
    s = torch.full((-(-K // group), N), 2.0 ** -4, device="cuda")
    x = torch.zeros(2, K, dtype=torch.bfloat16, device="cuda")
    x[0, K - 1], x[1, K - 3000] = 1.0, 2.0
    y = int4_matvec(x, w, s, group)
    want = torch.stack((unpack(w[K - 1:])[0], 2 * unpack(w[K - 3000:K - 2999])[0])) * 2.0 ** -4
    assert torch.equal(y.double().cpu(), want)


# -------------------------------------------------------------------- the layer
class Layer:
    """A layer of random 4-bit experts and its 64-bit definition."""

    def __init__(self, d, F, Fs, E, group, st, k=1, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.d, self.F, self.Fs, self.E, self.group, self.k = d, F, Fs, E, group, k

        def weight(K, N):
            w = torch.randn(K, N, generator=g) * (0.5 / K ** 0.5)
            return [t.cuda() for t in quantize_int4_groups(w, group, TYPES[st])]

        self.Wr = (torch.randn(d, E, generator=g) * (1.5 / d ** 0.5)).to(torch.bfloat16).cuda() if E else None
        self.gu = [weight(d, 2 * F) for _ in range(E)]
        self.dn = [weight(F, d) for _ in range(E)]
        self.sgu, self.sdn = weight(d, 2 * Fs), weight(Fs, d)
        self.layer = L4MoE(d, F, Fs, E, "int4")
        if k > 1:
            self.layer.set_top_k(k)
        self.set_scales()

    def set_scales(self):
        self.layer.set_weight_scales([s for _, s in self.gu], [s for _, s in self.dn], self.sgu[1], self.sdn[1],
                                     group=self.group)

    def weights(self):
        return self.Wr, [w for w, _ in self.gu], [w for w, _ in self.dn], self.sgu[0], self.sdn[0]

    def tokens(self, T, seed=1):
        g = torch.Generator().manual_seed(seed)
        return torch.randn(T, self.d, generator=g).to(torch.bfloat16).cuda()

    def ffn(self, x, gate, gu, dn):
        """SwiGLU of the gated rows: the exact values and a bound on what the
        layer's fp32 sums, f16 hidden rows and fast exp may be off by."""
        q, s = unpack(gu[0]), each_row(gu[1], self.group, self.d)
        a = (x @ (q * s)) * gate
        ea = product_bound(x, q, s, -(-self.d // 32)) * gate
        ga, ua = a.chunk(2, dim=1)
        eg, eu = ea.chunk(2, dim=1)
        silu = ga * torch.sigmoid(ga)
        h = silu * ua
        # |silu'| <= 1.1; exp, divide and products: 2^-19 for |a| < 20; then half a step of f16
        eh = 1.1 * eg * (ua.abs() + eu) + silu.abs() * eu + 2.0 ** -19 * h.abs()
        eh = eh + (h.abs() + eh) * 2.0 ** -11 + 2.0 ** -25
        q, s = unpack(dn[0]), each_row(dn[1], self.group, q.shape[1] // 2)
        return h @ (q * s), eh @ (q * s).abs() + product_bound(h.abs() + eh, q, s, -(-h.shape[1] // 32))

    def check(self, out, x, idx, gate):
        """out against the definition with the layer's own routing."""
        xd, idx, gate = x.double().cpu(), idx.cpu().long(), gate.cpu().double()
        one = torch.ones(x.shape[0], 1, dtype=torch.float64)
        y, tol = self.ffn(xd, one, self.sgu, self.sdn)
        for e in range(self.E):
            n = torch.nonzero(idx == e).flatten()
            if len(n):
                t = n // self.k
                v, b = self.ffn(xd[t], gate[n][:, None], self.gu[e], self.dn[e])
                y.index_add_(0, t, v)
                tol.index_add_(0, t, b)
        tol = tol + half_step(y.abs() + tol, torch.bfloat16) + 2.0 ** -22 * y.abs()
        err = (out.double().cpu() - y).abs()
        assert bool((err <= tol).all()), float((err - tol).max())
        # the bound is not a loose one: it stays below the values' size
        assert float(tol.mean()) < 0.2 * float(y.abs().mean())

    def run_and_check(self, x):
        out = self.layer.forward(x, *self.weights())
        self.layer.check_device_status()
        if not self.E:
            self.check(out, x, torch.zeros(0), torch.zeros(0))
            return out
        r = self.layer.routing()
        logits = x.double().cpu() @ self.Wr.double().cpu()
        top = torch.sort(logits, dim=1, descending=True, stable=True)
        want = top.indices[:, :self.k].flatten()
        margin = (top.values[:, :-1] - top.values[:, 1:])[:, :self.k].amin(1).repeat_interleave(self.k) if self.E > self.k \
            else torch.full((want.numel(),), 1.0)
        keep = margin > 1e-4
        got = r["idx"].cpu().long()
        assert bool((got[keep] == want[keep]).all())
        lg = logits.repeat_interleave(self.k, 0).gather(1, got[:, None]).flatten()
        assert bool((r["gate"].cpu().double() - torch.sigmoid(lg)).abs().max() < 1e-5)
        self.check(out, x, got, r["gate"])
        return out


LAYERS = [  # d, F, Fs, E, k, group, scales, tokens
    (64, 64, 64, 2, 1, 32, "f32", (1, 2, 16)),
    (128, 192, 64, 4, 2, 64, "f16", (1, 7, 8, 9)),
    (256, 512, 512, 8, 2, 64, "f32", (8, 16)),
    (320, 128, 448, 5, 3, 128, "bf16", (3, 15)),
    (192, 256, 128, 3, 1, 256, "f16", (16, 17, 40)),
    (512, 320, 2112, 32, 4, 96, "bf16", (5, 16, 150)),
    (2112, 64, 128, 16, 1, 32, "f16", (1, 300)),
    (64, 0, 128, 0, 1, 32, "f32", (1, 16, 33)),
]


@pytest.mark.gpu
@pytest.mark.parametrize("d,F,Fs,E,k,group,st,tokens", LAYERS)
def test_layer(d, F, Fs, E, k, group, st, tokens):
    m = Layer(d, F, Fs, E, group, st, k)
    for T in tokens:
        m.run_and_check(m.tokens(T, seed=T))


@pytest.mark.gpu
@pytest.mark.parametrize("E", [6, 8])
def test_layer_whose_tokens_all_take_one_expert(E):
    m = Layer(128, 128, 64, E, 32, "f32", k=2)
    bias = torch.zeros(E, device="cuda")
    bias[2], bias[4] = 50.0, 25.0
    m.layer.set_router_bias(bias)
    for T in (16, 100):
        x = m.tokens(T)
        out = m.layer.forward(x, *m.weights())
        r = m.layer.routing()
        assert r["counts"].tolist() == [0, 0, T, 0, T] + [0] * (E - 5)
        assert r["offsets"].tolist() == [0, 0, 0, T, T] + [2 * T] * (E - 4)
        assert r["perm"].view(2, T).tolist() == [list(range(0, 2 * T, 2)), list(range(1, 2 * T, 2))]
        m.check(out, x, r["idx"], r["gate"])


@pytest.mark.gpu
@pytest.mark.parametrize("E,k,T", [(136, 4, 16), (256, 4, 16), (256, 1, 1), (8, 4, 9), (248, 2, 13), (128, 3, 16)])
def test_layer_with_many_experts(E, k, T):
    """More than 128 experts (two blocks of them in the routing), k up to 4."""
    m = Layer(128, 64, 64, E, 64, "bf16", k=k)
    x = m.tokens(T, seed=E)
    m.run_and_check(x)
    r = m.layer.routing()
    idx = r["idx"].cpu().long()
    assert torch.equal(r["counts"].cpu().long(), torch.bincount(idx, minlength=E))
    assert torch.equal(r["perm"].cpu().long(), torch.argsort(idx, stable=True))
    assert torch.equal(r["offsets"].cpu().long()[1:], torch.bincount(idx, minlength=E).cumsum(0))


@pytest.mark.gpu
@pytest.mark.parametrize("E", [4, 8])
def test_ties_and_nan_logits_route_as_the_layer_says(E):
    """Equal logits take the lower index, NaN only when no number is left."""
    m = Layer(64, 64, 64, E, 32, "f32", k=2)
    zero = m.weights()
    zero[0].zero_()
    x = m.tokens(5)
    m.layer.forward(x, *zero)
    assert m.layer.routing()["idx"].tolist() == [0, 1] * 5
    bias = torch.full((E,), float("nan"), device="cuda")
    bias[3] = -float("inf")
    m.layer.set_router_bias(bias)
    m.layer.forward(x, *zero)
    assert m.layer.routing()["idx"].tolist() == [3, 0] * 5


@pytest.mark.gpu
def test_tokens_past_f16s_range_and_not_finite_tokens():
    """Rows of x beyond 65504 get a power of two; an infinite token is its own row's matter."""
    m = Layer(128, 64, 64, 8, 32, "f16")
    m.gu = [[w, s * 1e-6] for w, s in m.gu]
    m.sgu = [m.sgu[0], m.sgu[1] * 1e-6]
    m.gu, m.sgu = [[w, s.clamp(min=6e-8)] for w, s in m.gu], [m.sgu[0], m.sgu[1].clamp(min=6e-8)]
    m.set_scales()
    x = m.tokens(9)
    x[::2] *= 2.0 ** 18
    out = m.run_and_check(x)
    x[3, 5] = float("inf")
    bad = m.layer.forward(x, *m.weights())
    keep = [0, 1, 2, 4, 5, 6, 7, 8]
    assert torch.equal(bad[keep], out[keep]) and not bool(torch.isfinite(bad[3]).all())
    with pytest.raises(L4MoEError):
        m.layer.check_device_status()


@pytest.mark.gpu
def test_empty_batch_other_streams_and_two_layers_at_once():
    a, b = Layer(256, 128, 128, 8, 64, "f16", seed=1), Layer(256, 192, 64, 16, 32, "bf16", k=2, seed=2)
    assert a.layer.bind(*a.weights()).forward(a.tokens(0)).shape == (0, 256)
    xa, xb = a.tokens(16), b.tokens(7)
    want = a.run_and_check(xa), b.run_and_check(xb)
    ba, bb = a.layer.bind(*a.weights()), b.layer.bind(*b.weights())
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [torch.empty_like(w) for w in want]
    for _ in range(30):
        ba.forward(xa, out=outs[0], stream=s1)
        bb.forward(xb, out=outs[1], stream=s2.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


@pytest.mark.gpu
def test_a_decode_step_with_its_router_watched_and_an_output_head():
    """The three together: the layer's experts, the losses and counts of its
    own routing, and a 4-bit output matrix, captured and replayed."""
    from sparse_moe_transformer_router_b200.router_loss import router_loss
    m = Layer(256, 128, 128, 16, 64, "f16", k=2)
    bound = m.layer.bind(*m.weights())
    g = torch.Generator().manual_seed(4)
    head = [t.cuda() for t in quantize_int4_groups(torch.randn(256, 1024, generator=g) * 0.05, 64, torch.float16)]
    x = m.tokens(12)
    routing = None

    def step():
        h = bound.forward(x)
        idx = m.layer.routing()["idx"]
        r = router_loss(x.float() @ m.Wr.float(), 2, idx=idx)
        return h, r, int4_matvec(h, head[0], head[1], 64)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, r, logits = step()
    for seed in (1, 2):
        x.copy_(m.tokens(12, seed=seed))
        graph.replay()
        torch.cuda.synchronize()
        routing = m.layer.routing()
        m.check(h, x, routing["idx"], routing["gate"])
        check(logits, h, head[0], head[1], 64)
        assert torch.equal(r.counts, routing["counts"]) and r.rows.item() == 12
        f = routing["counts"].double() / 24
        P = torch.softmax(x.double() @ m.Wr.double(), 1).mean(0)
        assert abs(r.balance.item() - float(16 * (f * P).sum())) < 1e-4


@pytest.mark.gpu
def test_column_scales_as_one_group():
    """Group scales that cover a whole column are the column scales: both
    paths of the layer agree to their roundings."""
    m = Layer(128, 192, 64, 4, 192, "f32")
    x = m.tokens(12)
    grouped = m.run_and_check(x)
    # group 192 >= d = 128 and = F: one row of scales each; Fs = 64 too
    column = L4MoE(128, 192, 64, 4, "int4")
    column.set_weight_scales([s[0].contiguous() for _, s in m.gu], [s[0].contiguous() for _, s in m.dn],
                             m.sgu[1][0].contiguous(), m.sdn[1][0].contiguous())
    out = column.forward(x, *m.weights())
    r = column.routing()
    m.check(out, x, r["idx"], r["gate"])
    # and one handle may change from one kind of scales to the other
    m.layer.set_weight_scales([s[0].contiguous() for _, s in m.gu], [s[0].contiguous() for _, s in m.dn],
                              m.sgu[1][0].contiguous(), m.sdn[1][0].contiguous())
    assert torch.equal(m.layer.forward(x, *m.weights()), out)
    m.set_scales()
    assert torch.equal(m.layer.forward(x, *m.weights()), grouped)


@pytest.mark.gpu
def test_bound_static_host_and_captured_calls_agree():
    m = Layer(256, 128, 192, 8, 64, "bf16", k=2)
    x = m.tokens(11)
    want = m.run_and_check(x)
    bound = m.layer.bind(*m.weights())
    assert torch.equal(bound.forward(x), want)
    out = torch.empty_like(want)
    assert bound.forward(x, out=out) is out and torch.equal(out, want)
    out = torch.empty_like(want)
    m.layer.forward_static(x, *m.weights(), out)
    assert torch.equal(out, want)
    host_in, host_out = x.cpu().pin_memory(), torch.empty(x.shape, dtype=x.dtype).pin_memory()
    m.layer.forward_host(host_in, *m.weights(), host_out)
    m.layer.check_device_status()
    assert torch.equal(host_out, want.cpu())
    torch.cuda.synchronize()
    graphs = []
    for call in (lambda: bound.forward(x, out=out), lambda: m.layer.forward_static(x, *m.weights(), out)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    for seed in (5, 6):
        x.copy_(m.tokens(11, seed=seed))
        want = m.layer.forward(x, *m.weights())
        for g in graphs:
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
    with pytest.raises(ValueError, match="dtype"):
        bound.forward(x.float())
    with pytest.raises(ValueError, match="shape"):
        m.layer.bind(m.Wr[:, :4].contiguous(), *m.weights()[1:])


@pytest.mark.gpu
def test_hidden_values_past_f16_are_reported():
    m = Layer(64, 64, 64, 2, 32, "f32")
    x = m.tokens(4) * 3e4
    m.layer.forward(x, *m.weights())
    with pytest.raises(L4MoEError) as err:
        m.layer.check_device_status()
    assert err.value.status == binding.ERR_RANGE
    m.run_and_check(m.tokens(4))


@pytest.mark.gpu
def test_layer_refusals():
    m = Layer(64, 64, 64, 2, 32, "f32")
    lib, h = m.layer._lib, m.layer._h
    arr = (ctypes.c_void_p * 2)(256, 256)
    off = (ctypes.c_void_p * 2)(256, 264)
    assert lib.l4moe_set_group_scales(h, 32, 0, arr, arr, None, 256) == binding.ERR_ARG
    assert lib.l4moe_set_group_scales(h, 33, 0, arr, arr, 256, 256) == binding.ERR_ARG
    assert lib.l4moe_set_group_scales(h, 32, 4, arr, arr, 256, 256) == binding.ERR_DTYPE
    assert lib.l4moe_set_group_scales(h, 32, 0, arr, off, 256, 256) == binding.ERR_ALIGN
    other = L4MoE(64, 64, 64, 2, "int8")
    assert lib.l4moe_set_group_scales(other._h, 32, 0, arr, arr, 256, 256) == binding.ERR_DTYPE
    m.run_and_check(m.tokens(3))  # the refused calls changed nothing


@pytest.mark.gpu
@pytest.mark.parametrize("E,k,T", [(4, 2, 174_800), (0, 1, 524_289)])
def test_a_batch_past_the_units_of_a_launch_is_refused_before_anything_runs(E, k, T):
    """The grid's y axis holds 65535 units of up to 8 rows: at most min(E, T k)
    + T k / 8 of routed rows and T / 8 of the shared expert's."""
    m = Layer(64, 64 if E else 0, 64, E, 32, "f16", k)
    few = m.tokens(5)
    want = m.run_and_check(few)
    routed = {n: v.clone() for n, v in m.layer.routing().items()} if E else {}
    launches = m.layer.launch_count
    x = torch.zeros(T, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(x, 7.0)
    with pytest.raises(L4MoEError, match="batch too long") as err:
        m.layer.forward(x, *m.weights(), out=out)
    assert err.value.status == binding.ERR_ARG
    assert m.layer.launch_count == launches and bool((out == 7.0).all())
    if E:
        assert all(torch.equal(v, routed[n]) for n, v in m.layer.routing().items())
    m.layer.check_device_status()
    assert torch.equal(m.layer.forward(few, *m.weights()), want)
