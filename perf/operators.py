"""Measured cases of three operators of a mixture-of-experts layer.

- ``router_loss``: the router's balance loss, z loss and per-expert counts over
  T tokens of E logits, and the gradient of the logits.
- ``int4_matvec``: products of a few tokens with a 4-bit weight that has one
  scale per group of input rows and output column.
- ``layer``: the whole feed-forward layer (router, routed and shared SwiGLU
  experts) for a few tokens, its 4-bit experts with such group scales.

``run`` computes a case in its plain form (elementary torch operations in 32
bits) or, where ``own`` is true, through the package's entry points.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
BALANCE, Z = 1e-2, 1e-3  # the weights of the two losses


# ------------------------------------------------------------------ the cases
def _loss(name, T, E, k, dtype, score="softmax", mask=False, given=False, backward=True):
    return {"name": name, "op": "router_loss", "T": T, "E": E, "k": k, "dtype": dtype, "score": score,
            "mask": mask, "given": given, "backward": backward}


def _matvec(name, T, K, N, group, dtype, scales):
    return {"name": name, "op": "int4_matvec", "T": T, "K": K, "N": N, "group": group, "dtype": dtype,
            "scales": scales}


def _layer(name, T, E, k, d, F, Fs, group, scales):
    return {"name": name, "op": "layer", "T": T, "E": E, "k": k, "d": d, "F": F, "Fs": Fs, "group": group,
            "scales": scales}


def listed():
    return [
        # a training step's router of 16 experts, one 4096-token batch
        _loss("loss_T4096_E16", 4096, 16, 1, "bf16"),
        # 128 experts, fp32 logits, a 16384-token batch with padding
        _loss("loss_T16384_E128_f32_mask", 16384, 128, 1, "f32", mask=True),
        # the most experts, four per token, sigmoid scores, a long batch
        _loss("loss_T65536_E256_sigmoid_k4", 65536, 256, 4, "bf16", score="sigmoid"),
        # counts and losses alone, of a routing made elsewhere (monitoring a running layer)
        _loss("loss_T8191_E100_given_fwd", 8191, 100, 2, "f16", given=True, backward=False),
        # the smallest call: a few tokens, four experts
        _loss("loss_T64_E4_f32", 64, 4, 2, "f32"),
        # one token through a gate/up matrix
        _matvec("matvec_T1_5120x16384_g128", 1, 5120, 16384, 128, "bf16", "f16"),
        # a full small batch through a down matrix, finer groups
        _matvec("matvec_T16_8192x5120_g64_f16", 16, 8192, 5120, 64, "f16", "f16"),
        # odd sizes: rows that are no multiple of a group, columns of no vector
        _matvec("matvec_T5_1001x1234_g32", 5, 1001, 1234, 32, "bf16", "f32"),
        # one token through an output head
        _matvec("matvec_T1_5120x202048_g128", 1, 5120, 202048, 128, "bf16", "bf16"),
        # decode of one token, 128 experts
        _layer("layer_T1_E128_g128", 1, 128, 1, 5120, 8192, 8192, 128, "f16"),
        # decode of sixteen tokens, 16 experts, fine groups
        _layer("layer_T16_E16_g32", 16, 16, 1, 5120, 8192, 8192, 32, "bf16"),
        # a small layer, two experts per token, fp32 scales
        _layer("layer_T8_E8_k2_small", 8, 8, 2, 256, 512, 512, 64, "f32"),
    ]


def _spread(rng, lo, hi):
    """A whole number, even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("router_loss", "int4_matvec", "layer"))
    if op == "router_loss":
        E = _spread(rng, 2, 256)
        c = _loss("", _spread(rng, 1, 65536), E, rng.randint(1, min(4, E)), rng.choice(("f32", "bf16", "f16")),
                  rng.choice(("softmax", "sigmoid")), rng.random() < 0.5, rng.random() < 0.3, rng.random() < 0.8)
    elif op == "int4_matvec":
        K = _spread(rng, 64, 16384)
        N = 2 * _spread(rng, 32, 16384)
        if rng.random() < 0.6:  # most matrices have round sizes
            K, N = max(64, K // 64 * 64), max(64, N // 64 * 64)
        c = _matvec("", rng.randint(1, 16), K, N, rng.choice((32, 64, 96, 128, 256)), rng.choice(("bf16", "f16")),
                    rng.choice(("f32", "bf16", "f16")))
    else:
        E = _spread(rng, 2, 64)
        k = rng.randint(1, min(2, E))
        c = _layer("", rng.randint(1, 16 // k), E, k, 64 * _spread(rng, 2, 80), 64 * _spread(rng, 2, 128),
                   64 * _spread(rng, 2, 128), rng.choice((32, 64, 128, 256)), rng.choice(("f32", "bf16", "f16")))
    del c["name"]
    return c


# ----------------------------------------------------------------- the inputs
def _codes(K, N, gen):
    """4-bit codes of normal weights, two per byte along the columns (the even column in the low nibble)."""
    q = torch.randn(K, N, generator=gen, device="cuda").mul_(2.6).round_().clamp_(-7, 7).to(torch.int8)
    q &= 15
    return (q[:, 0::2] | (q[:, 1::2] << 4)).view(torch.uint8)


def _scales(K, N, group, std, dtype, gen):
    s = torch.rand(-(-K // group), N, generator=gen, device="cuda").mul_(0.5).add_(0.75)
    return s.mul_(std / 2.6).to(TYPES[dtype])


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(1_000_003 * seed + 17)
    s = {"case": case}
    if case["op"] == "router_loss":
        T, E = case["T"], case["E"]
        # logits of about unit spread, some experts preferred
        lean = torch.randn(E, generator=gen, device="cuda")
        s["logits"] = (torch.randn(T, E, generator=gen, device="cuda") * 1.4 + lean).to(TYPES[case["dtype"]])
        # the loss's own gradient: 1, or the loss scale of training in f16
        s["up"] = torch.tensor(65536.0 if case["dtype"] == "f16" else 1.0, device="cuda")
        s["mask"] = torch.rand(T, generator=gen, device="cuda") < 0.9 if case["mask"] else None
        s["idx"] = None
        if case["given"]:
            # a routing with noise, and some entries dropped (-1)
            noisy = s["logits"].float() + torch.rand(T, E, generator=gen, device="cuda")
            idx = torch.sort(noisy, dim=1, descending=True, stable=True)[1][:, :case["k"]].to(torch.int32)
            s["idx"] = idx.masked_fill(torch.rand(T, case["k"], generator=gen, device="cuda") < 0.05, -1).contiguous()
    elif case["op"] == "int4_matvec":
        T, K, N = case["T"], case["K"], case["N"]
        s["x"] = torch.randn(T, K, generator=gen, device="cuda").to(TYPES[case["dtype"]])
        s["w"] = torch.cat([_codes(min(512, K - r), N, gen) for r in range(0, K, 512)])
        s["s"] = _scales(K, N, case["group"], 0.02, case["scales"], gen)
    else:
        T, E, d, F, Fs, g = (case[n] for n in ("T", "E", "d", "F", "Fs", "group"))
        s["x"] = torch.randn(T, d, generator=gen, device="cuda").to(torch.bfloat16)
        s["Wr"] = torch.randn(d, E, generator=gen, device="cuda").mul_(1.5 / math.sqrt(d)).to(torch.bfloat16)
        std = 0.02 * math.sqrt(5120 / d)
        s["gu"] = torch.stack([_codes(d, 2 * F, gen) for _ in range(E)])
        s["dn"] = torch.stack([_codes(F, d, gen) for _ in range(E)])
        s["sgu"], s["sdn"] = _codes(d, 2 * Fs, gen), _codes(Fs, d, gen)
        s["s_gu"] = torch.stack([_scales(d, 2 * F, g, std, case["scales"], gen) for _ in range(E)])
        s["s_dn"] = torch.stack([_scales(F, d, g, std, case["scales"], gen) for _ in range(E)])
        s["ss_gu"] = _scales(d, 2 * Fs, g, std, case["scales"], gen)
        s["ss_dn"] = _scales(Fs, d, g, std, case["scales"], gen)
        if own:  # the layer's handle, as a serving program keeps it
            from sparse_moe_transformer_router_b200.binding import L4MoE
            layer = L4MoE(d, F, Fs, E, "int4")
            layer.set_top_k(case["k"])
            layer.set_weight_scales(list(s["s_gu"]), list(s["s_dn"]), s["ss_gu"], s["ss_dn"], group=g)
            s["layer"] = layer.bind(s["Wr"], list(s["gu"]), list(s["dn"]), s["sgu"], s["sdn"])
    return s


# -------------------------------------------------------------- the plain forms
def _unpack(w):
    """Packed codes [..., K, N / 2] -> fp32 codes [..., K, N]."""
    pair = torch.stack((w & 15, w >> 4), dim=-1).flatten(-2).to(torch.int8)
    return ((pair ^ 8) - 8).float()


def _weight(w, s, group):
    """fp32 weights [..., K, N] of packed codes and group scales."""
    return _unpack(w).mul_(s.float().repeat_interleave(group, dim=-2)[..., :w.shape[-2], :])


def _plain_loss(s):
    c = s["case"]
    E, k = c["E"], c["k"]
    l = s["logits"].float()
    live = (l != -math.inf).any(1) if s["mask"] is None else (l != -math.inf).any(1) & s["mask"]
    n = live.sum().clamp(min=1)
    idx = s["idx"].long() if s["idx"] is not None else torch.sort(l, dim=1, descending=True, stable=True)[1][:, :k]
    hit = (idx.unsqueeze(2) == torch.arange(E, device=l.device)).sum(1)           # [T, E]
    counts = (hit * live.unsqueeze(1)).sum(0)
    f = counts.float() / (k * n)
    m = l.amax(1, keepdim=True)
    e = torch.exp(l - m)
    lse = (m + torch.log(e.sum(1, keepdim=True)))
    soft = e / e.sum(1, keepdim=True)
    if c["score"] == "sigmoid":
        sig = 1 / (1 + torch.exp(-l))
        p, slope = sig / sig.sum(1, keepdim=True), 1 - sig
    else:
        p, slope = soft, torch.ones_like(l)
    w = live.unsqueeze(1)
    zero = torch.zeros((), device=l.device)
    P = torch.where(w, p, zero).double().sum(0) / n                              # long sums in 64 bits
    balance = (E * (f.double() * P).sum()).float()
    z = (torch.where(w, lse * lse, zero).double().sum() / n).float()
    out = {"loss": BALANCE * balance + Z * z, "balance": balance, "z": z, "counts": counts.to(torch.int32)}
    if c["backward"]:
        g = BALANCE * E / n * p * slope * (f - (f * p).sum(1, keepdim=True)) + Z * 2 / n * lse * soft
        out["dlogits"] = torch.where(w, s["up"] * g, zero).to(s["logits"].dtype)
    return out


def _plain_matvec(s):
    return (s["x"].float() @ _weight(s["w"], s["s"], s["case"]["group"])).to(s["x"].dtype)


def _swiglu(x, gu, sgu, dn, sdn, group):
    """x [n, d] times one weight each (or one for all): fp32 [n, d]."""
    a = x.unsqueeze(-2) @ _weight(gu, sgu, group)
    gate, up = a.chunk(2, dim=-1)
    h = gate / (1 + torch.exp(-gate)) * up
    return (h @ _weight(dn, sdn, group)).squeeze(-2)


def _plain_layer(s):
    c = s["case"]
    x = s["x"].float()
    val, idx = torch.sort(x @ s["Wr"].float(), dim=1, descending=True, stable=True)
    val, idx = val[:, :c["k"]].reshape(-1), idx[:, :c["k"]].reshape(-1)
    gated = x.repeat_interleave(c["k"], 0) * (1 / (1 + torch.exp(-val))).unsqueeze(1)
    y = _swiglu(gated, s["gu"][idx], s["s_gu"][idx], s["dn"][idx], s["s_dn"][idx], c["group"])
    shared = _swiglu(x, s["sgu"], s["ss_gu"], s["sdn"], s["ss_dn"], c["group"])
    return (shared + y.view(c["T"], c["k"], -1).sum(1)).to(torch.bfloat16)


def run(state):
    c = state["case"]
    if not own:
        return {"router_loss": _plain_loss, "int4_matvec": _plain_matvec, "layer": _plain_layer}[c["op"]](state)
    if c["op"] == "router_loss":
        from sparse_moe_transformer_router_b200.router_loss import router_loss
        r = router_loss(state["logits"], c["k"], balance=BALANCE, z=Z, score=c["score"], mask=state["mask"],
                        idx=state["idx"])
        out = {"loss": r.loss, "balance": r.balance, "z": r.z, "counts": r.counts}
        if c["backward"]:
            out["dlogits"] = r.grad(state["up"])
        return out
    if c["op"] == "int4_matvec":
        from sparse_moe_transformer_router_b200.int4 import int4_matvec
        return int4_matvec(state["x"], state["w"], state["s"], c["group"])
    return state["layer"].forward(state["x"])


# --------------------------------------------------------------------- the work
def work(case):
    if case["op"] == "router_loss":
        n = case["T"] * case["E"]
        b = n * BYTES[case["dtype"]] + 4 * case["E"] + (case["T"] if case["mask"] else 0)
        b += 4 * case["T"] * case["k"] if case["given"] else 0
        if case["backward"]:
            b += n * BYTES[case["dtype"]]
        return {"bytes": b, "flops": n * (16 if case["backward"] else 8)}
    if case["op"] == "int4_matvec":
        T, K, N = case["T"], case["K"], case["N"]
        b = K * N // 2 + -(-K // case["group"]) * N * BYTES[case["scales"]] + 2 * T * (K + N)
        return {"bytes": b, "flops": 2 * T * K * N}
    T, E, k, d, F, Fs, g = (case[n] for n in ("T", "E", "k", "d", "F", "Fs", "group"))
    ss = BYTES[case["scales"]]

    def ffn(w):  # the codes and scales of one expert of width w
        return 3 * d * w // 2 + ss * (-(-d // g) * 2 * w + -(-w // g) * d)

    # the experts that T * k even draws touch
    touched = E * (1 - (1 - 1 / E) ** (T * k))
    return {"bytes": touched * ffn(F) + ffn(Fs) + 2 * d * E + 4 * T * d,
            "flops": 2 * T * d * E + 6 * T * d * (k * F + Fs)}


# ------------------------------------------------------ the definition in 64 bits
def _table():
    """The two codes of every byte, in 64 bits."""
    t = [[(b & 15) - 16 * ((b & 15) > 7), (b >> 4) - 16 * ((b >> 4) > 7)] for b in range(256)]
    return torch.tensor(t, dtype=torch.float64, device="cuda")


def _product64(x, w, s, group):
    """x [n, K] (64 bits) times the weight of packed codes w [K, N / 2], in column blocks."""
    table, K = _table(), w.shape[0]
    out = []
    for c in range(0, w.shape[1], 4096):
        q = table[w[:, c:c + 4096].int()].reshape(K, -1)
        r = torch.arange(K, device="cuda") // group
        out.append(x @ (q * s[:, 2 * c:2 * c + 8192].double()[r]))
    return torch.cat(out, 1)


def _exact_loss(s):
    c = s["case"]
    l = s["logits"].double()
    T, E = l.shape
    keep = ~torch.isneginf(l).all(1)
    if s["mask"] is not None:
        keep = keep & s["mask"]
    l, n = l[keep], max(1, int(keep.sum()))
    if s["idx"] is not None:
        chosen = s["idx"][keep].long()
    else:
        chosen = torch.argsort(-l, dim=1, stable=True)[:, :c["k"]]
    chosen = chosen.flatten()
    counts = torch.bincount(chosen[chosen >= 0], minlength=E)
    f = counts.double() / (c["k"] * n)
    lse = torch.logsumexp(l, 1)
    soft = torch.exp(l - lse[:, None])
    p = torch.softmax(-torch.log1p(torch.exp(-l)), 1) if c["score"] == "sigmoid" else soft
    balance, z = E * torch.dot(f, p.sum(0) / n), (lse ** 2).sum() / n
    out = {"loss": BALANCE * balance + Z * z, "balance": balance, "z": z, "counts": None}
    if c["backward"]:
        d = p * (f - (p @ f)[:, None])                    # of the score's logarithm
        if c["score"] == "sigmoid":
            d = d * torch.sigmoid(-l)
        g = torch.zeros(T, E, dtype=torch.float64, device="cuda")
        g[keep] = BALANCE * E / n * d + 2 * Z / n * lse[:, None] * soft
        out["dlogits"] = g * float(s["up"])
    return out


def _exact_layer(s):
    c = s["case"]
    x = s["x"].double()
    logits = x @ s["Wr"].double()
    order = torch.argsort(-logits, dim=1, stable=True)

    def ffn(rows, gu, s_gu, dn, s_dn):
        a = _product64(rows, gu, s_gu, c["group"])
        half = a.shape[1] // 2
        return _product64(a[:, :half] * torch.sigmoid(a[:, :half]) * a[:, half:], dn, s_dn, c["group"])

    out = ffn(x, s["sgu"], s["ss_gu"], s["sdn"], s["ss_dn"])
    for e in range(c["E"]):
        t, j = torch.nonzero(order[:, :c["k"]] == e, as_tuple=True)
        if len(t):
            g = torch.sigmoid(logits[t, e])
            out[t] += ffn(x[t] * g[:, None], s["gu"][e], s["s_gu"][e], s["dn"][e], s["s_dn"][e])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "router_loss":
        return _exact_loss(s)
    if case["op"] == "int4_matvec":
        return _product64(s["x"].double(), s["w"], s["s"], case["group"])
    return _exact_layer(s)
