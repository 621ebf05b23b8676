"""Measured calls of the scored expert router and of the MXFP4 operators.

Five operators: the scored router (sigmoid or softmax scores, a balance bias, expert groups, top-k,
renormalised weights), its gradient, the MXFP4 quantizer with the decoder, the dense MXFP4 product
and the routed experts' grouped MXFP4 products (gate+up with SiLU, and down).  ``run`` computes
them in plain torch operations, or through the framework when ``own`` is set.

MXFP4 tensors: codes uint8 [rows, K/2] (two E2M1 codes per byte, the even element in the low
nibble) and scales uint8 [rows, K/32] (E8M0: 2**(byte - 127), 255 = NaN).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ---------------------------------------------------------------------------------------

def listed():
    router = dict(op="router", bias=True, groups=8, topk_groups=4, group_top=2, renorm=True, scale=2.5)
    return [
        # decode step of eight sequences: 384 experts, six chosen, grouped sigmoid scores with a balance bias
        dict(router, name="router_decode_t8", T=8, E=384, k=6, score="sigmoid", dtype="f32"),
        # the same router over an 8192-token prompt
        dict(router, name="router_prefill_t8192", T=8192, E=384, k=6, score="sigmoid", dtype="f32"),
        # ragged batch, plain softmax without groups or bias, bf16 logits, an odd number of experts
        dict(name="router_softmax_t1531", op="router", T=1531, E=101, k=7, score="softmax", dtype="bf16", bias=False,
             groups=1, topk_groups=1, group_top=1, renorm=False, scale=1.0),
        # training step: gradient of the renormalised sigmoid weights over an 8192-token batch
        dict(name="router_grad_t8192", op="router_grad", T=8192, E=384, k=6, score="sigmoid", dtype="f32",
             renorm=True, scale=2.5),
        # training step: softmax weights kept as they are (every logit has a gradient), ragged batch
        dict(name="router_grad_softmax_t1531", op="router_grad", T=1531, E=384, k=6, score="softmax", dtype="bf16",
             renorm=False, scale=1.0),
        # activations of a decode step
        dict(name="quantize_decode_8x7168", op="quantize", rows=8, cols=7168, dtype="bf16"),
        # the experts' hidden states of an 8192-token prompt, six experts a token
        dict(name="quantize_prefill_49152x2048", op="quantize", rows=49152, cols=2048, dtype="bf16"),
        # shared expert's down projection at decode
        dict(name="linear_decode_m8", op="linear", M=8, N=7168, K=2048),
        # projection of a large ragged prompt
        dict(name="linear_prefill_m16381", op="linear", M=16381, N=4096, K=7168),
        # gate+up of a decode step: the 48 experts that one GPU holds of 384
        dict(name="experts_up_decode_t8", op="experts_up", T=8, E=384, local=48, k=6, H=7168, I=2048, zipf=False),
        # down projection of a short prompt over all 384 experts, about eight rows each
        dict(name="experts_down_t512", op="experts_down", T=512, E=384, local=384, k=6, H=7168, I=2048, zipf=False),
        # gate+up of a long prompt, skewed routing: experts of no row, of a few and of thousands
        dict(name="experts_up_prefill_t8192", op="experts_up", T=8192, E=384, local=384, k=6, H=7168, I=2048,
             zipf=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["router", "router_grad", "quantize", "linear", "experts_up", "experts_down"])
    if op in ("router", "router_grad"):
        c = dict(op=op, T=_log_int(rng, 1, 8192), score=rng.choice(["sigmoid", "softmax"]),
                 dtype=rng.choice(["f32", "bf16"]), renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]))
        groups = rng.choice([1, 1, 2, 4, 8]) if op == "router" else 1
        per = rng.randint(max(1, -(-16 // groups)), 384 // groups)
        c["E"] = groups * per
        if op == "router":
            tg = rng.randint(max(1, groups // 2), groups)
            c.update(bias=rng.random() < 0.7, groups=groups, topk_groups=tg, group_top=rng.choice([1, 2]))
            c["k"] = rng.randint(1, min(8, tg * per))
        else:
            c["k"] = rng.randint(2, 8)  # one renormalised weight alone has no gradient
        return c
    if op == "quantize":
        cols = 32 * _log_int(rng, 4, 224)
        rows = _log_int(rng, 1, min(49152, 49152 * 2048 // cols))
        return dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "linear":
        return dict(op=op, M=_log_int(rng, 1, 16381), N=16 * _log_int(rng, 4, 256), K=128 * _log_int(rng, 1, 56))
    H, I = 256 * _log_int(rng, 1, 28), 128 * _log_int(rng, 1, 16)
    E = rng.choice([8, 16, 32, 48, 96])
    return dict(op=op, T=_log_int(rng, 1, 8192), E=E, local=rng.choice([E, max(1, E // 4)]), k=rng.randint(1, 6), H=H,
                I=I, zipf=rng.random() < 0.5)


# ---- inputs --------------------------------------------------------------------------------------

def _gen(seed, stream):
    g = torch.Generator(device=DEV)
    g.manual_seed((int(seed) * 1_000_003 + stream * 10_007) & 0x7FFF_FFFF_FFFF)
    return g


def _normal(shape, seed, stream, std=1.0):
    return torch.randn(shape, generator=_gen(seed, stream), device=DEV) * std


def _pow2(e):
    """2**e in float64, exactly, for whole e in the normal range."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _encode(x):
    """Codes and scales of float32 x [rows, K], for inputs that a program has already quantized."""
    b = x.reshape(x.shape[0], -1, 32)
    amax = b.abs().amax(-1)
    e = (torch.frexp(amax).exponent - 3).clamp(min=-127)
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    a = b.abs() * _pow2(-e[..., None])
    mag = sum((a > t).to(torch.uint8) for t in (0.25, 1.25, 2.5, 5.0)) + sum((a >= t).to(torch.uint8) for t in
                                                                               (0.75, 1.75, 3.5))
    c = (mag | (b < 0).to(torch.uint8) << 3).reshape(x.shape[0], -1, 2)
    return (c[..., 0] | c[..., 1] << 4).contiguous(), (e + 127).to(torch.uint8)


def _weights(E, N, K, seed, stream):
    """MXFP4 weights of E matrices [N, K], N(0, 0.02)."""
    codes = torch.empty(E, N, K // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(E, N, K // 32, dtype=torch.uint8, device=DEV)
    for e in range(E):
        codes[e], scales[e] = _encode(_normal((N, K), seed, stream + e, 0.02))
    return codes, scales


def _routing(case, seed):
    """Local rows by expert: counts [local], offsets [local + 1] and the token of each row (-1: unused)."""
    g = np.random.default_rng([int(seed), 1])
    T, E, k = case["T"], case["E"], case["k"]
    z = g.standard_normal((T, E), dtype=np.float32)
    if case["zipf"]:
        z -= (1.2 * np.log(1 + g.permutation(E))).astype(np.float32)
    ids = np.argpartition(-z, k - 1, axis=1)[:, :k]
    tok, ex = np.repeat(np.arange(T), k), ids.reshape(-1)
    keep = ex < case["local"]
    tok, ex = tok[keep], ex[keep]
    order = np.argsort(ex, kind="stable")
    counts = np.bincount(ex, minlength=case["local"]).astype(np.int32)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    row_token = np.full(T * k, -1, np.int32)
    row_token[:len(order)] = tok[order]
    return counts, offsets, row_token


def _rows_of(case):
    return max(1, case["T"] * case["k"])


def prepare(case, seed):
    op, s = case["op"], dict(case)
    f32, i32, u8 = (dict(dtype=d, device=DEV) for d in (torch.float32, torch.int32, torch.uint8))
    if op == "router":
        T, E, k = case["T"], case["E"], case["k"]
        s["logits"] = _normal((T, E), seed, 0).to(DTYPES[case["dtype"]])
        s["balance"] = _normal((E,), seed, 1, 0.1) if case["bias"] else None
        s["ids"], s["weights"] = torch.empty(T, k, **i32), torch.empty(T, k, **f32)
    elif op == "router_grad":
        T, E, k = case["T"], case["E"], case["k"]
        s["logits"] = _normal((T, E), seed, 0).to(DTYPES[case["dtype"]])
        s["ids"] = torch.rand((T, E), generator=_gen(seed, 2), device=DEV).topk(k, 1).indices.to(torch.int32)
        s["grad"] = _normal((T, k), seed, 3)
        s["grad_logits"] = torch.empty_like(s["logits"])
    elif op == "quantize":
        rows, cols = case["rows"], case["cols"]
        s["x"] = _normal((rows, cols), seed, 0, 0.09).to(DTYPES[case["dtype"]])
        s["codes"], s["scales"] = torch.empty(rows, cols // 2, **u8), torch.empty(rows, cols // 32, **u8)
        s["values"] = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    elif op == "linear":
        s["a_codes"], s["a_scales"] = _encode(_normal((case["M"], case["K"]), seed, 0, 0.09))
        s["w_codes"], s["w_scales"] = (t[0] for t in _weights(1, case["N"], case["K"], seed, 1))
        s["out"] = torch.empty(case["M"], case["N"], dtype=torch.bfloat16, device=DEV)
    else:
        H, I, L = case["H"], case["I"], case["local"]
        counts, offsets, row_token = _routing(case, seed)
        s["rows"] = counts.tolist()
        s["counts"], s["offsets"], s["row_token"] = (torch.from_numpy(a).to(DEV) for a in (counts, offsets, row_token))
        up = op == "experts_up"
        n, width = (case["T"], H) if up else (_rows_of(case), I)
        s["a_codes"], s["a_scales"] = _encode(_normal((n, width), seed, 0, 0.09))
        s["w_codes"], s["w_scales"] = _weights(L, 2 * I if up else H, width, seed, 1)
        s["out"] = torch.zeros(_rows_of(case), I if up else H, dtype=torch.bfloat16, device=DEV)
    return s


# ---- one pass ------------------------------------------------------------------------------------

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from nvfp4_block_scaled_top_amd import megamoe as mm

    op = s["op"]
    if op == "router":
        mm.moe_router_scores(s["logits"], s["k"], s["ids"], s["weights"], bias=s["balance"], score=s["score"],
                             n_group=s["groups"], topk_group=s["topk_groups"], group_top=s["group_top"],
                             renormalize=s["renorm"], scale=s["scale"])
        return {"ids": s["ids"], "weights": s["weights"]}
    if op == "router_grad":
        mm.moe_router_scores_bwd(s["logits"], s["ids"], s["grad"], s["grad_logits"], score=s["score"],
                                 renormalize=s["renorm"], scale=s["scale"])
        return {"grad_logits": s["grad_logits"]}
    if op == "quantize":
        mm.mxfp4_quantize_act(s["x"], s["codes"], s["scales"])
        mm.mxfp4_dequantize(s["codes"], s["scales"], s["values"])
        return {"values": s["values"], "scales": s["scales"]}
    if op == "linear":
        mm.mxfp4_linear(s["a_codes"], s["a_scales"], s["w_codes"], s["w_scales"], s["out"])
    elif op == "experts_up":
        mm.moe_grouped_gemm_l1_silu_mxfp4(s["a_codes"], s["a_scales"], s["row_token"], s["offsets"], s["counts"],
                                          s["w_codes"], s["w_scales"], s["out"], max_rows_per_expert=s["T"])
    else:
        mm.moe_grouped_gemm_l2_mxfp4(s["a_codes"], s["a_scales"], s["offsets"], s["counts"], s["w_codes"],
                                     s["w_scales"], s["out"], max_rows_per_expert=s["T"])
    return {"out": s["out"]}


def _scores(logits, kind):
    z = logits.double()
    return torch.sigmoid(z) if kind == "sigmoid" else torch.softmax(z, -1)


def _plain_router(s):
    T, E, G, k = s["T"], s["E"], s["groups"], s["k"]
    score = _scores(s["logits"], s["score"])
    choice = score.float() if s["balance"] is None else score.float() + s["balance"]
    if s["topk_groups"] < G:
        best = choice.view(T, G, E // G).topk(min(s["group_top"], E // G), -1).values.sum(-1)
        kept = torch.sort(best, dim=-1, descending=True, stable=True).indices[:, :s["topk_groups"]]
        mask = torch.zeros(T, G, dtype=torch.bool, device=choice.device).scatter_(1, kept, True)
        choice = choice.masked_fill(~mask.repeat_interleave(E // G, 1), float("-inf"))
    ids = torch.sort(choice, dim=-1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, ids)
    if s["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return {"ids": ids.to(torch.int32), "weights": (w * s["scale"]).float()}


def _plain_router_grad(s):
    ids, score = s["ids"].long(), _scores(s["logits"], s["score"])
    p, g = score.gather(1, ids), s["grad"].double() * s["scale"]
    if s["renorm"]:
        total = p.sum(-1, keepdim=True)
        g = (g - (g * p).sum(-1, keepdim=True) / total) / total
    if s["score"] == "sigmoid":
        dz = torch.zeros_like(score).scatter_(1, ids, g * p * (1 - p))
    else:
        dz = torch.zeros_like(score).scatter_(1, ids, g)
        dz = score * (dz - (g * p).sum(-1, keepdim=True))
    return {"grad_logits": dz.to(s["logits"].dtype)}


def _plain_quantize(s):
    b = s["x"].float().view(s["rows"], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.where(amax > 0, (torch.frexp(amax).exponent - 3).clamp(min=-127), -127)
    a = b.abs() * _pow2(-e)  # in 64 bits, where the division by the scale is exact
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = (torch.round(a / step) * step).clamp(max=6)
    values = q * _pow2(e) * torch.sign(b)
    return {"values": values.view(s["rows"], -1).bfloat16(), "scales": (e[..., 0] + 127).to(torch.uint8)}


def _decode(codes, scales):
    """float32 values [rows, K] of MXFP4 codes [rows, K/2] and scales [rows, K/32]."""
    table = torch.tensor(E2M1, device=codes.device)
    v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).view(codes.shape[0], -1, 32)
    return (v * _pow2(scales.int() - 127).float()[..., None]).view(codes.shape[0], -1)


def _silu_mul(z):
    gate, up = z.chunk(2, -1)
    return gate / (1 + torch.exp(-gate)) * up


def _plain_experts(s, up):
    a = _decode(s["a_codes"], s["a_scales"])
    out, r = torch.zeros_like(s["out"]), 0
    for e, n in enumerate(s["rows"]):  # one product an expert: their row counts differ
        if n:
            x = a[s["row_token"][r:r + n]] if up else a[r:r + n]
            z = x @ _decode(s["w_codes"][e], s["w_scales"][e]).t()
            out[r:r + n] = (_silu_mul(z) if up else z).bfloat16()
            r += n
    return {"out": out}


def _run_plain(s):
    op = s["op"]
    if op == "router":
        return _plain_router(s)
    if op == "router_grad":
        return _plain_router_grad(s)
    if op == "quantize":
        return _plain_quantize(s)
    if op == "linear":
        a, w = _decode(s["a_codes"], s["a_scales"]), _decode(s["w_codes"], s["w_scales"])
        return {"out": (a @ w.t()).bfloat16()}
    return _plain_experts(s, op == "experts_up")


# ---- bytes and operations of one pass --------------------------------------------------------------

def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4}
    if op == "router":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * size[case["dtype"]] + T * k * 8 + (E * 4 if case["bias"] else 0), "flops": 8 * T * E}
    if op == "router_grad":
        T, E, k, b = case["T"], case["E"], case["k"], size[case["dtype"]]
        # sigmoid scores need the chosen logits alone, softmax scores all of them
        read = T * k * b if case["score"] == "sigmoid" else T * E * b
        return {"bytes": read + T * k * 8 + T * E * b, "flops": (8 * T * E if case["score"] == "softmax" else 12 * T * k)}
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * size[case["dtype"]] + n * 2 + n // 32, "flops": 4 * n}
    per = 0.5 + 1 / 32  # bytes of an MXFP4 element with its share of the scale
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * K * per + 2 * M * N, "flops": 2 * M * N * K}
    counts, _, row_token = _routing(case, 0)
    rows, active, H, I = int(counts.sum()), int((counts > 0).sum()), case["H"], case["I"]
    if op == "experts_up":
        tokens = len(np.unique(row_token[row_token >= 0]))
        return {"bytes": max(1, active * 2 * I * H * per + tokens * H * per + rows * I * 2), "flops": 4 * rows * I * H}
    return {"bytes": max(1, active * H * I * per + rows * I * per + rows * H * 2), "flops": 2 * rows * I * H}


# ---- the definitions in 64 bits ---------------------------------------------------------------------

def _exact_values(codes, scales):
    """float64 values from the fields of each code: sign, two exponent bits (bias 1), one mantissa bit."""
    n = torch.empty(codes.shape[0], codes.shape[1], 2, dtype=torch.int32, device=codes.device)
    n[..., 0], n[..., 1] = codes.int() % 16, codes.int() // 16
    sign, ex, man = 1 - 2 * (n // 8), n // 2 % 4, n % 2
    mag = torch.where(ex == 0, man * 0.5, (1 + 0.5 * man) * 2.0 ** (ex - 1).double())
    block = torch.from_numpy(np.ldexp(1.0, scales.cpu().numpy().astype(np.int32) - 127)).to(DEV).repeat_interleave(32, 1)
    return (sign * mag).view(codes.shape[0], -1) * block


def _exact_softmax(z):
    e = torch.exp(z - z.max(1, keepdim=True).values)
    return e / e.sum(1, keepdim=True)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "router":
        # the choice is made of whole numbers; the weights follow from it in 64 bits
        z = s["logits"].double()
        p = 1 / (1 + torch.exp(-z)) if case["score"] == "sigmoid" else _exact_softmax(z)
        key = p.float() if s["balance"] is None else p.float() + s["balance"]
        key = key.cpu().numpy()
        p, T, G = p.cpu().numpy(), case["T"], case["groups"]
        if case["topk_groups"] < G:
            by = np.sort(key.reshape(T, G, -1), -1)[..., ::-1][..., :case["group_top"]]
            rank = np.argsort(np.argsort(-by.sum(-1, dtype=np.float32), 1, kind="stable"), 1, kind="stable")
            key = np.where(np.repeat(rank < case["topk_groups"], case["E"] // G, 1), key, -np.inf)
        ids = np.argsort(-key, 1, kind="stable")[:, :case["k"]]
        w = np.take_along_axis(p, ids, 1)
        w = case["scale"] * (w / w.sum(1, keepdims=True) if case["renorm"] else w)
        return {"ids": ids.astype(np.int32), "weights": w}
    if op == "router_grad":
        # through the Jacobian of the weights with respect to the logits, one chosen expert at a time
        z, ids, g = s["logits"].double(), s["ids"].long(), s["grad"].double() * case["scale"]
        p = 1 / (1 + torch.exp(-z)) if case["score"] == "sigmoid" else _exact_softmax(z)
        chosen, dz = torch.gather(p, 1, ids), torch.zeros_like(z)
        total = chosen.sum(1)
        for j in range(case["k"]):
            up = g[:, j]
            if case["renorm"]:
                up = (g[:, j] * (total - chosen[:, j]) - (g * chosen).sum(1) + g[:, j] * chosen[:, j]) / total ** 2
            if case["score"] == "sigmoid":
                dz[torch.arange(len(z)), ids[:, j]] += up * chosen[:, j] * (1 - chosen[:, j])
            else:
                dz -= (up * chosen[:, j])[:, None] * p
                dz[torch.arange(len(z)), ids[:, j]] += up * chosen[:, j]
        return {"grad_logits": dz}
    if op == "quantize":
        # the nearest of the eight magnitudes, by distance; of two equally near ones the even code
        b = s["x"].double().view(-1, 32)
        e = torch.from_numpy(np.frexp(b.abs().amax(1).cpu().numpy())[1]).to(DEV) - 3
        e = torch.where(b.abs().amax(1) > 0, e, -127).clamp(min=-127)
        unit = torch.from_numpy(np.ldexp(1.0, e.cpu().numpy())).to(DEV)[:, None]
        a = b.abs() / unit
        best, near = torch.zeros_like(a), a.clone()
        for i in (2, 4, 6, 1, 3, 5, 7):
            d = (a - E2M1[i]).abs()
            best, near = torch.where(d < near, E2M1[i], best), torch.minimum(d, near)
        v = torch.copysign(best, b) * unit
        return {"values": v.view(case["rows"], -1), "scales": (e + 127).to(torch.uint8).view(case["rows"], -1)}
    if op == "linear":
        return {"out": _exact_values(s["a_codes"], s["a_scales"]) @ _exact_values(s["w_codes"], s["w_scales"]).T}
    a = _exact_values(s["a_codes"], s["a_scales"])
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    starts = s["offsets"].tolist()
    for e in range(case["local"]):
        rows = torch.arange(starts[e], starts[e + 1], device=DEV)
        if len(rows):
            src = s["row_token"][rows].long() if op == "experts_up" else rows
            z = torch.mm(a[src], _exact_values(s["w_codes"][e], s["w_scales"][e]).T)
            if op == "experts_up":
                g, u = z[:, :case["I"]], z[:, case["I"]:]
                z = g * torch.sigmoid(g) * u
            out[rows] = z
    return {"out": out}
