"""Measured calls of the experts' 16-bit products with their gradients, and of the 8-bit integer operators.

Five operators: the grouped product of ragged experts in bf16 or fp16, its gradients (with respect to the
rows and to the weights), the 8-bit quantizer by rows with its decoder, the dense 8-bit product and the
routed experts' grouped 8-bit products (gate+up with SiLU, and down).  ``run`` computes them in plain torch
operations, or through the framework when ``own`` is set.

8-bit tensors: codes int8 [rows, K] and one float32 scale a row; an element's value is code * scale.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---- cases ---------------------------------------------------------------------------------------

def listed():
    return [
        # gate+up of a decode step of eight sequences on unquantized weights: the 48 experts one GPU holds of 384
        dict(name="grouped_decode_t8", op="grouped", T=8, E=384, local=48, k=6, K=7168, N=4096, dtype="bf16", gather=True,
             zipf=False),
        # down projection of a 1000-token batch over 64 experts, about 94 rows each
        dict(name="grouped_t1000", op="grouped", T=1000, E=64, local=64, k=6, K=2048, N=7168, dtype="f16", gather=False,
             zipf=False),
        # gate+up of an 8192-token batch, skewed routing: experts of a few rows and of thousands
        dict(name="grouped_t8192", op="grouped", T=8192, E=48, local=48, k=6, K=7168, N=4096, dtype="bf16", gather=True,
             zipf=True),
        # backward of a small layer on a short batch, odd widths
        dict(name="grouped_grad_t61", op="grouped_grad", T=61, E=8, local=8, k=2, K=520, N=1032, dtype="f16", dw="f16",
             gather=False, zipf=False),
        # backward of gate+up in a training step over 48 experts, skewed routing, float32 weight gradients
        dict(name="grouped_grad_t4096", op="grouped_grad", T=4096, E=48, local=48, k=6, K=7168, N=4096, dtype="bf16",
             dw="f32", gather=True, zipf=True),
        # activations of a decode step
        dict(name="quantize_decode_8x7168", op="quantize", rows=8, cols=7168, dtype="bf16"),
        # the experts' hidden states of an 8192-token prompt, six experts a token
        dict(name="quantize_prefill_49152x2048", op="quantize", rows=49152, cols=2048, dtype="bf16"),
        # shared expert's down projection at decode
        dict(name="linear_decode_m8", op="linear", M=8, N=7168, K=2048, dtype="bf16"),
        # projection of a large ragged prompt
        dict(name="linear_prefill_m16381", op="linear", M=16381, N=4096, K=7168, dtype="bf16"),
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
    op = rng.choice(["grouped", "grouped", "grouped_grad", "grouped_grad", "quantize", "linear", "experts_up",
                     "experts_down"])
    if op in ("grouped", "grouped_grad"):
        E = rng.choice([1, 4, 8, 16, 48, 64])
        c = dict(op=op, T=_log_int(rng, 1, 8192 if op == "grouped" else 4096), E=E, local=rng.choice([E, max(1, E // 4)]),
                 k=rng.randint(1, min(6, E)), K=8 * _log_int(rng, 2, 896), N=8 * _log_int(rng, 2, 512),
                 dtype=rng.choice(["bf16", "f16"]), gather=rng.random() < 0.5, zipf=rng.random() < 0.5)
        if op == "grouped_grad":
            c["dw"] = rng.choice([c["dtype"], "f32"])
        return c
    if op == "quantize":
        cols = 16 * _log_int(rng, 4, 448)
        rows = _log_int(rng, 1, min(49152, 49152 * 2048 // cols))
        return dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["bf16", "f16", "f32"]))
    if op == "linear":
        return dict(op=op, M=_log_int(rng, 1, 16381), N=8 * _log_int(rng, 4, 512), K=16 * _log_int(rng, 2, 448),
                    dtype=rng.choice(["bf16", "f16"]))
    H, I = 16 * _log_int(rng, 4, 448), 16 * _log_int(rng, 4, 128)
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


def _experts(E, N, K, seed, stream, std, dtype):
    w = torch.empty(E, N, K, dtype=dtype, device=DEV)
    for e in range(E):
        w[e] = _normal((N, K), seed, stream + e, std)
    return w


def _encode(x):
    """Codes and scales of float32 x [rows, K], for inputs that a program has already quantized."""
    amax = x.abs().amax(-1)
    scale = amax / 127
    return torch.round(x * (127 / amax)[:, None]).to(torch.int8), scale


def _coded(E, N, K, seed, stream):
    """8-bit weights of E matrices [N, K], N(0, 0.02), a scale for each channel."""
    codes = torch.empty(E, N, K, dtype=torch.int8, device=DEV)
    scales = torch.empty(E, N, dtype=torch.float32, device=DEV)
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


def prepare(case, seed):
    op, s = case["op"], dict(case)
    if op == "quantize":
        rows, cols = case["rows"], case["cols"]
        s["x"] = _normal((rows, cols), seed, 0, 0.09).to(DTYPES[case["dtype"]])
        s["codes"] = torch.empty(rows, cols, dtype=torch.int8, device=DEV)
        s["scales"] = torch.empty(rows, dtype=torch.float32, device=DEV)
        s["values"] = torch.empty_like(s["x"])
        return s
    if op == "linear":
        s["a_codes"], s["a_scales"] = _encode(_normal((case["M"], case["K"]), seed, 0, 0.09))
        s["w_codes"], s["w_scales"] = (t[0] for t in _coded(1, case["N"], case["K"], seed, 1))
        s["out"] = torch.empty(case["M"], case["N"], dtype=DTYPES[case["dtype"]], device=DEV)
        return s
    counts, offsets, row_token = _routing(case, seed)
    s["rows"] = counts.tolist()
    s["counts"], s["offsets"], s["row_token"] = (torch.from_numpy(a).to(DEV) for a in (counts, offsets, row_token))
    cap, L = len(row_token), case["local"]
    if op in ("grouped", "grouped_grad"):
        K, N, dt = case["K"], case["N"], DTYPES[case["dtype"]]
        s["x"] = _normal((case["T"] if case["gather"] else cap, K), seed, 0).to(dt)
        s["w"] = _experts(L, N, K, seed, 2, 0.02, dt)
        if op == "grouped":
            s["out"] = torch.zeros(cap, N, dtype=dt, device=DEV)
        else:
            s["dy"] = _normal((cap, N), seed, 1, 0.02).to(dt)
            s["dx"] = torch.zeros(cap, K, dtype=dt, device=DEV)
            s["dweight"] = torch.empty(L, N, K, dtype=DTYPES[case["dw"]], device=DEV)
        return s
    up, H, I = op == "experts_up", case["H"], case["I"]
    n, width = (case["T"], H) if up else (cap, I)
    s["a_codes"], s["a_scales"] = _encode(_normal((n, width), seed, 0, 0.09))
    s["w_codes"], s["w_scales"] = _coded(L, 2 * I if up else H, width, seed, 1)
    s["out"] = torch.zeros(cap, I if up else H, dtype=torch.bfloat16, device=DEV)
    return s


# ---- one pass ------------------------------------------------------------------------------------

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from nvfp4_block_scaled_top_amd import megamoe as mm

    op = s["op"]
    if op == "quantize":
        mm.int8_quantize_act(s["x"], s["codes"], s["scales"])
        mm.int8_dequantize(s["codes"], s["scales"], s["values"])
        return {"values": s["values"], "scales": s["scales"]}
    if op == "grouped":
        mm.moe_grouped_gemm(s["x"], s["w"], s["offsets"], s["counts"], s["out"],
                            row_token=s["row_token"] if s["gather"] else None, max_rows_per_expert=s["T"])
    elif op == "grouped_grad":
        mm.moe_grouped_gemm_dgrad(s["dy"], s["w"], s["offsets"], s["counts"], s["dx"])
        mm.moe_grouped_gemm_wgrad(s["dy"], s["x"], s["offsets"], s["counts"], s["dweight"],
                                  row_token=s["row_token"] if s["gather"] else None)
        return {"dx": s["dx"], "dweight": s["dweight"]}
    elif op == "linear":
        mm.int8_linear(s["a_codes"], s["a_scales"], s["w_codes"], s["w_scales"], s["out"])
    elif op == "experts_up":
        mm.moe_grouped_gemm_l1_silu_int8(s["a_codes"], s["a_scales"], s["row_token"], s["offsets"], s["counts"],
                                         s["w_codes"], s["w_scales"], s["out"], max_rows_per_expert=s["T"])
    else:
        mm.moe_grouped_gemm_l2_int8(s["a_codes"], s["a_scales"], s["offsets"], s["counts"], s["w_codes"],
                                    s["w_scales"], s["out"], max_rows_per_expert=s["T"])
    return {"out": s["out"]}


def _spans(s):
    """(expert, its rows, the rows of the operand that they read), for the experts that have any."""
    r = 0
    for e, n in enumerate(s["rows"]):
        if n:
            at = slice(r, r + n)
            yield e, at, s["row_token"][at] if s.get("gather", s["op"] == "experts_up") else at
            r += n


def _plain_quantize(s):
    x = s["x"].double()  # in 64 bits, where a code next to a border falls on its own side
    amax = x.abs().amax(-1, keepdim=True)
    scale = amax.float() / 127
    q = torch.where(amax > 0, torch.round(x * 127 / amax), 0.0)
    return {"values": (q.float() * scale).to(s["x"].dtype), "scales": scale[:, 0]}


def _silu_mul(z):
    gate, up = z.chunk(2, -1)
    return gate / (1 + torch.exp(-gate)) * up


def _coded_product(a, sa, w, sw):
    return a.float() @ w.float().t() * sa[:, None] * sw


def _run_plain(s):
    op = s["op"]
    if op == "quantize":
        return _plain_quantize(s)
    if op == "linear":
        return {"out": _coded_product(s["a_codes"], s["a_scales"], s["w_codes"], s["w_scales"]).to(s["out"].dtype)}
    if op == "grouped":
        out = torch.zeros_like(s["out"])
        for e, at, src in _spans(s):  # one product an expert: their row counts differ
            out[at] = (s["x"][src].float() @ s["w"][e].float().t()).to(out.dtype)
        return {"out": out}
    if op == "grouped_grad":
        dx, dw = torch.zeros_like(s["dx"]), torch.zeros_like(s["dweight"])
        for e, at, src in _spans(s):
            dy = s["dy"][at].float()
            dx[at] = (dy @ s["w"][e].float()).to(dx.dtype)
            dw[e] = (dy.t() @ s["x"][src].float()).to(dw.dtype)
        return {"dx": dx, "dweight": dw}
    out = torch.zeros_like(s["out"])
    for e, at, src in _spans(s):
        z = _coded_product(s["a_codes"][src], s["a_scales"][src], s["w_codes"][e], s["w_scales"][e])
        out[at] = (_silu_mul(z) if op == "experts_up" else z).bfloat16()
    return {"out": out}


# ---- bytes and operations of one pass --------------------------------------------------------------

def work(case):
    op = case["op"]
    size = {"bf16": 2, "f16": 2, "f32": 4}
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (2 * size[case["dtype"]] + 1) + 4 * case["rows"], "flops": 4 * n}
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * (K + 4) + 2 * M * N, "flops": 2 * M * N * K}
    counts, _, row_token = _routing(case, 0)
    rows, active = int(counts.sum()), int((counts > 0).sum())
    tokens = len(np.unique(row_token[row_token >= 0]))
    if op in ("grouped", "grouped_grad"):
        K, N = case["K"], case["N"]
        read = tokens if case["gather"] else rows
        if op == "grouped":
            return {"bytes": max(1, 2 * (active * N * K + read * K + rows * N)), "flops": 2 * rows * N * K}
        return {"bytes": 2 * (active * N * K + read * K + rows * (N + K)) + case["local"] * N * K * size[case["dw"]],
                "flops": 4 * rows * N * K}
    H, I = case["H"], case["I"]
    if op == "experts_up":
        return {"bytes": max(1, active * 2 * I * (H + 4) + tokens * (H + 4) + rows * I * 2), "flops": 4 * rows * I * H}
    return {"bytes": max(1, active * H * (I + 4) + rows * (I + 4) + rows * H * 2), "flops": 2 * rows * I * H}


# ---- the definitions in 64 bits ---------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        # the whole number nearest to 127 x / amax, of two equally near ones the even one
        x = s["x"].cpu().numpy() if case["dtype"] != "bf16" else s["x"].float().cpu().numpy()
        x = x.astype(np.float64)
        amax = np.abs(x).max(1, keepdims=True)
        unit = np.where(amax > 0, amax, 1.0)
        return {"values": np.rint(127.0 * x / unit) * (amax / 127.0), "scales": amax[:, 0] / 127.0}
    if op == "linear":
        a = s["a_codes"].double() * s["a_scales"].double()[:, None]
        w = s["w_codes"].double() * s["w_scales"].double()[:, None]
        return {"out": torch.mm(a, w.T)}
    starts, tokens = s["offsets"].tolist(), s["row_token"].long()
    if op == "grouped_grad":
        dx = torch.zeros(s["dx"].shape, dtype=torch.float64, device=DEV)
        dw = torch.zeros(s["dweight"].shape, dtype=torch.float64, device=DEV)
    else:
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    for e in range(case["local"]):
        rows = torch.arange(starts[e], starts[e + 1], device=DEV)
        if len(rows) == 0:
            continue
        if op in ("grouped", "grouped_grad"):
            x = s["x"].index_select(0, tokens[rows] if case["gather"] else rows).double()
            w = s["w"][e].double()
            if op == "grouped":
                out[rows] = torch.mm(x, w.T)
            else:
                dy = s["dy"].index_select(0, rows).double()
                dx[rows] = torch.mm(dy, w)
                dw[e] = torch.mm(dy.T, x)
            continue
        src = tokens[rows] if op == "experts_up" else rows
        a = s["a_codes"][src].double() * s["a_scales"][src].double()[:, None]
        z = torch.mm(a, (s["w_codes"][e].double() * s["w_scales"][e].double()[:, None]).T)
        if op == "experts_up":
            g, u = z[:, :case["I"]], z[:, case["I"]:]
            z = g * torch.sigmoid(g) * u
        out[rows] = z
    return {"dx": dx, "dweight": dw} if op == "grouped_grad" else {"out": out}
