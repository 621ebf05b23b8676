"""16-bit experts' products and their gradients on the GPU against a float64 reference.

Products of bf16 or fp16 numbers are exact in fp32; n of them are summed with an error of at most n * 2^-24
times the sum of their magnitudes (each addition rounds a partial sum no larger than that by half a step), and
the result is rounded once to the output (2^-8 bf16, 2^-11 fp16, 2^-24 fp32, relative)."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_top_amd import layer, megamoe as mm

from gpu_util import DEV

pytestmark = pytest.mark.gpu

STEP = {torch.bfloat16: (2.0 ** -8, 2.0 ** -133), torch.float16: (2.0 ** -11, 2.0 ** -24), torch.float32: (2.0 ** -24, 2.0 ** -149)}
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def normal(gen, *shape, std=1.0, dtype=BF):
    return (torch.randn(shape, generator=gen, device=DEV) * std).to(dtype)


def accept(out, ref, mag, n):
    """out against the float64 ref of n products with the summed magnitudes mag."""
    half, tiny = STEP[out.dtype]
    got = out.double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    bound = ref.abs() * half + mag * (n * 2.0 ** -24) * (1 + half) + tiny
    err = (got - ref).abs()
    err = torch.where(got == ref, torch.zeros_like(err), err)  # equal infinities
    assert bool(((err <= bound) | torch.isnan(ref)).all()), float((err / bound).nan_to_num().max())


def tables(counts, P, T, seed):
    """Offsets and tokens of the rows by expert (each token at most once an expert), unused rows -1."""
    rng = np.random.default_rng(seed)
    counts = np.array(counts, np.int32)
    poff = np.concatenate([[0], np.cumsum((counts + P - 1) // P * P)]).astype(np.int32)
    row_token = np.full(int(poff[-1]) + 5, -1, np.int32)
    for e, c in enumerate(counts):
        row_token[poff[e]:poff[e] + c] = np.sort(rng.permutation(T)[:c])
    return counts, poff, row_token


def on(a):
    return torch.from_numpy(a).to(DEV)


CASES = [  # rows by expert, P, K, N
    ([3, 0, 1, 16, 0, 17], 1, 256, 128),
    ([0, 0, 0], 8, 64, 40),
    ([1], 1, 8, 8),
    ([5, 2], 1, 24, 16),
    ([40, 64, 65, 128, 129, 0, 256, 257, 2], 16, 392, 136),
    ([300, 0, 5, 33], 128, 1160, 264),
    ([2] * 48, 1, 1024, 256),
    ([0] * 500 + [7, 600, 0, 20], 1, 256, 256),
    ([16] * 3 + [15] * 3 + [31, 32], 1, 640, 520),
    ([300, 0, 70, 20, 500, 129, 17, 260, 16, 190, 3], 8, 1096, 648),
    ([1100, 33, 0, 450], 1, 1408, 904),
    ([2100, 100, 40, 2060, 64, 130], 1, 64, 2056),
    ([2100, 0, 40, 2060], 1, 200, 1032),
    ([1, 16, 0, 15, 4, 0, 0, 16, 16, 31, 2, 8, 16, 0, 5, 16, 1, 20, 16], 1, 7168, 2048),
    ([9, 4, 0, 12], 1, 2048, 7168),
]


def setup(i, dtype, gather):
    counts, P, K, N = CASES[i]
    T = max(max(counts), 1) + 7
    counts, poff, rt = tables(counts, P, T, i)
    gen = torch.Generator(device=DEV).manual_seed(i)
    cap, E = len(rt), len(counts)
    x = normal(gen, T if gather else cap, K, dtype=dtype)
    w = torch.full((E, N, K), float("nan"), dtype=dtype, device=DEV)  # of experts without rows: never read
    for e in np.nonzero(counts)[0]:
        w[e] = normal(gen, N, K, std=0.05, dtype=dtype)
    dy = normal(gen, cap, N, std=0.1, dtype=dtype)
    free = torch.ones(cap, dtype=torch.bool, device=DEV)
    for e in np.nonzero(counts)[0]:
        free[poff[e]:poff[e] + counts[e]] = False
    dy[free] = float("nan")  # rows that hold no assignment are not read
    if not gather:
        x[free] = float("nan")
    return counts, poff, rt, K, N, x, w, dy, free


def spans(counts, poff, rt, gather):
    for e in np.nonzero(counts)[0]:
        at = slice(int(poff[e]), int(poff[e] + counts[e]))
        yield int(e), at, on(rt[at]).long() if gather else at


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_product(i, dtype, gather):
    counts, poff, rt, K, N, x, w, dy, free = setup(i, dtype, gather)
    outs = []
    for bound in (0, 1, 10 ** 6):
        y = torch.full((len(rt), N), 7.0, dtype=dtype, device=DEV)
        mm.moe_grouped_gemm(x, w, on(poff), on(counts), y, row_token=on(rt) if gather else None, max_rows_per_expert=bound)
        outs.append(y)
    torch.cuda.synchronize()
    for y in outs:
        for e, at, src in spans(counts, poff, rt, gather):
            a, b = x[src].double(), w[e].double().t()
            accept(y[at], a @ b, a.abs() @ b.abs(), K)
        assert torch.all(y[free] == 7.0)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_rows_gradient(i, dtype):
    counts, poff, rt, K, N, x, w, dy, free = setup(i, dtype, False)
    dx = torch.full((len(rt), K), 7.0, dtype=dtype, device=DEV)
    mm.moe_grouped_gemm_dgrad(dy, w, on(poff), on(counts), dx)
    torch.cuda.synchronize()
    for e, at, _ in spans(counts, poff, rt, False):
        g, b = dy[at].double(), w[e].double()
        accept(dx[at], g @ b, g.abs() @ b.abs(), N)
    assert torch.all(dx[free] == 7.0)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("dtype,dwt", [(BF, BF), (BF, F32), (HF, HF), (HF, F32)])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_weights_gradient(i, dtype, dwt, gather):
    counts, poff, rt, K, N, x, w, dy, free = setup(i, dtype, gather)
    E = len(counts)
    dw = torch.full((E, N, K), float("nan"), dtype=dwt, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(99)
    old = normal(gen, E, N, K, dtype=dwt)
    acc = old.clone()
    kw = dict(row_token=on(rt) if gather else None)
    mm.moe_grouped_gemm_wgrad(dy, x, on(poff), on(counts), dw, **kw)
    mm.moe_grouped_gemm_wgrad(dy, x, on(poff), on(counts), acc, accumulate=True, **kw)
    torch.cuda.synchronize()
    for e, at, src in spans(counts, poff, rt, gather):
        g, a = dy[at].double().t(), x[src].double()
        ref, mag, n = g @ a, g.abs() @ a.abs(), int(counts[e])
        accept(dw[e], ref, mag, n)
        # the float32 sum of the old value and the total adds a rounding
        accept(acc[e], old[e].double() + ref, mag + (old[e].double().abs() + mag) / n, n)
    none = torch.from_numpy(counts == 0).to(DEV)
    assert not dw[none].any() and not torch.isnan(dw[none]).any()
    assert torch.equal(acc[none], old[none])


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("dtype,dwt", [(BF, F32), (HF, HF)])
@pytest.mark.parametrize("counts,K,N", [
    ([3584, 1, 0, 3583, 127, 129], 40, 696),   # an expert's tokens fill what is kept of them,
    ([5, 3585, 0, 128, 4], 40, 696),           # or are one too many
    ("ragged", 64, 64),                        # several experts a workgroup
    ("ragged", 8, 72),
])
def test_weights_gradient_of_small_matrices(counts, K, N, dtype, dwt, gather):
    if counts == "ragged":
        counts = np.random.default_rng(5).integers(0, 300, 1024).tolist()
    T = max(counts) + 9
    counts, poff, rt = tables(counts, 1, T, 3)
    gen = torch.Generator(device=DEV).manual_seed(K)
    x, dy = normal(gen, T if gather else len(rt), K, dtype=dtype), normal(gen, len(rt), N, std=0.1, dtype=dtype)
    old = normal(gen, len(counts), N, K, dtype=dwt)
    dw, acc = torch.full_like(old, float("nan")), old.clone()
    kw = dict(row_token=on(rt) if gather else None)
    mm.moe_grouped_gemm_wgrad(dy, x, on(poff), on(counts), dw, **kw)
    mm.moe_grouped_gemm_wgrad(dy, x, on(poff), on(counts), acc, accumulate=True, **kw)
    torch.cuda.synchronize()
    for e, at, src in spans(counts, poff, rt, gather):
        g, a = dy[at].double().t(), x[src].double()
        accept(dw[e], g @ a, g.abs() @ a.abs(), int(counts[e]))
        accept(acc[e], g @ a + old[e].double(), g.abs() @ a.abs() + old[e].double().abs(), int(counts[e]) + 1)
    none = on(counts == 0)
    assert not dw[none].any() and torch.equal(acc[none], old[none])


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("bound", [0, 3])
def test_all_the_experts_there_can_be(bound, gather):
    """1024 experts of 0 to 3 rows, a few of more, and with them the last lists' places."""
    counts = np.random.default_rng(6).integers(0, 4, 1024)
    counts[[0, 500, 1023]] = 300, 70, 140
    counts, poff, rt = tables(counts, 1, 310, 4)
    gen = torch.Generator(device=DEV).manual_seed(7)
    K, N, cap = 136, 72, len(rt)
    x, w, dy = normal(gen, 310 if gather else cap, K), normal(gen, 1024, N, K), normal(gen, cap, N)
    y, dx = torch.full((cap, N), 7.0, dtype=BF, device=DEV), torch.full((cap, K), 7.0, dtype=BF, device=DEV)
    mm.moe_grouped_gemm(x, w, on(poff), on(counts), y, row_token=on(rt) if gather else None, max_rows_per_expert=bound)
    mm.moe_grouped_gemm_dgrad(dy, w, on(poff), on(counts), dx)
    torch.cuda.synchronize()
    for e, at, src in spans(counts, poff, rt, gather):
        a, b, g = x[src].double(), w[e].double(), dy[at].double()
        accept(y[at], a @ b.t(), a.abs() @ b.t().abs(), K)
        accept(dx[at], g @ b, g.abs() @ b.abs(), N)
    assert torch.all(y[poff[-1]:] == 7.0) and torch.all(dx[poff[-1]:] == 7.0)


def test_gradients_agree_with_differences():
    """A loss that is linear in each factor: halves of central differences of the product itself, in fp32 sums of
    values that bf16 holds exactly (small whole numbers)."""
    counts, poff, rt = tables([5, 0, 18, 70], 1, 80, 3)
    gen = torch.Generator(device=DEV).manual_seed(1)
    K, N, cap = 40, 24, len(rt)
    whole = lambda *s: torch.randint(-3, 4, s, generator=gen, device=DEV).to(BF)  # noqa: E731
    x, w, dy = whole(80, K), whole(4, N, K), whole(cap, N)
    used = torch.from_numpy(rt >= 0).to(DEV)
    tab = on(poff), on(counts)

    def loss(x, w):
        y = torch.zeros(cap, N, dtype=HF, device=DEV)
        mm.moe_grouped_gemm(x.to(HF), w.to(HF), *tab, y, row_token=on(rt))
        return float((y.double() * dy.double())[used].sum())
    dx, dw = torch.zeros(cap, K, dtype=BF, device=DEV), torch.empty(4, N, K, device=DEV)
    mm.moe_grouped_gemm_dgrad(dy, w, *tab, dx)
    mm.moe_grouped_gemm_wgrad(dy, x, *tab, dw, row_token=on(rt))
    gx = torch.zeros(80, K, dtype=torch.float64, device=DEV)
    gx.index_add_(0, on(rt)[used].long(), dx[used].double())
    rng = np.random.default_rng(0)
    for t, g in ((x, gx), (w, dw)):
        for _ in range(12):
            i = tuple(int(rng.integers(n)) for n in t.shape)
            d = []
            for step in (1, -1):
                t[i] += step
                d.append(loss(x, w))
                t[i] -= step
            # dx of a token is a sum of rows rounded to bf16: at most 3 rows of magnitude up to 216
            assert abs((d[0] - d[1]) / 2 - float(g[i])) <= (3 * 216 * 2.0 ** -8 if t is x else 0), (i, d, float(g[i]))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("rows", [4, 40, 300])
def test_infinities_and_nan_stay_in_their_rows(rows, dtype):
    """A NaN row of x, an infinite weight, values beyond fp16 and subnormals: each output as float64 has it."""
    gen = torch.Generator(device=DEV).manual_seed(rows)
    K, N = 136, 72
    counts, poff, rt = tables([rows, rows + 3], 1, 400, rows)
    x, w = normal(gen, 400, K, dtype=dtype), normal(gen, 2, N, K, dtype=dtype)
    t = on(rt)[:3].long()
    x[t[0], 5] = float("nan")
    x[t[1]] = torch.finfo(dtype).tiny / 4 if dtype == HF else torch.finfo(dtype).tiny
    x[t[2], 7] = float("inf")
    w[1, 9, 3] = float("-inf")
    w[0, 11] = torch.finfo(dtype).max if dtype == HF else 1e30
    y = torch.zeros(len(rt), N, dtype=dtype, device=DEV)
    mm.moe_grouped_gemm(x, w, on(poff), on(counts), y, row_token=on(rt))
    for e, at, src in spans(counts, poff, rt, True):
        a, b = x[src].double(), w[e].double().t()
        ref = (a.cpu() @ b.cpu()).to(DEV)
        mag = torch.nan_to_num(a.abs(), nan=0, posinf=0) @ torch.nan_to_num(b.abs(), nan=0, posinf=0)
        over = ref.abs() > torch.finfo(dtype).max * (1 + 2.0 ** -9)
        got = y[at]
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        assert torch.equal(got[over].double(), torch.sign(ref[over]) * float("inf"))
        near = torch.isnan(ref) | over | (ref.abs() > torch.finfo(dtype).max * (1 - 2.0 ** -9))
        accept(torch.where(near, 0, got), torch.where(near, 0.0, ref), torch.where(near, 0.0, mag), K)


def test_offsets_past_32_bits():
    """x, y, dy and dx beyond 2^32 elements' bytes, weights beyond 4 GB, rows at both ends."""
    gen = torch.Generator(device=DEV).manual_seed(2)
    K, N, E = 4096, 4104, 150
    counts = np.zeros(E, np.int32)
    counts[[0, 3, 70, 149]] = [600000, 20, 300, 5]
    poff = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    cap = int(poff[-1])
    assert 2 * cap * K > 2 ** 32 and E * N * K * 2 > 2 ** 32
    x, w = normal(gen, cap, K), torch.empty(E, N, K, dtype=BF, device=DEV)
    for e in (0, 3, 70, 149):
        w[e] = normal(gen, N, K, std=0.05)
    y = torch.full((cap, N), float("nan"), dtype=BF, device=DEV)
    mm.moe_grouped_gemm(x, w, on(poff), on(counts), y)
    dx = torch.full((cap, K), float("nan"), dtype=BF, device=DEV)
    mm.moe_grouped_gemm_dgrad(y, w, on(poff), on(counts), dx)
    pick = torch.tensor([0, 1, 255, 256, 300001, 524287, 524288, 599999, 600000, 600019, 600020, 600319, 600320, cap - 1], device=DEV)
    for r in pick.tolist():
        e = int(np.searchsorted(poff, r, side="right")) - 1
        e = max(i for i in range(E) if poff[i] <= r and counts[i] > 0 and r < poff[i] + counts[i])
        a, b = x[r:r + 1].double(), w[e].double().t()
        accept(y[r:r + 1], a @ b, a.abs() @ b.abs(), K)
        g = y[r:r + 1].double()
        accept(dx[r:r + 1], g @ b.t(), g.abs() @ b.t().abs(), N)
    assert not torch.isnan(y.view(-1)[::4099]).any() and not torch.isnan(dx.view(-1)[::4099]).any()
    del dx, w
    dw = torch.empty(E, N, K, dtype=BF, device=DEV)  # beyond 2^31 elements
    mm.moe_grouped_gemm_wgrad(y, x, on(poff), on(counts), dw)
    for e in (3, 70, 149):
        at = slice(int(poff[e]), int(poff[e] + counts[e]))
        g, a = y[at].double().t(), x[at].double()
        accept(dw[e], g @ a, g.abs() @ a.abs(), int(counts[e]))
    assert not dw[1].any() and not dw[148].any()


def test_unaligned_buffers_and_repeats():
    """Operands and outputs at an odd multiple of 16 bytes: the same bits, call after call."""
    counts, poff, rt = tables([5, 40, 300, 0, 17], 1, 310, 8)
    gen = torch.Generator(device=DEV).manual_seed(8)
    K, N, cap, tab = 520, 264, len(rt), (on(poff), on(counts))

    def at(t):
        v = torch.empty(t.numel() + 8, dtype=t.dtype, device=DEV)[8:].view(t.shape)
        return v.copy_(t)
    x, w, dy = normal(gen, 310, K), normal(gen, 5, N, K), normal(gen, cap, N)
    res = []
    for f in (lambda t: t, lambda t: t, at):
        y, dx, dw = (f(torch.zeros(s, dtype=BF, device=DEV)) for s in ((cap, N), (cap, K), (5, N, K)))
        mm.moe_grouped_gemm(f(x), f(w), *tab, y, row_token=on(rt))
        mm.moe_grouped_gemm_dgrad(f(dy), f(w), *tab, dx)
        mm.moe_grouped_gemm_wgrad(f(dy), f(x), *tab, dw, row_token=on(rt))
        res.append((y, dx, dw))
    for other in res[1:]:
        assert all(torch.equal(a, b) for a, b in zip(res[0], other))


# ---- as they are used together ---------------------------------------------------------------------

def experts_step(L, x, ids, wts, w13, w2, dout, s=None):
    """Forward and backward of the routed experts on unquantized weights, SiLU in torch operations: route, gate+up,
    SiLU(g) * u, down, combine; then the gradients of both weights and of the tokens, in bf16."""
    T, k = ids.shape
    with torch.cuda.stream(s) if s is not None else torch.cuda.stream(torch.cuda.current_stream()):
        mm.moe_route_permute(ids, 0, L.E, L.P, L.counts, L.expert_offsets, L.padded_offsets, L.row_token, L.token_rows,
                             L.sched, L.route_ws)
        tab = L.padded_offsets, L.counts
        I = w2.shape[2]
        z = torch.zeros(L.M_cap, 2 * I, dtype=BF, device=DEV)
        mm.moe_grouped_gemm(x, w13, *tab, z, row_token=L.row_token, max_rows_per_expert=T)
        g, u = z[:, :I].float(), z[:, I:].float()
        sig = torch.sigmoid(g)
        h = (g * sig * u).to(BF)
        y = torch.zeros(L.M_cap, x.shape[1], dtype=BF, device=DEV)
        mm.moe_grouped_gemm(h, w2, *tab, y, max_rows_per_expert=T)
        out = torch.empty_like(x)
        mm.moe_combine(y, L.token_rows, wts, out)
        rows = L.token_rows.view(T, k).long()
        dy = torch.zeros_like(y)
        dy[rows.reshape(-1)] = (wts.unsqueeze(-1) * dout.float().unsqueeze(1)).reshape(T * k, -1).to(BF)
        dh, dw2 = torch.zeros_like(h), torch.empty_like(w2, dtype=F32)
        mm.moe_grouped_gemm_dgrad(dy, w2, *tab, dh)
        mm.moe_grouped_gemm_wgrad(dy, h, *tab, dw2)
        dhf = dh.float()
        dz = torch.cat([dhf * u * sig * (1 + g * (1 - sig)), dhf * g * sig], 1).to(BF)
        dxr, dw13 = torch.zeros(L.M_cap, x.shape[1], dtype=BF, device=DEV), torch.empty_like(w13, dtype=F32)
        mm.moe_grouped_gemm_dgrad(dz, w13, *tab, dxr)
        mm.moe_grouped_gemm_wgrad(dz, x, *tab, dw13, row_token=L.row_token)
        dx = torch.empty_like(x)
        mm.moe_combine(dxr, L.token_rows, torch.ones_like(wts), dx)
    return out, dx, dw13, dw2


@pytest.mark.parametrize("T,E,k,stream", [(3, 6, 2, False), (150, 5, 2, True), (700, 9, 3, False)])
def test_training_step_of_the_experts(T, E, k, stream):
    """Against the same step in float64 by automatic differentiation.  The five bf16 roundings on the way (z, h, dy,
    dh, dz) are 2^-8 each; a product of them over independent terms is compared in the norm: 5 * 2^-8 of each
    gradient's, and 3 * 2^-8 of the output's."""
    gen = torch.Generator(device=DEV).manual_seed(T)
    H, I = 264, 136
    x, w13, w2 = normal(gen, T, H), normal(gen, E, 2 * I, H, std=0.06), normal(gen, E, H, I, std=0.08)
    dout = normal(gen, T, H)
    ids = torch.rand(T, E, generator=gen, device=DEV).topk(k, 1).indices.to(torch.int32)
    wts = torch.rand(T, k, generator=gen, device=DEV)
    L = layer.MXMoELayer(T, k, E, 256, 128, 1, device=DEV)
    s = torch.cuda.Stream() if stream else None
    if s is not None:
        s.wait_stream(torch.cuda.current_stream())
    got = experts_step(L, x, ids, wts, w13, w2, dout, s)
    torch.cuda.synchronize()
    xd, w13d, w2d = (t.double().cpu().requires_grad_() for t in (x, w13, w2))
    out = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            z = w13d[e] @ xd[t]
            out[t] = out[t] + float(wts[t, j]) * (w2d[e] @ (torch.nn.functional.silu(z[:I]) * z[I:]))
    out.backward(dout.double().cpu())
    for a, b, n in zip(got, (out.detach(), xd.grad, w13d.grad, w2d.grad), (3, 5, 5, 5)):
        assert float((a.double().cpu() - b).norm()) <= n * 2.0 ** -8 * float(b.norm())


@pytest.mark.parametrize("T", [5, 200])
def test_calls_captured_and_on_two_streams(T):
    """A captured forward and backward replayed on new inputs, with eager calls on another stream in between."""
    gen = torch.Generator(device=DEV).manual_seed(T)
    counts, poff, rt = tables([T, 0, T // 2, 1, T], 1, T, T)
    K, N, cap, tab = 520, 264, len(rt), (on(poff), on(counts), )
    x, w, dy, row = normal(gen, T, K), normal(gen, 5, N, K), normal(gen, cap, N), on(rt)

    def outputs():
        return [torch.zeros(cap, N, dtype=BF, device=DEV), torch.zeros(cap, K, dtype=BF, device=DEV),
                torch.zeros(5, N, K, device=DEV)]

    def step(o, stream=None):
        mm.moe_grouped_gemm(x, w, *tab, o[0], row_token=row, max_rows_per_expert=T, stream=stream)
        mm.moe_grouped_gemm_dgrad(dy, w, *tab, o[1], stream=stream)
        mm.moe_grouped_gemm_wgrad(dy, x, *tab, o[2], row_token=row, stream=stream)
    a, b = outputs(), outputs()
    step(a)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(a)
    side = torch.cuda.Stream()
    for r in range(4):
        for t in (x, w, dy):
            t.copy_(torch.randn(t.shape, generator=gen, device=DEV))
        want = outputs()
        step(want)
        torch.cuda.synchronize()
        for o in a + b:
            o[: len(o) - 5 if o.shape[0] == cap else 5].fill_(3.0)
        torch.cuda.synchronize()
        g.replay()
        step(b, side)
        torch.cuda.synchronize()
        for o in (a, b):
            assert all(torch.equal(p[:cap - 5], q[:cap - 5]) for p, q in zip(o, want))


def test_captured_calls_on_other_counts():
    """One captured forward and backward, replayed on tables that each kernel's tiles and none would take."""
    gen = torch.Generator(device=DEV).manual_seed(12)
    K, N, T, E = 264, 136, 1400, 4
    cap = 1408
    x, w, dy = normal(gen, T, K), normal(gen, E, N, K), normal(gen, cap, N)
    poff, counts = (torch.zeros(n, dtype=torch.int32, device=DEV) for n in (E + 1, E))
    row = torch.zeros(cap, dtype=torch.int32, device=DEV)
    y, dx, dw = (torch.zeros(n, dtype=BF, device=DEV) for n in ((cap, N), (cap, K), (E, N, K)))

    def step():
        mm.moe_grouped_gemm(x, w, poff, counts, y, row_token=row)
        mm.moe_grouped_gemm_dgrad(dy, w, poff, counts, dx)
        mm.moe_grouped_gemm_wgrad(dy, x, poff, counts, dw, row_token=row)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for case in ([1, 0, 2, 3], [700, 0, 60, 300], [0, 0, 0, 0], [1400, 1, 1, 1], [128, 256, 64, 65]):
        cnt, po, rt = tables(case, 1, T, 5)
        rt = rt[:cap]
        counts.copy_(on(cnt))
        poff.copy_(on(po))
        row[:len(rt)].copy_(on(rt))
        for t in (y, dx, dw):
            t.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for e, at, src in spans(cnt, po, rt, True):
            a, b, d = x[src].double(), w[e].double(), dy[at].double()
            accept(y[at], a @ b.t(), a.abs() @ b.t().abs(), K)
            accept(dx[at], d @ b, d.abs() @ b.abs(), N)
            accept(dw[e], d.t() @ a, d.t().abs() @ a.abs(), case[e])
        assert torch.all(y[po[-1]:] == 7.0) and torch.all(dx[po[-1]:] == 7.0) and not dw[on(cnt == 0)].any()


def test_no_rows():
    """M_cap = 0: no product; weights' gradients become 0, or stay with accumulate."""
    bf = lambda *s: torch.zeros(*s, dtype=BF, device=DEV)  # noqa: E731
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device=DEV)  # noqa: E731
    mm.moe_grouped_gemm(bf(0, 64), bf(4, 32, 64), i32(5), i32(4), bf(0, 32), row_token=i32(0))
    mm.moe_grouped_gemm_dgrad(bf(0, 32), bf(4, 32, 64), i32(5), i32(4), bf(0, 64))
    dw = torch.full((4, 32, 64), 3.0, device=DEV)
    mm.moe_grouped_gemm_wgrad(bf(0, 32), bf(0, 64), i32(5), i32(4), dw, accumulate=True)
    assert torch.all(dw == 3.0)
    mm.moe_grouped_gemm_wgrad(bf(0, 32), bf(0, 64), i32(5), i32(4), dw)
    assert not dw.any()


def test_no_tokens_beside_padded_rows():
    """Gathering from no tokens, with room for rows: no product; weights' gradients become 0, or stay with accumulate."""
    counts, poff, rt = np.zeros(4, np.int32), np.zeros(5, np.int32), np.full(24, -1, np.int32)
    x, w = torch.empty(0, 64, dtype=BF, device=DEV), torch.zeros(4, 32, 64, dtype=BF, device=DEV)
    y, dw = torch.full((24, 32), 7.0, dtype=BF, device=DEV), torch.full((4, 32, 64), 3.0, device=DEV)
    tab = on(poff), on(counts)
    mm.moe_grouped_gemm(x, w, *tab, y, row_token=on(rt))
    mm.moe_grouped_gemm_wgrad(y, x, *tab, dw, row_token=on(rt), accumulate=True)
    assert torch.all(y == 7.0) and torch.all(dw == 3.0)
    mm.moe_grouped_gemm_wgrad(y, x, *tab, dw, row_token=on(rt))
    assert not dw.any()


MOST = 2 ** 31 - 1  # rows that a call can have


def repeated(block, rows):
    """block again and again, cut at `rows`."""
    t = torch.empty(rows, block.shape[1], dtype=block.dtype, device=DEV)
    for a in range(0, rows, len(block)):
        t[a:a + len(block)] = block[:rows - a]
    return t


def is_repeated(t, block):
    return all(torch.equal(t[a:a + len(block)], block[:len(t) - a]) for a in range(0, len(t), len(block)))


@pytest.mark.parametrize("bound", [0, 1])
def test_as_many_rows_as_there_can_be(bound):
    """One expert of 2^31 - 1 rows; whole numbers, whose sums bf16 holds exactly."""
    gen = torch.Generator(device=DEV).manual_seed(1)
    whole = lambda *s: torch.randint(-3, 4, s, generator=gen, device=DEV).to(BF)  # noqa: E731
    block, w = whole(1000003, 8), whole(2, 8, 8)
    tab = on(np.array([0, 0, MOST], np.int32)), on(np.array([0, MOST], np.int32))
    x = repeated(block, MOST)
    y = torch.full((MOST, 8), 7.5, dtype=BF, device=DEV)
    mm.moe_grouped_gemm(x, w, *tab, y, max_rows_per_expert=bound)
    assert is_repeated(y, (block.float() @ w[1].float().t()).to(BF))
    if bound == 0:
        y.fill_(7.5)
        mm.moe_grouped_gemm_dgrad(x, w, *tab, y)
        assert is_repeated(y, (block.float() @ w[1].float()).to(BF))


def test_weights_gradient_of_as_many_rows_as_there_can_be():
    """As above; all but a few rows of dy are 0, the last one not."""
    gen = torch.Generator(device=DEV).manual_seed(2)
    whole = lambda *s: torch.randint(-3, 4, s, generator=gen, device=DEV).to(BF)  # noqa: E731
    block, few = whole(1000003, 8), whole(64, 8)
    tab = on(np.array([0, MOST, MOST], np.int32)), on(np.array([MOST, 0], np.int32))
    x, dy = repeated(block, MOST), torch.zeros(MOST, 8, dtype=BF, device=DEV)
    at = torch.cat([torch.arange(0, MOST, MOST // 61, device=DEV)[:61], torch.tensor([MOST - 3, MOST - 2, MOST - 1], device=DEV)])
    dy[at] = few
    dw = torch.full((2, 8, 8), 7.5, device=DEV)
    mm.moe_grouped_gemm_wgrad(dy, x, *tab, dw)
    assert torch.equal(dw[0], few.float().t() @ block[at % len(block)].float()) and not dw[1].any()
