"""int8 quantizer, decoder and products on the GPU against the float64 oracle.

Quantizer and decoder: bit for bit.  Products: the integer sum is exact; it is rounded to fp32, multiplied by
two scales with a rounding each (3 * 2^-24 relative) and rounded once to the output (2^-8 for bf16, 2^-11 for
fp16).  SiLU(g) * u: g and u as above, passed on with |g SiLU'(g)| <= 1.1 |SiLU(g)| + 1.1 |g s(g)| (both at
most 1.1 |g|); the hardware exp2 and reciprocal are a step off each, the exponent's rounding adds |g| of them:
(6 + 2 |g|) * 2^-23 in all."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_top_amd import layer, megamoe as mm
from oracle import int8_oracle as Q
from oracle import mxfp4_oracle as X

from gpu_util import DEV, np_i32

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}  # a step of the smallest values
FP32 = 3 * 2.0 ** -24


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def host(t):
    with np.errstate(invalid="ignore"):
        return t.detach().cpu().double().numpy()


def operand(rng, rows, K, std=1.0):
    """Codes of a normal tensor with its scales, spread over a few binades from row to row."""
    c, s = Q.quantize((rng.standard_normal((rows, K)) * std).astype(np.float32).astype(np.float64))
    return c, (s * 2.0 ** rng.integers(-2, 3, rows)).astype(np.float32)


def accept(out, ref):
    got, dt = host(out), out.dtype
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    with np.errstate(invalid="ignore"):
        assert np.all((np.abs(got - ref) <= np.abs(ref) * (HALF[dt] + 2 * FP32) + TINY[dt]) | np.isnan(ref))


def accept_silu(out, g, u):
    got, dt = host(out), out.dtype
    ref = Q.silu(g) * u
    err = 1.1 * np.abs(g * u) * FP32 + np.abs(ref) * (FP32 + (6 + 2 * np.abs(g)) * 2.0 ** -23)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    with np.errstate(invalid="ignore"):
        assert np.all((np.abs(got - ref) <= np.abs(ref) * HALF[dt] + 1.01 * err + TINY[dt]) | np.isnan(ref))


def gate_up(a, sa, w, sw):
    z = Q.product(a, sa, w, sw)
    return np.split(z, 2, axis=1)


# ---- quantizer and decoder -------------------------------------------------------------------------

def check_quantize(xt, row_valid=None):
    rows, cols = xt.shape
    codes = torch.full((rows + 1, cols), 77, dtype=torch.int8, device=DEV)
    scales = torch.full((rows + 1,), 77.0, device=DEV)
    mm.int8_quantize_act(xt.to(DEV), codes[:rows], scales[:rows], row_valid=None if row_valid is None else dev(row_valid))
    torch.cuda.synchronize()
    x = xt.double().numpy()
    if row_valid is not None:
        x = np.where(row_valid[:, None] < 0, 0.0, x)
    rc, rs = Q.quantize(x)
    assert np.array_equal(codes[:rows].cpu().numpy(), rc)
    assert np.array_equal(scales[:rows].cpu().numpy(), rs, equal_nan=True)
    assert torch.all(codes[rows:] == 77) and torch.all(scales[rows:] == 77)  # behind the last row
    for dt in (torch.bfloat16, torch.float16, torch.float32):
        out = torch.full((rows + 1, cols), 7.0, dtype=dt, device=DEV)
        mm.int8_dequantize(codes[:rows], scales[:rows], out[:rows])
        with np.errstate(invalid="ignore", over="ignore"):
            want = torch.from_numpy(Q.dequantize(rc, rs)).to(dt)
        assert torch.equal(torch.nan_to_num(out[:rows].cpu(), nan=123.0), torch.nan_to_num(want, nan=123.0))
        assert torch.all(out[rows:] == 7.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(0, 32), (1, 16), (3, 48), (1, 7168), (8, 7168), (257, 1040), (33, 2064), (5, 4112),
                                       (3, 28688), (2, 30016), (2050, 528), (2049, 7184), (4100, 2048), (2100, 10000)])
def test_quantize_shapes(rows, cols, dtype):
    rng = np.random.default_rng(rows + cols)
    check_quantize(torch.from_numpy((rng.standard_normal((rows, cols)) * 0.09).astype(np.float32)).to(dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows", [40, 3000])
def test_quantize_borders_and_extremes(dtype, rows):
    """Quotients on a border and next to one, infinities, NaN, zeros of both signs, the largest, the smallest and
    subnormal values."""
    rng = np.random.default_rng(4)
    x = torch.from_numpy(rng.standard_normal((rows, 288)).astype(np.float32)).to(dtype)
    half = torch.arange(-127, 127).float() + 0.5       # borders under amax 127, and under its multiples
    for r, m in enumerate((1.0, 2.0, 0.25)):
        x[r, :254] = (half * m).to(dtype)
        x[r, 254:] = torch.tensor([127.0 * m] + [0.0] * 33).to(dtype)
    x[3, :254], x[3, 254:] = (half * (1 + 2.0 ** -7)).to(dtype), torch.tensor([127.0] + [1.0] * 33).to(dtype)
    bits = torch.tensor(half.numpy().view(np.int32) + np.tile([1, -1], 127).astype(np.int32)).view(torch.float32)
    x[4, :254], x[4, 254:] = bits.to(dtype), torch.tensor([127.0] + [2.0] * 33).to(dtype)
    fi = torch.finfo(dtype)
    x[5, 3], x[6, 287], x[7, 0] = float("inf"), float("-inf"), float("nan")
    x[8], x[9] = 0.0, -0.0
    x[10] *= fi.tiny
    x[11] = (x[11].float() * fi.tiny * 2.0 ** -3).to(dtype)
    x[12, :], x[13, :] = fi.max, -fi.max
    x[14] = 0
    x[14, 9] = fi.smallest_normal * (fi.eps if dtype != torch.bfloat16 else 2.0 ** -7)  # the smallest value
    x[15, 1:] = 0.0
    check_quantize(x)


def test_quantize_many_near_borders():
    """float32 rows whose quotients lie a step of float32 around borders."""
    rng = np.random.default_rng(6)
    amax = rng.uniform(0.5, 2.0, (500, 1)).astype(np.float32)
    n = rng.integers(0, 127, (500, 256)) + 0.5
    x = (n * amax.astype(np.float64) / 127).astype(np.float32)
    x = (x.view(np.int32) + rng.integers(-1, 2, x.shape).astype(np.int32)).view(np.float32)
    x[:, :1] = amax
    check_quantize(torch.from_numpy(x * rng.choice([-1, 1], x.shape).astype(np.float32)))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_quantize_every_16_bit_value(dtype):
    """Every finite value below each of some maxima: all borders that 16-bit rows can meet."""
    top = 0x7F80 if dtype == torch.bfloat16 else 0x7C00
    bits = torch.arange(top, dtype=torch.int32)
    rng = np.random.default_rng(11)
    most = np.concatenate([[1, 2, 127, 128, 254, top - 1], top - 1 - rng.integers(0, top // 4, 12), top // 2 + np.arange(12)])
    rows = [torch.where(bits <= int(m), bits, 0).to(torch.int16).view(dtype) for m in most]
    check_quantize(torch.stack(rows) * torch.where(bits % 3 == 0, -1.0, 1.0).to(dtype))


@pytest.mark.parametrize("rows", [70, 2500])
def test_quantize_skips_invalid_rows(rows):
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((rows, 256)).astype(np.float32)).to(torch.bfloat16)
    rv = rng.integers(-1, 3, rows).astype(np.int32)
    x[np.nonzero(rv < 0)[0][0]] = float("nan")
    check_quantize(x, rv)


def test_quantize_and_decode_past_32_bits():
    """2^32 elements and some: each row as the same row of a small tensor."""
    rows, cols = 2 ** 21 + 5, 2048
    gen = torch.Generator(device=DEV).manual_seed(8)
    few = (torch.randn(64, cols, generator=gen, device=DEV) * 0.3).to(torch.bfloat16)
    x = few.repeat(rows // 64 + 1, 1)[:rows]
    out = []
    for t in (few, x):
        c, s = torch.empty(t.shape, dtype=torch.int8, device=DEV), torch.empty(len(t), device=DEV)
        mm.int8_quantize_act(t, c, s)
        y = torch.empty_like(t)
        mm.int8_dequantize(c, s, y)
        out.append((c, s, y))
    for a in range(0, rows, 2 ** 17):
        n = min(2 ** 17, rows - a)
        for small, large in zip(*out):
            assert torch.equal(large[a:a + n], small.repeat(2 ** 11, *[1] * (small.dim() - 1))[:n])


# ---- dense products ------------------------------------------------------------------------------

SHAPES = [  # M, N, K
    (0, 64, 256), (1, 8, 16), (1, 7168, 2048), (5, 40, 48), (16, 256, 7168), (17, 264, 656), (32, 512, 1024),
    (33, 128, 128), (64, 72, 2192), (100, 4096, 512), (129, 520, 1152), (255, 256, 256), (256, 256, 512),
    (257, 1032, 912), (513, 2048, 1024), (1000, 296, 2048), (8, 4096, 16384), (3, 24, 131056), (300, 64, 65536),
    (1500, 1032, 896), (1400, 1064, 1152), (2060, 776, 640), (4200, 4104, 16), (4161, 4104, 400), (4353, 4112, 128),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear(M, N, K, dtype):
    rng = np.random.default_rng(M + N + K)
    (ac, as_), (wc, ws) = operand(rng, M, K, 0.09), operand(rng, N, K, 0.02)
    out = torch.full((M + 1, N), 7.0, dtype=dtype, device=DEV)
    mm.int8_linear(dev(ac), dev(as_), dev(wc), dev(ws), out[:M])
    torch.cuda.synchronize()
    assert torch.all(out[M:] == 7.0)
    accept(out[:M], Q.product(ac, as_, wc, ws))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,N,K", [(0, 32, 128), (1, 8, 16), (1, 2048, 7168), (7, 40, 400), (16, 128, 1024), (31, 136, 640),
                                   (64, 2048, 256), (130, 264, 1168), (257, 512, 2048), (520, 1032, 256), (1500, 520, 912),
                                   (1400, 568, 1152), (2060, 408, 512), (4200, 2056, 128), (4161, 2056, 16)])
def test_gate_up_silu(M, N, K, dtype):
    rng = np.random.default_rng(M + N + K + 1)
    (ac, as_), (wc, ws) = operand(rng, M, K, 0.3), operand(rng, 2 * N, K, 1.0 / np.sqrt(K))
    h = torch.full((M + 1, N), 7.0, dtype=dtype, device=DEV)
    mm.int8_linear_gate_up_silu(dev(ac), dev(as_), dev(wc), dev(ws), h[:M])
    torch.cuda.synchronize()
    assert torch.all(h[M:] == 7.0)
    accept_silu(h[:M], *gate_up(ac, as_, wc, ws))


@pytest.mark.parametrize("M", [3, 20, 70, 300, 1500])
def test_linear_every_code_and_full_sums(M):
    """Any codes, -128 among them, and rows whose sum is the largest an int32 meets here."""
    rng = np.random.default_rng(M)
    N, K = 72, 131056
    ac, wc = (rng.integers(-128, 128, (n, K)).astype(np.int8) for n in (M, N))
    ac[1], wc[2], wc[3] = -128, -128, 127
    as_, ws = (rng.uniform(0.5, 2, n).astype(np.float32) for n in (M, N))
    out = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    mm.int8_linear(dev(ac), dev(as_), dev(wc), dev(ws), out)
    accept(out, Q.product(ac, as_, wc, ws))


@pytest.mark.parametrize("M", [2, 20, 100, 300, 1500])
def test_linear_nan_and_infinite_scales_reach_their_outputs_only(M):
    rng = np.random.default_rng(M + 9)
    N, K = 1040, 640
    (ac, as_), (wc, ws) = operand(rng, M, K), operand(rng, N, K)
    as_[1], ws[17], ws[1000] = np.nan, np.nan, np.inf
    ac[1] = 0
    out = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    mm.int8_linear(dev(ac), dev(as_), dev(wc), dev(ws), out)
    got, ref = host(out), Q.product(ac, as_, wc, ws)
    want = np.zeros((M, N), bool)
    want[1], want[:, 17] = True, True
    want[:, 1000] |= np.isnan(ref[:, 1000])
    assert np.array_equal(np.isnan(got), want)
    assert np.array_equal(got[:, 1000][~want[:, 1000]], ref[:, 1000][~want[:, 1000]])
    keep = ~want
    keep[:, 1000] = False
    assert np.all(np.abs(got - ref)[keep] <= np.abs(ref)[keep] * (2.0 ** -8 + 2 * FP32))


def test_linear_repeats_and_unaligned_buffers():
    """Scales at any multiple of 4 bytes, codes and outputs at an odd multiple of 16: the same bits."""
    for M in (5, 40, 700):
        rng = np.random.default_rng(M)
        N, K = 1032, 1040
        (ac, as_), (wc, ws) = operand(rng, M, K), operand(rng, N, K)

        def at(a, o):
            buf = torch.empty(a.nbytes + 64, dtype=torch.int8, device=DEV)
            t = torch.from_numpy(a)
            v = buf[o:o + a.nbytes].view(t.dtype).view(t.shape)
            v.copy_(t)
            return v
        want, again = (torch.empty(M, N, dtype=torch.float16, device=DEV) for _ in range(2))
        mm.int8_linear(dev(ac), dev(as_), dev(wc), dev(ws), want)
        mm.int8_linear(dev(ac), dev(as_), dev(wc), dev(ws), again)
        out = torch.empty(M * N + 8, dtype=torch.float16, device=DEV)[8:].view(M, N)
        mm.int8_linear(at(ac, 16), at(as_, 4), at(wc, 48), at(ws, 12), out)
        assert torch.equal(out, want) and torch.equal(again, want)


@pytest.mark.parametrize("M,N,K", [(300000, 16, 16384), (300000, 264, 16384), (4, 300000, 16384), (600, 300000, 16384),
                                   (131077, 32784, 128)])
def test_linear_offsets_past_32_bits(M, N, K):
    """Codes beyond 4 GB and more than 2^32 outputs: samples against the oracle, ends included."""
    gen = torch.Generator(device=DEV).manual_seed(N)

    def big(rows):
        c = torch.randint(-127, 128, (rows, K), dtype=torch.int8, device=DEV, generator=gen)
        return c, torch.rand(rows, device=DEV, generator=gen) + 0.5
    (ac, as_), (wc, ws) = big(M), big(N)
    out = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    mm.int8_linear(ac, as_, wc, ws, out)
    torch.cuda.synchronize()
    rng = np.random.default_rng(1)
    pick = [torch.from_numpy(np.unique(np.concatenate([rng.choice(n, min(n, 20), replace=False), [0, n // 2, n - 1]])))
            for n in (M, N)]
    part = lambda t, i: t[i.to(DEV)].cpu().numpy()  # noqa: E731
    ref = Q.product(part(ac, pick[0]), part(as_, pick[0]), part(wc, pick[1]), part(ws, pick[1]))
    accept(out[pick[0].to(DEV)][:, pick[1].to(DEV)], ref)
    assert not torch.isnan(out.view(-1)[:: 4099]).any() and not torch.isnan(out[:, -1]).any()


@pytest.mark.parametrize("M", [2 ** 31 - 1, 2 ** 31 - 64])
def test_linear_of_as_many_rows_as_there_can_be(M):
    """The same rows again and again, whole sums that bf16 rounds once."""
    gen = torch.Generator(device=DEV).manual_seed(3)
    block, w = (torch.randint(-128, 128, (n, 16), dtype=torch.int8, device=DEV, generator=gen) for n in (1000003, 8))
    a, out = torch.empty(M, 16, dtype=torch.int8, device=DEV), torch.full((M, 8), 7.5, dtype=torch.bfloat16, device=DEV)
    for r in range(0, M, len(block)):
        a[r:r + len(block)] = block[:M - r]
    mm.int8_linear(a, torch.ones(M, device=DEV), w, torch.full((8,), 0.5, device=DEV), out)
    want = (block.float() @ w.float().t() * 0.5).to(torch.bfloat16)  # sums below 2^24: exact in float32
    assert all(torch.equal(out[r:r + len(block)], want[:M - r]) for r in range(0, M, len(block)))


# ---- experts -------------------------------------------------------------------------------------

def tables(counts, P, T, rng):
    """Routing tables for the given rows by expert, each token at most once an expert."""
    padded = (counts + P - 1) // P * P
    poff = np.concatenate([[0], np.cumsum(padded)]).astype(np.int32)
    row_token = np.full(int(poff[-1]) + 5, -1, np.int32)
    for e, c in enumerate(counts):
        row_token[poff[e]:poff[e] + c] = np.sort(rng.permutation(T)[:c])
    return poff, row_token


EXPERTS = [  # rows by expert, P, H, I
    ([3, 0, 1, 16, 0, 17], 1, 256, 128),
    ([0, 0, 0, 0], 8, 256, 128),
    ([1], 1, 16, 16),
    ([40, 64, 65, 128, 129, 0, 256, 257, 2], 16, 400, 144),
    ([300, 0, 5, 33], 128, 1168, 272),
    ([2] * 48, 1, 1024, 256),
    ([0] * 500 + [7, 600, 0, 20], 1, 256, 256),
    ([16] * 3 + [15] * 3 + [31, 32], 1, 640, 512),
    ([300, 0, 70, 20, 500, 129, 17, 260, 16, 190, 3], 8, 1152, 640),
    ([1100, 33, 0, 450], 1, 1408, 912),
    ([2100, 0, 40, 2060], 1, 256, 2064),
    ([2100, 100, 40, 2060, 64, 130], 1, 128, 2064),
    ([8, 1, 0, 15, 16, 0, 9, 7, 16, 3, 25, 0, 16, 16, 1], 1, 12288, 272),
    ([1, 16, 0, 15, 4, 0, 0, 16, 16, 31, 2, 8, 16, 0, 5, 16, 1, 20, 16], 1, 7168, 2048),
]


@pytest.mark.parametrize("bound", [0, 1, 10 ** 6])
@pytest.mark.parametrize("i", range(len(EXPERTS)))
def test_experts(i, bound):
    counts, P, H, I = EXPERTS[i]
    rng = np.random.default_rng(i)
    counts = np.array(counts, np.int32)
    E, T = len(counts), max(int(counts.max()), 1) + 7
    poff, row_token = tables(counts, P, T, rng)
    M_cap = len(row_token)
    (xc, xs), (hc, hs) = operand(rng, T, H, 0.3), operand(rng, M_cap, I, 0.3)
    w13c, w13s = np.zeros((E, 2 * I, H), np.int8), np.full((E, 2 * I), np.nan, np.float32)
    w2c, w2s = np.zeros((E, H, I), np.int8), np.full((E, H), np.nan, np.float32)
    used = np.nonzero(counts)[0]
    for e in used:  # the others hold NaN scales: never read
        w13c[e], w13s[e] = operand(rng, 2 * I, H, 1 / np.sqrt(H))
        w2c[e], w2s[e] = operand(rng, H, I, 0.1)
    hs[row_token < 0] = np.nan
    rt, po, ct = dev(row_token), dev(poff), dev(counts)
    h = torch.full((M_cap, I), 7.0, dtype=torch.bfloat16, device=DEV)
    y = torch.full((M_cap, H), 7.0, dtype=torch.bfloat16, device=DEV)
    mm.moe_grouped_gemm_l1_silu_int8(dev(xc), dev(xs), rt, po, ct, dev(w13c), dev(w13s), h, max_rows_per_expert=bound)
    mm.moe_grouped_gemm_l2_int8(dev(hc), dev(hs), po, ct, dev(w2c), dev(w2s), y, max_rows_per_expert=bound)
    torch.cuda.synchronize()
    free = np.ones(M_cap, bool)
    for e in used:
        r = np.arange(poff[e], poff[e] + counts[e])
        free[r] = False
        t = row_token[r]
        accept_silu(h[dev(r)], *gate_up(xc[t], xs[t], w13c[e], w13s[e]))
        accept(y[dev(r)], Q.product(hc[r], hs[r], w2c[e], w2s[e]))
    assert torch.all(h[dev(free)] == 7.0) and torch.all(y[dev(free)] == 7.0)  # rows without an assignment


def test_experts_no_rows():
    i8 = lambda *s: torch.zeros(*s, dtype=torch.int8, device=DEV)  # noqa: E731
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device=DEV)  # noqa: E731
    f32, bf = (lambda *s, d=d: torch.zeros(*s, dtype=d, device=DEV) for d in (torch.float32, torch.bfloat16))
    mm.moe_grouped_gemm_l1_silu_int8(i8(0, 256), f32(0), i32(0), i32(5), i32(4), i8(4, 256, 256), f32(4, 256), bf(0, 128))
    mm.moe_grouped_gemm_l2_int8(i8(0, 128), f32(0), i32(5), i32(4), i8(4, 256, 128), f32(4, 256), bf(0, 256))
    torch.cuda.synchronize()


# ---- the layer -----------------------------------------------------------------------------------

def make_layer(T, k, Eg, e0, E, H, I, P, seed):
    rng = np.random.default_rng(seed)
    W = layer.Int8MoEWeights.empty(E, H, I, device=DEV)
    for e in range(E):
        w13, w2 = (torch.from_numpy(rng.standard_normal(s).astype(np.float32) * 0.1).bfloat16().to(DEV)
                   for s in ((2 * I, H), (H, I)))
        layer.quantize_expert_int8_into(W, e, w13, w2)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32) * 0.5).bfloat16().to(DEV)
    z = torch.from_numpy(rng.standard_normal((T, Eg)).astype(np.float32)).to(DEV)
    return W, x, z, layer.Int8MoELayer(T, k, E, H, I, P, expert_begin=e0, device=DEV)


@pytest.mark.parametrize("T,P,stream", [(1, 1, False), (8, 1, True), (300, 16, False)])
def test_layer_steps_agree_with_the_oracle(T, P, stream):
    """The whole layer from logits: routing and the quantized h bit for bit against the oracle given
    the stage's own inputs, products and combine within their bounds."""
    k, Eg, e0, E, H, I = 4, 32, 4, 20, 528, 272
    W, x, z, L = make_layer(T, k, Eg, e0, E, H, I, P, T)
    bias = torch.linspace(-0.1, 0.1, Eg, device=DEV)
    s = torch.cuda.Stream() if stream else None
    if s is not None:
        s.wait_stream(torch.cuda.current_stream())
    out = L.forward_scores(x, z, W, bias=bias, score="sigmoid", n_group=4, topk_group=2, scale=2.5, stream=s)
    torch.cuda.synchronize()
    ids, _ = X.router(z.cpu().numpy(), k, bias.cpu().numpy(), "sigmoid", 4, 2, 2, True, 2.5)
    assert np.array_equal(np_i32(L.topk_ids), ids)
    counts, poff, rt = np_i32(L.counts), np_i32(L.padded_offsets), np_i32(L.row_token)
    xc, xs = Q.quantize(host(x))
    assert np.array_equal(L.x_codes.cpu().numpy(), xc) and np.array_equal(L.x_scales.cpu().numpy(), xs)
    valid = rt >= 0
    hc, hs = Q.quantize(np.where(valid[:, None], host(L.h), 0.0))
    assert np.array_equal(L.h_codes.cpu().numpy(), hc) and np.array_equal(L.h_scales.cpu().numpy(), hs)
    n = lambda t: t.cpu().numpy()  # noqa: E731
    for e in np.nonzero(counts)[0]:
        r = np.arange(poff[e], poff[e] + counts[e])
        accept_silu(L.h[dev(r)], *gate_up(xc[rt[r]], xs[rt[r]], n(W.w13_codes[e]), n(W.w13_scales[e])))
        accept(L.y[dev(r)], Q.product(hc[r], hs[r], n(W.w2_codes[e]), n(W.w2_scales[e])))
    y = host(L.y)
    tr, w = np_i32(L.token_rows).reshape(T, k), L.topk_weights.cpu().numpy().astype(np.float64)
    terms = [np.where(tr[:, j:j + 1] >= 0, w[:, j:j + 1] * y[np.maximum(tr[:, j], 0)], 0.0) for j in range(k)]
    ref, mag = sum(terms), sum(np.abs(t) for t in terms)
    assert np.all(np.abs(host(out) - ref) <= np.abs(ref) * 2.0 ** -8 + mag * (k + 1) * 2.0 ** -24 * 1.01 + 2.0 ** -133)


def test_layer_from_ids_equals_layer_from_logits():
    W, x, z, L = make_layer(40, 3, 16, 0, 16, 256, 128, 1, 77)
    a = L.forward_scores(x, z, W, score="softmax", renormalize=False).clone()
    ids, w = L.topk_ids.clone(), L.topk_weights.clone()
    L.out.fill_(float("nan"))
    assert torch.equal(L.forward(x, ids, w, W), a)


@pytest.mark.parametrize("T", [12, 200])
def test_layer_same_expert_twice(T):
    """A token that names an expert twice has two equal rows there; an expert then has more rows than T."""
    W, x, _, L = make_layer(T, 2, 8, 0, 8, 256, 128, 1, T)
    ids = torch.full((T, 2), 3, dtype=torch.int32, device=DEV)
    w = torch.tensor([[0.75, -0.25]], device=DEV).expand(T, 2).contiguous()
    out = L.forward(x, ids, w, W).clone()
    assert int(L.counts[3]) == 2 * T and int(L.counts.sum()) == 2 * T
    y = L.y[L.token_rows.view(T, 2).long()]
    assert torch.equal(y[:, 0], y[:, 1])
    assert torch.equal(out, (y[:, 0].float() * 0.5).to(torch.bfloat16))  # 0.75 y - 0.25 y, exact


@pytest.mark.parametrize("T", [0, 2, 100])
def test_layer_captured_and_two_layers_at_once(T):
    """One captured forward replayed on new inputs, with eager work of a second layer on another stream
    in between; both give what an eager forward alone gives."""
    k, Eg, E, H, I = 4, 24, 24, 512, 256
    W, x, z, L = make_layer(T, k, Eg, 0, E, H, I, 1, 5)
    L2 = layer.Int8MoELayer(T, k, E, H, I, 1, device=DEV)
    kw = dict(score="sigmoid", n_group=4, topk_group=2)
    L.forward_scores(x, z, W, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.forward_scores(x, z, W, **kw)
    side = torch.cuda.Stream()
    for r in range(4):
        gen = torch.Generator(device=DEV).manual_seed(r)
        x.copy_(torch.randn(x.shape, generator=gen, device=DEV) * 0.5)
        z.copy_(torch.randn(z.shape, generator=gen, device=DEV))
        torch.cuda.synchronize()
        want = L2.forward_scores(x, z, W, **kw).clone()
        L.out.fill_(3.0)
        L.h.fill_(3.0)
        L2.out.fill_(3.0)
        torch.cuda.synchronize()
        g.replay()
        L2.forward_scores(x, z, W, stream=side, **kw)
        torch.cuda.synchronize()
        assert torch.equal(L.out, want) and torch.equal(L2.out, want)


@pytest.mark.parametrize("P", [1, 16])
@pytest.mark.parametrize("kind", ["int8", "mxfp4"])
def test_layer_without_tokens(kind, P):
    """A rank that got no token: an empty output, and the rows that padding leaves room for are not written."""
    cls, W = {"int8": (layer.Int8MoELayer, layer.Int8MoEWeights), "mxfp4": (layer.MXMoELayer, layer.MXMoEWeights)}[kind]
    w = W.empty(8, 256, 128, device=DEV)
    for t in (w.w13_codes, w.w13_scales, w.w2_codes, w.w2_scales):
        t.zero_()
    L = cls(0, 2, 8, 256, 128, P, device=DEV)
    L.h.fill_(7.0)
    x, z = torch.empty(0, 256, dtype=torch.bfloat16, device=DEV), torch.empty(0, 8, device=DEV)
    ids, wts = torch.empty(0, 2, dtype=torch.int32, device=DEV), torch.empty(0, 2, device=DEV)
    assert L.forward(x, ids, wts, w).shape == (0, 256) and L.forward_scores(x, z, w).shape == (0, 256)
    torch.cuda.synchronize()
    assert not L.counts.any() and torch.all(L.h == 7.0) and len(L.h) == (8 * (P - 1))


# ---- one result whatever kernel runs -----------------------------------------------------------------

@pytest.mark.parametrize("i", range(len(EXPERTS)))
def test_experts_bits_do_not_depend_on_the_bound(i):
    """The caller's bound changes which kernel runs (stream or tiles, m-tiles of 4, 8 or 16 rows), not a bit."""
    counts, P, H, I = EXPERTS[i]
    rng = np.random.default_rng(100 + i)
    counts = np.array(counts, np.int32)
    E, T = len(counts), max(int(counts.max()), 1) + 7
    poff, row_token = tables(counts, P, T, rng)
    M_cap, gen = len(row_token), torch.Generator(device=DEV).manual_seed(i)
    code = lambda *s: torch.randint(-127, 128, s, dtype=torch.int8, device=DEV, generator=gen)  # noqa: E731
    scale = lambda *s, m=1.0: (torch.rand(s, device=DEV, generator=gen) + 0.5) * m  # noqa: E731
    x, xs, hc, hs = code(T, H), scale(T, m=0.01), code(M_cap, I), scale(M_cap, m=0.01)
    w13, w13s, w2, w2s = code(E, 2 * I, H), scale(E, 2 * I, m=0.02 / H ** 0.5), code(E, H, I), scale(E, H, m=0.01)
    rt, po, ct = dev(row_token), dev(poff), dev(counts)
    first = None
    for bound in (0, 1, 5, 16, 10 ** 6):
        h, y = (torch.full((M_cap, n), 7.0, dtype=torch.bfloat16, device=DEV) for n in (I, H))
        mm.moe_grouped_gemm_l1_silu_int8(x, xs, rt, po, ct, w13, w13s, h, max_rows_per_expert=bound)
        mm.moe_grouped_gemm_l2_int8(hc, hs, po, ct, w2, w2s, y, max_rows_per_expert=bound)
        first = first or (h, y)
        assert torch.equal(h, first[0]) and torch.equal(y, first[1]), bound


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,K", [(48, 48), (528, 1040), (272, 7168), (4096, 2048)])
def test_dense_bits_do_not_depend_on_the_rows(N, K, dtype):
    """The first rows of a call of many as in a call of few: stream, tiles of 64 x 64, tiles of 256 columns."""
    gen = torch.Generator(device=DEV).manual_seed(N)
    M = 4200
    a, w = (torch.randint(-127, 128, (n, K), dtype=torch.int8, device=DEV, generator=gen) for n in (M, N))
    sa, sw = torch.rand(M, device=DEV, generator=gen) * 0.02, torch.rand(N, device=DEV, generator=gen) * 0.02 / K ** 0.5
    whole, wide = torch.empty(M, N, dtype=dtype, device=DEV), torch.empty(M, N // 2, dtype=dtype, device=DEV)
    mm.int8_linear(a, sa, w, sw, whole)
    mm.int8_linear_gate_up_silu(a, sa, w, sw, wide)
    for m in (1, 4, 7, 16, 17, 40, 200, 1500):
        out, h = torch.empty(m, N, dtype=dtype, device=DEV), torch.empty(m, N // 2, dtype=dtype, device=DEV)
        mm.int8_linear(a[:m], sa[:m], w, sw, out)
        mm.int8_linear_gate_up_silu(a[:m], sa[:m], w, sw, h)
        assert torch.equal(out, whole[:m]) and torch.equal(h, wide[:m]), m


@pytest.mark.parametrize("rows,cols", [(5 * 2 ** 20 + 3, 2064), (5 * 2 ** 20 + 3, 64)])
def test_quantize_and_decode_beyond_one_grid(rows, cols):
    """More rows, and pieces of output, than a grid has places for: a workgroup a row, and a wave a row."""
    gen = torch.Generator(device=DEV).manual_seed(9)
    few = (torch.randn(10007, cols, generator=gen, device=DEV) * 0.3).to(torch.bfloat16)
    x, row_valid = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV), torch.zeros(rows, dtype=torch.int32, device=DEV)
    for a in range(0, rows, len(few)):
        x[a:a + len(few)] = few[:rows - a]
    row_valid[rows - 2] = -1
    c, s = torch.full((rows, cols), 77, dtype=torch.int8, device=DEV), torch.full((rows,), 77.0, device=DEV)
    mm.int8_quantize_act(x, c, s, row_valid=row_valid)
    x.fill_(7.0)
    mm.int8_dequantize(c, s, x)
    fc, fs = Q.quantize(host(few))
    small = dev(fc), dev(fs), torch.from_numpy(Q.dequantize(fc, fs)).to(torch.bfloat16).to(DEV)
    for t, f in zip((c, s, x), small):
        assert not t[rows - 2].any()
        t[rows - 2] = f[(rows - 2) % len(few)]
        assert all(torch.equal(t[a:a + len(few)], f[:rows - a]) for a in range(0, rows, len(few)))
