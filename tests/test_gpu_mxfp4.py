"""MXFP4 quantizer, decoder and products on the GPU against the float64 oracle.

Quantizer and decoder: bit for bit.  Products: the operands are exact, so an output is off by the fp32
accumulation, at most K * 2^-24 times the sum of the products' magnitudes (each of the at most K
additions rounds a partial sum no larger than that by half a step), and by one rounding to bf16
(2^-8 relative).  SiLU(g) * u: the errors of g and u pass with |SiLU'| <= 1.1; the hardware exp2 and
reciprocal are a step off each, the exponent's rounding adds |g| of them: (6 + 2 |g|) * 2^-23 in all."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_top_amd import layer, megamoe as mm
from oracle import mxfp4_oracle as X

from gpu_util import DEV, np_i32

pytestmark = pytest.mark.gpu

TINY = 2.0 ** -133  # outputs below the normal range of fp32


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def bf16_np(t):
    with np.errstate(invalid="ignore"):  # signalling NaN
        return t.detach().float().cpu().numpy().astype(np.float64)


def bf16_round(a):
    return torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16)


def quantized(rng, rows, K, std):
    return X.quantize(bf16_np(bf16_round(rng.standard_normal((rows, K)) * std)))


def accept(got, ref, zabs, K):
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    err = np.abs(got - ref)
    assert np.all((err <= np.abs(ref) * 2.0 ** -8 + zabs * K * 2.0 ** -24 * (1 + 2.0 ** -8) + TINY) | np.isnan(ref))


def accept_silu(got, h, g, u, gabs, uabs, K):
    dg, du = gabs * K * 2.0 ** -24, uabs * K * 2.0 ** -24
    err = 1.1 * dg * np.abs(u) + np.abs(X.silu(g)) * du + 1.1 * dg * du + np.abs(h) * (6 + 2 * np.abs(g)) * 2.0 ** -23
    assert np.array_equal(np.isnan(got), np.isnan(h))
    assert np.all((np.abs(got - h) <= np.abs(h) * 2.0 ** -8 + err * (1 + 2.0 ** -8) + TINY) | np.isnan(h))


# ---- quantizer and decoder -------------------------------------------------------------------------

def check_quantize(xt, row_valid=None):
    rows, cols = xt.shape
    codes = torch.full((rows + 1, cols // 2), 0xAB, dtype=torch.uint8, device=DEV)
    scales = torch.full((rows + 1, cols // 32), 0xCD, dtype=torch.uint8, device=DEV)
    rv = None if row_valid is None else dev(row_valid)
    mm.mxfp4_quantize_act(xt.to(DEV), codes[:rows], scales[:rows], row_valid=rv)
    torch.cuda.synchronize()
    rc, rs = X.quantize(xt.double().numpy())
    if row_valid is not None:
        rc[row_valid < 0], rs[row_valid < 0] = 0, 0
    assert np.array_equal(np_i32(codes[:rows]), rc) and np.array_equal(np_i32(scales[:rows]), rs)
    assert torch.all(codes[rows:] == 0xAB) and torch.all(scales[rows:] == 0xCD)  # behind the last row
    return codes[:rows], scales[:rows]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(0, 32), (1, 32), (3, 96), (1, 7168), (8, 7168), (257, 1056), (4100, 2048)])
def test_quantize_shapes(rows, cols, dtype):
    rng = np.random.default_rng(rows + cols)
    x = torch.from_numpy((rng.standard_normal((rows, cols)) * 0.09).astype(np.float32)).to(dtype)
    check_quantize(x)


def test_quantize_every_bf16_value():
    """Every finite bf16 value as an element of blocks whose largest value sits 0 to 4 binades above it,
    and on its own."""
    bits = np.arange(1 << 16, dtype=np.uint16)
    bits = bits[(bits & 0x7F80) != 0x7F80]
    v = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16)
    x = torch.zeros(len(bits), 96, dtype=torch.bfloat16)
    x[:, 5] = v
    for j in range(1, 3):
        x[:, 32 * j + 7] = v
        big = (bits & 0x7F80).astype(np.int64) + 0x80 * (1 if j == 1 else 4) + 0x35
        big[big >= 0x7F80] = 0x7F7F
        x[:, 32 * j + 30] = torch.from_numpy(big.astype(np.uint16).view(np.int16)).view(torch.bfloat16)
    codes, scales = check_quantize(x)
    out = torch.empty(len(bits), 96, dtype=torch.bfloat16, device=DEV)
    mm.mxfp4_dequantize(codes, scales, out)
    ref = X.decode(np_i32(codes).astype(np.uint8), np_i32(scales).astype(np.uint8))
    got = bf16_np(out)
    fits = np.abs(ref) < 2.0 ** 128 * (1 - 2.0 ** -8)
    assert np.array_equal(got[fits], ref[fits])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_extremes(dtype):
    """Infinities, NaN, zeros of both signs, subnormals, the largest and the smallest values, ties."""
    rng = np.random.default_rng(4)
    x = torch.from_numpy(rng.standard_normal((12, 64)).astype(np.float32))
    x[0, 3], x[0, 40] = float("inf"), float("-inf")
    x[1, 63] = float("nan")
    x[2] = 0.0
    x[3] = -0.0
    x[4] *= 2.0 ** -140
    x[5] = x[5] * 2.0 ** -125
    x[6] = torch.finfo(dtype).max
    x[7] = -torch.finfo(dtype).max
    x[8, :32] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0] * 4)
    x[9, 5] = torch.finfo(torch.float32).tiny
    x[10, 1:] = 0.0
    check_quantize(x.to(dtype))


def test_quantize_skips_invalid_rows():
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((70, 256)).astype(np.float32)).to(torch.bfloat16)
    rv = rng.integers(-1, 3, 70).astype(np.int32)
    x[np.nonzero(rv < 0)[0][0]] = float("nan")
    check_quantize(x, rv)


def test_dequantize_every_code_and_scale():
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))       # every pair of codes under every scale
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, 1)
    out = torch.empty(256, 512, dtype=torch.bfloat16, device=DEV)
    mm.mxfp4_dequantize(dev(codes), dev(scales), out)
    torch.cuda.synchronize()
    ref = X.decode(codes, scales)
    got = bf16_np(out)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    big = np.abs(ref) >= 2.0 ** 128
    assert np.array_equal(got[big], np.sign(ref[big]) * np.inf)
    rest = ~big & ~np.isnan(ref)
    assert np.array_equal(got[rest], ref[rest])


# ---- dense products ------------------------------------------------------------------------------

SHAPES = [  # M, N, K
    (0, 64, 256), (1, 16, 128), (1, 7168, 2048), (5, 48, 384), (16, 256, 7168), (17, 272, 640), (32, 512, 1024),
    (33, 128, 128), (64, 80, 2176), (100, 4096, 512), (129, 528, 1152), (255, 256, 256), (256, 256, 512),
    (257, 1040, 896), (513, 2048, 1024), (1000, 304, 2048), (8, 4096, 16384),
    (13, 48, 9088), (9, 32, 20480), (3, 16, 40448), (5, 32, 40576),  # long reductions, few rows
    # enough tiles for the tile kernel: last rows of each tile height, column edges, K of whole and half
    # stages, with and without 16-byte scale pieces, of one stage and of two (with tiles beyond one a CU)
    (1500, 1040, 896), (1400, 1072, 1152), (2060, 784, 640), (1537, 1040, 1024), (1500, 1040, 256),
    (4200, 4112, 128), (4161, 4112, 384), (4353, 4112, 512),
]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear(M, N, K):
    rng = np.random.default_rng(M + N + K)
    (ac, as_), (wc, ws) = quantized(rng, M, K, 0.09), quantized(rng, N, K, 0.02)
    out = torch.full((M + 1, N), 7.0, dtype=torch.bfloat16, device=DEV)
    mm.mxfp4_linear(dev(ac), dev(as_), dev(wc), dev(ws), out[:M])
    torch.cuda.synchronize()
    assert torch.all(out[M:] == 7.0)
    ref, zabs = X.product(X.decode(ac, as_), X.decode(wc, ws))
    accept(bf16_np(out[:M]), ref, zabs, K)


@pytest.mark.parametrize("M,N,K", [(0, 32, 128), (1, 16, 128), (1, 2048, 7168), (7, 48, 384), (16, 128, 1024),
                                   (31, 144, 640), (64, 2048, 256), (130, 272, 1152), (257, 512, 2048),
                                   (520, 1040, 256), (1500, 528, 896), (1400, 560, 1152), (2060, 400, 512),
                                   (4200, 2064, 128), (4161, 2064, 384)])
def test_gate_up_silu(M, N, K):
    rng = np.random.default_rng(M + N + K + 1)
    (ac, as_), (wc, ws) = quantized(rng, M, K, 0.5), quantized(rng, 2 * N, K, 0.1)
    out = torch.full((M + 1, N), 7.0, dtype=torch.bfloat16, device=DEV)
    mm.mxfp4_linear_gate_up_silu(dev(ac), dev(as_), dev(wc), dev(ws), out[:M])
    torch.cuda.synchronize()
    assert torch.all(out[M:] == 7.0)
    accept_silu(bf16_np(out[:M]), *X.gate_up(X.decode(ac, as_), X.decode(wc, ws)), K)


@pytest.mark.parametrize("M,N", [(3, 64), (40, 64), (300, 64), (1500, 1040)])
def test_linear_random_codes_and_scales(M, N):
    """Every code, scales over sixty binades, zero blocks and zero rows."""
    rng = np.random.default_rng(M)
    K = 768
    ac, wc = (rng.integers(0, 256, (n, K // 2)).astype(np.uint8) for n in (M, N))
    as_, ws = (rng.integers(97, 157, (n, K // 32)).astype(np.uint8) for n in (M, N))
    ac[1] = 0
    wc[2, 16:32] = 0x88  # minus zero
    out = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    mm.mxfp4_linear(dev(ac), dev(as_), dev(wc), dev(ws), out)
    torch.cuda.synchronize()
    ref, zabs = X.product(X.decode(ac, as_), X.decode(wc, ws))
    accept(bf16_np(out), ref, zabs, K)


@pytest.mark.parametrize("M,N", [(2, 48), (20, 48), (300, 48), (1500, 1040)])
def test_linear_nan_scales_reach_their_outputs_only(M, N):
    rng = np.random.default_rng(M + 9)
    K = 640
    (ac, as_), (wc, ws) = quantized(rng, M, K, 1.0), quantized(rng, N, K, 1.0)
    as_[1, K // 32 - 1] = 255
    ws[17, 0] = 255
    out = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    mm.mxfp4_linear(dev(ac), dev(as_), dev(wc), dev(ws), out)
    torch.cuda.synchronize()
    got = bf16_np(out)
    want = np.zeros((M, N), bool)
    want[1], want[:, 17] = True, True
    assert np.array_equal(np.isnan(got), want)
    ref, zabs = X.product(np.nan_to_num(X.decode(ac, as_)), np.nan_to_num(X.decode(wc, ws)))
    accept(np.where(want, 0, got), np.where(want, 0, ref), zabs, K)


def test_linear_large_is_repeatable_and_matches_samples():
    rng = np.random.default_rng(31)
    M, N, K = 4111, 2064, 7168
    xt = torch.from_numpy((rng.standard_normal((M, K)) * 0.09).astype(np.float32)).to(torch.bfloat16).to(DEV)
    ac, as_ = torch.empty(M, K // 2, dtype=torch.uint8, device=DEV), torch.empty(M, K // 32, dtype=torch.uint8, device=DEV)
    mm.mxfp4_quantize_act(xt, ac, as_)
    wc, ws = quantized(rng, N, K, 0.02)
    wct, wst = dev(wc), dev(ws)
    out, again = (torch.empty(M, N, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    mm.mxfp4_linear(ac, as_, wct, wst, out)
    mm.mxfp4_linear(ac, as_, wct, wst, again)
    torch.cuda.synchronize()
    assert torch.equal(out, again)
    rows = np.unique(np.concatenate([rng.choice(M, 40, replace=False), [0, M - 1]]))
    a = X.decode(np_i32(ac)[rows].astype(np.uint8), np_i32(as_)[rows].astype(np.uint8))
    ref, zabs = X.product(a, X.decode(wc, ws))
    accept(bf16_np(out)[rows], ref, zabs, K)


@pytest.mark.parametrize("off", [4, 8, 12])
@pytest.mark.parametrize("M", [5, 700])
def test_linear_scales_aligned_to_words(M, off):
    """Scales at any multiple of 4, codes and outputs at an odd multiple of 16: the same bits."""
    rng = np.random.default_rng(M + off)
    N, K = 2064, 1024
    (ac, as_), (wc, ws) = quantized(rng, M, K, 0.5), quantized(rng, N, K, 0.1)

    def at(a, o):
        buf = torch.empty(a.size + 64, dtype=torch.uint8, device=DEV)
        v = buf[o:o + a.size].view(a.shape)
        v.copy_(torch.from_numpy(a))
        return v
    want = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    mm.mxfp4_linear(dev(ac), dev(as_), dev(wc), dev(ws), want)
    out = torch.empty(M * N + 8, dtype=torch.bfloat16, device=DEV)[8:].view(M, N)
    mm.mxfp4_linear(at(ac, 16), at(as_, off), at(wc, 48), at(ws, 16 - off), out)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("M,N,K", [(300000, 16, 32768), (300000, 256, 32768), (4, 300000, 32768), (600, 300000, 32768),
                                   (131077, 32784, 128)])
def test_linear_offsets_past_32_bits(M, N, K):
    """Codes beyond 4 GB and more than 2^32 outputs: samples against the oracle, ends included."""
    gen = torch.Generator(device=DEV).manual_seed(N)

    def operand(rows):
        c = torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, device=DEV, generator=gen)
        return c, torch.randint(118, 124, (rows, K // 32), dtype=torch.uint8, device=DEV, generator=gen)
    (ac, as_), (wc, ws) = operand(M), operand(N)
    out = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    mm.mxfp4_linear(ac, as_, wc, ws, out)
    torch.cuda.synchronize()
    rng = np.random.default_rng(1)
    pick = [torch.from_numpy(np.unique(np.concatenate([rng.choice(n, min(n, 20), replace=False), [0, n // 2, n - 1]])))
            for n in (M, N)]
    part = lambda t, i: t[i.to(DEV)].cpu().numpy()  # noqa: E731
    ref, zabs = X.product(X.decode(part(ac, pick[0]), part(as_, pick[0])), X.decode(part(wc, pick[1]), part(ws, pick[1])))
    got = out[pick[0].to(DEV)][:, pick[1].to(DEV)]
    accept(bf16_np(got), ref, zabs, K)
    assert not torch.isnan(out.view(-1)[:: 4099]).any() and not torch.isnan(out[:, -1]).any()


def test_quantize_and_decode_past_32_bits():
    """2^32 elements and some: each row as the same row of a small tensor."""
    rows, cols = 2 ** 21 + 5, 2048
    gen = torch.Generator(device=DEV).manual_seed(8)
    few = (torch.randn(64, cols, generator=gen, device=DEV) * 0.3).to(torch.bfloat16)
    x = few.repeat(rows // 64 + 1, 1)[:rows]
    out = []
    for t in (few, x):
        c, s = (torch.empty(len(t), cols // n, dtype=torch.uint8, device=DEV) for n in (2, 32))
        mm.mxfp4_quantize_act(t, c, s)
        y = torch.empty_like(t)
        mm.mxfp4_dequantize(c, s, y)
        out.append((c, s, y))
    for a in range(0, rows, 2 ** 17):
        n = min(2 ** 17, rows - a)
        for small, large in zip(*out):
            assert torch.equal(large[a:a + n], small.repeat(2 ** 11, 1)[:n])


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
    ([1], 1, 128, 16),
    ([40, 64, 65, 128, 129, 0, 256, 257, 2], 16, 384, 144),
    ([300, 0, 5, 33], 128, 1152, 272),
    ([2] * 48, 1, 1024, 256),
    ([0] * 500 + [7, 600, 0, 20], 1, 256, 256),
    ([16] * 3 + [15] * 3 + [31, 32], 1, 640, 512),
    # enough tiles for the tile kernel beside small experts: every tile height, half stages, several
    # tiles a workgroup with one and two stages
    ([300, 0, 70, 20, 500, 129, 17, 260, 16, 190, 3], 8, 1152, 640),
    ([1100, 33, 0, 450], 1, 1408, 896),
    ([1100, 33, 0, 450], 16, 512, 720),
    ([2100, 0, 40, 2060], 1, 256, 2064),
    ([2100, 0, 40, 2060], 1, 384, 2064),
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
    xc, xs = quantized(rng, T, H, 0.5)
    down = I % 128 == 0  # L2's reduction; L1 alone takes any multiple of 16
    hc, hs = quantized(rng, M_cap, I if down else 128, 0.5)
    used = np.nonzero(counts)[0]
    w13c, w13s = np.zeros((E, 2 * I, H // 2), np.uint8), np.full((E, 2 * I, H // 32), 255, np.uint8)
    w2c, w2s = np.zeros((E, H, I // 2), np.uint8), np.full((E, H, I // 32), 255, np.uint8)
    for e in used:  # the others hold NaN scales: never read
        w13c[e], w13s[e] = quantized(rng, 2 * I, H, 0.1)
        if down:
            w2c[e], w2s[e] = quantized(rng, H, I, 0.1)
    rt, po, ct = dev(row_token), dev(poff), dev(counts)
    h = torch.full((M_cap, I), 7.0, dtype=torch.bfloat16, device=DEV)
    mm.moe_grouped_gemm_l1_silu_mxfp4(dev(xc), dev(xs), rt, po, ct, dev(w13c), dev(w13s), h, max_rows_per_expert=bound)
    y = torch.full((M_cap, H), 7.0, dtype=torch.bfloat16, device=DEV)
    if down:
        mm.moe_grouped_gemm_l2_mxfp4(dev(hc), dev(hs), po, ct, dev(w2c), dev(w2s), y, max_rows_per_expert=bound)
    torch.cuda.synchronize()
    hg, yg, free = bf16_np(h), bf16_np(y), np.ones(M_cap, bool)
    xv, hv = X.decode(xc, xs), X.decode(hc, hs)
    for e in used:
        r = np.arange(poff[e], poff[e] + counts[e])
        free[r] = False
        accept_silu(hg[r], *X.gate_up(xv[row_token[r]], X.decode(w13c[e], w13s[e])), H)
        if down:
            ref, zabs = X.product(hv[r], X.decode(w2c[e], w2s[e]))
            accept(yg[r], ref, zabs, I)
    assert np.all(hg[free] == 7.0) and np.all(yg[free] == 7.0)  # rows without an assignment: as they were


def random_operand(rng, *shape):
    """Any codes under scales over six binades around 2^-5: sums of a few units at the lengths used here."""
    *rows, K = shape
    return rng.integers(0, 256, (*rows, K // 2), dtype=np.uint8), rng.integers(119, 125, (*rows, K // 32), dtype=np.uint8)


# Reductions that the small kernel splits over its waves, with m-tiles of 16, 8 and 4 token rows.  With some 20
# m-tiles of 17 or 18 groups a workgroup has more than one group, and many cross into the next m-tile or expert
# (empty ones between them).
LONG = [
    (2688, [3, 0, 16, 1, 0, 0, 15, 16, 9, 5, 16, 0, 1, 12, 16, 33, 7, 16, 0, 2, 40]),
    (2816, [16] * 12 + [0] * 70 + [15, 0, 1] * 3 + [17]),
    (7168, [1, 16, 0, 15, 4, 0, 0, 16, 16, 31, 2, 8, 16, 0, 5, 16, 1, 20, 16]),
    (12288, [8, 1, 0, 15, 16, 0, 9, 7, 16, 3, 25, 0, 16, 16, 1]),
    (24576, [4, 0, 1, 15, 16, 3, 0, 5, 16, 18, 2]),
]


@pytest.mark.parametrize("bound", [0, 1])
@pytest.mark.parametrize("K,counts", LONG, ids=[str(K) for K, _ in LONG])
def test_experts_long_reductions(K, counts, bound):
    rng = np.random.default_rng(K)
    counts = np.array(counts, np.int32)
    E, T, I, H = len(counts), int(counts.max()) + 3, 144, 272
    poff, row_token = tables(counts, 1, T, rng)
    M_cap = len(row_token)
    (xc, xs), (hc, hs) = random_operand(rng, T, K), random_operand(rng, M_cap, K)
    (w13c, w13s), (w2c, w2s) = random_operand(rng, E, 2 * I, K), random_operand(rng, E, H, K)
    used = np.nonzero(counts)[0]
    w13s[counts == 0] = w2s[counts == 0] = 255  # never read
    rt, po, ct = dev(row_token), dev(poff), dev(counts)
    h = torch.full((M_cap, I), 7.0, dtype=torch.bfloat16, device=DEV)
    y = torch.full((M_cap, H), 7.0, dtype=torch.bfloat16, device=DEV)
    mm.moe_grouped_gemm_l1_silu_mxfp4(dev(xc), dev(xs), rt, po, ct, dev(w13c), dev(w13s), h, max_rows_per_expert=bound)
    mm.moe_grouped_gemm_l2_mxfp4(dev(hc), dev(hs), po, ct, dev(w2c), dev(w2s), y, max_rows_per_expert=bound)
    torch.cuda.synchronize()
    hg, yg, free = bf16_np(h), bf16_np(y), np.ones(M_cap, bool)
    xv, hv = X.decode(xc, xs), X.decode(hc, hs)
    for e in used:
        r = np.arange(poff[e], poff[e] + counts[e])
        free[r] = False
        accept_silu(hg[r], *X.gate_up(xv[row_token[r]], X.decode(w13c[e], w13s[e])), K)
        ref, zabs = X.product(hv[r], X.decode(w2c[e], w2s[e]))
        accept(yg[r], ref, zabs, K)
    assert np.all(hg[free] == 7.0) and np.all(yg[free] == 7.0)


@pytest.mark.parametrize("M,K", [(40, 2688), (47, 7168), (21, 12288), (11, 24576)])
def test_linear_long_reductions_of_several_m_tiles(M, K):
    """The same kernel on a dense call of three m-tiles and more, 387 groups of weight rows and 390 of gate+up."""
    rng = np.random.default_rng(M + K)
    N, I = 2064, 1040
    (ac, as_), (wc, ws) = random_operand(rng, M, K), random_operand(rng, 2 * I, K)
    out = torch.full((M + 1, N), 7.0, dtype=torch.bfloat16, device=DEV)
    h = torch.full((M + 1, I), 7.0, dtype=torch.bfloat16, device=DEV)
    a, w = (dev(ac), dev(as_)), (dev(wc), dev(ws))
    mm.mxfp4_linear(*a, w[0][:N], w[1][:N], out[:M])
    mm.mxfp4_linear_gate_up_silu(*a, *w, h[:M])
    torch.cuda.synchronize()
    assert torch.all(out[M:] == 7.0) and torch.all(h[M:] == 7.0)
    av, wv = X.decode(ac, as_), X.decode(wc, ws)
    accept(bf16_np(out[:M]), *X.product(av, wv[:N]), K)
    accept_silu(bf16_np(h[:M]), *X.gate_up(av, wv), K)


def test_experts_no_rows():
    """M_cap = 0: nothing is enqueued."""
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device=DEV)  # noqa: E731
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device=DEV)  # noqa: E731
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    mm.moe_grouped_gemm_l1_silu_mxfp4(u8(0, 128), u8(0, 8), i32(0), i32(5), i32(4), u8(4, 256, 128), u8(4, 256, 8),
                                      bf(0, 128))
    mm.moe_grouped_gemm_l2_mxfp4(u8(0, 64), u8(0, 4), i32(5), i32(4), u8(4, 256, 64), u8(4, 256, 4), bf(0, 256))
    torch.cuda.synchronize()


# ---- the layer -----------------------------------------------------------------------------------

def make_layer(T, k, Eg, e0, E, H, I, P, seed):
    rng = np.random.default_rng(seed)
    W = layer.MXMoEWeights.empty(E, H, I, device=DEV)
    for e in range(E):
        w13, w2 = (bf16_round(rng.standard_normal(s) * 0.1).to(DEV) for s in ((2 * I, H), (H, I)))
        layer.quantize_expert_mx_into(W, e, w13, w2)
    x = bf16_round(rng.standard_normal((T, H)) * 0.5).to(DEV)
    z = torch.from_numpy(rng.standard_normal((T, Eg)).astype(np.float32)).to(DEV)
    return W, x, z, layer.MXMoELayer(T, k, E, H, I, P, expert_begin=e0, device=DEV)


@pytest.mark.parametrize("T,P,stream", [(1, 1, False), (8, 1, True), (300, 16, False)])
def test_layer_steps_agree_with_the_oracle(T, P, stream):
    """The whole layer from logits: routing and the quantized h bit for bit against the oracle given
    the stage's own inputs, products and combine within their bounds."""
    k, Eg, e0, E, H, I = 4, 32, 4, 20, 512, 256
    W, x, z, L = make_layer(T, k, Eg, e0, E, H, I, P, T)
    bias = torch.linspace(-0.1, 0.1, Eg, device=DEV)
    s = torch.cuda.Stream() if stream else None
    if s is not None:
        s.wait_stream(torch.cuda.current_stream())
    out = L.forward_scores(x, z, W, bias=bias, score="sigmoid", n_group=4, topk_group=2, scale=2.5, stream=s)
    torch.cuda.synchronize()
    ids, wts = X.router(z.cpu().numpy(), k, bias.cpu().numpy(), "sigmoid", 4, 2, 2, True, 2.5)
    assert np.array_equal(np_i32(L.topk_ids), ids)
    counts, poff, rt = np_i32(L.counts), np_i32(L.padded_offsets), np_i32(L.row_token)
    xc, xs = X.quantize(bf16_np(x))
    assert np.array_equal(np_i32(L.x_codes), xc) and np.array_equal(np_i32(L.x_scales), xs)
    u8 = lambda t: np_i32(t).astype(np.uint8)  # noqa: E731
    h, y, xv = bf16_np(L.h), bf16_np(L.y), X.decode(xc, xs)
    valid = rt >= 0
    hc, hs = X.quantize(np.where(valid[:, None], h, 0.0))
    hc[~valid], hs[~valid] = 0, 0
    assert np.array_equal(u8(L.h_codes), hc) and np.array_equal(u8(L.h_scales), hs)
    hv = X.decode(hc, hs)
    for e in np.nonzero(counts)[0]:
        r = np.arange(poff[e], poff[e] + counts[e])
        accept_silu(h[r], *X.gate_up(xv[rt[r]], X.decode(u8(W.w13_codes[e]), u8(W.w13_scales[e]))), H)
        ref, zabs = X.product(hv[r], X.decode(u8(W.w2_codes[e]), u8(W.w2_scales[e])))
        accept(y[r], ref, zabs, I)
    tr, w = np_i32(L.token_rows).reshape(T, k), L.topk_weights.cpu().numpy().astype(np.float64)
    ref = sum(np.where(tr[:, j:j + 1] >= 0, w[:, j:j + 1] * y[np.maximum(tr[:, j], 0)], 0.0) for j in range(k))
    mag = sum(np.where(tr[:, j:j + 1] >= 0, np.abs(w[:, j:j + 1] * y[np.maximum(tr[:, j], 0)]), 0.0) for j in range(k))
    assert np.all(np.abs(bf16_np(out) - ref) <= np.abs(ref) * 2.0 ** -8 + mag * (k + 1) * 2.0 ** -24 * 1.01 + TINY)


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
    hv, rows = X.decode(np_i32(L.h_codes).astype(np.uint8), np_i32(L.h_scales).astype(np.uint8)), np_i32(L.token_rows)[::2]
    ref, zabs = X.product(hv[rows], X.decode(np_i32(W.w2_codes[3]).astype(np.uint8), np_i32(W.w2_scales[3]).astype(np.uint8)))
    accept(bf16_np(y[:, 0]), ref, zabs, 128)
    assert torch.equal(out, (y[:, 0].float() * 0.5).to(torch.bfloat16))  # 0.75 y - 0.25 y, exact


@pytest.mark.parametrize("T", [0, 2, 100])
def test_layer_captured_and_two_layers_at_once(T):
    """One captured forward replayed on new inputs, with eager work of a second layer on another stream
    in between; both give what an eager forward alone gives."""
    k, Eg, E, H, I = 4, 24, 24, 512, 256
    W, x, z, L = make_layer(T, k, Eg, 0, E, H, I, 1, 5)
    L2 = layer.MXMoELayer(T, k, E, H, I, 1, device=DEV)
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
