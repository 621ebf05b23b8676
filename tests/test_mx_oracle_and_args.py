"""The oracle of the scored router and the MXFP4 operators against brute force and differences, and
the refusals of their entry points (host checks, no GPU needed)."""
import os

import numpy as np
import pytest
import torch

from nvfp4_block_scaled_top_amd import layer, megamoe as mm
from oracle import mxfp4_oracle as X


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mm.library_path()):
        from nvfp4_block_scaled_top_amd import build_lib
        build_lib.build()
    return mm.lib()


FAKE = 0x1000  # never dereferenced: every call below fails its host-side checks
ODD = FAKE + 2


def test_oracle_quantizer_is_nearest_point():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((64, 96)) * np.exp2(rng.integers(-20, 20, (64, 1)).astype(float))
    x[0] = 0.0
    x[1, :32] = np.tile([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], 4)  # every tie at scale 1
    codes, scales = X.quantize(x)
    v = X.decode(codes, scales)
    unit = np.repeat(np.ldexp(1.0, scales.astype(int) - 127), 32, -1)
    points = np.concatenate([X.E2M1, -X.E2M1])
    best = np.abs(np.abs(x)[..., None] / unit[..., None] - X.E2M1).min(-1)
    assert np.array_equal(np.abs(np.abs(x) - np.abs(v)) / unit, best)
    assert np.isin(v / unit, points).all() and np.all((v == 0) | (np.sign(v) == np.sign(x)))
    assert v[1, :8].tolist() == [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0]
    amax = np.abs(x).reshape(64, 3, 32).max(-1)
    assert np.array_equal(scales[1:], (np.floor(np.log2(amax[1:])) - 2 + 127).astype(np.uint8))
    assert not scales[0].any() and not codes[0].any()


def test_oracle_quantizer_extremes():
    x = np.zeros((4, 32))
    x[0, 3], x[1, 5] = np.inf, np.nan
    x[2, 0] = 2.0 ** -133          # the smallest bf16: below half a step of the smallest scale
    x[3, 0], x[3, 1] = 2.0 ** -126, -3 * 2.0 ** -128
    codes, scales = X.quantize(x)
    assert scales[:, 0].tolist() == [255, 255, 0, 0]
    assert not codes[:3].any()
    assert X.decode(codes, scales)[3, :2].tolist() == [2.0 ** -126, -3 * 2.0 ** -128]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_oracle_router_gradient_by_differences(score, renormalize):
    rng = np.random.default_rng(3)
    z = rng.standard_normal((5, 24))
    ids, _ = X.router(z, 4, None, score, 4, 2, 2, renormalize, 2.5)
    grad = rng.standard_normal((5, 4))

    def loss(zz):
        s = X.scores(zz, score)
        p = np.take_along_axis(s, ids, 1)
        w = 2.5 * (p / p.sum(1, keepdims=True) if renormalize else p)
        return (w * grad).sum(1)

    got = X.router_bwd(z, ids, grad, score, renormalize, 2.5)
    h = 1e-5
    for e in range(24):
        d = np.zeros((5, 24))
        d[:, e] = h
        diff = (loss(z + d) - loss(z - d)) / (2 * h)
        # central difference: third derivatives of order 10 times h^2 / 6, and the sums' rounding over h
        assert np.abs(diff - got[:, e]).max() <= 1e-8


def test_oracle_router_masks():
    z = np.zeros((3, 8))
    z[0] = -np.inf
    z[1, 2:] = np.nan
    z[2, 4:] = -np.inf
    ids, w = X.router(z, 3, score="softmax", n_group=2, topk_group=1, group_top=2)
    assert ids.tolist() == [[-1, -1, -1], [0, 1, -1], [0, 1, 2]]
    assert w[0].tolist() == [0, 0, 0] and w[1].tolist() == [0.5, 0.5, 0]


def test_oracle_router_group_sums_that_overflow():
    """A group whose sum of choices is -inf in float32 is still before one without an available expert."""
    z = np.zeros((1, 12), np.float32)
    z[0, :4] = -np.inf
    bias = np.full(12, -3e38, np.float32)
    for top, want in ((2, [4, 5]), (1, [4, 5])):
        ids, w = X.router(z, 2, bias, "sigmoid", 3, 1, top)
        assert ids.tolist() == [want] and w.tolist() == [[0.5, 0.5]]


FAR = [0.0, -40.0, -700.0, -709.0, -720.0, -744.0, -746.0, -1e4, -1e30]


@pytest.mark.parametrize("far", FAR)
def test_oracle_gradient_far_from_the_largest_logit(far):
    """Two chosen logits, `far` below the row's largest (softmax) or 0 (sigmoid): n_1 = 1 / (1 + e^(z_2 - z_1))
    of scores that are e^z up to a common factor; dw_1 = -dw_2 = scale * n_1 n_2 (g_1 - g_2)."""
    z = np.array([[0.0, far - 1.0, far - 1.75, -3.0]])
    ids, grad = np.array([[1, 2]]), np.array([[1.0, -0.5]])
    d = z[0, 2] - z[0, 1]  # as rounded
    n = 1 / (1 + np.exp(d))
    want = 2.5 * n * (1 - n) * 1.5
    got = X.router_bwd(z, ids, grad, "softmax", True, 2.5)[0]
    assert np.all(np.abs(got - [0, want, -want, 0]) <= want * 2.0 ** -40)
    if far <= -40.0:
        z[0, 0] = -3.0
        got = X.router_bwd(z, ids, grad, "sigmoid", True, 2.5)[0]
        assert np.all(np.abs(got - [0, want, -want, 0]) <= want * 2.0 ** -40)


@pytest.mark.parametrize("far", FAR)
def test_oracle_weights_far_from_the_largest_logit(far):
    """A bias that forces two experts, `far` below the row's largest logit (softmax) or 0 (sigmoid)."""
    z = np.array([[0.0, far - 1.0, far - 1.75, -3.0]], np.float32)
    bias = np.array([0, 5, 4, 0], np.float32)
    n = 1 / (1 + np.exp(float(z[0, 2]) - float(z[0, 1])))
    for score in ("softmax", "sigmoid") if far <= -40.0 else ("softmax",):
        ids, w = X.router(z, 2, bias, score, scale=2.5)
        assert ids.tolist() == [[1, 2]]
        assert np.all(np.abs(w[0] - [2.5 * n, 2.5 * (1 - n)]) <= 2.5 * 2.0 ** -40)


def test_oracle_sigmoid_gradient_of_large_logits():
    """s (1 - s) = 1 / (2 cosh(z / 2))^2."""
    z = np.array([[-60.0, -20, -1, 0, 1, 20, 30, 36, 37, 40, 60, 100, 700]])
    ids = np.arange(z.shape[1])[None]
    got = X.router_bwd(z, ids, np.ones(ids.shape), "sigmoid", False, 1.0)
    want = 1 / (2 * np.cosh(z / 2)) ** 2
    assert np.all(np.abs(got - want) <= want * 2.0 ** -40)


@pytest.mark.parametrize("gap", [0.0, 20.0, 37.0, 60.0, 700.0])
def test_oracle_renormalized_gradient_of_a_dominant_expert(gap):
    """Two slots: n_0 n_1 (g_0 - g_1), of either sign."""
    z, ids, g = np.array([[0.5 - gap, 0.5, -1.0]]), np.array([[0, 1]]), np.array([[1.0, -2.0]])
    want = 3 / (2 * np.cosh(gap / 2)) ** 2
    assert np.all(np.abs(X.router_bwd(z, ids, g, "softmax", True, 1.0)[0] - [want, -want, 0]) <= want * 2.0 ** -40)
    r = np.exp(0.5 - gap) / (1 + np.exp(0.5 - gap)) * (1 + np.exp(-0.5))  # s_0 / s_1
    want = 3 * r / (1 + r) ** 2 * np.array([1 / (1 + np.exp(0.5 - gap)), -1 / (1 + np.exp(0.5)), 0])
    assert np.all(np.abs(X.router_bwd(z, ids, g, "sigmoid", True, 1.0)[0] - want) <= np.abs(want) * 2.0 ** -40)
    for score in ("softmax", "sigmoid"):
        assert not X.router_bwd(z, ids[:, :1], g[:, :1], score, True, 1.0).any()


@pytest.mark.parametrize("gap", [0.0, 20.0, 37.0, 60.0, 700.0])
def test_oracle_softmax_gradient_of_a_dominant_expert(gap):
    """Two experts: s_0 (1 - s_0) = 1 / (2 cosh(gap / 2))^2, of either sign."""
    got = X.router_bwd(np.array([[0.0, -gap]]), np.array([[0]]), np.array([[1.0]]), "softmax", False, 1.0)[0]
    want = 1 / (2 * np.cosh(gap / 2)) ** 2
    assert np.all(np.abs(got - [want, -want]) <= want * 2.0 ** -40)


def test_scores_reject_bad_args(lib):
    f = lib.moe_router_scores

    def call(logits=FAKE, dtype=1, T=4, E=384, k=6, bias=None, score=1, n_group=8, topk_group=4, group_top=2, scale=1.0,
             ids=FAKE, w=FAKE):
        return f(logits, dtype, T, E, k, bias, score, n_group, topk_group, group_top, 1, scale, ids, w, None)

    assert call(dtype=2) == -2 and call(dtype=-1) == -2
    assert call(score=2) == -2
    assert call(T=-1) == -2 and call(k=0) == -2 and call(k=65) == -2
    assert call(E=1032) == -2 and call(E=0) == -2
    assert call(n_group=7) == -2                  # does not divide 384
    assert call(n_group=0) == -2 and call(n_group=96, topk_group=1) == -2
    assert call(topk_group=9) == -2 and call(topk_group=0) == -2
    assert call(E=16, n_group=8, topk_group=2, k=5) == -2  # more than the kept groups hold
    assert call(group_top=3) == -2 and call(group_top=0) == -2
    assert call(scale=float("inf")) == -2 and call(scale=float("nan")) == -2
    assert call(logits=None) == -1 and call(ids=None) == -1 and call(w=None) == -1
    b = lib.moe_router_scores_bwd
    assert b(FAKE, 3, 4, 384, 6, 1, 1, 1.0, FAKE, FAKE, FAKE, None) == -2
    assert b(FAKE, 1, 4, 384, 6, 5, 1, 1.0, FAKE, FAKE, FAKE, None) == -2
    assert b(FAKE, 1, 4, 384, 0, 1, 1, 1.0, FAKE, FAKE, FAKE, None) == -2
    assert b(FAKE, 1, 4, 384, 6, 1, 1, float("nan"), FAKE, FAKE, FAKE, None) == -2
    assert b(FAKE, 1, 4, 384, 6, 1, 1, 1.0, FAKE, None, FAKE, None) == -1
    assert b(FAKE, 1, 4, 384, 6, 1, 1, 1.0, FAKE, FAKE, None, None) == -1
    r = lib.moe_route_scores
    ok = [FAKE] * 6
    assert r(FAKE, 1, 4, 384, 6, None, 1, 7, 1, 2, 1, 1.0, 0, 48, 1, 0, FAKE, FAKE, *ok, FAKE, 4096, None) == -2
    assert r(FAKE, 1, 4, 384, 6, None, 1, 8, 4, 2, 1, 1.0, 0, 0, 1, 0, FAKE, FAKE, *ok, FAKE, 4096, None) == -2
    assert r(FAKE, 1, 4, 384, 6, None, 1, 8, 4, 2, 1, 1.0, 0, 48, 1, 0, FAKE, FAKE, *ok, FAKE, 4, None) == -3
    assert r(None, 1, 4, 384, 6, None, 1, 8, 4, 2, 1, 1.0, 0, 48, 1, 0, FAKE, FAKE, *ok, FAKE, 4096, None) == -1


def test_scores_reject_misaligned_pointers(lib):
    """Every array at its elements' alignment: 4 bytes, 2 for bf16 logits."""
    def fwd(logits=FAKE, dtype=1, bias=FAKE, ids=FAKE, w=FAKE):
        return lib.moe_router_scores(logits, dtype, 4, 384, 6, bias, 1, 8, 4, 2, 1, 1.0, ids, w, None)

    def route(logits=FAKE, dtype=1, bias=FAKE, ids=FAKE, w=FAKE):
        return lib.moe_route_scores(logits, dtype, 4, 384, 6, bias, 1, 8, 4, 2, 1, 1.0, 0, 48, 1, 0, ids, w, *[FAKE] * 6,
                                    FAKE, 4096, None)

    def bwd(logits=FAKE, dtype=1, ids=FAKE, grad=FAKE, out=FAKE):
        return lib.moe_router_scores_bwd(logits, dtype, 4, 384, 6, 1, 1, 1.0, ids, grad, out, None)

    for f in (fwd, route):
        for name in ("logits", "bias", "ids", "w"):
            assert f(**{name: ODD}) == -6 and f(dtype=0, **{name: FAKE + 1}) == -6
    for name in ("logits", "ids", "grad", "out"):
        assert bwd(**{name: ODD}) == -6 and bwd(dtype=0, **{name: FAKE + 1}) == -6
    # bf16 logits at 2 bytes: the next check is the first to refuse
    assert lib.moe_router_scores(ODD, 0, 4, 384, 6, None, 1, 8, 4, 2, 1, 1.0, FAKE, ODD, None) == -6
    assert lib.moe_route_scores(ODD, 0, 4, 384, 6, None, 1, 8, 4, 2, 1, 1.0, 0, 0, 1, 0, FAKE, FAKE, *[FAKE] * 6, FAKE,
                                4096, None) == -2


def test_mxfp4_reject_bad_args(lib):
    q, d = lib.mxfp4_quantize_act, lib.mxfp4_dequantize
    assert q(FAKE, 0, 4, 48, None, FAKE, FAKE, None) == -2     # cols % 32
    assert q(FAKE, 0, 4, 0, None, FAKE, FAKE, None) == -2
    assert q(FAKE, 0, -1, 64, None, FAKE, FAKE, None) == -2
    assert q(FAKE, 2, 4, 64, None, FAKE, FAKE, None) == -2     # dtype
    assert q(FAKE, 0, 1 << 40, 64, None, FAKE, FAKE, None) == -2
    assert q(None, 0, 4, 64, None, FAKE, FAKE, None) == -1
    assert q(ODD, 0, 4, 64, None, FAKE, FAKE, None) == -6
    assert q(FAKE, 0, 4, 64, None, ODD, FAKE, None) == -6
    assert d(FAKE, FAKE, 4, 40, FAKE, None) == -2
    assert d(FAKE, None, 4, 64, FAKE, None) == -1
    assert d(FAKE, FAKE, 4, 64, ODD, None) == -6
    for lin, n in ((lib.mxfp4_linear, 64), (lib.mxfp4_linear_gate_up_silu, 64)):
        assert lin(FAKE, FAKE, 4, 192, FAKE, FAKE, n, FAKE, None) == -2   # K % 128
        assert lin(FAKE, FAKE, 4, 0, FAKE, FAKE, n, FAKE, None) == -2
        assert lin(FAKE, FAKE, 4, 256, FAKE, FAKE, 24, FAKE, None) == -2  # N % 16
        assert lin(FAKE, FAKE, 4, 256, FAKE, FAKE, 0, FAKE, None) == -2
        assert lin(FAKE, FAKE, 1 << 31, 256, FAKE, FAKE, n, FAKE, None) == -2
        assert lin(FAKE, FAKE, -1, 256, FAKE, FAKE, n, FAKE, None) == -2
        assert lin(FAKE, FAKE, 4, 256, FAKE, None, n, FAKE, None) == -1
        assert lin(FAKE, FAKE, 4, 256, FAKE, FAKE, n, None, None) == -1
        assert lin(FAKE, ODD, 4, 256, FAKE, FAKE, n, FAKE, None) == -6
        assert lin(FAKE, FAKE, 4, 256, FAKE, FAKE, n, ODD, None) == -6
        assert lin(FAKE, FAKE, 1 << 30, 256, FAKE, FAKE, n, FAKE, None) == -2     # 2^37 bytes of A
        assert lin(FAKE, FAKE, 4, 1 << 17, FAKE, FAKE, 1 << 20, FAKE, None) == -2  # 2^36 of W
    assert q(FAKE, 0, 1 << 31, 64, None, FAKE, FAKE, None) == -2 and d(FAKE, FAKE, 1 << 31, 64, FAKE, None) == -2
    l1, l2 = lib.moe_grouped_gemm_l1_silu_mxfp4, lib.moe_grouped_gemm_l2_mxfp4
    a7, a6 = [FAKE] * 7, [FAKE] * 6
    assert l1(*a7, 8, 192, 128, 64, 0, FAKE, None) == -2       # H % 128
    assert l1(*a7, 8, 256, 120, 64, 0, FAKE, None) == -2       # I % 16
    assert l1(*a7, 0, 256, 128, 64, 0, FAKE, None) == -2 and l1(*a7, 1025, 256, 128, 64, 0, FAKE, None) == -2
    assert l1(*a7, 8, 256, 128, -1, 0, FAKE, None) == -2 and l1(*a7, 8, 256, 128, 64, -1, FAKE, None) == -2
    assert l1(*a7, 8, 1 << 17, 1 << 19, 64, 0, FAKE, None) == -2  # 2^36 bytes an expert
    assert l2(*a6, 8, 1 << 20, 1 << 17, 64, 0, FAKE, None) == -2
    assert l1(*a7, 8, 256, 128, 1 << 30, 0, FAKE, None) == -2
    assert l1(*a7, 8, 256, 128, 64, 0, None, None) == -1
    assert l1(FAKE, FAKE, None, *[FAKE] * 4, 8, 256, 128, 64, 0, FAKE, None) == -1
    assert l1(*a7, 8, 256, 128, 64, 0, ODD, None) == -6
    assert l2(*a6, 8, 256, 96, 64, 0, FAKE, None) == -2        # I % 128
    assert l2(*a6, 8, 248, 128, 64, 0, FAKE, None) == -2
    assert l2(FAKE, FAKE, FAKE, None, FAKE, FAKE, 8, 256, 128, 64, 0, FAKE, None) == -1
    assert l2(*a6, 8, 256, 128, 64, 0, None, None) == -1


def test_mxfp4_products_refuse_reductions_of_2_30(lib):
    """A lane's 32-bit offset of 7 weight rows of K / 2 bytes, and K rounded up to a stage, hold K below 2^30.
    (Every operand here is below 2^36 bytes: K alone refuses the call.)"""
    for K in (1 << 30, 1227133568, 2 ** 31 - 512, 2 ** 31 - 384, 2 ** 31 - 256, 2 ** 31 - 128):
        assert lib.mxfp4_linear(FAKE, FAKE, 1, K, FAKE, FAKE, 16, FAKE, None) == -2
        assert lib.mxfp4_linear_gate_up_silu(FAKE, FAKE, 1, K, FAKE, FAKE, 16, FAKE, None) == -2
        assert lib.moe_grouped_gemm_l1_silu_mxfp4(*[FAKE] * 7, 8, K, 16, 1, 0, FAKE, None) == -2
        assert lib.moe_grouped_gemm_l2_mxfp4(*[FAKE] * 6, 8, 16, K, 1, 0, FAKE, None) == -2
    K = (1 << 30) - 128  # accepted: the next check is the first to refuse
    assert 7 * (K // 2) + 16 * 8 < 2 ** 32 and K + 511 < 2 ** 31
    assert lib.mxfp4_linear(FAKE, FAKE, 1, K, FAKE, None, 16, FAKE, None) == -1


def test_binding_refuses_wrong_tensors():
    """The binding's own checks come before the library: type, shape, device."""
    z = torch.zeros(4, 8)
    ids, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(mm.MegaMoEError, match="GPU"):
        mm.moe_router_scores(z, 2, ids, w)
    with pytest.raises(mm.MegaMoEError, match="score"):
        mm.moe_router_scores(z, 2, ids, w, score="tanh")
    with pytest.raises(mm.MegaMoEError, match="logits is"):
        mm.moe_router_scores(z.double(), 2, ids, w)
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    with pytest.raises(mm.MegaMoEError, match="GPU"):
        mm.mxfp4_quantize_act(z.bfloat16(), u8(4, 4), u8(4, 1))
    with pytest.raises(mm.MegaMoEError, match="x is"):
        mm.mxfp4_quantize_act(z.half(), u8(4, 4), u8(4, 1))


def test_binding_refuses_more_token_codes_than_offsets_reach():
    """x of 2^36 bytes of codes beside an output of a few rows (meta tensors: nothing is allocated)."""
    def meta(*s, d=torch.uint8):
        return torch.empty(*s, dtype=d, device="meta")

    def call(T, H=256):
        mm.moe_grouped_gemm_l1_silu_mxfp4(meta(T, H // 2), meta(T, H // 32), meta(64, d=torch.int32), meta(5, d=torch.int32),
                                          meta(4, d=torch.int32), meta(4, 256, H // 2), meta(4, 256, H // 32),
                                          meta(64, 128, d=torch.bfloat16))
    with pytest.raises(mm.MegaMoEError, match="2\\^36"):
        call(1 << 29)
    with pytest.raises(mm.MegaMoEError, match="GPU"):
        call((1 << 29) - 1)


def test_mx_layer_weight_shapes():
    w = layer.MXMoEWeights.empty(4, 256, 128, device="cpu")
    assert (w.num_experts, w.hidden, w.intermediate) == (4, 256, 128)
    assert w.w13_scales.shape == (4, 256, 8) and w.w2_scales.shape == (4, 256, 4)
    assert w.nbytes_expert() == 256 * 256 // 2 + 256 * 8 + 256 * 128 // 2 + 256 * 4
