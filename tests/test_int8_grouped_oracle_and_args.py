"""The oracle of the int8 and 16-bit expert operators against closed forms and differences, and the refusals of
their entry points and binding (no GPU)."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_top_amd import layer, megamoe as mm
from oracle import int8_oracle as Q

FAKE, ODD = 0x10000, 0x10000 + 2  # never dereferenced: every check comes first


@pytest.fixture(scope="module")
def lib():
    return mm.lib()


# ---- oracle --------------------------------------------------------------------------------------

def test_oracle_quantizer_ties_extremes_and_zeros():
    # amax 127 * 2: a quotient is x / 2, and odd x are borders
    c, s = Q.quantize(np.array([[254.0, 1, 3, 5, -1, -3, 253, 0], [0] * 8, [1e-40, -1e-40, 5e-41, 0, 0, 0, 0, 0]]))
    assert c[0].tolist() == [127, 0, 2, 2, 0, -2, 126, 0] and s[0] == 2.0
    assert not c[1].any() and s[1] == 0
    assert c[2].tolist()[:2] == [127, -127]
    c, s = Q.quantize(np.array([[1.0, np.inf], [np.nan, 2.0], [-3.0, 3.0]]))
    assert not c[:2].any() and np.isnan(s[:2]).all() and c[2].tolist() == [-127, 127]


def test_oracle_quantizer_is_within_half_a_step():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((50, 96)).astype(np.float32).astype(np.float64)
    c, s = Q.quantize(x)
    step = np.abs(x).max(1, keepdims=True) / 127
    assert np.all(np.abs(c * step - x) <= step * (0.5 + 1e-9)) and np.abs(c.astype(int)).max() == 127
    assert np.array_equal(Q.dequantize(c, s), c.astype(np.float32) * s[:, None])


def test_oracle_product_counts_whole_numbers():
    a, w = np.full((2, 5), -128, np.int8), np.full((3, 5), 127, np.int8)
    got = Q.product(a, np.array([1.0, 0.5], np.float32), w, np.array([1.0, 2.0, 4.0], np.float32))
    assert np.array_equal(got, -81280.0 * np.array([[1], [0.5]]) * [1, 2, 4])


def test_oracle_gradients_agree_with_differences():
    rng = np.random.default_rng(2)
    counts, offsets = np.array([3, 0, 2]), np.array([0, 4, 4])
    tokens = np.array([1, 0, 3, -1, 2, 1])
    x, w = rng.standard_normal((4, 5)), rng.standard_normal((3, 6, 5))
    dy = rng.standard_normal((6, 6))

    def loss(x, w):
        return sum((dy[r] * y).sum() for r, y, _ in Q.grouped(x, w, offsets, counts, tokens).values())
    gx, gw = np.zeros_like(x), np.zeros_like(w)
    for e, (r, dx, _, dw, _) in Q.grouped_grads(x, w, dy, offsets, counts, tokens).items():
        np.add.at(gx, tokens[r], dx)
        gw[e] = dw
    for t, g in ((x, gx), (w, gw)):
        for i in np.ndindex(*t.shape):  # the loss is linear in each entry: a difference is exact up to rounding
            d = []
            for step in (0.5, -0.5):
                t[i] += step
                d.append(loss(x, w))
                t[i] -= step
            assert abs(d[0] - d[1] - g[i]) < 1e-11


# ---- refusals ------------------------------------------------------------------------------------

def test_int8_quantizer_refuses_bad_args(lib):
    q, d = lib.int8_quantize_act, lib.int8_dequantize
    assert q(FAKE, 0, 4, 40, None, FAKE, FAKE, None) == -2     # cols % 16
    assert q(FAKE, 0, 4, 0, None, FAKE, FAKE, None) == -2 and q(FAKE, 0, -1, 64, None, FAKE, FAKE, None) == -2
    assert q(FAKE, 3, 4, 64, None, FAKE, FAKE, None) == -2 and q(FAKE, -1, 4, 64, None, FAKE, FAKE, None) == -2
    assert q(FAKE, 0, 1, 1 << 30, None, FAKE, FAKE, None) == -2
    assert q(FAKE, 0, 1 << 31, 64, None, FAKE, FAKE, None) == -2  # 2^37 elements
    assert q(None, 0, 4, 64, None, FAKE, FAKE, None) == -1 and q(FAKE, 0, 4, 64, None, None, FAKE, None) == -1
    assert q(FAKE, 0, 4, 64, None, FAKE, None, None) == -1
    assert q(FAKE + 8, 0, 4, 64, None, FAKE, FAKE, None) == -6 and q(FAKE, 0, 4, 64, None, FAKE + 8, FAKE, None) == -6
    assert q(FAKE, 0, 4, 64, None, FAKE, ODD, None) == -6 and q(FAKE, 0, 4, 64, ODD, FAKE, FAKE, None) == -6
    assert d(FAKE, FAKE, 4, 40, 0, FAKE, None) == -2 and d(FAKE, FAKE, 4, 64, 3, FAKE, None) == -2
    assert d(FAKE, FAKE, -1, 64, 0, FAKE, None) == -2 and d(FAKE, FAKE, 1 << 31, 64, 0, FAKE, None) == -2
    assert d(None, FAKE, 4, 64, 0, FAKE, None) == -1 and d(FAKE, None, 4, 64, 0, FAKE, None) == -1
    assert d(FAKE, FAKE, 4, 64, 0, None, None) == -1
    assert d(FAKE + 8, FAKE, 4, 64, 0, FAKE, None) == -6 and d(FAKE, ODD, 4, 64, 0, FAKE, None) == -6
    assert d(FAKE, FAKE, 4, 64, 0, FAKE + 8, None) == -6


@pytest.mark.parametrize("cols", [16, 48, 7168, (1 << 30) - 16])
def test_int8_quantizer_takes_all_sizes_below_its_limit(lib, cols):
    """The most rows that keep a tensor below 2^37 elements, and one more.  Without pointers the next check refuses."""
    most = ((1 << 37) - 1) // cols
    for rows, rc in ((most, -1), (most + 1, -2)):
        assert lib.int8_quantize_act(None, 0, rows, cols, None, FAKE, FAKE, None) == rc
        assert lib.int8_dequantize(None, FAKE, rows, cols, 0, FAKE, None) == rc


@pytest.mark.parametrize("name", ["int8_linear", "int8_linear_gate_up_silu"])
def test_int8_dense_products_refuse_bad_args(lib, name):
    def call(a=FAKE, sa=FAKE, M=4, K=256, w=FAKE, sw=FAKE, N=64, dtype=0, out=FAKE):
        return getattr(lib, name)(a, sa, M, K, w, sw, N, dtype, out, None)
    for bad in (dict(K=24), dict(K=0), dict(K=8), dict(K=1 << 17), dict(N=12), dict(N=0), dict(N=1 << 22), dict(M=-1),
                dict(M=1 << 31), dict(dtype=1), dict(dtype=3), dict(dtype=-1), dict(M=1 << 20, K=1 << 16)):
        assert call(**bad) == -2, bad
    for arg in ("a", "sa", "w", "sw", "out"):
        assert call(**{arg: None}) == -1
        assert call(**{arg: ODD}) == -6
    for arg in ("a", "w", "out"):
        assert call(**{arg: FAKE + 8}) == -6
    assert call(K=(1 << 17) - 16, sw=None) == -1  # the longest: the next check is the first to refuse
    assert 2 ** 14 * ((1 << 17) - 16) < 2 ** 31


def test_int8_expert_products_refuse_bad_args(lib):
    def l1(x=FAKE, xs=FAKE, rt=FAKE, po=FAKE, ct=FAKE, w=FAKE, ws=FAKE, E=8, H=256, I=128, M=64, bound=0, h=FAKE):
        return lib.moe_grouped_gemm_l1_silu_int8(x, xs, rt, po, ct, w, ws, E, H, I, M, bound, h, None)

    def l2(x=FAKE, xs=FAKE, po=FAKE, ct=FAKE, w=FAKE, ws=FAKE, E=8, H=128, I=256, M=64, bound=0, h=FAKE):
        return lib.moe_grouped_gemm_l2_int8(x, xs, po, ct, w, ws, E, H, I, M, bound, h, None)
    for f, red, out in ((l1, "H", "I"), (l2, "I", "H")):
        for bad in ({red: 40}, {red: 1 << 17}, {out: 4}, {out: 20}, {out: 1 << 22}, dict(E=0), dict(E=1025), dict(M=-1),
                    dict(M=1 << 31), dict(bound=-1), {"M": 1 << 28}):
            assert f(**bad) == -2, bad
        for arg in ("x", "xs", "po", "ct", "w", "ws", "h"):
            assert f(**{arg: None}) == -1 and f(**{arg: ODD}) == -6
    assert l1(rt=None) == -1 and l1(rt=ODD) == -6


def test_grouped_products_refuse_bad_args(lib):
    def fwd(x=FAKE, dtype=0, rt=None, po=FAKE, ct=FAKE, w=FAKE, E=8, K=256, N=128, M=64, bound=0, out=FAKE):
        return lib.moe_grouped_gemm(x, dtype, rt, po, ct, w, E, K, N, M, bound, out, None)

    def dgrad(x=FAKE, dtype=0, po=FAKE, ct=FAKE, w=FAKE, E=8, K=256, N=128, M=64, out=FAKE):
        return lib.moe_grouped_gemm_dgrad(x, dtype, po, ct, w, E, K, N, M, out, None)

    def wgrad(x=FAKE, w=FAKE, dtype=0, rt=None, po=FAKE, ct=FAKE, E=8, K=256, N=128, M=64, dwt=0, acc=0, out=FAKE):
        return lib.moe_grouped_gemm_wgrad(x, w, dtype, rt, po, ct, E, K, N, M, dwt, acc, out, None)
    for f in (fwd, dgrad, wgrad):
        for bad in (dict(K=4), dict(K=252), dict(K=0), dict(K=1 << 22), dict(N=4), dict(N=132), dict(N=1 << 22), dict(E=0),
                    dict(E=1025), dict(M=-1), dict(M=1 << 31), dict(dtype=1), dict(dtype=3), dict(dtype=-1)):
            assert f(**bad) == -2, (f.__name__, bad)
        for arg in ("x", "po", "ct", "w", "out"):
            assert f(**{arg: None}) == -1 and f(**{arg: ODD}) == -6, (f.__name__, arg)
        for arg in ("x", "w", "out"):
            assert f(**{arg: FAKE + 8}) == -6
    assert fwd(bound=-1) == -2
    assert fwd(rt=ODD) == -6 and wgrad(rt=ODD) == -6
    assert wgrad(dtype=0, dwt=2) == -2 and wgrad(dtype=2, dwt=0) == -2 and wgrad(dwt=4) == -2
    # rows of 2^36 bytes and more
    assert fwd(K=1 << 16, M=1 << 19) == -2 and dgrad(N=1 << 16, M=1 << 19) == -2
    assert wgrad(K=1 << 16, M=1 << 19) == -2 and wgrad(N=1 << 16, M=1 << 19) == -2


def test_binding_refuses_wrong_tensors():
    i8, i32 = (lambda *s, d=d: torch.zeros(*s, dtype=d) for d in (torch.int8, torch.int32))
    f32, bf = torch.zeros, lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    with pytest.raises(mm.MegaMoEError, match="GPU"):
        mm.int8_quantize_act(bf(4, 32), i8(4, 32), f32(4))
    with pytest.raises(mm.MegaMoEError, match="x is"):
        mm.int8_quantize_act(bf(4, 32).double(), i8(4, 32), f32(4))
    meta = lambda *s, d=torch.bfloat16: torch.empty(*s, dtype=d, device="meta")  # noqa: E731
    with pytest.raises(mm.MegaMoEError, match="GPU"):
        mm.int8_linear(i8(4, 32), f32(4), i8(8, 32), f32(8), bf(4, 8))
    with pytest.raises(mm.MegaMoEError, match="GPU"):
        mm.moe_grouped_gemm(bf(4, 32), bf(2, 8, 32), i32(3), i32(2), bf(4, 8))
    with pytest.raises(mm.MegaMoEError, match="x is"):
        mm.moe_grouped_gemm(f32(4, 32), bf(2, 8, 32), i32(3), i32(2), bf(4, 8))
    with pytest.raises(mm.MegaMoEError, match="GPU"):
        mm.moe_grouped_gemm_dgrad(bf(4, 8), bf(2, 8, 32), i32(3), i32(2), bf(4, 32))
    with pytest.raises(mm.MegaMoEError, match="GPU"):
        mm.moe_grouped_gemm_wgrad(bf(4, 8), bf(4, 32), i32(3), i32(2), bf(2, 8, 32))
    # a gathered tensor of 2^36 bytes beside an output of a few rows (meta tensors: nothing is allocated)
    tables = meta(5, d=torch.int32), meta(4, d=torch.int32)
    rt, T = meta(64, d=torch.int32), 1 << 27
    for rows, match in ((T, "2\\^36"), (T - 1, "GPU")):
        with pytest.raises(mm.MegaMoEError, match=match):
            mm.moe_grouped_gemm(meta(rows, 256), meta(4, 128, 256), *tables, meta(64, 128), row_token=rt)
        with pytest.raises(mm.MegaMoEError, match=match):
            mm.moe_grouped_gemm_wgrad(meta(64, 128), meta(rows, 256), *tables, meta(4, 128, 256), row_token=rt)
        with pytest.raises(mm.MegaMoEError, match=match):
            mm.moe_grouped_gemm_l1_silu_int8(meta(rows, 512, d=torch.int8), meta(rows, d=torch.float32), rt, *tables,
                                             meta(4, 256, 512, d=torch.int8), meta(4, 256, d=torch.float32), meta(64, 128))


def test_int8_layer_weight_shapes():
    w = layer.Int8MoEWeights.empty(4, 256, 128, device="cpu")
    assert (w.num_experts, w.hidden, w.intermediate) == (4, 256, 128)
    assert w.w13_scales.shape == (4, 256) and w.w2_scales.shape == (4, 256)
    assert w.nbytes_expert() == 256 * 256 + 256 * 4 + 256 * 128 + 256 * 4


@pytest.mark.parametrize("other", [torch.float16, torch.float32])
def test_calls_on_bf16_refuse_other_types(other, monkeypatch):
    """The products, their gradients and the decoder write float16 too; a call that knows only bf16 has to refuse it
    (it would take the bits for bf16).  Every other argument is taken as it is here, CPU tensors too: each call ends at
    the refusal."""
    monkeypatch.setattr(mm, "_ptr", lambda t: None if t is None else t.data_ptr())
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    bad = lambda *s: torch.zeros(*s, dtype=other)  # noqa: E731
    i32, u8, f32 = (lambda *s, d=d: torch.zeros(*s, dtype=d) for d in (torch.int32, torch.uint8, torch.float32))
    rows, w, parts = i32(8), f32(4, 2), f32(mm.L1_AMAX_PARTS)
    dense = u8(4, 32), u8(4, 4), f32(1), u8(64, 32), u8(64, 4), f32(1)
    routed = u8(4, 32), u8(4, 4), f32(1)
    w13, w2 = (u8(2, 128, 32), u8(2, 128, 4), f32(2)), (u8(2, 64, 32), u8(2, 64, 4), f32(2))
    tabs = [i32(3)] * 3
    calls = {
        "y_bf16": [lambda: mm.moe_combine(bad(8, 64), rows, w, bf(4, 64)),
                   lambda: mm.moe_combine_shared(bad(8, 64), rows, w, bf(4, 64), bf(4, 64)),
                   lambda: mm.moe_grouped_gemm_l2(*routed, *tabs, *w2, bad(8, 64))],
        "out_bf16": [lambda: mm.moe_combine(bf(8, 64), rows, w, bad(4, 64)),
                     lambda: mm.moe_combine_shared(bf(8, 64), rows, w, bf(4, 64), bad(4, 64)),
                     lambda: mm.nvfp4_linear(*dense, bad(4, 64), u8(64))],
        "y_shared_bf16": [lambda: mm.moe_combine_shared(bf(8, 64), rows, w, bad(4, 64), bf(4, 64))],
        "x_bf16": [lambda: mm.nvfp4_quantize_act(bad(4, 64), u8(4, 32), u8(4, 4), f32(1)),
                   lambda: mm.nvfp4_quantize_act_gs(bad(4, 64), f32(1), u8(4, 32), u8(4, 4)),
                   lambda: layer.quantize_matrix(bad(4, 64), u8(4, 32), u8(4, 4), f32(1))],
        "h_bf16": [lambda: mm.nvfp4_linear_gate_up_silu(*dense, bad(4, 32), parts, u8(64)),
                   lambda: mm.moe_grouped_gemm_l1_silu(*routed, i32(8), *tabs, *w13, bad(8, 64), parts)],
    }
    for name, fs in calls.items():
        for f in fs:
            with pytest.raises(mm.MegaMoEError, match=f"{name} is {other}"):
                f()


def test_combine_refuses_tensors_that_hold_too_little():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    rows, w = torch.zeros(8, dtype=torch.int32), torch.zeros(4, 2)
    for y, r, wt, out, match in ((bf(8, 32), rows, w, bf(4, 64), "y_bf16 has"), (bf(8, 64), rows, w, bf(3, 64), "out_bf16 has"),
                                 (bf(8, 64), rows[:7], w, bf(4, 64), "token_rows 7"), (bf(8, 64), rows.long(), w, bf(4, 64), "int64"),
                                 (bf(8, 64), rows, w.double(), bf(4, 64), "float64"), (bf(8, 64), rows, w, bf(4, 64), "GPU")):
        with pytest.raises(mm.MegaMoEError, match=match):
            mm.moe_combine(y, r, wt, out)
    for sh in (bf(3, 64), bf(4, 32)):
        with pytest.raises(mm.MegaMoEError, match="y_shared_bf16 has"):
            mm.moe_combine_shared(bf(8, 64), rows, w, sh, bf(4, 64))
