"""Scored router and its gradient on the GPU against the float64 oracle.

ids: equal.  Weights: float64 arithmetic and one rounding to float32, so within half a step
(2^-24 relative) of the oracle's, plus 2^-40 for the two sides' float64 exponentials and sums, plus half
of the smallest float32 subnormal.  Gradients: one rounding to the logits' type (2^-24 or 2^-8 relative),
plus 2^-40 times the magnitudes that the formula subtracts."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_top_amd import layer, megamoe as mm
from oracle import mxfp4_oracle as X
from oracle import nvfp4_oracle as O

from gpu_util import DEV, np_i32

pytestmark = pytest.mark.gpu

F32_TINY = 2.0 ** -150


def to_dev(z, dtype):
    t = torch.from_numpy(np.ascontiguousarray(z, np.float32)).to(dtype)
    return t.to(DEV), t.float().numpy()


def run(z, k, bias=None, dtype=torch.float32, **kw):
    zt, zh = to_dev(z, dtype)
    T = zt.shape[0]
    ids = torch.full((T + 1, k), -7, dtype=torch.int32, device=DEV)
    w = torch.full((T + 1, k), -1.0, device=DEV)
    bt = None if bias is None else torch.from_numpy(bias).to(DEV)
    mm.moe_router_scores(zt, k, ids[:T], w[:T], bias=bt, **kw)
    torch.cuda.synchronize()
    assert np.all(np_i32(ids[T:]) == -7) and torch.all(w[T:] == -1.0)
    return np_i32(ids[:T]), w[:T].cpu().numpy(), zh


def check(z, k, bias=None, dtype=torch.float32, **kw):
    ids, w, zh = run(z, k, bias, dtype, **kw)
    ref_ids, ref_w = X.router(zh, k, bias, **kw)
    assert np.array_equal(ids, ref_ids)
    assert np.all(np.abs(w - ref_w) <= np.abs(ref_w) * (2.0 ** -24 + 2.0 ** -40) + F32_TINY)
    return ids, w


CASES = [  # T, E, k, n_group, topk_group, group_top
    (0, 384, 6, 8, 4, 2), (1, 1, 1, 1, 1, 1), (1, 384, 6, 8, 4, 2), (9, 384, 6, 1, 1, 2), (5, 64, 64, 1, 1, 1),
    (3, 1024, 64, 1, 1, 1), (7, 1024, 8, 64, 3, 2), (33, 101, 7, 1, 1, 1), (6, 60, 5, 3, 2, 1), (4, 33, 4, 33, 7, 2),
    (2, 990, 9, 33, 2, 2), (130, 256, 8, 8, 4, 2), (5, 66, 3, 2, 1, 2), (3, 514, 2, 1, 1, 1),
]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k,n_group,topk_group,group_top", CASES)
def test_shapes(T, E, k, n_group, topk_group, group_top, score):
    rng = np.random.default_rng(T * 7 + E + k)
    z = rng.standard_normal((T, E)) * 2
    bias = (rng.standard_normal(E) * 0.2).astype(np.float32)
    kw = dict(score=score, n_group=n_group, topk_group=topk_group, group_top=group_top)
    for dtype in (torch.float32, torch.bfloat16):
        for b in (None, bias):
            for renorm, scale in ((True, 2.5), (False, 1.0)):
                check(z, k, b, dtype, renormalize=renorm, scale=scale, **kw)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_masks_and_extremes(score):
    """-inf and NaN logits and biases (experts that may not be chosen), rows that leave nothing or
    less than k, the lowest and the largest floats, infinities, exact ties of experts and groups."""
    rng = np.random.default_rng(11)
    E, k, lowest = 48, 6, float(np.finfo(np.float32).min)
    z = rng.standard_normal((16, E)).astype(np.float32)
    z[0] = -np.inf
    z[1] = np.nan
    z[2, 3:] = -np.inf
    z[3, ::2] = -np.inf
    z[4] = lowest
    z[5, 1:] = lowest
    z[6] = 0.0
    z[7, 7], z[7, 30] = np.inf, np.inf
    z[8, :24] = -np.inf            # half of the groups without an expert
    z[9, [5, 9, 13, 17]] = np.nan
    z[10] = np.round(z[10])        # many ties
    z[11] = 1e30
    z[12, 0] = 800.0
    z[13] = -1e4                   # every sigmoid underflows
    z[14, 8:] = -np.inf            # one group of eight is left
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
    bias[[2, 40]] = -np.inf
    bias[41] = np.nan
    bias[43] = np.inf
    for groups in (dict(), dict(n_group=6, topk_group=2, group_top=2), dict(n_group=6, topk_group=3, group_top=1)):
        for b in (None, bias, np.zeros(E, np.float32)):
            for renorm in (True, False):
                check(z, k, b, score=score, renormalize=renorm, **groups)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("group_top", [1, 2])
def test_groups_of_choices_at_the_ends_of_float32(score, group_top):
    """Sums of a group's choices that overflow to either infinity, beside groups with no available expert
    (before them, after them and between them) and groups with a single one."""
    rng = np.random.default_rng(17)
    E, low = 48, np.float32(-3e38)
    z = rng.standard_normal((12, E)).astype(np.float32)
    for t in range(12):
        z[t, 8 * (t % 6):8 * (t % 6) + 8] = -np.inf
        z[t, 8 * (t // 3):8 * (t // 3) + (8 if t % 2 else 7)] = -np.inf
    for bias in (np.full(E, low), np.full(E, -low), np.where(np.arange(E) % 16 < 8, low, np.float32(-1e-3)),
                 np.where(np.arange(E) % 8 < 7, low, np.float32(0)), np.full(E, np.finfo(np.float32).min)):
        for topk_group in (1, 2, 4):
            check(z, 5, bias.astype(np.float32), score=score, n_group=6, topk_group=topk_group, group_top=group_top)


def test_large_batch_matches_oracle_on_samples_and_is_repeatable():
    rng = np.random.default_rng(5)
    z = rng.standard_normal((8192, 384)).astype(np.float32)
    bias = (rng.standard_normal(384) * 0.1).astype(np.float32)
    kw = dict(score="sigmoid", n_group=8, topk_group=4, group_top=2, renormalize=True, scale=2.5)
    ids, w, _ = run(z, 6, bias, **kw)
    again = run(z, 6, bias, **kw)
    assert np.array_equal(ids, again[0]) and np.array_equal(w, again[1])
    rows = rng.choice(8192, 200, replace=False)
    ref_ids, ref_w = X.router(z[rows], 6, bias, **kw)
    assert np.array_equal(ids[rows], ref_ids)
    assert np.all(np.abs(w[rows] - ref_w) <= ref_w * (2.0 ** -24 + 2.0 ** -40))


def test_softmax_without_options_matches_the_plain_router():
    rng = np.random.default_rng(6)
    z = (rng.standard_normal((300, 384)) * 2).astype(np.float32)
    ids, w, _ = run(z, 6, score="softmax", renormalize=False)
    zt = torch.from_numpy(z).to(DEV)
    ids2, w2 = torch.empty(300, 6, dtype=torch.int32, device=DEV), torch.empty(300, 6, device=DEV)
    mm.moe_router_topk(zt, 6, ids2, w2)
    assert np.array_equal(ids, np_i32(ids2))
    assert np.all(np.abs(w - w2.cpu().numpy()) <= w * 2.0 ** -23)  # half a step each


# ---- gradient ------------------------------------------------------------------------------------

def run_bwd(z, ids, grad, dtype=torch.float32, **kw):
    zt, zh = to_dev(z, dtype)
    out = torch.full_like(zt, 3.0)
    mm.moe_router_scores_bwd(zt, torch.from_numpy(ids).to(DEV), torch.from_numpy(grad).to(DEV), out, **kw)
    torch.cuda.synchronize()
    return out, zh, zt


def check_bwd(z, ids, grad, dtype=torch.float32, **kw):
    out, zh, zt = run_bwd(z, ids, grad, dtype, **kw)
    got = out.float().cpu().numpy().astype(np.float64)
    ref = X.router_bwd(zh, ids, grad, **kw)
    half = 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8
    tiny = F32_TINY if dtype == torch.float32 else 2.0 ** -134
    # what is subtracted: at most 2 * scale * k * max|grad| (times a score of at most 1, over S)
    inside = (ids >= 0) & (ids < zh.shape[1])
    s = np.take_along_axis(X.scores(zh, kw["score"]), np.where(inside, ids, 0), 1) * inside
    S = s.sum(1, keepdims=True) if kw["renormalize"] else np.ones((len(z), 1))
    size = 2 * abs(kw["scale"]) * ids.shape[1] * np.abs(grad).max(initial=0) / np.where(S > 0, S, 1)
    assert np.all(np.abs(got - ref) <= np.abs(ref) * half + size * 2.0 ** -40 + tiny)
    return out, zt


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,E,k", [(0, 384, 6), (1, 1, 1), (1, 384, 6), (33, 101, 7), (5, 64, 64), (3, 1024, 64),
                                   (130, 130, 8), (9, 1000, 3)])
def test_gradient(T, E, k, score, renormalize):
    rng = np.random.default_rng(T + E + k)
    z = rng.standard_normal((T, E)) * 2
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32) if T else np.zeros((0, k), np.int32)
    grad = rng.standard_normal((T, k)).astype(np.float32)
    for dtype in (torch.float32, torch.bfloat16):
        for scale in (1.0, 2.5):
            check_bwd(z, ids, grad, dtype, score=score, renormalize=renormalize, scale=scale)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient_empty_slots_repeats_and_masks(score, renormalize):
    """Slots without an expert (-1 and beyond the range), an expert named twice, masked logits, rows
    with nothing to give (every score zero, no slot)."""
    rng = np.random.default_rng(2)
    z = rng.standard_normal((8, 40)).astype(np.float32)
    ids = np.stack([rng.permutation(40)[:5] for _ in range(8)]).astype(np.int32)
    grad = rng.standard_normal((8, 5)).astype(np.float32)
    ids[0, 2:] = -1
    ids[1] = -1
    ids[2, 1] = ids[2, 3]
    ids[3, 0], ids[3, 4] = 40, 2 ** 31 - 1
    z[4, ids[4, 0]] = -np.inf
    z[5] = -np.inf
    z[6] = np.nan
    z[7] = -1e4
    check_bwd(z, ids, grad, score=score, renormalize=renormalize, scale=2.5)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_gradient_matches_differences_of_the_forward(score):
    """Central differences of the kernel's own weights.  A weight (at most 2.5) is off by 2^-24 of itself,
    so a difference over 2h = 2^-7 by 5 * 2^-24 * 6 / 2^-7 at most; the third derivative adds h^2 / 6
    times at most 6 * 2.5."""
    rng = np.random.default_rng(8)
    z = rng.standard_normal((4, 32)).astype(np.float32)
    kw = dict(score=score, renormalize=True, scale=2.5)
    ids, _, _ = run(z, 6, n_group=4, topk_group=4, **kw)
    grad = rng.uniform(-1, 1, (4, 6)).astype(np.float32)
    got = run_bwd(z, ids, grad, **kw)[0].cpu().numpy()
    h = 2.0 ** -8
    bias = np.full((4, 32), 0, np.float32)
    for e in range(32):
        both = []
        for sign in (1, -1):
            zz = z.copy()
            zz[:, e] += np.float32(sign * h)
            # keep the choice: rows are run one at a time with a bias that forces their ids
            rows = []
            for t in range(4):
                b = bias[t].copy()
                b[ids[t]] = 100.0 - np.arange(6)
                i2, w2, _ = run(zz[t:t + 1], 6, b, **kw)
                assert np.array_equal(i2[0], ids[t])
                rows.append(float((w2[0].astype(np.float64) * grad[t]).sum()))
            both.append(np.array(rows))
        step = ((z[:, e] + np.float32(h)).astype(np.float64) - (z[:, e] - np.float32(h)).astype(np.float64))
        diff = (both[0] - both[1]) / step
        assert np.all(np.abs(diff - got[:, e]) <= 30 * 2.0 ** -24 / 2.0 ** -7 + h * h / 6 * 15)


def test_gradient_in_place():
    """grad_logits may be the logits' own memory."""
    rng = np.random.default_rng(9)
    z = rng.standard_normal((70, 384)).astype(np.float32)
    ids = np.stack([rng.permutation(384)[:6] for _ in range(70)]).astype(np.int32)
    grad = rng.standard_normal((70, 6)).astype(np.float32)
    for score in ("sigmoid", "softmax"):
        kw = dict(score=score, renormalize=True, scale=2.5)
        want = run_bwd(z, ids, grad, **kw)[0]
        zt = torch.from_numpy(z).to(DEV)
        mm.moe_router_scores_bwd(zt, torch.from_numpy(ids).to(DEV), torch.from_numpy(grad).to(DEV), zt, **kw)
        torch.cuda.synchronize()
        assert torch.equal(zt, want)


@pytest.mark.parametrize("T,E,k,dtype", [(2 ** 26 + 3, 2, 1, torch.bfloat16), (2 ** 22 + 3, 1024, 8, torch.float32)])
def test_more_tokens_than_a_grid_and_logits_past_32_bits(T, E, k, dtype):
    """Every row is one of 1009 rows, so the expected output is a table's."""
    gen = torch.Generator(device=DEV).manual_seed(3)
    few = torch.randn(1009, E, generator=gen, device=DEV).to(dtype)
    which = torch.arange(T, device=DEV) % 1009
    kw = dict(score="softmax", renormalize=False, scale=1.5)
    z = few[which]
    g = torch.ones(1, k, device=DEV).expand(T, k).contiguous()
    out = []
    for rows in (few, z):
        ids = torch.full((len(rows), k), -7, dtype=torch.int32, device=DEV)
        w = torch.full((len(rows), k), 9.0, device=DEV)
        mm.moe_router_scores(rows, k, ids, w, **kw)
        out.append((ids, w))
    grad = torch.empty_like(few)
    mm.moe_router_scores_bwd(few, out[0][0], g[:1009], grad, **kw)
    mm.moe_router_scores_bwd(z, out[1][0], g, z, **kw)  # in place
    step = 2 ** 21
    for a in range(0, T, step):
        i = which[a:a + step]
        assert torch.equal(out[1][0][a:a + step], out[0][0][i]) and torch.equal(out[1][1][a:a + step], out[0][1][i])
        assert torch.equal(z[a:a + step], grad[i])


# Chosen logits far below the row's largest (softmax) or 0 (sigmoid): their scores are float64 subnormals from 709
# on and 0 from 745 on.  One row each.
FAR = [0.0, 30.0, 41.0, 42.0, 100.0, 700.0, 706.0, 709.0, 712.0, 720.0, 736.0, 744.0, 745.5, 750.0, 800.0, 1e4, 1e30]


def far_rows(seed, dtype):
    """float32 logits [len(FAR), 40], representable in dtype, and the ids of 5 of them: 0 the largest logit,
    the chosen ones FAR below it, within 3 of each other."""
    rng = np.random.default_rng(seed)
    z = -rng.uniform(0.5, 4, (len(FAR), 40))
    z[:, 0] = 0.0
    ids = np.stack([1 + rng.permutation(39)[:5] for _ in FAR]).astype(np.int32)
    for t, far in enumerate(FAR):
        z[t, ids[t]] -= far
    return torch.from_numpy(z.astype(np.float32)).to(dtype).float().numpy(), ids


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_renormalized_weights_far_from_the_largest_logit(score, dtype):
    """A bias of a row's own forces its experts, so a token a call."""
    z, ids = far_rows(20, dtype)
    if score == "sigmoid":
        z[:, 0] = -1.0
    for t in range(len(z)):
        bias = np.zeros(40, np.float32)
        bias[ids[t]] = 100.0 - np.arange(5)
        got, w = check(z[t:t + 1], 5, bias, dtype, score=score, renormalize=True, scale=2.5)
        assert np.array_equal(got[0], ids[t]) and abs(w.sum() - 2.5) <= 5 * 2.5 * 2.0 ** -24
        check(z[t:t + 1], 5, bias, dtype, score=score, renormalize=False, scale=2.5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_renormalized_gradient_far_from_the_largest_logit(score, dtype):
    """Within one rounding of scale * n_j (g_j - sum g n) f_j, f_j <= 1, whose shares n_j of either side are off by
    less than 2^-42 of themselves (an exponent of at most 800 in float64, and sums of 5)."""
    z, ids = far_rows(21, dtype)
    if score == "sigmoid":
        z[:, 0] = -1.0
    rng = np.random.default_rng(22)
    grad = rng.standard_normal(ids.shape).astype(np.float32)
    ids[3, 2] = ids[3, 0]     # an expert named twice
    ids[9, 1] = -1
    z[10, ids[10, 4]] = -np.inf
    kw = dict(score=score, renormalize=True, scale=2.5)
    out, zh, _ = run_bwd(z, ids, grad, dtype, **kw)
    got, ref = out.float().cpu().numpy().astype(np.float64), X.router_bwd(zh, ids, grad, **kw)
    half, tiny = (2.0 ** -24, F32_TINY) if dtype == torch.float32 else (2.0 ** -8, 2.0 ** -134)
    n = np.zeros_like(ref)
    for t in range(len(ids)):
        at = [e for e in ids[t] if e >= 0]
        np.add.at(n[t], at, X.shares(zh[t, at], score))
    size = 2 * 2.5 * np.abs(grad).max(1, keepdims=True) * n
    assert np.isfinite(got).all()
    assert np.all(np.abs(got - ref) <= np.abs(ref) * half + size * 2.0 ** -40 + tiny)
    named = np.zeros_like(n, bool)
    for t in range(len(ids)):
        named[t, ids[t][ids[t] >= 0]] = True
    assert np.all(got[~named] == 0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sigmoid_gradient_of_large_logits(dtype):
    """grad * s (1 - s) has no cancellation of its own: one rounding, and 2^-40 for the two sides' float64.
    Renormalised, g_j - sum g n may cancel: 2^-40 of what is subtracted."""
    z = np.concatenate([np.arange(-64, 65), [-705.0, -100.0, 72.5, 88.0, 100.0, 705.0, 1e30, -1e30]])
    z = torch.from_numpy(np.tile(z, (3, 1)).astype(np.float32)).to(dtype).float().numpy()
    rng = np.random.default_rng(14)
    ids = np.concatenate([rng.permutation(z.shape[1]), [0] * 55])[:192].reshape(3, 64).astype(np.int32)
    grad = rng.standard_normal(ids.shape).astype(np.float32)
    half, tiny = (2.0 ** -24, F32_TINY) if dtype == torch.float32 else (2.0 ** -8, 2.0 ** -134)
    for rows in (slice(0, 2), slice(2, 3)):  # ids named once; one of them named often
        for renormalize in (False, True):
            kw = dict(score="sigmoid", renormalize=renormalize, scale=2.5)
            out, zh, _ = run_bwd(z[rows], ids[rows], grad[rows], dtype, **kw)
            got, ref = out.float().cpu().numpy().astype(np.float64), X.router_bwd(zh, ids[rows], grad[rows], **kw)
            size = np.zeros_like(ref)
            with np.errstate(over="ignore"):
                slope = X.scores(zh, "sigmoid") / (1 + np.exp(zh.astype(np.float64)))
            for t, at in enumerate(ids[rows]):
                s = X.scores(zh[t:t + 1], "sigmoid")[0, at]
                np.add.at(size[t], at, 2.5 * np.abs(grad[rows][t]) if not renormalize else
                          2 * 2.5 * np.abs(grad[rows][t]).max() / s.sum())
            assert np.all(np.abs(got - ref) <= np.abs(ref) * half + size * slope * 2.0 ** -40 + tiny)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k", [(2, 1), (40, 1), (40, 5), (300, 8), (1024, 3)])
def test_softmax_gradient_of_a_dominant_expert(E, k, dtype):
    """One logit up to 700 above the others, named by the slots or not, once or twice, or shared by two experts.
    With x its expert and G the slots' gradients by expert: s_e ((G_e - G_x) - sum_{i != x} (G_i - G_x) s_i), one
    rounding, and 2^-40 of what is summed."""
    rng = np.random.default_rng(E + k)
    gaps = [0.0, 5.0, 20.0, 30.0, 36.0, 37.0, 38.0, 50.0, 80.0, 100.0, 700.0]
    z = rng.standard_normal((4 * len(gaps), E))
    x = rng.integers(0, E, len(z))
    ids = np.stack([rng.permutation(E)[:k] for _ in z]).astype(np.int32)
    for t in range(len(z)):
        z[t] -= z[t].max() + gaps[t // 4]
        z[t, x[t]] = 0.5
        if t % 4 < 3:
            ids[t, 0] = x[t]
        if t % 4 == 1:
            ids[t, k - 1] = x[t]
        if t % 4 == 2:
            z[t, (x[t] + 1) % E] = 0.5
    grad = rng.standard_normal(ids.shape).astype(np.float32)
    kw = dict(score="softmax", renormalize=False, scale=2.5)
    out, zh, _ = run_bwd(z, ids, grad, dtype, **kw)
    got, ref = out.float().cpu().numpy().astype(np.float64), X.router_bwd(zh, ids, grad, **kw)
    half, tiny = (2.0 ** -24, F32_TINY) if dtype == torch.float32 else (2.0 ** -8, 2.0 ** -134)
    s, G = X.scores(zh, "softmax"), np.zeros_like(ref)
    for t, at in enumerate(ids):
        np.add.at(G[t], at, 2.5 * grad[t].astype(np.float64))
    top = zh.argmax(1)[:, None]
    Gx, sx = np.take_along_axis(G, top, 1), np.copy(s)
    np.put_along_axis(sx, top, 0.0, 1)
    size = s * (np.abs(G - Gx) + (sx * (np.abs(G) + np.abs(Gx))).sum(1, keepdims=True))
    assert np.all(np.abs(got - ref) <= np.abs(ref) * half + size * 2.0 ** -40 + tiny)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k", [(2, 1), (2, 2), (40, 1), (40, 5), (1024, 64)])
def test_renormalized_gradient_of_a_dominant_expert(E, k, score, dtype):
    """One chosen logit up to 700 above the other chosen ones, in any slot: with x its slot,
    scale * n_j f_j ((g_j - g_x) - sum_{i != x} n_i (g_i - g_x)), one rounding, and 2^-40 of what is summed.  One slot
    alone: exactly 0."""
    rng = np.random.default_rng(E + k + 1)
    gaps = np.repeat([0.0, 5.0, 20.0, 30.0, 36.0, 37.0, 38.0, 50.0, 80.0, 100.0, 700.0], 3)
    z = rng.standard_normal((len(gaps), E)) - 4 - gaps[:, None]
    ids = np.stack([rng.permutation(E)[:k] for _ in z]).astype(np.int32)
    x = rng.integers(0, k, (len(z), 1))
    np.put_along_axis(z, np.take_along_axis(ids, x, 1), 0.5, 1)
    grad = rng.standard_normal(ids.shape).astype(np.float32)
    kw = dict(score=score, renormalize=True, scale=2.5)
    out, zh, _ = run_bwd(z, ids, grad, dtype, **kw)
    got, ref = out.float().cpu().numpy().astype(np.float64), X.router_bwd(zh, ids, grad, **kw)
    half, tiny = (2.0 ** -24, F32_TINY) if dtype == torch.float32 else (2.0 ** -8, 2.0 ** -134)
    n = np.stack([X.shares(zh[t, ids[t]], score) for t in range(len(z))])
    h = np.abs(grad.astype(np.float64) - np.take_along_axis(grad, x, 1))
    part = 2.5 * n * (h + (n * h).sum(1, keepdims=True))
    if score == "sigmoid":
        part = part / (1 + np.exp(np.take_along_axis(zh, ids, 1).astype(np.float64)))
    size = np.zeros_like(ref)
    np.put_along_axis(size, ids, part, 1)
    assert np.all(np.abs(got - ref) <= np.abs(ref) * half + size * 2.0 ** -40 + tiny)
    if k == 1:
        assert not got.any()


# ---- with the routing step -----------------------------------------------------------------------

@pytest.mark.parametrize("T,P", [(0, 1), (1, 1), (8, 128), (700, 8)])
def test_route_scores_tables(T, P):
    rng = np.random.default_rng(T)
    z = rng.standard_normal((T, 96)).astype(np.float32)
    z[: T // 4, 20:] = -np.inf       # fewer local experts, and slots that stay empty
    z[: T // 8, 3:] = -np.inf
    L = layer.MXMoELayer(T, 4, 24, 256, 128, P, expert_begin=8, device=DEV)
    mm.moe_route_scores(torch.from_numpy(z).to(DEV), 4, 8, 24, P, L.topk_ids, L.topk_weights, L.counts,
                        L.expert_offsets, L.padded_offsets, L.row_token, L.token_rows, L.sched, L.route_ws,
                        score="sigmoid", n_group=4, topk_group=2)
    torch.cuda.synchronize()
    ids, _ = X.router(z, 4, None, "sigmoid", 4, 2)
    assert np.array_equal(np_i32(L.topk_ids), ids)
    counts, eoff, poff, row_token, token_rows = O.route(ids, 8, 24, P)[:5]
    assert np.array_equal(np_i32(L.counts), counts) and np.array_equal(np_i32(L.expert_offsets), eoff)
    assert np.array_equal(np_i32(L.padded_offsets), poff)
    assert np.array_equal(np_i32(L.row_token), row_token)
    assert np.array_equal(np_i32(L.token_rows).reshape(T, 4), np.asarray(token_rows).reshape(T, 4))


def test_other_stream_and_captured_graph():
    """On a stream of its own, and captured once and replayed on new inputs in the same buffers."""
    rng = np.random.default_rng(12)
    zs = [rng.standard_normal((50, 384)).astype(np.float32) for _ in range(4)]
    grad = rng.standard_normal((50, 6)).astype(np.float32)
    kw = dict(score="softmax", renormalize=True, scale=2.5)
    zt = torch.from_numpy(zs[0]).to(DEV)
    gt = torch.from_numpy(grad).to(DEV)
    ids, w = torch.empty(50, 6, dtype=torch.int32, device=DEV), torch.empty(50, 6, device=DEV)
    dz = torch.empty_like(zt)

    def step(stream=None):
        mm.moe_router_scores(zt, 6, ids, w, n_group=8, topk_group=4, stream=stream, **kw)
        mm.moe_router_scores_bwd(zt, ids, gt, dz, stream=stream, **kw)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    step(s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for z in zs:
        zt.copy_(torch.from_numpy(z))
        ids.fill_(-5)
        dz.fill_(9.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        ref_ids, _ = X.router(z, 6, None, n_group=8, topk_group=4, **kw)
        assert np.array_equal(np_i32(ids), ref_ids)
        eager = run_bwd(z, ref_ids, grad, **kw)[0]
        assert torch.equal(dz, eager)
