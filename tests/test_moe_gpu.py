"""Routed expert layer on the GPU against plain 64-bit forms (tests/_moe.py): routing and its
gradient, the plan, dispatch, combine and its gradients, the SwiGLU and its backward pass from the
8-bit checkpoint, and a whole layer of them with the grouped GEMMs, forward and backward."""
import numpy as np
import pytest
import torch

import oracle
from fp8_fine_grained_fp8q_b200 import ops, synth
from tests import _moe
from tests._moe import ELEM, U16, U32
from tests._util import bf16_dev, check_gemm, f32_dev, host, u8_dev

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def bf16(x):
    """float array -> (device tensor, the values it holds in binary64)."""
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)
    return t.cuda(), t.double().numpy()


def ok():
    assert ops.device_status() == ops.DEV_OK


def make_plan(idx, E):
    return ops.MoePlan(*(i32(a) for a in _moe.plan(idx, E)))


# -- routing ------------------------------------------------------------------------------------- #

ROUTES = [  # T, E, k, n_group, topk_group
    (1, 256, 8, 8, 4), (37, 256, 8, 8, 4), (5, 1, 1, 1, 1), (9, 7, 7, 1, 1), (33, 60, 4, 1, 1), (6, 96, 6, 4, 2),
    (3, 1024, 32, 32, 5), (4, 1000, 8, 10, 3), (130, 64, 1, 32, 3), (2, 33, 2, 11, 11), (5, 320, 20, 5, 1),
]


def check_route(logits, dtype, k, bias=None, **kw):
    t = torch.from_numpy(logits.astype(np.float32)).to(dtype).cuda()
    b = None if bias is None else f32_dev(bias)
    idx, w = ops.moe_route(t, k, bias=b, **kw)
    ok()
    ref_idx, ref_w = _moe.route(t.double().cpu().numpy(), k, None if bias is None else np.float32(bias), **kw)
    assert np.array_equal(host(idx), ref_idx)
    got = host(w).astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(ref_w))
    fine = ~np.isnan(ref_w)
    # One value to ELEM, and 2^-149 / 2 where fp32 has no smaller number.
    assert (np.abs(got - ref_w)[fine] <= ELEM * np.abs(ref_w[fine]) + 2.0 ** -149).all()
    return t, idx, w


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("shape", ROUTES)
def test_route_and_its_gradient(shape, score, with_bias, dtype):
    T, E, k, ng, kg = shape
    rng = np.random.default_rng(E + T)
    logits = 2 * rng.normal(size=(T, E))
    bias = 0.1 * rng.normal(size=E) if with_bias else None
    for renorm, scale in ((True, 2.5), (False, 1.0)):
        t, idx, w = check_route(logits, dtype, k, bias, score=score, n_group=ng, topk_group=kg, renormalize=renorm,
                                scale=scale)
        dw = rng.normal(size=(T, k)).astype(np.float32)
        got = ops.moe_route_backward(f32_dev(dw), w, idx, t, score=score, renormalize=renorm, scale=scale)
        ok()
        assert got.dtype == dtype
        ref, mag = _moe.route_backward(dw, host(idx), t.double().cpu().numpy(), score, renorm, scale)
        # Each term to ELEM (w, p and the score are single values to that), a sum of k more of them to k U32,
        # and the rounding of a bf16 result.
        tol = (4 * ELEM + 2 * k * U32) * mag + 1e-37
        if dtype == torch.bfloat16:
            tol = tol + U16 * (np.abs(ref) + tol)
        assert (np.abs(host(got) - ref) <= tol).all()


def test_route_orders_keys_that_fp32_cannot_tell_apart():
    # Scores 1e-8 apart under a bias of 0.3: their fp32 sums are equal, their binary64 sums are not.
    rng = np.random.default_rng(1)
    T, E = 64, 64
    logits = np.stack([3.0 + rng.permutation(E) * 2.0 ** -22 for _ in range(T)]).astype(np.float32)
    bias = np.full(E, 0.3, np.float32)
    for score in ("sigmoid", "softmax"):
        check_route(logits, torch.float32, 8, bias, score=score)
        check_route(logits, torch.float32, 8, bias, score=score, n_group=8, topk_group=3)
    # Scores and biases that cancel to within an fp32 step of each other, in pairs of groups.
    x = rng.normal(size=(T, E // 2)).astype(np.float32)
    s = 1 / (1 + np.exp(-x.astype(np.float64)))
    logits = np.concatenate([x, np.zeros_like(x)], 1)
    for t in range(0, T, 8):
        bias = np.concatenate([np.zeros(E // 2), s[t] - 0.5]).astype(np.float32)
        check_route(logits[t:t + 1], torch.float32, 12, bias, n_group=16, topk_group=9)


@pytest.mark.parametrize("E", [24, 64, 96, 256, 288, 1024])
@pytest.mark.parametrize("unit", [2.0 ** -22, -2.0 ** -22, 2.0 ** -149])
def test_route_orders_logits_one_step_apart(E, unit):
    # Neighbouring fp32 numbers around +-3, and the smallest there are: with and without groups, whole in a
    # warp's lanes or not, and with a bias that leaves the order to binary64.
    rng = np.random.default_rng(E)
    start = 0.0 if unit == 2.0 ** -149 else 3.0 * np.sign(unit)
    logits = np.stack([start + rng.permutation(E) * unit for _ in range(40)]).astype(np.float32)
    for score in ("sigmoid", "softmax"):
        for n_group, topk_group in ((1, 1), (8, 3), (3, 2) if E % 3 == 0 else (4, 3), (2, 1)):
            check_route(logits, torch.float32, 8, score=score, n_group=n_group, topk_group=topk_group)
            if unit != 2.0 ** -149:      # (sums that binary64 tells apart)
                bias = np.full(E, -0.7, np.float32)
                check_route(logits, torch.float32, 8, bias, score=score, n_group=n_group, topk_group=topk_group)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("k", [1, 8, 31, 32])
@pytest.mark.parametrize("E", [48, 64, 128, 256, 600, 1024])
def test_route_near_tie_at_the_last_place(E, k, score):
    # k - 1 keys far above, two within a few fp32 steps of each other at places k and k + 1, the rest far below: the
    # larger of the two is chosen, at the lower index or the higher.  The experts of the last of four groups are
    # the lowest of all, so that the choice of three groups leaves the pair in.
    rng = np.random.default_rng(E + k)
    inside = rng.permutation(E // 4 * 3)
    far, (lo, hi) = inside[:k - 1], np.sort(inside[k - 1:k + 1])
    steps = np.repeat(np.arange(1, 8), 2)
    logits = np.empty((14, E), np.float32)
    logits[:] = -2.0 - rng.random((14, E))
    logits[:, E // 4 * 3:] -= 8.0
    logits[:, far] = 3.0 + 0.5 * rng.permuted(np.tile(np.arange(k - 1), (14, 1)), axis=1)
    up = np.where(np.arange(14) % 2, hi, lo)
    logits[:, lo] = logits[:, hi] = 1.0
    logits[np.arange(14), up] = 1.0 + steps * 2.0 ** -23
    groups = [dict(n_group=1, topk_group=1), dict(n_group=4, topk_group=3)]
    for g in groups:
        _, idx, _ = check_route(logits, torch.float32, k, score=score, **g)
        assert (host(idx)[:, k - 1] == up).all()
    # The same with a bias that sets the far keys apart: the pair's scores differ by less than fp32 holds.
    bias = np.full(E, -2.0, np.float32)
    bias[far], bias[[lo, hi]], bias[E // 4 * 3:] = 1.0 + 0.5 * np.arange(k - 1), -0.7, -9.0
    for g in groups:
        _, idx, _ = check_route(logits, torch.float32, k, bias, score=score, **g)
        assert (host(idx)[:, k - 1] == up).all()
    # Equal logits whose biases are one step apart, and exactly equal ones.
    logits[:, [lo, hi]] = 1.0
    for e in (lo, hi, None):
        b = bias.copy()
        if e is not None:
            b[e] = np.nextafter(b[e], np.float32(0))
        for dtype in (torch.float32, torch.bfloat16):
            for g in groups:
                _, idx, _ = check_route(logits, dtype, k, b, score=score, **g)
                assert (host(idx)[:, k - 1] == (lo if e is None else e)).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E", [64, 96, 256, 1024])
def test_route_equal_inputs_around_a_near_tie(E, score):
    # A smaller logit at the lowest index, one fp32 step below `copies` equal ones behind it, `inside` of which
    # are among the first k by the index: all the places go to the equal ones, in the order of the index.
    rng = np.random.default_rng(E)
    k = 8
    rows, want = [], []
    for inside in (1, 2, 5, 8):
        for copies in (inside, inside + 1, inside + 30, E - 1 - k):
            at = np.sort(rng.permutation(E)[:copies + 1 + k - inside])
            far, at = at[:k - inside], at[k - inside:]
            l = np.full(E, -2.0, np.float32) - rng.random(E).astype(np.float32)
            l[far], l[at[0]], l[at[1:]] = 3.0, 1.0, 1.0 + 2.0 ** -23
            rows.append(l)
            want.append(np.concatenate([far, at[1:]])[:k])
    logits = np.stack(rows)
    for bias in (None, np.full(E, -0.7, np.float32)):
        _, idx, _ = check_route(logits, torch.float32, k, bias, score=score)
        assert (host(idx) == want).all()
        check_route(logits, torch.float32, k, bias, score=score, n_group=8, topk_group=5)
        check_route(logits, torch.float32, 32, bias, score=score, n_group=8, topk_group=6)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,n_group", [(64, 8), (64, 32), (96, 8), (512, 8), (40, 20)])
def test_route_one_input_everywhere_and_masks(E, n_group, dtype):
    # Rows of one value, some of it masked, with groups that have two experts left, one or none.  The biases
    # leave sums of a few 1e-9, of either sign: a group's two keys are then more than another's one, or less.
    rng = np.random.default_rng(E + n_group)
    per = E // n_group
    for x in (0.0, 1.0, -0.375, 2.5, -40.0):
        l = np.full((12, E), x, np.float32)
        l[1, rng.random(E) < 0.5] = -INF
        l[2, ::per] = -INF
        l[3, per:] = -INF
        l[4, :-per] = -INF
        l[5] = -INF
        l[6, rng.random(E) < 0.9] = -INF
        for g in range(n_group):                 # two, one or no expert left
            left = rng.permutation(per)[:(7, 2, 1, 0)[g % 4]]
            l[7 + g % 3, g * per:(g + 1) * per] = -INF
            l[7 + g % 3, g * per + left] = x
            l[11, g * per:(g + 1) * per] = -INF
            l[11, g * per + left] = x
        near = np.float32(_moe.sigmoid(np.float64(x)))
        for score in ("sigmoid", "softmax"):
            for kg in (n_group // 2, n_group - 1):
                for k in (1, min(8, kg * per), min(32, kg * per)):
                    for b in (None, 0.0, 0.3, -near, -np.nextafter(near, np.float32(1)), -np.nextafter(near, np.float32(0))):
                        check_route(l, dtype, k, None if b is None else np.full(E, b, np.float32), score=score,
                                    n_group=n_group, topk_group=kg)


@pytest.mark.parametrize("E,n_group,topk_group", [(256, 8, 4), (256, 16, 5), (128, 4, 2), (384, 12, 4), (512, 8, 8)])
def test_route_many_tokens(E, n_group, topk_group):
    # Enough tokens for every kind of near tie.
    rng = np.random.default_rng(E + n_group)
    for dtype in (torch.float32, torch.bfloat16):
        logits = rng.normal(size=(3000, E))
        for bias in (None, np.zeros(E), 0.05 * rng.normal(size=E)):
            for score in ("sigmoid", "softmax"):
                t = torch.from_numpy(logits.astype(np.float32)).to(dtype).cuda()
                b = None if bias is None else f32_dev(bias)
                idx, _ = ops.moe_route(t, 8, bias=b, score=score, n_group=n_group, topk_group=topk_group)
                ok()
                # The definition in torch's binary64, with sorts that keep the order of equals.
                l = t.double()
                key = l if bias is None else (torch.sigmoid(l) if score == "sigmoid" else torch.softmax(l, -1)) + b.double()
                per = key.view(-1, n_group, E // n_group)
                best = per.amax(-1) if bias is None else per.topk(2, -1).values.sum(-1)
                kept = torch.sort(best, dim=-1, descending=True, stable=True).indices[:, :topk_group]
                allowed = torch.zeros_like(best, dtype=torch.bool).scatter_(1, kept, True)
                key = per.masked_fill(~allowed[:, :, None], -INF).view(-1, E)
                want = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, :8]
                assert torch.equal(idx.long(), want)


@pytest.mark.parametrize("E,k", [(8, 8), (64, 32), (256, 8), (1024, 32)])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("spread", [1.0, 6.0, 40.0])
def test_route_weights_to_the_error_that_is_stated(spread, score, renorm, E, k):
    # In units of U32.  One score: an exponential of 2 steps (4) and of a difference d rounded once (d), one more
    # exponential (2, being at most half of its sum), a sum and a quotient: 8 + d, and with the scale 9 + d.
    # Renormalised, the sum of k of them is off by their mean of that, weighted with the scores (sum of p d < 2 for at
    # most 32), and by 5 additions, and a quotient and the scale add 2: 25 + d.  softmax as it is: the sum of E fast
    # exponentials is off by (2 + 1.2 d) 2 + d each, again weighted (sum of p d < 4.5 for at most 1024: 19.3), and by
    # 37 additions; with the chosen one's 4 + d, a quotient and the scale 62.3 + d.  All are below the header's 64 + d.
    # Below 2^-126 the exponential is off by 2 steps of 2^-149 and the quotient by half of one, times the scale.
    rng = np.random.default_rng(E + k)
    l = (spread * rng.normal(size=(200, E))).astype(np.float32)
    idx, w = ops.moe_route(f32_dev(l), k, score=score, renormalize=renorm, scale=2.5)
    ok()
    ref_idx, ref = _moe.route(l, k, score=score, renormalize=renorm, scale=2.5)
    assert np.array_equal(host(idx), ref_idx)
    x = np.take_along_axis(l.astype(np.float64), ref_idx, 1)
    top = np.minimum(x[:, :1], 0.0) if score == "sigmoid" else x[:, :1]      # idx is in descending order
    d = np.maximum(top - x, 0.0)
    steps = 25 + d if renorm else 9 + np.zeros_like(d) if score == "sigmoid" else 62.3 + d
    assert (np.abs(host(w) - ref) <= steps * (1 + ELEM) * U32 * ref + 3.5 * 2.0 ** -147).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_ties_go_to_the_lower_index(dtype):
    T, E = 5, 96
    flat = np.zeros((T, E))
    for bias in (None, np.zeros(E), np.full(E, 0.25)):
        _, idx, _ = check_route(flat, dtype, 6, bias, n_group=4, topk_group=2)
        assert (host(idx) == np.arange(6)).all()
    steps = np.random.default_rng(2).integers(0, 3, size=(T, E)) * 0.5   # many equal logits
    for score in ("sigmoid", "softmax"):
        for bias in (None, np.random.default_rng(3).integers(0, 2, E) * 0.125):
            check_route(steps, dtype, 8, bias, score=score)
            check_route(steps, dtype, 8, bias, score=score, n_group=12, topk_group=3)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_masks_nan_and_extremes(score, with_bias, dtype):
    rng = np.random.default_rng(4)
    T, E, k = 14, 64, 6
    l = rng.normal(size=(T, E))
    l[0, :] = -INF                      # nothing left at all
    l[1, 5:] = -INF                     # fewer than k left
    l[2, 8:16] = -INF                   # a whole group of the 8
    l[3, ::2] = -INF
    l[4, 17] = NAN
    l[5, 30] = INF
    l[6, :] = NAN
    l[7] = -200 - 50 * rng.random(E)    # every sigmoid underflows fp32
    l[8] = -3e38
    l[9] = 3e38
    l[10, 3] = 1e5
    l[11] *= 300
    l[12, 1:] = -INF                    # one expert
    l[13] = np.where(np.arange(E) < 60, -INF, -90.0)
    bias = 0.1 * rng.normal(size=E) if with_bias else None
    for renorm in (True, False):
        for ng, kg in ((1, 1), (8, 3)):
            t, idx, w = check_route(l, dtype, k, bias, score=score, renormalize=renorm, n_group=ng, topk_group=kg)
            dw = rng.normal(size=(T, k)).astype(np.float32)
            d = host(ops.moe_route_backward(f32_dev(dw), w, idx, t, score=score, renormalize=renorm))
            ok()
            rows = [0, 1, 2, 3, 7, 8, 9, 10, 11, 12, 13]
            ref, mag = _moe.route_backward(dw, host(idx), t.double().cpu().numpy(), score, renorm)
            tol = (4 * ELEM + 2 * k * U32) * mag + 1e-37
            if dtype == torch.bfloat16:
                tol = tol + U16 * (np.abs(ref) + tol)
            assert (np.abs(d - ref)[rows] <= tol[rows]).all()
            assert np.isnan(d[[4, 5, 6]]).any(axis=1).all()      # an unusable logit is not hidden


def test_route_bias_masks_too():
    rng = np.random.default_rng(8)
    l, bias = rng.normal(size=(6, 32)), 0.1 * rng.normal(size=32)
    bias[3:29] = -INF
    check_route(l, torch.float32, 8, bias)
    check_route(l, torch.float32, 8, bias, n_group=4, topk_group=2)
    bias[7] = NAN
    _, _, w = check_route(l, torch.float32, 8, bias)
    assert bool(torch.isnan(w).all())


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E", [64, 96, 512])
def test_route_masks_of_the_lowest_value(E, score):
    # A mask of fp32's lowest finite number is a key like any other: below every ordinary one, above -inf.  The
    # sum of two of them leaves fp32.
    rng = np.random.default_rng(E)
    low = float(torch.finfo(torch.float32).min)
    per = E // 8
    l = rng.normal(size=(40, E)).astype(np.float32)
    masked = l.copy()
    masked[:, rng.random(E) < 0.4] = low
    masked[1] = low
    masked[2, per:] = low
    masked[3, :per], masked[3, per:] = -INF, low
    masked[4, per + 1:] = -INF
    masked[4, :per] = low
    for ng, kg in ((1, 1), (8, 3), (4, 2)):
        for k in (6, min(32, kg * E // ng - 2)):
            check_route(masked, torch.float32, k, score=score, n_group=ng, topk_group=kg)
    high = -low
    for group in ([-INF, low, 0, low, -INF, 0, low, -INF], [low, -INF, low, low, 0, 0.1, -0.1, low],
                  [low] * 8, [low, low / 2, low / 4, low, -INF, low / 2, low, low], [high, 0, high / 2, high, 0, 0, high, 0]):
        bias = np.repeat(np.asarray(group, np.float64), per)
        for some in (False, True):
            if some:         # one ordinary expert in the masked groups too
                bias[per // 2::per] = 0.25
            for ng, kg in ((1, 1), (8, 3), (8, 5), (8, 7), (4, 2)):
                for k in (6, min(32, kg * E // ng - 2)):
                    check_route(l, torch.float32, k, bias, score=score, n_group=ng, topk_group=kg)
        bias = np.where(rng.random(E) < 0.5, low, bias)
        check_route(l, torch.float32, 6, bias, score=score, n_group=8, topk_group=3)


def test_route_backward_same_expert_twice_masked_gradients_and_bad_index():
    rng = np.random.default_rng(9)
    l, k = rng.normal(size=(3, 16)).astype(np.float32), 3
    idx = np.array([[4, 4, 7], [0, 15, 2], [1, 2, 3]], np.int32)
    dw = rng.normal(size=(3, k)).astype(np.float32)
    for score in ("sigmoid", "softmax"):
        for renorm in (True, False):
            s = [_moe.scores(r.astype(np.float64), score) for r in l]
            w = np.stack([_moe.weights_of(l[t].astype(np.float64), idx[t], s[t][1], s[t][0], score, renorm, 1.0)
                          for t in range(3)]).astype(np.float32)
            got = host(ops.moe_route_backward(f32_dev(dw), f32_dev(w), i32(idx), f32_dev(l), score=score,
                                              renormalize=renorm))
            ok()
            ref, mag = _moe.route_backward(dw, idx, l, score, renorm)
            assert (np.abs(got - ref) <= (4 * ELEM + 2 * k * U32) * mag + 1e-37).all()
    # A slot of weight zero takes no part, whatever its gradient says.
    w = np.full((3, k), 0.5, np.float32)
    w[:, 2] = 0.0
    dw[:, 2] = NAN
    got = host(ops.moe_route_backward(f32_dev(dw), f32_dev(w), i32(idx), f32_dev(l)))
    assert np.isfinite(got).all()
    bad = idx.copy()
    bad[1, 1] = 16
    ops.moe_route_backward(f32_dev(dw), f32_dev(w), i32(bad), f32_dev(l))
    assert ops.device_status() == ops.DEV_BAD_INDEX


# -- plan ------------------------------------------------------------------------------------------ #

@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 256), (4, 8, 256), (5, 7, 3), (33, 1, 1024), (1000, 6, 60),
                                   (1025, 8, 1024), (5003, 4, 96), (8192, 8, 256), (40000, 8, 128), (70001, 3, 7)])
def test_plan_is_the_stable_sort(T, k, E):
    rng = np.random.default_rng(T + k)
    for idx in (rng.integers(0, E, size=(T, k)), np.full((T, k), E - 1), np.arange(T * k).reshape(T, k) % E):
        idx = idx.astype(np.int32)
        plan = ops.moe_plan(i32(idx), E)
        ok()
        for got, want in zip(plan, _moe.plan(idx, E)):
            assert np.array_equal(host(got), want)


def test_plan_bad_expert_and_no_tokens():
    for value in (-1, 16, 1 << 30):
        idx = np.random.default_rng(0).integers(0, 16, size=(5000, 4)).astype(np.int32)
        idx[4321, 2] = value
        plan = ops.moe_plan(i32(idx), 16)
        assert ops.device_status() == ops.DEV_BAD_INDEX
        assert not host(plan.offsets).any() and (host(plan.slots) == -1).all() and (host(plan.rows) == -1).all()
    plan = ops.moe_plan(torch.empty(0, 4, dtype=torch.int32, device="cuda"), 16)
    ok()
    assert host(plan.offsets).tolist() == [0] * 17 and plan.slots.numel() == 0


# -- dispatch --------------------------------------------------------------------------------------- #

def dispatch(xbits, plan, weights=None, both=True, cap=None):
    M, C, E = plan.rows.numel(), xbits.shape[1], plan.offsets.numel() - 1
    cap = ops.ragged_capacity(M, E) if cap is None else cap
    q = torch.full((M, C), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.full((C // 128, M), NAN, device="cuda")
    qt = torch.full((C, cap), 0xA5, dtype=torch.uint8, device="cuda") if both else None
    st = torch.full((cap // 128, C), NAN, device="cuda") if both else None
    ops.moe_dispatch(bf16_dev(xbits), plan, weights=weights, transposed=both, Kcap=cap, q=q, s=s, qt=qt, st=st)
    return q, s, qt, st


def same_bits(got, want, what):
    a, b = host(got), np.asarray(want)
    assert np.array_equal(a.view(np.uint32) if a.dtype == np.float32 else a,
                          b.view(np.uint32) if b.dtype == np.float32 else b), what


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("T,k,E,C", [(1, 1, 1, 128), (1, 8, 256, 384), (37, 8, 16, 256), (300, 2, 3, 640),
                                     (129, 1, 5, 128), (64, 32, 40, 256), (513, 3, 1024, 128),
                                     (40, 11, 30, 896), (33, 31, 31, 128), (200, 5, 9, 1152)])
def test_dispatch_is_the_quantisers_of_the_gathered_rows(T, k, E, C, weighted):
    rng = np.random.default_rng(T * k)
    idx = _moe.distinct(rng, T, k, E)
    if E > 4:
        idx[idx == 2] = 3                                          # an expert without rows, and duplicates
    off, slots, rows = _moe.plan(idx, E)
    plan = ops.MoePlan(i32(off), i32(slots), i32(rows))
    bits = synth.activations_channel_outliers(T, C, seed=T)
    bits[0, :128] = 0                                              # a group of zeros
    v = synth.bf16_bits_to_f32(bits)[slots // k]
    w = None
    if weighted:
        w = (rng.random((T, k)) - 0.3).astype(np.float32)
        w[0, 0] = 0.0
        v = (v * w.reshape(-1)[slots][:, None]).astype(np.float32)
        w = f32_dev(w)
    else:
        want = oracle.quant_1x128(bits[slots // k])
        assert np.array_equal(want[0], _moe.quant_rows(v)[0])
    wq, ws = _moe.quant_rows(v)
    wqt, wst = _moe.quant_cols(v, off)
    q, s, _, _ = dispatch(bits, plan, w, both=False)
    ok()
    same_bits(q, wq, "codes")
    same_bits(s, ws, "scales")
    q, s, qt, st = dispatch(bits, plan, w)
    ok()
    same_bits(q, wq, "codes, both forms")
    same_bits(s, ws, "scales, both forms")
    K = wqt.shape[1]
    same_bits(qt[:, :K], wqt, "transposed codes")
    same_bits(st[:K // 128], wst, "transposed scales")
    assert bool((qt[:, K:] == 0xA5).all()) and bool(torch.isnan(st[K // 128:]).all()), "the tail was written"


@pytest.mark.parametrize("weighted", [False, True])
def test_dispatch_many_tiles_a_cta(weighted):
    # 300 experts of 0 to some 200 rows, 9 channel blocks: every CTA of the 128x1 form walks over several items of
    # one to four blocks, in groups of more than 64 rows and of fewer.
    T, k, E, C = 3001, 4, 300, 1152
    rng = np.random.default_rng(5)
    popular = np.exp(1.5 * rng.normal(size=E))
    idx = np.argsort(-(np.log(popular) + rng.gumbel(size=(T, E))), axis=1)[:, :k].astype(np.int32)
    off, slots, rows = _moe.plan(idx, E)
    sizes = np.diff(off) % 128
    assert ((sizes > 0) & (sizes <= 64)).sum() > 50 and (sizes > 64).sum() > 20
    bits = synth.activations_channel_outliers(T, C, seed=2)
    v = synth.bf16_bits_to_f32(bits)[slots // k]
    w = None
    if weighted:
        w = (rng.random((T, k)) - 0.3).astype(np.float32)
        v = (v * w.reshape(-1)[slots][:, None]).astype(np.float32)
        w = f32_dev(w)
    q, s, qt, st = dispatch(bits, ops.MoePlan(i32(off), i32(slots), i32(rows)), w)
    ok()
    for got, want in zip((q, s), _moe.quant_rows(v)):
        same_bits(got, want, "rows")
    wqt, wst = _moe.quant_cols(v, off)
    K = wqt.shape[1]
    assert K // 128 * 3 > 2 * 3 * 148
    same_bits(qt[:, :K], wqt, "transposed codes")
    same_bits(st[:K // 128], wst, "transposed scales")
    assert bool((qt[:, K:] == 0xA5).all()) and bool(torch.isnan(st[K // 128:]).all()), "the tail was written"


@pytest.mark.parametrize("weighted", [False, True])
def test_dispatch_nan_and_infinity_show(weighted):
    x = np.zeros((3, 128), np.float32)
    x[0, 3], x[0, 4], x[0, 100] = NAN, 2.0, -NAN
    x[1, 7], x[1, 8] = INF, -3.0
    x[2, 3], x[2, 4] = 5.0, NAN
    t, _ = bf16(x)
    idx = np.zeros((3, 1), np.int32)
    w = f32_dev(np.ones((3, 1), np.float32)) if weighted else None
    for both in (False, True):
        q, s, qt, st = ops.moe_dispatch(t, make_plan(idx, 1), weights=w, transposed=both)
        ok()
        v = t.float().cpu().numpy()
        wq, ws = _moe.quant_rows(v)
        same_bits(s, ws, "scales")
        # A NaN stays one and does not touch its neighbours; an infinity makes its group's scale infinite, and
        # with it the whole group NaN.
        with np.errstate(invalid="ignore"):
            got, want = _moe.decode_rows(host(q), host(s)), _moe.decode_rows(wq, ws)
            assert np.array_equal(got, want, equal_nan=True)
            assert np.isnan(got[[0, 0, 1, 2], [3, 100, 7, 4]]).all() and np.isnan(got).sum() == 3 + 128
            if both:
                wq, ws = _moe.quant_cols(v, np.array([0, 3]))
                same_bits(st[:1], ws, "column scales")
                got, want = _moe.decode_cols(host(qt)[:, :128], host(st)[:1]), _moe.decode_cols(wq, ws)
                assert np.array_equal(got, want, equal_nan=True)
                assert abs(got[3, 2] - 5.0) < 1e-6 and np.isnan(got[3, 0]) and np.isnan(got[7, 1])


def test_dispatch_bad_plans():
    T, k, E, C = 20, 2, 4, 128
    idx = _moe.distinct(np.random.default_rng(0), T, k, E)
    off, slots, rows = _moe.plan(idx, E)
    bits = synth.output_grad(T, C, seed=1)
    bad = rows.copy()
    bad[3, 1] = T * k
    q, s, _, _ = dispatch(bits, ops.MoePlan(i32(off), i32(slots), i32(bad)), both=False)
    assert ops.device_status() == ops.DEV_BAD_INDEX
    assert (host(q)[rows[3, 1]] == 0xA5).all() and np.isnan(host(s)[:, rows[3, 1]]).all()
    bad = slots.copy()
    bad[5] = -7
    _, _, qt, _ = dispatch(bits, ops.MoePlan(i32(off), i32(bad), i32(rows)))
    at = [128 * g + r for g, n in enumerate(np.diff(off)) for r in range(n)]       # padded columns of the rows
    assert ops.device_status() == ops.DEV_BAD_INDEX and not host(qt)[:, at[5]].any() and host(qt)[:, at[4]].any()
    for o in ([0, 5, 3, 30, 40], [1, 5, 9, 30, 40], [0, 5, 9, 30, 41], [0, -2000000000, 2000000000, 30, 40]):
        q, s, qt, st = dispatch(bits, ops.MoePlan(i32(o), i32(slots), i32(rows)))
        assert ops.device_status() == ops.DEV_BAD_OFFSETS
        assert bool((q == 0xA5).all()) and bool((qt == 0xA5).all()) and bool(torch.isnan(st).all())
    q, _, qt, _ = dispatch(bits, ops.MoePlan(i32(off), i32(slots), i32(rows)), cap=256)   # four experts: four groups
    assert ops.device_status() == ops.DEV_BAD_OFFSETS and bool((q == 0xA5).all())
    # The empty plan of a bad routing is refused by every reader.
    idx[0, 0] = 99
    plan = ops.moe_plan(i32(idx), E)
    assert ops.device_status() == ops.DEV_BAD_INDEX
    q, _, _, _ = dispatch(bits, plan, both=False)
    assert ops.device_status() == ops.DEV_BAD_INDEX and bool((q == 0xA5).all())
    q, _, _, _ = dispatch(bits, plan)
    assert ops.device_status() == ops.DEV_BAD_OFFSETS and bool((q == 0xA5).all())


# -- combine ----------------------------------------------------------------------------------------- #

@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("with_add", [False, True])
@pytest.mark.parametrize("T,k,C", [(1, 1, 8), (1, 8, 7168), (37, 8, 256), (129, 3, 2056), (300, 1, 128), (5, 32, 1000)])
def test_combine_and_its_weight_gradient(T, k, C, with_add, weighted):
    rng = np.random.default_rng(T + C)
    idx = rng.integers(0, 6, size=(T, k)).astype(np.int32)
    _, slots, rows = _moe.plan(idx, 6)
    plan = make_plan(idx, 6)
    y, yv = bf16(rng.normal(size=(T * k, C)))
    add, av = bf16(3 * rng.normal(size=(T, C))) if with_add else (None, 0.0)
    w = (rng.random((T, k)) - 0.2).astype(np.float32) if weighted else None
    out = ops.moe_combine(y, plan, weights=None if w is None else f32_dev(w), add=add)
    ok()
    terms = yv[rows] * (1.0 if w is None else w.astype(np.float64)[:, :, None])
    ref, mag = av + terms.sum(1), np.abs(av) + np.abs(terms).sum(1)
    tol = 2 * (k + 1) * U32 * mag                      # k + 1 fused steps of at most half a step of the sum so far
    assert (np.abs(host(out) - ref) <= tol + U16 * (np.abs(ref) + tol)).all()

    dout, dv = bf16(1e-3 * rng.normal(size=(T, C)))
    dw = ops.moe_combine_dweight(dout, y, plan)
    ok()
    prod = dv[:, None, :] * yv[rows]
    # C products summed in any order: at most C steps, each within U32 of the sum of magnitudes.
    assert (np.abs(host(dw) - prod.sum(2)) <= min(C, 128) * U32 * np.abs(prod).sum(2) + 1e-37).all()


def test_combine_leaves_out_zero_weights_and_bad_rows():
    T, k, C = 3, 2, 64
    idx = np.array([[0, 1], [1, 0], [0, 1]], np.int32)
    off, slots, rows = _moe.plan(idx, 2)
    yv = np.random.default_rng(0).normal(size=(T * k, C))
    yv[rows[0, 1]] = INF
    yv[rows[1, 0], 5] = NAN
    y, yv = bf16(yv)
    w = np.array([[0.5, 0.0], [0.25, 1.0], [0.0, 0.0]], np.float32)
    plan = ops.MoePlan(i32(off), i32(slots), i32(rows))
    out = host(ops.moe_combine(y, plan, weights=f32_dev(w)))
    ok()
    assert (np.abs(out[0] - 0.5 * yv[rows[0, 0]]) <= U16 * np.abs(out[0]) + 1e-30).all()
    assert np.isnan(out[1, 5]) and np.isfinite(np.delete(out[1], 5)).all()
    assert not out[2].any()
    bad = rows.copy()
    bad[2] = [-1, T * k]
    out = host(ops.moe_combine(y, ops.MoePlan(i32(off), i32(slots), i32(bad))))
    assert ops.device_status() == ops.DEV_BAD_INDEX and not out[2].any()
    dout, _ = bf16(np.ones((T, C)))
    dw = host(ops.moe_combine_dweight(dout, y, ops.MoePlan(i32(off), i32(slots), i32(bad))))
    assert ops.device_status() == ops.DEV_BAD_INDEX and not dw[2].any()


# -- SwiGLU ------------------------------------------------------------------------------------------- #

@pytest.mark.parametrize("M,I", [(1, 128), (8, 2048), (37, 256), (129, 384), (1000, 128)])
def test_swiglu_quant(M, I):
    rng = np.random.default_rng(M + I)
    hv = rng.normal(size=(M, 2 * I)) * np.where(rng.random((M, 2 * I)) < 0.01, 8, 1)
    hv[0, :128] = 0.0                                      # a = 0: a group of zeros
    hv[-1, I - 128:I] = -24.0                              # silu ~ -1e-9
    h, hv = bf16(np.clip(hv, -24, 24))
    q, s, hq, hs = ops.swiglu_quant(h)
    ok()
    ref = _moe.swiglu(hv)
    _moe.check_quantised(host(q), host(s), ref, ELEM * np.abs(ref) + 1e-37, what="a")
    wq, ws = _moe.quant_rows(hv.astype(np.float32))
    same_bits(hq, wq, "checkpoint codes")
    same_bits(hs, ws, "checkpoint scales")
    q2, s2, none_q, none_s = ops.swiglu_quant(h, checkpoint=False)
    assert none_q is None and none_s is None and torch.equal(q, q2) and torch.equal(s, s2)


def test_swiglu_far_gates_nan_and_infinity():
    hv = np.zeros((4, 256), np.float32)
    hv[0, :128], hv[0, 128:] = 300.0, 2.0                  # silu(300) = 300
    hv[1, :128], hv[1, 128:] = -300.0, 2.0                 # silu(-300) = -0
    hv[2, 5], hv[2, 128:] = NAN, 1.0
    hv[3, :128], hv[3, 128:], hv[3, 7] = 1.0, 1.0, INF
    h, _ = bf16(hv)
    q, s, hq, hs = ops.swiglu_quant(h)
    ok()
    got = _moe.decode_rows(host(q), host(s))
    assert np.allclose(got[0], 600.0, rtol=1e-3) and not got[1].any()
    assert np.isnan(got[2, 5]) and np.isfinite(np.delete(got[2], 5)).all()
    assert np.isnan(got[3, 7])
    back = _moe.decode_rows(host(hq), host(hs))
    assert np.isnan(back[2, 5]) and np.isnan(back[3, 7]) and np.allclose(back[1, :128], -300.0, rtol=1e-3)


def swiglu_problem(M, I, seed):
    rng = np.random.default_rng(seed)
    h = np.clip(3 * rng.normal(size=(M, 2 * I)), -24, 24).astype(np.float32)
    hq, hs = _moe.quant_rows(h)
    da = synth.output_grad(M, I, seed=seed)
    return da, hq, hs


@pytest.mark.parametrize("counts,I", [([1], 128), ([1, 0, 127, 129, 300, 5], 256), ([0, 0, 7], 128), ([256, 128], 384),
                                      (None, 128), (None, 1408)])
def test_swiglu_backward_from_the_checkpoint(counts, I):
    M = sum(counts) if counts else 333
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32) if counts else np.array([0, M], np.int32)
    da, hq, hs = swiglu_problem(M, I, seed=M + I)
    cap = ops.ragged_capacity(M, len(counts)) if counts else 128 * ((M + 127) // 128)
    bufs = {n: torch.full(sh, 0xA5, dtype=torch.uint8, device="cuda")
            for n, sh in (("q", (M, 2 * I)), ("qt", (2 * I, cap)), ("aqt", (I, cap)))}
    bufs |= {n: torch.full(sh, NAN, device="cuda")
             for n, sh in (("s", (2 * I // 128, M)), ("st", (cap // 128, 2 * I)), ("ast", (cap // 128, I)))}
    ops.swiglu_backward_quant(bf16_dev(da), u8_dev(hq), f32_dev(hs), offsets=i32(off) if counts else None, Kcap=cap,
                              **bufs)
    ok()
    h = (oracle.e4m3_decode(hq.reshape(-1)).reshape(hq.shape) * np.repeat(hs.T, 128, axis=1)).astype(np.float32)
    # code * scale is one fp32 product in the kernel and here.
    (dg, du, a), (eg, eu, ea) = _moe.swiglu_backward(synth.bf16_bits_to_f32(da).astype(np.float64),
                                                     h[:, :I].astype(np.float64), h[:, I:].astype(np.float64))
    dh, eh = np.concatenate([dg, du], 1), np.concatenate([eg, eu], 1)
    _moe.check_quantised(host(bufs["q"]), host(bufs["s"]), dh, eh, what="dh")
    pad = lambda v: np.ascontiguousarray(_moe.padded_rows(v, off).T)   # noqa: E731
    K = pad(a).shape[1]
    # Columns: groups run along the padded rows, one scale for (group, column).
    for name, v, e in (("", dh, eh), ("a", a, ea)):
        qt, st = host(bufs[name + "qt"]), host(bufs[name + "st"])
        _moe.check_quantised(np.ascontiguousarray(qt[:, :K]), np.ascontiguousarray(st[:K // 128]), pad(v), pad(e),
                             what=name + "t")
        assert (qt[:, K:] == 0xA5).all() and np.isnan(st[K // 128:]).all(), "the tail was written"
        padding = pad(np.ones((M, 1)))[0] == 0
        assert not qt[:, :K][:, padding].any(), "padding must hold zero codes"


def test_swiglu_backward_many_tiles_a_cta():
    # More than four tiles a CTA, groups of more than 64 rows and of fewer one after another.
    rng = np.random.default_rng(7)
    counts = rng.integers(0, 200, size=60)
    counts[[3, 17, 18]] = 0, 64, 65
    off, I = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), 1152
    M = int(off[-1])
    assert sum(-(-n // 128) for n in counts) * (I // 128) > 4 * 148
    da, hq, hs = swiglu_problem(M, I, seed=8)
    args = bf16_dev(da), u8_dev(hq), f32_dev(hs)
    q, s, qt, st, aqt, ast = got = ops.swiglu_backward_quant(*args, offsets=i32(off))
    again = ops.swiglu_backward_quant(*args, offsets=i32(off))
    ok()
    h = (oracle.e4m3_decode(hq.reshape(-1)).reshape(hq.shape) * np.repeat(hs.T, 128, axis=1)).astype(np.float32)
    (dg, du, a), (eg, eu, ea) = _moe.swiglu_backward(synth.bf16_bits_to_f32(da).astype(np.float64),
                                                     h[:, :I].astype(np.float64), h[:, I:].astype(np.float64))
    dh, eh = np.concatenate([dg, du], 1), np.concatenate([eg, eu], 1)
    _moe.check_quantised(host(q), host(s), dh, eh, what="dh")
    padding = _moe.padded_rows(np.ones((M, 1)), off)[:, 0] == 0
    K = padding.size
    for codes, scales, v, e, what in ((qt, st, dh, eh, "dh, transposed"), (aqt, ast, a, ea, "a, transposed")):
        codes, scales = np.ascontiguousarray(host(codes)[:, :K]), np.ascontiguousarray(host(scales)[:K // 128])
        _moe.check_quantised(codes, scales, np.ascontiguousarray(_moe.padded_rows(v, off).T),
                             np.ascontiguousarray(_moe.padded_rows(e, off).T), what=what)
        assert not codes[:, padding].any(), "padding must hold zero codes"
    for x, y, rows in zip(got, again, (True, True, False, False, False, False)):
        if not rows:                # what lies behind the last group is not written
            x, y = (x[:, :K], y[:, :K]) if x.dtype == torch.uint8 else (x[:K // 128], y[:K // 128])
        assert torch.equal(x, y)


def test_swiglu_backward_bad_offsets_write_nothing():
    M, I = 40, 128
    da, hq, hs = swiglu_problem(M, I, 3)
    for o, cap in (([0, 30, 20, 40], 512), ([0, 10, 20, 41], 512), ([0, 10, 20, 40], 256)):
        q = torch.full((M, 2 * I), 0xA5, dtype=torch.uint8, device="cuda")
        aqt = torch.full((I, cap), 0xA5, dtype=torch.uint8, device="cuda")
        ops.swiglu_backward_quant(bf16_dev(da), u8_dev(hq), f32_dev(hs), offsets=i32(o), Kcap=cap, q=q, aqt=aqt)
        assert ops.device_status() == ops.DEV_BAD_OFFSETS
        assert bool((q == 0xA5).all()) and bool((aqt == 0xA5).all())


# -- refusals of the binding ------------------------------------------------------------------------- #

def test_binding_refusals():
    T, k, E, C = 4, 2, 8, 256
    logits = torch.zeros(T, E, device="cuda")
    idx, w = ops.moe_route(logits, k)
    plan = ops.moe_plan(idx, E)
    x = torch.zeros(T, C, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(T * k, C, dtype=torch.bfloat16, device="cuda")
    for exc, call in [
        (TypeError, lambda: ops.moe_route(logits.double(), k)),
        (ValueError, lambda: ops.moe_route(logits.t(), k)),
        (ValueError, lambda: ops.moe_route(logits, k, score="relu")),
        (ValueError, lambda: ops.moe_route(logits, 0)),
        (ops.Fp8qError, lambda: ops.moe_route(logits, 9)),
        (ops.Fp8qError, lambda: ops.moe_route(logits, k, n_group=3, topk_group=1)),
        (ValueError, lambda: ops.moe_route(logits, k, bias=torch.zeros(E + 1, device="cuda"))),
        (ValueError, lambda: ops.moe_route(logits, k, bias=torch.zeros(E))),
        (TypeError, lambda: ops.moe_plan(idx.long(), E)),
        (ValueError, lambda: ops.moe_route_backward(w[:2], w, idx, logits)),
        (ValueError, lambda: ops.moe_dispatch(x[:3], plan)),
        (ValueError, lambda: ops.moe_dispatch(x, plan, weights=w.t())),
        (ValueError, lambda: ops.moe_dispatch(x, plan._replace(slots=plan.slots[:3]))),
        (ops.Fp8qError, lambda: ops.moe_dispatch(x[:, :192].contiguous(), plan)),
        (ValueError, lambda: ops.moe_combine(y[:5], plan)),
        (ValueError, lambda: ops.moe_combine(y, plan, add=y)),
        (ValueError, lambda: ops.moe_combine_dweight(x, y[:, :128].contiguous(), plan)),
        (ValueError, lambda: ops.swiglu_quant(x[:, :255].contiguous())),
        (ops.Fp8qError, lambda: ops.swiglu_quant(x[:, :128].contiguous())),
        (ValueError, lambda: ops.swiglu_backward_quant(x, torch.zeros(T, C, dtype=torch.uint8, device="cuda"),
                                                       torch.zeros(2, T, device="cuda"))),
    ]:
        with pytest.raises(exc):
            call()
    ok()


# -- together ------------------------------------------------------------------------------------------ #

class Layer:
    """An expert layer out of these operators and the grouped GEMMs: weights and inputs of a seed."""

    def __init__(self, T=97, E=6, k=2, C=256, I=128, seed=11):
        rng = np.random.default_rng(seed)
        self.T, self.E, self.k, self.C, self.I = T, E, k, C, I
        self.x, self.xv = bf16(rng.normal(size=(T, C)))
        self.logits = f32_dev(rng.normal(size=(T, E)) - 5.0 * (np.arange(E) == 4))   # expert 4: hardly a token
        self.bias = f32_dev(0.05 * rng.normal(size=E))
        self.w1 = [bf16(rng.normal(size=(2 * I, C)) / C ** 0.5) for _ in range(E)]
        self.w2 = [bf16(rng.normal(size=(C, I)) / I ** 0.5) for _ in range(E)]
        self.w1q, self.w1s = (torch.stack(a) for a in zip(*(ops.weight_128x128(w)[:2] for w, _ in self.w1)))
        self.w2q, self.w2s = (torch.stack(a) for a in zip(*(ops.weight_128x128(w)[:2] for w, _ in self.w2)))
        self.shared, self.sv = bf16(rng.normal(size=(T, C)))
        self.dout, self.dv = bf16(rng.normal(size=(T, C)))
        self.route = dict(score="sigmoid", renormalize=True, scale=2.5)

    def step(self):
        M = self.T * self.k
        idx, w = ops.moe_route(self.logits, self.k, bias=self.bias, n_group=3, topk_group=2, **self.route)
        plan = ops.moe_plan(idx, self.E)
        xq, xs, xqt, xst = ops.moe_dispatch(self.x, plan, transposed=True)
        h = ops.grouped_gemm_blockscaled(xq, xs, self.w1q, self.w1s, plan.offsets)
        aq, as_, hq, hs = ops.swiglu_quant(h)
        y = ops.grouped_gemm_blockscaled(aq, as_, self.w2q, self.w2s, plan.offsets)
        out = ops.moe_combine(y, plan, weights=w, add=self.shared)
        # backward
        dyq, dys, dyqt, dyst = ops.moe_dispatch(self.dout, plan, weights=w, transposed=True)
        dw = ops.moe_combine_dweight(self.dout, y, plan)
        dlogits = ops.moe_route_backward(dw, w, idx, self.logits, **self.route)
        da = ops.grouped_gemm_blockscaled_dgrad(dyq, dys, self.w2q, self.w2s, plan.offsets)
        dhq, dhs, dhqt, dhst, aqt, ast = ops.swiglu_backward_quant(da, hq, hs, offsets=plan.offsets)
        dw2 = ops.grouped_gemm_blockscaled_wgrad(dyqt, dyst, aqt, ast, plan.offsets, M)
        dxr = ops.grouped_gemm_blockscaled_dgrad(dhq, dhs, self.w1q, self.w1s, plan.offsets)
        dw1 = ops.grouped_gemm_blockscaled_wgrad(dhqt, dhst, xqt, xst, plan.offsets, M)
        dx = ops.moe_combine(dxr, plan)
        return dict(idx=idx, w=w, out=out, dx=dx, dlogits=dlogits, dw1=dw1, dw2=dw2, h=h, y=y, da=da, dxr=dxr)

    def plain(self, idx):
        """The layer and its gradients in binary64, with the same choice of experts."""
        T, k, I = self.T, self.k, self.I
        l = host(self.logits).astype(np.float64)
        s = 1 / (1 + np.exp(-l))
        p = np.take_along_axis(s, idx, 1)
        w = 2.5 * p / p.sum(1, keepdims=True)
        out, dx, dw = self.sv.copy(), np.zeros_like(self.xv), np.zeros((T, k))
        dw1, dw2 = np.zeros((self.E, 2 * I, self.C)), np.zeros((self.E, self.C, I))
        for t in range(T):
            for j, e in enumerate(idx[t]):
                h = self.w1[e][1] @ self.xv[t]
                (dg, du, a), _ = _moe.swiglu_backward(self.w2[e][1].T @ (w[t, j] * self.dv[t]), h[:I], h[I:])
                y = self.w2[e][1] @ a
                out[t] += w[t, j] * y
                dw[t, j] = self.dv[t] @ y
                dh = np.concatenate([dg, du])
                dx[t] += self.w1[e][1].T @ dh
                dw1[e] += np.outer(dh, self.xv[t])
                dw2[e] += np.outer(w[t, j] * self.dv[t], a)
        dl, _ = _moe.route_backward(dw, idx, l, **self.route)
        return dict(w=w, out=out, dx=dx, dlogits=dl, dw1=dw1, dw2=dw2)


def test_a_layer_forward_and_backward():
    layer = Layer()
    got = layer.step()
    ok()
    idx = host(got["idx"])
    assert np.array_equal(idx, _moe.route(host(layer.logits), layer.k, host(layer.bias), n_group=3, topk_group=2,
                                          **layer.route)[0])
    ref = layer.plain(idx)
    for name, want in ref.items():
        have = host(got[name]).astype(np.float64)
        assert have.shape == want.shape
        err = np.linalg.norm(have - want) / np.linalg.norm(want)
        # Every operand of a product is off by at most half an E4M3 step (2^-4) of itself; at most six such
        # roundings lie between the inputs and any result, and in a sum they add as independent errors do:
        # sqrt(6) 2^-4 = 0.153 of the norm.  The weights come from fp32 alone.
        assert err <= (ELEM if name == "w" else 0.153), f"{name}: {err:.3g}"


def test_a_layer_is_repeatable_captured_and_on_another_stream():
    layer = Layer(T=130, seed=12)
    first = layer.step()
    again = layer.step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = layer.step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = layer.step()
    for v in captured.values():
        v.zero_()
    graph.replay()
    torch.cuda.synchronize()
    ok()
    for name, v in first.items():
        for o in (again, other, captured):
            assert torch.equal(v, o[name]), name
    # The same graph on other inputs.
    fresh = Layer(T=130, seed=13)
    for name in ("x", "logits", "bias", "shared", "dout", "w1q", "w1s", "w2q", "w2s"):
        getattr(layer, name).copy_(getattr(fresh, name))
    graph.replay()
    want = fresh.step()
    torch.cuda.synchronize()
    ok()
    for name, v in want.items():
        assert torch.equal(v, captured[name]), name


def test_a_single_token_through_the_layer():
    layer = Layer(T=1, E=16, k=8, seed=14)
    layer.route["score"] = "softmax"
    idx, w = ops.moe_route(layer.logits, 8, **layer.route)
    plan = ops.moe_plan(idx, 16)
    xq, xs, _, _ = ops.moe_dispatch(layer.x, plan)
    h = ops.grouped_gemm_blockscaled(xq, xs, layer.w1q, layer.w1s, plan.offsets)
    aq, as_, _, _ = ops.swiglu_quant(h, checkpoint=False)
    y = ops.grouped_gemm_blockscaled(aq, as_, layer.w2q, layer.w2s, plan.offsets)
    out = host(ops.moe_combine(y, plan, weights=w))
    ok()
    want = np.zeros((1, layer.C))
    for j, e in enumerate(host(idx)[0]):
        h = layer.w1[e][1] @ layer.xv[0]
        want[0] += host(w)[0, j] * (layer.w2[e][1] @ _moe.swiglu(h[None])[0])
    assert np.linalg.norm(out - want) <= 0.153 * np.linalg.norm(want)


def test_two_layers_on_two_streams_at_once():
    layers = [Layer(T=300, seed=s) for s in (21, 22)]
    want = [l.step() for l in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    got = [[], []]
    for _ in range(3):
        for i, (l, st) in enumerate(zip(layers, streams)):
            with torch.cuda.stream(st):
                got[i].append(l.step())
    torch.cuda.synchronize()
    ok()
    for i in range(2):
        for g in got[i]:
            for name, v in want[i].items():
                assert torch.equal(v, g[name]), name


def test_the_public_ways_to_device_and_stream_do_too(monkeypatch):
    layer = Layer(T=60, seed=15)
    want = layer.step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert ops._stream_now(0) == ops._public_stream(0) == side.cuda_stream
    monkeypatch.setattr(ops, "_device_now", torch.cuda.current_device)
    monkeypatch.setattr(ops, "_stream_now", ops._public_stream)
    with torch.cuda.stream(side):
        got = layer.step()
    side.synchronize()
    ok()
    for name, v in want.items():
        assert torch.equal(v, got[name]), name


FIRST_USE = """
import torch
from fp8_fine_grained_fp8q_b200 import ops
x = torch.randn(130, 256, device="cuda").to(torch.bfloat16)
logits, bias = torch.randn(130, 16, device="cuda"), torch.zeros(16, device="cuda")
h, dw = torch.randn(520, 512, device="cuda").to(torch.bfloat16), torch.randn(130, 4, device="cuda")

def step():
    idx, w = ops.moe_route(logits, 4, bias=bias, n_group=4, topk_group=2)
    plan = ops.moe_plan(idx, 16)
    q = ops.moe_dispatch(x, plan, weights=w, transposed=True)
    a = ops.swiglu_quant(h)
    b = ops.swiglu_backward_quant(h[:, :256].contiguous(), a[2], a[3], offsets=plan.offsets)
    y = h[:, 256:].contiguous()
    out = ops.moe_combine(y, plan, weights=w, add=x)
    d = ops.moe_route_backward(ops.moe_combine_dweight(out, y, plan), w, idx, logits)
    return [idx, w, *plan, *q[:2], *a, *b[:2], out, d]

g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    captured = step()
g.replay()
torch.cuda.synchronize()
assert ops.device_status() == ops.DEV_OK
assert all(torch.equal(p, q) for p, q in zip(captured, step()))
print("same")
"""


def test_first_use_inside_a_capture():
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_USE], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr


def test_no_tokens_anywhere():
    E, k, C, I = 6, 2, 256, 128
    bf = lambda *shape: torch.empty(*shape, dtype=torch.bfloat16, device="cuda")   # noqa: E731
    idx, w = ops.moe_route(torch.empty(0, E, device="cuda"), k)
    plan = ops.moe_plan(idx, E)
    q, s, qt, st = ops.moe_dispatch(bf(0, C), plan, weights=w, transposed=True)
    y = bf(0, C)
    out, dw = ops.moe_combine(y, plan, weights=w), ops.moe_combine_dweight(bf(0, C), y, plan)
    d = ops.moe_route_backward(dw, w, idx, torch.empty(0, E, device="cuda"))
    a = ops.swiglu_quant(bf(0, 2 * I))
    g = ops.swiglu_backward_quant(bf(0, I), a[2], a[3], offsets=plan.offsets)
    ops.swiglu_backward_quant(bf(0, I), a[2], a[3])
    # The experts' weight gradients of no tokens are zero.
    dw1 = ops.grouped_gemm_blockscaled_wgrad(g[2], g[3], qt, st, plan.offsets, 0)
    ok()
    assert not host(plan.offsets).any() and not host(dw1).any()
    assert [tuple(t.shape) for t in (idx, q, out, dw, d, a[0])] == [(0, k), (0, C), (0, C), (0, k), (0, E), (0, I)]


# -- sizes whose offsets pass 32 bits, against the library's own quantisers ------------------------------ #

def test_dispatch_and_combine_past_32_bit_offsets():
    T, k, E, C = 70001, 8, 12, 7680                       # 4.3e9 codes in each form
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, C, generator=g, device="cuda", dtype=torch.bfloat16)
    idx = torch.rand(T, E, generator=g, device="cuda").topk(k).indices.to(torch.int32)
    plan = ops.moe_plan(idx, E)
    q, s, qt, st = ops.moe_dispatch(x, plan, transposed=True)
    ok()
    M = T * k
    at = torch.cat([torch.arange(512, device="cuda"), torch.arange(M - 640, M, device="cuda")])
    rows = x[(plan.slots[at] // k).long()].contiguous()
    wq, ws = ops.act_1x128(rows)
    assert torch.equal(q[at], wq) and torch.equal(s[:, at], ws)
    # The last expert's last whole groups, whose columns lie behind all others'.
    off = plan.offsets.tolist()
    groups = [-(-(b - a) // 128) for a, b in zip(off[:-1], off[1:])]
    n = off[E] - off[E - 1]
    lo = 128 * (n // 128 - 2)
    rows = x[(plan.slots[off[E - 1] + lo:off[E - 1] + lo + 256] // k).long()].contiguous()
    wqt, wst = ops.act_128x1_transposed(rows)
    first = sum(groups[:-1]) + lo // 128
    assert torch.equal(qt[:, 128 * first:128 * first + 256], wqt) and torch.equal(st[first:first + 2], wst)
    del qt, st, q, s
    y = torch.randn(M, C, generator=g, device="cuda", dtype=torch.bfloat16)
    out = ops.moe_combine(y, plan)
    dw = ops.moe_combine_dweight(x, y, plan)
    ok()
    for t in (0, T // 2, T - 1):
        r = y[plan.rows[t].long()].double()
        tol = 2 * (k + 1) * U32 * r.abs().sum(0)
        assert bool(((out[t].double() - r.sum(0)).abs() <= tol + U16 * (r.sum(0).abs() + tol)).all())
        p = r * x[t].double()
        assert bool(((dw[t].double() - p.sum(1)).abs() <= 128 * U32 * p.abs().sum(1)).all())


def test_swiglu_past_32_bit_offsets():
    M, I = 300001, 7296                                    # 4.4e9 codes of the checkpoint
    g = torch.Generator(device="cuda").manual_seed(2)
    h = torch.randn(M, 2 * I, generator=g, device="cuda", dtype=torch.bfloat16)
    q, s, hq, hs = ops.swiglu_quant(h)
    ok()
    for lo in (0, M - 200):
        tq, ts, thq, ths = ops.swiglu_quant(h[lo:lo + 200].contiguous())
        assert torch.equal(q[lo:lo + 200], tq) and torch.equal(s[:, lo:lo + 200], ts)
        assert torch.equal(hq[lo:lo + 200], thq) and torch.equal(hs[:, lo:lo + 200], ths)
    da = h[:, :I].contiguous()
    del h, q, s
    dq, ds, dqt, dst, aqt, ast = ops.swiglu_backward_quant(da, hq, hs)
    ok()
    lo = 128 * (M // 128 - 1)
    n = M - lo                                             # a whole group and the last, partial one
    want = ops.swiglu_backward_quant(da[lo:].contiguous(), hq[lo:].contiguous(), hs[:, lo:].contiguous())
    got = (dq[lo:], ds[:, lo:], dqt[:, lo:], dst[lo // 128:], aqt[:, lo:], ast[lo // 128:])
    assert n > 128 and all(torch.equal(a, b) for a, b in zip(got, want))
