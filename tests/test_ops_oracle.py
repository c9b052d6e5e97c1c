"""Pins of the float64 oracle of the feed-forward block and the distillation loss (CPU)."""

import math

import numpy as np
import pytest

from oracle import ops_oracle as R


def test_activations_hand_values():
    g = np.array([0.0, 1.0, -1.0])
    a, s = R.act_and_slope(g, "silu")
    e = math.exp(-1.0)
    assert np.allclose(a, [0.0, 1 / (1 + e), -e / (1 + e)], rtol=1e-15)
    assert s[0] == 0.5
    a, s = R.act_and_slope(g, "gelu")
    assert np.allclose(a, [0.0, 0.8413447460685429, -0.15865525393145707], rtol=1e-14) and s[0] == 0.5
    a, s = R.act_and_slope(g, "gelu_tanh")
    t = math.tanh(math.sqrt(2 / math.pi) * 1.044715)
    assert np.allclose(a, [0.0, 0.5 * (1 + t), -0.5 * (1 - t)], rtol=1e-14) and s[0] == 0.5


@pytest.mark.parametrize("act", R.ACTS)
def test_slopes_against_differences(act):
    g = np.linspace(-6, 6, 241)
    h = 1e-5
    num = (R.act_and_slope(g + h, act)[0] - R.act_and_slope(g - h, act)[0]) / (2 * h)
    # truncation h^2 |f'''| / 6 (below 1e-10), rounding 6 * 2^-53 / h (below 1e-10)
    assert np.max(np.abs(num - R.act_and_slope(g, act)[1])) < 2e-10


@pytest.mark.parametrize("act", R.ACTS)
def test_block_gradients_against_differences(act):
    rng = np.random.default_rng(1)
    x, wg, wu = rng.standard_normal((3, 4)), rng.standard_normal((5, 4)), rng.standard_normal((5, 4))
    dh = rng.standard_normal((3, 5))
    h, g, u = R.gated_ffn(x, wg, wu, act)
    grads = R.gated_ffn_grads(dh, x, wg, wu, g, u, act)[:3]
    eps = 1e-5
    for i, grad in enumerate(grads):
        args = [x, wg, wu]
        for idx in np.ndindex(grad.shape):
            vals = []
            for s in (eps, -eps):
                a = [t.copy() for t in args]
                a[i][idx] += s
                vals.append(np.sum(dh * R.gated_ffn(*a, act)[0]))
            assert abs((vals[0] - vals[1]) / (2 * eps) - grad[idx]) < 1e-7


def test_block_of_one():
    h, g, u = R.gated_ffn(np.array([[2.0]]), np.array([[0.0]]), np.array([[3.0]]), "silu")
    assert h[0, 0] == 0.0 and u[0, 0] == 6.0
    dx, dwg, dwu, _, _ = R.gated_ffn_grads(np.array([[1.0]]), np.array([[2.0]]), np.array([[0.0]]),
                                           np.array([[3.0]]), g, u, "silu")
    assert dx[0, 0] == 0.0 and dwg[0, 0] == 6.0 and dwu[0, 0] == 0.0


def test_loss_hand_values():
    # a uniform student over 4, the teacher's two entries equal: loss log 4 - log 2
    loss, stats, grad = R.distill_topk(np.zeros((1, 4)), np.array([[1, 3]]), np.array([[7.0, 7.0]]), np.ones(1), 1.0)
    assert abs(loss[0] - math.log(2.0)) < 1e-15 and stats[0].tolist() == [0.0, 4.0]
    assert np.allclose(grad, [[0.25, -0.25, 0.25, -0.25]], atol=1e-16)
    # the same with one entry given twice
    loss2, _, grad2 = R.distill_topk(np.zeros((1, 4)), np.array([[1, 1]]), np.array([[7.0, 7.0]]), np.ones(1), 1.0)
    assert abs(loss2[0] - math.log(2.0)) < 1e-15 and np.allclose(grad2, [[0.25, -0.75, 0.25, 0.25]])


def test_loss_is_zero_where_student_is_teacher():
    rng = np.random.default_rng(2)
    z = rng.standard_normal((3, 9))
    ids = np.tile(np.arange(9), (3, 1))
    loss, _, grad = R.distill_topk(z, ids, z + 5.0, np.ones(3), 1.7)
    assert np.max(np.abs(loss)) < 1e-14 and np.max(np.abs(grad)) < 1e-15


def test_absent_masked_and_bad_rows():
    z = np.full((4, 3), np.nan)
    z[3] = 0.0
    ids = np.array([[-1, -1], [0, 1], [0, 2], [0, 3]])
    vals = np.array([[1.0, 2.0], [1.0, 2.0], [-np.inf, -np.inf], [1.0, 1.0]])
    loss, _, grad = R.distill_topk(z, ids, vals, np.array([1.0, 0.0, 1.0, 1.0]), 1.0)
    assert np.array_equal(loss[:3], np.zeros(3)) and np.array_equal(grad[:3], np.zeros((3, 3)))
    assert np.isnan(loss[3]) and np.isnan(grad[3]).all()


def test_loss_gradient_against_differences():
    rng = np.random.default_rng(3)
    z = rng.standard_normal((2, 6))
    ids = np.array([[0, 4, -1], [5, 5, 2]])
    vals, w, t = rng.standard_normal((2, 3)), np.array([0.7, 1.9]), 1.6
    grad = R.distill_topk(z, ids, vals, w, t)[2]
    eps = 1e-5
    for idx in np.ndindex(z.shape):
        hi, lo = z.copy(), z.copy()
        hi[idx] += eps
        lo[idx] -= eps
        num = (R.distill_topk(hi, ids, vals, w, t)[0].sum() - R.distill_topk(lo, ids, vals, w, t)[0].sum()) / (2 * eps)
        assert abs(num - grad[idx]) < 1e-8


def test_every_logit_the_lowest_value():
    z = np.full((1, 8), np.finfo(np.float32).min, dtype=np.float64)
    loss, _, grad = R.distill_topk(z, np.array([[0, 1]]), np.array([[3.0, 3.0]]), np.ones(1), 1.0)
    assert abs(loss[0] - math.log(4.0)) < 1e-14 and np.allclose(grad[0], [-0.375] * 2 + [0.125] * 6)


def test_rows_of_ids_past_the_vocabulary_only():
    ids = np.array([[3, 3], [-1, 4], [5, -1], [-1, -1], [9, 9]])
    vals = np.array([[1.0, 2.0], [1.0, 2.0], [-np.inf, 0.0], [1.0, 1.0], [0.0, 0.0]])
    loss, _, grad = R.distill_topk(np.zeros((5, 3)), ids, vals, np.array([1.0, 1.0, 1.0, 1.0, 0.0]), 1.0)
    assert np.isnan(loss[:3]).all() and np.isnan(grad[:3]).all()
    assert not loss[3:].any() and not grad[3:].any()
