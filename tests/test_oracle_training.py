"""Pins of the training-step oracle: closed forms, and gradients against
central differences of the forward definitions (float64, CPU)."""
import numpy as np
import pytest

from oracle import training as ot


def _directional(f, x, d, h=1e-5):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


def test_embedding_gradient_is_the_lookup_transposed():
    rng = np.random.default_rng(0)
    W, ids = rng.standard_normal((7, 5)), np.array([3, 3, 0, -1, 7, 6, 3])
    dY, D = rng.standard_normal((7, 5)), rng.standard_normal((7, 5))
    f = lambda w: float((ot.embedding_lookup(w, ids, 1.7) * dY).sum())
    want = float((ot.embedding_grad(dY, ids, 7, 1.7) * D).sum())
    assert _directional(f, W, D) == pytest.approx(want, rel=1e-8)
    assert np.all(ot.embedding_lookup(W, ids)[3:5] == 0)


@pytest.mark.parametrize("offsets", [[0, 3, 3, 9], [2, 4, 8, 8], [0, 0, 0, 0]])
def test_expert_gradients_match_differences(offsets):
    rng = np.random.default_rng(1)
    X, W = rng.standard_normal((9, 4)), rng.standard_normal((3, 5, 4))
    dY = rng.standard_normal((9, 5))
    DX, DW = rng.standard_normal(X.shape), rng.standard_normal(W.shape)
    f = lambda x, w: float((ot.expert_linear(x, w, offsets) * dY).sum())
    assert _directional(lambda x: f(x, W), X, DX) == pytest.approx(
        float((ot.expert_linear_dgrad(dY, W, offsets) * DX).sum()), rel=1e-7, abs=1e-9)
    assert _directional(lambda w: f(X, w), W, DW) == pytest.approx(
        float((ot.expert_linear_wgrad(dY, X, offsets) * DW).sum()), rel=1e-7, abs=1e-9)


@pytest.mark.parametrize("temperature", [0.5, 1.0, 3.0])
def test_distill_gradient_matches_differences(temperature):
    rng = np.random.default_rng(2)
    S, t = rng.standard_normal((4, 11)), rng.standard_normal((4, 3))
    idx = np.array([[1, 4, 9], [2, 2, 5], [0, -1, 11], [10, 3, 0]])      # a repeated place, absent entries
    w = np.array([1.0, 0.3, 2.0, 0.7])
    D = rng.standard_normal(S.shape)
    f = lambda s: float(ot.distill_topk(s, idx, t, temperature, w)[0].sum())
    grad = ot.distill_topk(S, idx, t, temperature, w)[1]
    assert _directional(f, S, D) == pytest.approx(float((grad * D).sum()), rel=1e-6)
    assert np.allclose(grad.sum(1), 0, atol=1e-12)                       # q and p both sum to one


def test_distill_of_a_full_copy_is_zero_and_masks_follow_the_definition():
    S = np.array([[1.0, 2.0, -np.inf, 0.5], [0.0, 0.0, 0.0, 0.0], [np.nan] * 4, [-np.inf] * 4])
    idx = np.tile(np.arange(4), (4, 1))
    t = np.array([[1.0, 2.0, -np.inf, 0.5], [-np.inf] * 4, [0.0] * 4, [0.0] * 4])
    loss, grad, q, _ = ot.distill_topk(S, idx, t, 2.0, np.array([1.0, 1.0, 0.0, 1.0]))
    assert loss[0] == pytest.approx(0, abs=1e-15) and np.allclose(grad[0], 0, atol=1e-15) and q[0, 2] == 0
    assert loss[1] == 0 and np.all(grad[1] == 0) and loss[2] == 0 and np.all(grad[2] == 0)
    assert loss[3] == np.inf and np.allclose(grad[3], -2 * 0.25)
