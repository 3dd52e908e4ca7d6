"""Pins of oracle.head: closed forms, enumeration and central differences."""
import numpy as np
import pytest

from oracle import head as oh


def _problem(T=5, D=3, V=7, seed=0):
    rng = np.random.Generator(np.random.PCG64(seed))
    return rng, rng.normal(size=(T, D)), rng.normal(size=(V, D))


def test_two_tokens_closed_form():
    h, W = np.array([[1.0]]), np.array([[2.0], [0.0]])
    r = oh.token_logprobs(np.array([[0, 1]]), h, W, top_k=2)
    p = 1 / (1 + np.exp(-2.0))
    np.testing.assert_allclose(r["logp"][0], [np.log(p), np.log(1 - p)], rtol=1e-12)
    np.testing.assert_allclose(r["entropy"][0], -(p * np.log(p) + (1 - p) * np.log(1 - p)), rtol=1e-12)
    assert r["top_ids"].tolist() == [[0, 1]]


def test_equal_logits_uniform_and_lowest_ids_first():
    r = oh.token_logprobs(None, np.zeros((2, 3)), np.ones((6, 3)), top_k=4)
    np.testing.assert_allclose(r["entropy"], np.log(6.0), rtol=1e-12)
    assert r["top_ids"].tolist() == [[0, 1, 2, 3]] * 2


def _difference(f, x, eps=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += eps
        b[i] -= eps
        g[i] = (f(a) - f(b)) / (2 * eps)
    return g


@pytest.mark.parametrize("entropy", [False, True])
def test_logprob_gradients_against_differences(entropy):
    rng, h, W = _problem()
    ids = np.array([[1, 1], [6, -1], [0, 3], [-1, -1], [2, 5]])
    g = rng.normal(size=ids.shape)
    ge = rng.normal(size=5) if entropy else None

    def loss(h, W):
        r = oh.token_logprobs(ids, h, W)
        return np.sum(g * r["logp"]) + (np.sum(ge * r["entropy"]) if entropy else 0.0)

    G = oh.token_logprobs_grad(ids, h, W, g, ge)
    np.testing.assert_allclose(G @ W, _difference(lambda x: loss(x, W), h), rtol=1e-6, atol=1e-7)
    np.testing.assert_allclose(G.T @ h, _difference(lambda x: loss(h, x), W), rtol=1e-6, atol=1e-7)


def test_distillation_gradients_against_differences():
    rng, h, W = _problem(seed=1)
    y = np.array([0, 6, 3, 2, -1])
    tid = np.array([[0, 4, 4], [1, -1, -1], [-1, -1, -1], [5, 6, -1], [1, 2, 3]])
    z = rng.normal(size=tid.shape)
    z[1, 1] = np.nan
    z[3, 1] = -np.inf
    w = np.array([1.0, 0.5, 2.0, 1.0, 0.0])

    def loss(h, W):
        return 3.0 * oh.topk_distill(y, tid, z, h, W, 0.4, w)["losses"][2]

    G = oh.topk_distill(y, tid, z, h, W, 0.4, w, grad_scale=3.0)["G"]
    np.testing.assert_allclose(G @ W, _difference(lambda x: loss(x, W), h), rtol=1e-6, atol=1e-7)
    np.testing.assert_allclose(G.T @ h, _difference(lambda x: loss(h, x), W), rtol=1e-6, atol=1e-7)


def test_distillation_of_every_token_is_the_full_cross_entropy():
    """With all V tokens present the term is the cross-entropy to the teacher's whole softmax, and a teacher
    equal to the student leaves no distillation gradient."""
    rng, h, W = _problem(T=4, seed=2)
    l = oh.head_logits(h, W)
    tid = np.tile(np.arange(7), (4, 1))
    r = oh.topk_distill(np.zeros(4, int), tid, l, h, W, alpha_d=1.0)
    logq, _ = oh.log_softmax(l)
    np.testing.assert_allclose(r["stats"][2], -np.sum(np.exp(logq) * logq, axis=1), rtol=1e-12)
    np.testing.assert_allclose(r["G"], 0.0, atol=1e-15)


def test_alpha_zero_is_the_plain_cross_entropy():
    rng, h, W = _problem(seed=3)
    y = np.array([0, 1, 2, 3, 4])
    r = oh.topk_distill(y, np.full((5, 2), 6), np.zeros((5, 2)), h, W, alpha_d=0.0)
    logq, _ = oh.log_softmax(oh.head_logits(h, W))
    np.testing.assert_allclose(r["losses"][2], -np.mean(logq[np.arange(5), y]), rtol=1e-12)
