"""Pins of oracle/scoring.py: small cases by hand, and the gradient against
central differences of the loss (float64)."""
import numpy as np
import pytest

from oracle import scoring as O


def test_log_probabilities_of_known_values():
    W = np.eye(4)
    H = np.log(np.array([[1.0, 2.0, 4.0, 1.0], [1.0, 1.0, 1.0, 1.0]]))
    lp, ent, lse, ids, best = O.vocab_logprobs(H, W, np.array([[2, -1], [3, 9]]), 3)
    assert np.allclose(lse, np.log([8.0, 4.0]))
    assert np.allclose(lp[0], [np.log(0.5), 0.0]) and lp[1, 0] == pytest.approx(np.log(0.25))
    assert np.isnan(lp[1, 1])
    # -(1/8 log 1/8) * 2 - 1/4 log 1/4 - 1/2 log 1/2
    assert np.allclose(ent, [np.log(2) * (2 * 3 / 8 + 2 / 4 + 1 / 2), np.log(4)])
    assert ids.tolist() == [[2, 1, 0], [0, 1, 2]]       # equal ones: the lower word first
    assert np.allclose(np.exp(best), [[0.5, 0.25, 0.125], [0.25, 0.25, 0.25]])


def test_divergence_of_known_values():
    W = np.eye(4)
    H = np.log(np.array([[1.0, 2.0, 4.0, 1.0]] * 3))
    ids = np.array([[2, 1], [2, -1], [-1, -1]])
    # the student's own probabilities: nothing to lose
    logq = np.log([[0.5, 0.25], [0.5, 0.5], [0.5, 0.5]])
    loss, lse, rest, hit = O.vocab_distill(H, W, ids, logq)
    assert np.allclose(loss, 0) and np.allclose(lse, [np.log(8)] * 2 + [0])
    assert np.allclose(rest, [np.log(2), np.log(4), 0]) and hit[1, 1] == 0 and (hit[2] == 0).all()
    # without a tail the two words are the whole: 2/3 log(4/3) + 1/3 log(4/3); one word: log 2
    loss, _, rest, _ = O.vocab_distill(H, W, ids, logq, tail=False)
    assert np.allclose(loss, [np.log(4 / 3), np.log(2), 0]) and np.allclose(rest[:2], np.log(8))
    assert np.allclose(O.vocab_distill(H, W, ids, logq + 3.0, tail=False)[0], loss)
    # every word listed, one twice
    full = np.array([[0, 1, 2, 3, 3]])
    lq = np.log([[0.125, 0.25, 0.5, 0.0625, 0.0625]])
    loss, _, rest, _ = O.vocab_distill(H[:1], W, full, lq)
    assert rest[0] == -np.inf and loss[0] == pytest.approx(-0.125 * np.log(2))


def test_divergence_from_all_words_is_the_whole_divergence():
    rng = np.random.default_rng(0)
    H, W = rng.standard_normal((3, 6)), rng.standard_normal((9, 6))
    zt = 2 * rng.standard_normal((3, 9))
    logq = zt - O.lse_of(zt)[:, None]
    ids = np.stack([rng.permutation(9) for _ in range(3)])
    logp = O.logits(H, W) - O.lse_of(O.logits(H, W))[:, None]
    want = (np.exp(logq) * (logq - logp)).sum(1)
    listed = np.take_along_axis(logq, ids, 1)
    for tail in (True, False):
        assert np.allclose(O.vocab_distill(H, W, ids, listed, tail=tail)[0], want)
    # fewer words bound it from below (joining outcomes loses divergence)
    assert (O.vocab_distill(H, W, ids[:, :4], listed[:, :4])[0] <= want + 1e-12).all()


@pytest.mark.parametrize("tail", [True, False])
def test_gradient_against_differences(tail):
    rng = np.random.default_rng(3)
    T, V, d, K, scale = 5, 11, 4, 4, 0.7
    H, W = rng.standard_normal((T, d)), rng.standard_normal((V, d))
    ids = np.stack([rng.choice(V, K, replace=False) for _ in range(T)])
    ids[1, 2:] = -1
    ids[2] = -1
    ids[3] = [5, 7, 5, 5]          # one word listed three times
    logq = np.log(rng.dirichlet(np.ones(K + 1), T)[:, :K])
    dl = rng.standard_normal(T)

    def f(H, W):
        return (dl * O.vocab_distill(H, W, ids, logq, scale, tail)[0]).sum()

    dH, dW, _ = O.vocab_distill_backward(H, W, ids, logq, dl, scale, tail)
    assert (dH[2] == 0).all()
    h = 1e-5
    for k, g in enumerate((dH, dW)):
        for i in np.ndindex(g.shape):
            args = [H.copy(), W.copy()]
            args[k][i] += h
            up = f(*args)
            args[k][i] -= 2 * h
            assert abs((up - f(*args)) / (2 * h) - g[i]) <= 1e-7 * (1 + abs(g[i]))
