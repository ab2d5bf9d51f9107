"""Pins of oracle/tuning.py: exact small cases, and gradients against central
differences of the formulas (float64, so a difference quotient with step h is
off by about h^2 of the third derivative plus 1e-16 / h)."""
import numpy as np
import pytest

from oracle import tuning as O


def test_checkpoint_of_known_values():
    x = np.zeros((3, 40))
    x[0, :4] = [127.0, -126.5, 0.5, 1.5]         # step 1; ties go to even
    x[0, 32] = 2.0 ** -130                        # below the least step
    x[1, 0], x[1, 33] = 127.5, np.inf             # step 2; a group that is not finite
    x[2, 5] = -3.0e38                             # (3.0e38 <= 127 2^121 < 2^128)
    c, e = O.act8_quantize(x)
    assert e.tolist() == [[127, 1], [128, 255], [127 + 121, 1]]
    assert c[0, :4].tolist() == [127, -126, 0, 2] and c[0, 32] == 0
    assert c[1, 0] == 64 and (c[1, 32:] == 0).all()
    v = O.act8_values(c, e)
    assert v[1, 0] == 128.0 and np.isnan(v[1, 32:]).all()
    assert abs(v[2, 5] - x[2, 5]) <= 2.0 ** 120


@pytest.mark.parametrize("top", [121, 9])
def test_checkpoint_step_is_the_least_that_holds(top):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((50, 64)) * np.exp2(rng.integers(-20, 8, (50, 1)))
    c, e = O.act8_quantize(x, top)
    step = O.act8_steps(e)
    big = np.abs(x.reshape(50, 2, 32)).max(-1)
    assert (big <= 127 * step).all() and (big > 127 * step / 2).all()
    assert (np.abs(O.act8_values(c, e) - x) <= np.repeat(step, 32, 1) / 2).all()


def test_layer_gradient_against_differences():
    rng = np.random.default_rng(1)
    m, n, r, T = 7, 9, 5, 4
    SU, SV = np.sign(rng.standard_normal((m, r))), np.sign(rng.standard_normal((n, r)))
    s1, s2 = rng.uniform(0.5, 2, m), rng.uniform(0.5, 2, n)
    x, c = rng.standard_normal((T, n)), rng.standard_normal((T, m))

    def f(x, s1, s2):   # a loss with dL/dy = c + y
        y = s1 * (((x * s2) @ SV) @ SU.T)
        return (c * y).sum() + 0.5 * (y * y).sum()

    y = s1 * (((x * s2) @ SV) @ SU.T)
    got = O.layer_backward(SU, SV, s1, s2, x, c + y)
    h = 1e-5
    for k, (arg, d) in enumerate(zip((x, s1, s2), got)):
        for i in np.ndindex(arg.shape):
            lo, hi = arg.copy(), arg.copy()
            lo[i] -= h
            hi[i] += h
            args = [x, s1, s2]
            a = f(*[hi if j == k else v for j, v in enumerate(args)])
            b = f(*[lo if j == k else v for j, v in enumerate(args)])
            assert abs((a - b) / (2 * h) - d[i]) <= 1e-6 * (1 + abs(d[i]))


def test_loss_gradient_against_differences():
    rng = np.random.default_rng(2)
    T, V, d, scale = 5, 11, 6, 0.7
    H, W = rng.standard_normal((T, d)), rng.standard_normal((V, d))
    labels = np.array([3, -100, 0, 10, -1])
    H[1] = np.nan   # an ignored row may hold anything
    dl = rng.standard_normal(T)
    loss, lse = O.vocab_loss(H, W, labels, scale)
    assert (loss[[1, 4]] == 0).all() and (lse[[1, 4]] == 0).all()
    dH, dW, _ = O.vocab_loss_backward(H, W, labels, dl, scale)
    assert (dH[[1, 4]] == 0).all()
    h = 1e-5
    for arg, grad in ((H, dH), (W, dW)):
        for i in np.ndindex(arg.shape):
            if arg is H and labels[i[0]] < 0:
                continue
            keep = arg[i]
            arg[i] = keep + h
            a = (dl * O.vocab_loss(H, W, labels, scale)[0]).sum()
            arg[i] = keep - h
            b = (dl * O.vocab_loss(H, W, labels, scale)[0]).sum()
            arg[i] = keep
            assert abs((a - b) / (2 * h) - grad[i]) <= 1e-7 * (1 + abs(grad[i]))


def test_loss_of_one_word_is_zero():
    loss, lse = O.vocab_loss(np.array([[2.0]]), np.array([[3.0]]), np.array([0]))
    assert loss[0] == 0.0 and lse[0] == 6.0
