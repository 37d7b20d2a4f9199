"""The oracle of the operators between the GEMMs, against differences of the
functions whose gradients it states and against worked values (CPU only)."""
import numpy as np
import pytest

from oracle import rowops as R


def differences(f, x, h=1e-5):
    """Central differences of a scalar function."""
    g = np.empty_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


def close(a, b, tol=1e-7):
    assert np.max(np.abs(a - b)) <= tol * max(1.0, np.max(np.abs(b)))


@pytest.mark.parametrize("affine", [False, True])
def test_layer_norm_gradient(affine):
    rng = np.random.default_rng(1)
    X, dY = rng.standard_normal((3, 7)), rng.standard_normal((3, 7))
    g, b = (rng.standard_normal(7), rng.standard_normal(7)) if affine else (np.ones(7), np.zeros(7))

    def loss(x, g, b):
        m, r = R.ln_stats64(x, 1e-2)
        return float(np.sum(dY * ((x - m[:, None]) * r[:, None] * g + b)))

    m, r = R.ln_stats64(X, 1e-2)
    dX, dg, db, _ = R.ln_bwd64(dY, X, m, r, g if affine else None)
    close(dX, differences(lambda x: loss(x, g, b), X))
    close(dg, differences(lambda v: loss(X, v, b), g))
    close(db, differences(lambda v: loss(X, g, v), b))


def test_gelu_gradient():
    x = np.linspace(-9, 9, 401)
    h = 1e-5
    close(R.act_grad64(x, "gelu"), (R.gelu64(x + h) - R.gelu64(x - h)) / (2 * h))
    assert R.act_grad64(np.array([0.0]), "gelu")[0] == 0.5
    assert np.max(np.abs(R.act_grad64(np.array([-1e30, 1e30]), "gelu") - [0.0, 1.0])) < 1e-300


def test_logprob_gradient():
    rng = np.random.default_rng(2)
    X = rng.standard_normal((3, 6))
    t, g, gh = np.array([1, -100, 5]), rng.standard_normal(3), rng.standard_normal(3)

    def loss(x):
        lp, h, _, _, _ = R.logprobs64(x, t)
        return float(np.sum(g * lp + gh * h))

    _, h, lse, _, _ = R.logprobs64(X, t)
    close(R.logprobs_bwd64(X, t, lse, h, g, gh), differences(loss, X))


def test_logprob_conventions():
    inf = np.inf
    X = np.array([[-inf, -inf, -inf], [0.0, -inf, 0.0], [1.0, np.nan, 0.0], [2.0, 2.0, 1.0]])
    lp, h, lse, top, tlp = R.logprobs64(X, [1, 2, 0, -1], topk=2)
    assert lse[0] == -inf and h[0] == 0 and lp[0] == -inf and list(top[0]) == [0, 1]
    assert abs(lp[1] + np.log(2)) < 1e-15 and abs(h[1] - np.log(2)) < 1e-15 and list(top[1]) == [0, 2]
    assert np.isnan(lse[2]) and np.isnan(lp[2]) and list(top[2]) == [0, 2]
    assert lp[3] == 0 and list(top[3]) == [0, 1] and tlp[3][0] == tlp[3][1]


def test_checkpoint_rule():
    X = np.array([[127.0, -63.5, 0.0, np.inf, 1.0, 2.0]], dtype=np.float32)
    Q, S = R.checkpoint_i8(X, 3)
    assert list(Q[0]) == [127, -63, 0, 0, 0, 0] and S[0, 0] == 1.0 and np.isnan(S[0, 1])
    Y = R.checkpoint_restore(Q, S, 3)
    assert list(Y[0, :3]) == [127.0, -63.0, 0.0] and np.isnan(Y[0, 3:]).all()
    # 127 * RN(a/127) is above a by up to 2^-23 of it: finite for all but the last few values of binary32
    big = np.float32(np.finfo(np.float32).max * (1 - 2.0 ** -22))
    Q, S = R.checkpoint_i8(np.array([[big, -big]], dtype=np.float32), 32)
    assert np.isfinite(R.checkpoint_restore(Q, S, 32)).all()
