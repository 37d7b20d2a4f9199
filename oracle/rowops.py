"""The operators between the GEMMs in numpy: layer norm, 8-bit activation
checkpoints, log probabilities of given tokens.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

Every function takes the values as float64 or float32 arrays and states what
it returns: the formula in binary64 (``*64``), or the library's definition
with each binary32 step rounded on its own (the others).
"""
import numpy as np

from . import ref

F32 = np.float32
U = 2.0 ** -24                 # half a step of binary32, relative


# ---- layer norm -------------------------------------------------------------
def ln_stats64(X, eps):
    """mean and rstd of each row in binary64."""
    X = np.asarray(X, dtype=np.float64)
    mean = X.mean(axis=1)
    var = np.square(X - mean[:, None]).mean(axis=1)
    return mean, 1.0 / np.sqrt(var + eps)


def ln_values(X, mean, rstd, gamma=None, beta=None):
    """RN(RN(RN(RN(x - mean) * rstd) * gamma) + beta) from binary32 statistics."""
    X = np.asarray(X, dtype=F32)
    g = np.ones(X.shape[1], dtype=F32) if gamma is None else np.asarray(gamma, dtype=F32)
    b = np.zeros(X.shape[1], dtype=F32) if beta is None else np.asarray(beta, dtype=F32)
    xh = (X - np.asarray(mean, dtype=F32)[:, None]).astype(F32) * np.asarray(rstd, dtype=F32)[:, None]
    return ((xh.astype(F32) * g).astype(F32) + b).astype(F32)


def ln_bwd64(dY, X, mean, rstd, gamma=None):
    """(dX, dgamma, dbeta, bounds) in binary64 from given statistics.  bounds
    holds how far the library's binary32 steps may be off: for dX one bound a
    value, for dgamma and dbeta one a column."""
    dY, X = np.asarray(dY, np.float64), np.asarray(X, np.float64)
    mean, rstd = np.asarray(mean, np.float64)[:, None], np.asarray(rstd, np.float64)[:, None]
    n = X.shape[1]
    w = dY if gamma is None else dY * np.asarray(gamma, np.float64)
    xh = (X - mean) * rstd
    c1 = w.mean(axis=1, keepdims=True)
    c2 = (w * xh).mean(axis=1, keepdims=True)
    dX = rstd * (w - c1 - xh * c2)
    # relative errors, in units of U: w 1, xh 2, w*xh 3, c1 1 + those of w, c2 1 + 3
    m1, m2 = np.abs(w).mean(axis=1, keepdims=True), np.abs(w * xh).mean(axis=1, keepdims=True)
    a = np.abs(w) + m1 + np.abs(c1)                       # w - c1 before its own rounding
    b = 3 * np.abs(xh * c2) + np.abs(xh) * (3 * m2 + np.abs(c2))   # xh * c2 with its rounding
    total = a + b + 3 * (np.abs(w - c1) + np.abs(xh * c2))         # two subtractions, the last product
    bound = 1.01 * U * np.abs(rstd) * total + 2.0 ** -148
    dgamma, dbeta = (dY * xh).sum(axis=0), dY.sum(axis=0)
    sg, sb = np.abs(dY * xh).sum(axis=0), np.abs(dY).sum(axis=0)
    e64 = 2.0 ** -52 * max(X.shape[0], 1)
    return dX, dgamma, dbeta, (bound, 1.01 * U * (np.abs(dgamma) + 2 * sg) + e64 * sg,
                               1.01 * U * np.abs(dbeta) + e64 * sb)


# ---- checkpoints ------------------------------------------------------------
def checkpoint_i8(X, group):
    """Codes and scales of each group of columns (ref.quantize_rows' rule); a
    group with an infinity or a NaN: scale NaN, codes 0."""
    X = np.asarray(X, dtype=F32)
    rows, cols = X.shape
    n = -(-cols // group) if group else 1
    Q = np.zeros((rows, cols), dtype=np.int8)
    S = np.empty((rows, n), dtype=F32)
    for g in range(n):
        sl = slice(g * group, (g + 1) * group) if group else slice(None)
        part = X[:, sl]
        bad = ~np.isfinite(part).all(axis=1)
        q, s = ref.quantize_rows(np.where(bad[:, None], F32(0), part))
        Q[:, sl] = q
        S[:, g] = np.where(bad, F32(np.nan), s)
    return Q, S


def checkpoint_restore(Q, S, group):
    """RN(q * s)."""
    Q = np.asarray(Q)
    column = np.arange(Q.shape[1]) // group if group else np.zeros(Q.shape[1], dtype=np.int64)
    return (Q.astype(F32) * np.asarray(S, dtype=F32).reshape(Q.shape[0], -1)[:, column]).astype(F32)


def gelu64(x):
    u = np.sqrt(2 / np.pi) * (x + 0.044715 * x ** 3)
    return 0.5 * x * (1 + np.tanh(u))


def act_grad64(x, act):
    """The derivative of the activation function in binary64."""
    x = np.asarray(x, dtype=np.float64)
    if act == "relu":
        return (x > 0).astype(np.float64)
    c, a = np.sqrt(2 / np.pi), 0.044715
    z = np.minimum(np.abs(2 * c * (x + a * x ** 3)), 700.0)
    e = np.exp(-z)
    p = np.where(x < 0, e, 1.0) / (1 + e)
    with np.errstate(over="ignore"):
        rest = x * (e / (1 + e) ** 2) * 2 * c * (1 + 3 * a * x * x)
    return p + np.where(z >= 700.0, 0.0, rest)


# ---- log probabilities ------------------------------------------------------
def logprobs64(X, targets, topk=0):
    """(logprob, entropy, lse, top_index, top_logprob) in binary64, with the
    library's conventions for missing tokens, -inf and NaN."""
    X = np.asarray(X, dtype=np.float64)
    rows, vocab = X.shape
    lp = np.full((rows, vocab), -np.inf)
    lse, ent = np.empty(rows), np.empty(rows)
    for i in range(rows):
        x = X[i]
        if np.isnan(x).any() or (x == np.inf).any():
            lse[i] = ent[i] = np.nan
            lp[i] = np.nan
            continue
        m = x.max()
        if m == -np.inf:
            lse[i], ent[i] = -np.inf, 0.0
            continue
        e = np.exp(x - m)
        s = e.sum()
        lse[i] = m + np.log(s)
        lp[i] = x - m - np.log(s)
        live = e > 0
        ent[i] = -(e[live] / s * lp[i][live]).sum()
    targets = np.asarray(targets)
    given = (targets >= 0) & (targets < vocab)
    logprob = np.where(given, lp[np.arange(rows), np.where(given, targets, 0)], 0.0)
    order = np.argsort(-np.where(np.isnan(X), -np.inf, X), axis=1, kind="stable")[:, :topk]
    return logprob, ent, lse, order, np.take_along_axis(lp, order, axis=1)


def logprobs_bwd64(X, targets, lse, entropy, g, gh):
    """The gradient in binary64 from given lse and entropy."""
    X = np.asarray(X, dtype=np.float64)
    rows, vocab = X.shape
    lse = np.asarray(lse, np.float64)[:, None]
    dead = np.abs(lse) >= 2.0 ** 24
    lp = X - np.where(dead, 0.0, lse)
    p = np.where(dead, 0.0, np.exp(lp))
    lp = np.where(np.isneginf(lp), 0.0, lp)
    d = np.zeros((rows, vocab))
    if gh is not None:
        d -= np.asarray(gh, np.float64)[:, None] * p * (lp + np.asarray(entropy, np.float64)[:, None])
    if g is not None:
        targets = np.asarray(targets)
        given = (targets >= 0) & (targets < vocab)
        gg = np.where(given, np.asarray(g, np.float64), 0.0)
        d -= gg[:, None] * p
        d[np.arange(rows)[given], targets[given]] += np.where(dead[given, 0], 0.0, gg[given])
    return d
