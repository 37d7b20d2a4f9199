"""References in 64 bits and helpers for the tests of the two ends of a
training step (head.hip, embedding.hip); numpy, none of the library's code."""
import numpy as np
import torch

U32 = 2.0 ** -24            # half a step of binary32, relative
LOG2E = 1.4426950408889634


def codes(rng, rows, k, scale=None, zero_rows=()):
    """Random codes (-127 ... 127) and positive binary32 scales."""
    q = rng.integers(-127, 128, size=(rows, k)).astype(np.int8)
    for r in zero_rows:
        q[r % max(rows, 1)] = 0
    s = (rng.uniform(0.5, 1.5, size=rows) * (scale if scale is not None else 1.0)).astype(np.float32)
    return q, s


def padded(q, extra=0):
    """Codes on the GPU in rows of whole 16 bytes and `extra` times 16 more; what is behind a row is not 0."""
    rows, k = q.shape
    ld = max((k + 15) // 16 * 16, 16) + 16 * extra
    buf = torch.full((rows, ld), 85, dtype=torch.int8, device="cuda")
    buf[:, :k] = torch.from_numpy(q).cuda()
    return buf[:, :k]


def logits(qa, sa, qb, sb):
    """RN(RN(RN(acc) s_row) s_col) as float64 (binary32 values)."""
    acc = qa.astype(np.int64) @ qb.astype(np.int64).T
    with np.errstate(over="ignore", invalid="ignore"):
        y = acc.astype(np.float32) * sa[:, None].astype(np.float32)
        return (y * sb[None, :].astype(np.float32)).astype(np.float64)


def logsumexp(x):
    m = x.max(axis=1, keepdims=True)
    return (m + np.log(np.exp(x - m).sum(axis=1, keepdims=True)))[:, 0]


def logprobs(x, t):
    """(logprob, lse) of the rows of x in 64 bits."""
    lse = logsumexp(x)
    lp = np.zeros(len(x))
    real = (t >= 0) & (t < x.shape[1])
    lp[real] = x[real, t[real]] - lse[real]
    return lp, lse


def lse_bound(x):
    """How far the computed log-sum-exp may be from the exact one.

    In units of U32: the rounded argument of an exponential, t = (x - m) log2 e
    to half a step, is |t| ln 2 of its value, weighted by p; the exponential
    2 (1 ulp) and the rescalings of a tile's sums 6; a lane's 64 additions and
    the joining ones 72; binary32's log2 e is off by 0.23 units, which moves the
    exponents' scale: 0.23 (|lse| + sum p |x|).  Then lse's own rounding, |lse|.
    """
    lse = logsumexp(x)
    p = np.exp(x - lse[:, None])
    far = (p * np.abs(x - x.max(axis=1, keepdims=True))).sum(axis=1)
    size = (p * np.abs(x)).sum(axis=1)
    return U32 * (80 + far + 0.23 * (np.abs(lse) + size) + np.abs(lse)) * 1.01


def head_grads(qa, sa, qb, sb, t, lse, g, gl, terms, own=False):
    """(dA, dBt) in 64 bits for the given binary32 lse, and how far the computed
    ones may be before their outputs' rounding.

    A value of T: p's argument to half a step (|t| ln 2 units of U32, |t| the
    distance from lse in powers of two), the exponential and the row's factor
    2 + 2, products and the given token's sum 8; its rounding to one f16 2^-11 or
    to two 2^-22, and 2^-37 of the largest (|g| + |gl|) s_row s_col (with own: of
    the value's own, where all are within 2^24 of the largest).  Sums: one
    binary32 rounding for each 16 products and term, planes and scaling 8.
    """
    x = logits(qa, sa, qb, sb)
    m, n = x.shape
    with np.errstate(over="ignore"):
        p = np.exp(x - lse[:, None].astype(np.float64))
    real = (t >= 0) & (t < n)
    gi = np.where(real, g.astype(np.float64), 0.0) if g is not None else np.zeros(m)
    li = gl.astype(np.float64) if gl is not None else np.zeros(m)
    big = np.abs(lse) >= 2.0 ** 24
    gi, li = np.where(big, 0.0, gi), np.where(big, 0.0, li)
    p = np.where(big[:, None], 0.0, p)
    G = p * (li - gi)[:, None]
    size = p * (np.abs(li) + np.abs(gi))[:, None]           # what p's errors scale with
    one = np.zeros_like(x)
    one[np.flatnonzero(real), t[real]] = gi[real]
    G = G + one
    size = size + np.abs(one)
    a, b = sa[:, None].astype(np.float64) * qa, sb[:, None].astype(np.float64) * qb
    away = np.where(p > 0, np.abs(x - lse[:, None]), 0.0)
    bound_a = (np.abs(gi) + np.abs(li)) * sa
    largest = bound_a[:, None] * sb[None, :] if own else bound_a.max(initial=0.0) * sb.max(initial=0.0)
    rounding = 2.0 ** -11 if terms == 1 else 2.0 ** -22
    # in values of G s_row s_col
    offT = size * sa[:, None] * sb[None, :] * (U32 * (away + 12) + rounding) + 2.0 ** -37 * largest
    aq, bq = np.abs(qa.astype(np.float64)), np.abs(qb.astype(np.float64))
    sizeT = size * sa[:, None] * sb[None, :]
    off_a = (offT @ bq + sizeT @ bq * 2 * U32 * (terms * -(-n // 16) + 8)) / sa[:, None]
    off_b = (offT.T @ aq + sizeT.T @ aq * 2 * U32 * (terms * -(-m // 16) + 8)) / sb[:, None]
    return G @ b, G.T @ a, off_a, off_b


def embedding(w, tokens, alpha, pos, positions, dtype):
    """RN(RN(alpha w) + p) in binary32, as `dtype`; w: binary32 values, a torch tensor on the CPU."""
    vocab = w.shape[0]
    real = (tokens >= 0) & (tokens < vocab)
    y = w[tokens.clamp(0, max(vocab - 1, 0))] * torch.tensor(alpha, dtype=torch.float32)
    if pos is not None:
        there = (positions >= 0) & (positions < pos.shape[0])
        p = pos.float()[positions.clamp(0, pos.shape[0] - 1)]
        y = torch.where(there[:, None], y + p, y)
    return torch.where(real[:, None], y, torch.zeros(())).to(dtype)


def embedding_bwd(dy, tokens, vocab, alpha, add=None):
    """(dW, sum of the absolute values) in 64 bits."""
    real = (tokens >= 0) & (tokens < vocab)
    dw, size = np.zeros((vocab, dy.shape[1])), np.zeros((vocab, dy.shape[1]))
    np.add.at(dw, tokens[real], dy[real])
    np.add.at(size, tokens[real], np.abs(dy[real]))
    a = float(np.float32(alpha))
    dw, size = dw * a, size * abs(a)
    return (dw, size) if add is None else (dw + add, size + np.abs(add))
