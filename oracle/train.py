"""The training step's operators beside the GEMMs (oracle; test
infrastructure only): the router with its balance loss, the combine over
partly routed tokens and its backward pass, the expert activation with an
MXFP8 checkpoint, and the weight gradient over MXFP8 rows.

The pages the library follows have no router, no loss and no backward pass
but the weight gradient; these are the plain definitions in float64, as
include/moe_train.h states them. The forward functions share nothing with the
gradient functions but the scores, so central differences of the first pin
the second (tests/test_oracle_train.py).

Each function that a GPU result in fp32 is compared with also returns, where
cancellation matters, the size of the terms that were added up ("size"): the
rounding errors of a computation in fp32 are relative to it.
"""

import numpy as np

from .gemm import relu2, silu
from .quant import mx_dequantize_e4m3, mx_quantize_e4m3


def _exp(x):
    with np.errstate(over="ignore", invalid="ignore"):
        return np.exp(x)


def log_scores(z, score):
    """a with softmax(a) the probabilities: z, or log sigmoid(z)."""
    z = np.asarray(z, dtype=np.float64)
    if score == "softmax":
        return z
    with np.errstate(invalid="ignore"):
        return np.where(z > 0, 0.0, z) - np.log1p(_exp(-np.abs(z)))


def softmax_lse(a):
    """(softmax over the last axis, log of the sum of exponentials); a row of
    -inf gives zeros and -inf."""
    with np.errstate(invalid="ignore", divide="ignore"):
        m = a.max(axis=-1, keepdims=True)
        m0 = np.where(np.isneginf(m), 0.0, m)
        e = _exp(a - m0)
        s = e.sum(axis=-1, keepdims=True)
        q = np.where(s > 0, e / np.where(s == 0, 1.0, s), 0.0)
        q = np.where(np.isnan(s), np.nan, q)
        return q, (m0 + np.log(s))[..., 0]


def choose(z, top_k, mask=None):
    """The chosen experts [T, top_k]: by logit, largest first, ties lowest
    expert first; -inf and NaN never; -1 in places left over and padded rows."""
    z = np.asarray(z, dtype=np.float64)
    key = np.where(np.isnan(z), -np.inf, z)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :top_k]
    ids = np.where(np.isneginf(np.take_along_axis(key, ids, 1)), -1, ids)
    if mask is not None:
        ids = np.where(np.asarray(mask)[:, None] != 0, ids, -1)
    return ids.astype(np.int32)


def chosen_scores(z, ids, score, renormalize):
    """v [T, top_k]: the chosen experts' scores, 0 in places of -1."""
    a = log_scores(z, score)
    ix = np.maximum(ids, 0)
    on = ids >= 0
    if renormalize:
        v, _ = softmax_lse(np.where(on, np.take_along_axis(a, ix, 1), -np.inf))
        return v
    v = np.take_along_axis(softmax_lse(a)[0], ix, 1) if score == "softmax" else \
        _exp(np.take_along_axis(a, ix, 1))
    return np.where(on, v, 0.0)


def routed_rows(z, mask=None):
    z = np.asarray(z, dtype=np.float64)
    live = ~np.isneginf(z).all(axis=1)
    return live if mask is None else live & (np.asarray(mask) != 0)


def losses(z, ids, score, mask=None, counts=None):
    """(counts [E], n, prob_sum [E], [balance loss, z loss]). counts may be
    given (held constant, as the gradient does)."""
    z = np.asarray(z, dtype=np.float64)
    E, k = z.shape[1], ids.shape[1]
    live = routed_rows(z, mask)
    n = int(live.sum())
    if counts is None:
        counts = np.bincount(ids[ids >= 0], minlength=E)
    if n == 0:
        return counts, 0, np.zeros(E), np.zeros(2)
    q, lse = softmax_lse(log_scores(z, score))
    p = q[live].sum(axis=0)
    zl = (lse[live] ** 2).sum() / n if score == "softmax" else 0.0
    return counts, n, p, np.array([E / (k * n * n) * (counts * p).sum(), zl])


def route(z, top_k, score="softmax", renormalize=True, scale=1.0, mask=None):
    """(ids, w, counts, n, prob_sum, losses).
    Pinned: closed forms on uniform and one-hot logits, a scalar loop, ties,
    masked experts and rows."""
    ids = choose(z, top_k, mask)
    w = scale * chosen_scores(z, ids, score, renormalize)
    return (ids, w) + losses(z, ids, score, mask)


def route_backward(z, ids, dw, score="softmax", renormalize=True, scale=1.0, counts=None, n=0, dlosses=None):
    """(dlogits, size) [T, E]. Pinned: central differences of route()."""
    z = np.asarray(z, dtype=np.float64)
    T, E = z.shape
    k = ids.shape[1]
    live = ids[:, 0] >= 0
    on = (ids >= 0) & (ids < E)
    ids = np.where(on, ids, -1)
    a = log_scores(z, score)
    q, lse = softmax_lse(a)
    v = chosen_scores(z, ids, score, renormalize)
    g = np.where(on, scale * np.asarray(dw, dtype=np.float64), 0.0)
    gv = (g * v).sum(axis=1, keepdims=True)
    u = v * (g - gv) if renormalize else v * g
    us = v * (np.abs(g) + np.abs(g * v).sum(axis=1, keepdims=True)) if renormalize else np.abs(u)
    common = np.zeros((T, 1))
    size = np.zeros((T, 1))
    if score == "softmax" and not renormalize:
        common, size = common - u.sum(axis=1, keepdims=True), size + us.sum(axis=1, keepdims=True)
    c = np.zeros(E)
    if dlosses is not None and n > 0:
        c = dlosses[0] * E / (k * n * n) * np.asarray(counts, dtype=np.float64)
        if score == "softmax":
            zt = 2 * dlosses[1] * np.where(live, lse, 0.0)[:, None] / n
            common, size = common + zt, size + np.abs(zt)
    common = common + c[None, :] - (q * c).sum(axis=1, keepdims=True)
    size = size + np.abs(c)[None, :] + (q * np.abs(c)).sum(axis=1, keepdims=True)
    da, size = q * common, q * size
    rows = np.repeat(np.arange(T), k).reshape(T, k)
    np.add.at(da, (rows[on], ids[on]), u[on])
    np.add.at(size, (rows[on], ids[on]), us[on])
    if score == "sigmoid":
        f = 1.0 / (1.0 + _exp(z))
        da, size = da * f, size * f
    return np.where(live[:, None], da, 0.0), np.where(live[:, None], size, 0.0)


def combine_routed(c, topk_w, ids, num_experts):
    """y[t] = sum over the routed slots of w * c. Pinned: gemm.combine with
    the unrouted slots' rows and weights zero."""
    T, k = ids.shape
    on = (ids >= 0) & (ids < num_experts)
    y = np.zeros((T, c.shape[1]))
    for t in range(T):
        for j in range(k):
            if on[t, j]:
                y[t] += float(topk_w[t, j]) * c[t * k + j]
    return y


def combine_backward(dy, c, topk_w, ids=None, num_experts=0):
    """(dC, dtopk_w, size of the dot products). Pinned: linearity in dy and
    differences of combine_routed."""
    T, k = topk_w.shape
    on = np.ones((T, k), dtype=bool) if ids is None else (ids >= 0) & (ids < num_experts)
    dc = np.zeros((T * k, dy.shape[1]))
    dw, size = np.zeros((T, k)), np.zeros((T, k))
    for t, j in zip(*np.nonzero(on)):
        dc[t * k + j] = topk_w[t, j] * dy[t]
        dw[t, j] = (dy[t] * c[t * k + j]).sum()
        size[t, j] = np.abs(dy[t] * c[t * k + j]).sum()
    return dc, dw, size


def act(pre, activation):
    """h = swiglu(pre) or max(pre, 0)^2 over float64 rows."""
    if activation == "relu2":
        return relu2(pre)
    half = pre.shape[1] // 2
    return silu(pre[:, :half]) * pre[:, half:]


def act_mxfp8(pre, activation):
    """(h, codes, scales). Pinned: its parts are (gemm, quant)."""
    return (act(pre, activation),) + mx_quantize_e4m3(pre)


def act_backward(codes, scales, dh, activation):
    """(dpre, h, size of dpre's terms) from the checkpoint.
    Pinned: central differences of act() at the decoded values."""
    v = mx_dequantize_e4m3(codes, scales)
    dh = np.asarray(dh, dtype=np.float64)
    if activation == "relu2":
        d = np.where(v > 0, 2 * v * dh, 0.0)
        return d, relu2(v), np.abs(d)
    half = v.shape[1] // 2
    g, u = v[:, :half], v[:, half:]
    s = 1.0 / (1.0 + _exp(-g))
    dg, du = dh * u * s * (1 + g * (1 - s)), dh * g * s
    size = np.abs(dh * u) * s * (1 + np.abs(g) * (1 - s))
    return np.concatenate([dg, du], 1), g * s * u, np.concatenate([size, np.abs(du)], 1)


def wgrad_mxfp8_expert(codes, scales, grad, topk_ids, top_k, expert):
    """(dW[expert], size) [N, K]; grad float64 [S, N].
    Pinned: wgrad.wgrad_expert on the decoded rows."""
    ids = np.asarray(topk_ids).reshape(-1).astype(np.int64)
    slots = np.nonzero(ids == int(expert))[0]
    x = mx_dequantize_e4m3(codes[slots // top_k], scales[slots // top_k])
    g = np.asarray(grad[slots], dtype=np.float64)
    return g.T @ x, np.abs(g).T @ np.abs(x)
