"""Pins for the oracle's training operators: closed forms, brute force and
central differences."""

import numpy as np
import pytest

from oracle import formats, gemm, quant, train, wgrad


def _logits(T, E, seed):
    return np.random.default_rng(seed).standard_normal((T, E)) * 1.5


def test_route_uniform_logits():
    # equal logits: the lowest experts are chosen, every probability is 1/E
    z = np.full((4, 8), 0.3)
    ids, w, counts, n, p, loss = train.route(z, 3)
    assert (ids == [0, 1, 2]).all() and n == 4
    np.testing.assert_allclose(w, 1 / 3)
    np.testing.assert_array_equal(counts, [4, 4, 4, 0, 0, 0, 0, 0])
    np.testing.assert_allclose(p, 4 / 8)
    np.testing.assert_allclose(loss, [1.0, (0.3 + np.log(8)) ** 2])
    _, w, *_ = train.route(z, 3, renormalize=False, scale=2.0)
    np.testing.assert_allclose(w, 2 / 8)
    _, w, _, _, p, loss = train.route(z, 3, score="sigmoid", renormalize=False)
    np.testing.assert_allclose(w, 1 / (1 + np.exp(-0.3)))
    np.testing.assert_allclose(p, 4 / 8)
    assert loss[1] == 0


def test_route_collapsed_router_has_the_largest_loss():
    # every token sends everything to expert 2: E * 1 * 1
    z = np.zeros((5, 6))
    z[:, 2] = 80.0
    ids, w, counts, n, p, loss = train.route(z, 1)
    assert (ids == 2).all() and counts[2] == 5
    np.testing.assert_allclose(loss[0], 6.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_scalar_loop(score, renorm):
    T, E, k = 7, 9, 4
    z = _logits(T, E, 1)
    mask = np.array([1, 1, 0, 1, 1, 0, 1])
    ids, w, counts, n, p, loss = train.route(z, k, score, renorm, 2.5, mask)
    f, P, zl = np.zeros(E), np.zeros(E), 0.0
    for t in range(T):
        if not mask[t]:
            assert (ids[t] == -1).all() and (w[t] == 0).all()
            continue
        s = [np.exp(x) for x in z[t]] if score == "softmax" else [1 / (1 + np.exp(-x)) for x in z[t]]
        order = sorted(range(E), key=lambda e: (-z[t, e], e))[:k]
        assert list(ids[t]) == order
        total = sum(s[e] for e in order) if renorm else (sum(s) if score == "softmax" else 1.0)
        for j, e in enumerate(order):
            assert abs(w[t, j] - 2.5 * s[e] / total) < 1e-12
            f[e] += 1 / (n * k)
        P += np.array(s) / sum(s) / n
        zl += np.log(sum(s)) ** 2 / n
    assert abs(loss[0] - E * (f * P).sum()) < 1e-12
    assert abs(loss[1] - (zl if score == "softmax" else 0)) < 1e-12


def test_route_masked_experts_and_rows():
    z = np.zeros((4, 5))
    z[0] = [-np.inf, 1.0, -np.inf, 2.0, -np.inf]
    z[1] = -np.inf
    z[2] = -3.38e38                       # masks of the type's lowest value are numbers
    z[3] = [np.nan, 0.0, 1.0, -np.inf, 2.0]
    ids, w, counts, n, p, loss = train.route(z, 3)
    assert list(ids[0]) == [3, 1, -1] and list(ids[1]) == [-1] * 3 and list(ids[2]) == [0, 1, 2]
    assert list(ids[3]) == [4, 2, 1] and n == 3
    np.testing.assert_allclose(w[0], [np.e / (1 + np.e), 1 / (1 + np.e), 0])
    np.testing.assert_allclose(w[2], 1 / 3)
    assert (w[1] == 0).all() and np.isfinite(w[3]).all() and np.isnan(p).all() and np.isnan(loss).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_differences(score, renorm):
    T, E, k = 6, 10, 3
    z = _logits(T, E, 2)
    mask = np.array([1, 1, 1, 0, 1, 1])
    rng = np.random.default_rng(3)
    dw, dl = rng.standard_normal((T, k)), np.array([0.7, -0.3])
    ids, _, counts, n, _, _ = train.route(z, k, score, renorm, 1.7, mask)

    def value(z):
        w = 1.7 * train.chosen_scores(z, ids, score, renorm)
        loss = train.losses(z, ids, score, mask, counts=counts)[3]
        return (w * dw * (ids >= 0)).sum() + (loss * dl).sum()

    got, size = train.route_backward(z, ids, dw, score, renorm, 1.7, counts, n, dl)
    assert (got[3] == 0).all() and (np.abs(got) <= size + 1e-15).all()
    for t in range(T):
        for e in range(E):
            d = np.zeros_like(z)
            d[t, e] = 1e-5
            assert abs((value(z + d) - value(z - d)) / 2e-5 - got[t, e]) < 1e-8


def test_route_backward_ignores_places_of_minus_one():
    z = np.array([[-np.inf, 1.0, -np.inf, 2.0]])
    ids, w, counts, n, _, _ = train.route(z, 3)
    g, _ = train.route_backward(z, ids, np.array([[1.0, 2.0, np.nan]]))
    v = w[0, :2]
    want = v * (np.array([1.0, 2.0]) - (v * [1.0, 2.0]).sum())
    np.testing.assert_allclose(g[0], [0, want[1], 0, want[0]])


def test_combine_routed_and_backward():
    T, k, N, E = 4, 3, 5, 6
    rng = np.random.default_rng(4)
    c, w = rng.standard_normal((T * k, N)), rng.random((T, k))
    ids = np.array([[0, 5, 2], [-1, 1, 6], [3, 4, 0], [-1, -1, -1]])
    on = (ids >= 0) & (ids < E)
    bad = c.copy()
    bad[~on.reshape(-1)] = np.nan
    y = train.combine_routed(bad, w, ids, E)
    np.testing.assert_allclose(y, gemm.combine(np.where(on.reshape(-1, 1), c, 0), w * on, k))
    dy = rng.standard_normal((T, N))
    dc, dw, _ = train.combine_backward(dy, bad, w, ids, E)
    assert (dc[~on.reshape(-1)] == 0).all() and (dw[~on] == 0).all()
    for t in range(T):
        for j in range(k):
            if on[t, j]:
                d = np.zeros_like(w)
                d[t, j] = 1.0
                np.testing.assert_allclose(dw[t, j], (dy * train.combine_routed(c, d, ids, E)).sum())
                np.testing.assert_allclose(dc[t * k + j], w[t, j] * dy[t])
    full, _, _ = train.combine_backward(dy, c, w)
    np.testing.assert_allclose(full, np.repeat(dy, k, 0) * w.reshape(-1, 1))


@pytest.mark.parametrize("activation", ["swiglu", "relu2"])
def test_act_backward_differences(activation):
    rng = np.random.default_rng(5)
    pre = rng.standard_normal((3, 128)) * 2
    h, q, s = train.act_mxfp8(pre, activation)
    rq, rs = quant.mx_quantize_e4m3(pre)
    assert np.array_equal(q, rq) and np.array_equal(s, rs)
    v = quant.mx_dequantize_e4m3(q, s)
    # half a step of E4M3 (2^-4 relative, 2^-10 of the scale when subnormal);
    # what lies in (448, 512) scales, which only a block's maximum's binade
    # reaches, saturates at 448 scales
    x = np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, axis=1)
    near = np.minimum(np.abs(pre), 448 * x)
    assert (np.abs(np.abs(v) - near) <= np.maximum(2.0 ** -4 * near, 2.0 ** -10 * x)).all()
    dh = rng.standard_normal(h.shape)
    d, h2, size = train.act_backward(q, s, dh, activation)
    np.testing.assert_allclose(h2, train.act(v, activation), atol=1e-15)
    assert (np.abs(d) <= size * (1 + 1e-12)).all()
    step = np.zeros_like(v)
    for i in range(0, 128, 5):
        step[:, i] = 1e-6
        num = (dh * (train.act(v + step, activation) - train.act(v - step, activation))).sum(1) / 2e-6
        np.testing.assert_allclose(d[:, i], num, rtol=1e-6, atol=1e-6)
        step[:, i] = 0


def test_act_closed_forms():
    # swiglu at g = 0: h = 0, dg = dh u / 2, du = 0; relu2 at +-3
    v = np.zeros((1, 64))
    v[0, 32:] = 2.0
    q, s = quant.mx_quantize_e4m3(v)
    d, h, _ = train.act_backward(q, s, np.ones((1, 32)), "swiglu")
    assert (h == 0).all() and (d[0, :32] == 1.0).all() and (d[0, 32:] == 0).all()
    q, s = quant.mx_quantize_e4m3(np.array([[3.0, -3.0] * 16]))
    d, h, _ = train.act_backward(q, s, np.ones((1, 32)), "relu2")
    assert list(d[0, :2]) == [6.0, 0.0] and list(h[0, :2]) == [9.0, 0.0]


def test_wgrad_mxfp8_is_wgrad_of_the_decoded_rows():
    T, k, E, N, K = 9, 2, 4, 5, 64
    rng = np.random.default_rng(6)
    q, s = quant.mx_quantize_e4m3(rng.standard_normal((T, K)))
    v = quant.mx_dequantize_e4m3(q, s)
    bits = (v.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    assert np.array_equal(formats.bf16_to_f64(bits), v)  # exact in bf16
    g = (rng.integers(-8, 9, (T * k, N)) / 4.0).astype(np.float32)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    for e in range(E):
        dw, size = train.wgrad_mxfp8_expert(q, s, g, ids, k, e)
        ref = wgrad.wgrad_expert(bits, (g.view(np.uint32) >> 16).astype(np.uint16), ids, k, e)
        np.testing.assert_allclose(dw, ref)
        assert (np.abs(dw) <= size + 1e-12).all()
