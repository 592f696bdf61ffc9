"""Pins for the oracle's block operators: known answers, closed forms and
central differences."""

import numpy as np
import pytest
import torch

from oracle import block, formats


def _hex(words):
    return " ".join(f"{int(w):08x}" for w in words)


@pytest.mark.parametrize("counter,key,answer", [
    ([0, 0, 0, 0], [0, 0], "6627e8d5 e169c58d bc57ac4c 9b00dbd8"),
    ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, "408f276d 41c83b0e a20bc7c6 6d5451fd"),
    ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
     "d16cfe09 94fdcceb 5001e420 24126ea1"),
])
def test_philox_known_answers(counter, key, answer):
    assert _hex(block.philox4x32(np.array(counter), key)) == answer


def test_dropout_bit_order():
    # piece 0 of key and offset 0: 16-bit numbers e8d5 6627 c58d e169 ac4c bc57 dbd8 9b00
    halves = [0xE8D5, 0x6627, 0xC58D, 0xE169, 0xAC4C, 0xBC57, 0xDBD8, 0x9B00]
    for p in (0.25, 0.5, 0.75):
        keep = block.dropout_keep(1, 8, p, 0, 0)
        assert list(keep[0]) == [h >= p * 65536 for h in halves]
    # offset and element number are the counter's halves, seed the key
    w = block.philox4x32(np.array([1, 0, 5, 7]), [9, 3])
    keep = block.dropout_keep(2, 8, 0.5, 9 + (3 << 32), 5 + (7 << 32))
    assert list(keep[1]) == [h >= 32768 for v in w for h in (int(v) & 0xFFFF, int(v) >> 16)]


def test_dropout_values():
    x = np.arange(1.0, 8 * 4096 + 1).reshape(8, 4096)
    assert (block.dropout(x, 0.0) == x).all()
    assert (block.dropout(x, 1.0, 1, 2) == 0).all()
    assert (block.dropout(x, 2.0 ** -18, 1, 2) == x).all()      # a threshold of 0
    y = block.dropout(x, 0.25, 11, 3)
    kept = y != 0
    np.testing.assert_allclose(y[kept], x[kept] / 0.75)
    n = x.size
    assert abs(kept.sum() - 0.75 * n) < 5 * np.sqrt(n * 0.75 * 0.25)
    # the mask belongs to the element's number, not to the shape
    assert (block.dropout_keep(4, 8192, 0.25, 11, 3).reshape(-1) == kept.reshape(-1)).all()
    assert (block.dropout_keep(8, 4096, 0.25, 11, 4) != kept).mean() > 0.3
    assert (block.dropout_keep(8, 4096, 0.25, 12, 3) != kept).mean() > 0.3


def test_rmsnorm_closed_forms():
    v = np.array([[3.0, -4.0, 0.0, 0.0]])
    np.testing.assert_allclose(block.rmsnorm(v, np.array([1.0, 2.0, 3.0, 4.0]), 0.0), [[1.2, -3.2, 0, 0]])
    np.testing.assert_allclose(block.rmsnorm(v, np.ones(4), 93.75), v / 10)   # mean square 6.25
    r = np.random.default_rng(1).standard_normal((5, 32))
    np.testing.assert_allclose((block.rmsnorm(r, np.ones(32), 0.0) ** 2).mean(axis=1), 1.0)
    np.testing.assert_allclose(block.rmsnorm(7 * r, np.ones(32), 0.0), block.rmsnorm(r, np.ones(32), 0.0))


def test_rmsnorm_backward_by_differences():
    g = np.random.default_rng(2)
    v, w, dy, dsum = g.standard_normal((4, 16)), g.standard_normal(16), g.standard_normal((4, 16)), g.standard_normal((4, 16))
    dv, dw = block.rmsnorm_backward(dy, v, w, 0.3, dsum)

    def loss(v, w):
        return (dy * block.rmsnorm(v, w, 0.3)).sum() + (dsum * v).sum()

    h = 1e-6
    for i in np.ndindex(4, 16):
        e = np.zeros((4, 16))
        e[i] = h
        assert abs((loss(v + e, w) - loss(v - e, w)) / (2 * h) - dv[i]) < 1e-7
    for i in range(16):
        e = np.zeros(16)
        e[i] = h
        assert abs((loss(v, w + e) - loss(v, w - e)) / (2 * h) - dw[i]) < 1e-7


def test_quantize_per_token():
    u = np.random.default_rng(3).standard_normal((6, 64)) * np.exp2(np.arange(6.0) * 7 - 20)[:, None]
    u[2] = 0
    q, s = block.quantize_per_token(u)
    np.testing.assert_allclose(s[[0, 1, 3]], np.abs(u).max(axis=1)[[0, 1, 3]] / 448)
    assert s[2] == 2.0 ** -126 and (q[2] == 0).all()
    ref = torch.from_numpy(u / s[:, None]).float().to(torch.float8_e4m3fn).float().double().numpy()
    np.testing.assert_array_equal(q, ref)


def test_quantize_mxfp8_is_the_rule_of_the_quantizer():
    u = np.random.default_rng(4).standard_normal((3, 64))
    q, s = block.quantize_mxfp8(u)
    top = np.abs(u.reshape(3, 2, 32)).max(axis=2)
    np.testing.assert_array_equal(s, np.floor(np.log2(top)) - 8 + 127)
    back = formats.e4m3_to_f64(q) * np.repeat(np.exp2(s.astype(float) - 127), 32, axis=1)
    assert (np.abs(back - u) <= np.maximum(2.0 ** -4 * np.abs(u), np.repeat(np.exp2(s - 137.0), 32, axis=1)) +
            np.repeat(64 * np.exp2(s - 127.0), 32, axis=1) * (np.abs(u) > 448 * np.repeat(np.exp2(s - 127.0), 32, axis=1))).all()


def _lora_case(S, G, R, K, N, div, seed):
    g = np.random.default_rng(seed)
    ids = g.integers(-1, G, S)
    return (g.standard_normal((S, N)), g.standard_normal((-(-S // div), K)), g.standard_normal((G, R, K)),
            g.standard_normal((G, N, R)), ids, g.standard_normal(G), div)


def test_lora_is_a_merged_weight():
    c, x, a, b, ids, scale, div = _lora_case(11, 3, 2, 5, 4, 2, 1)
    out, h = block.lora(c, x, a, b, ids, scale, div)
    for s, g in enumerate(ids):
        want = c[s] if g < 0 else c[s] + (scale[g] * b[g] @ a[g]) @ x[s // div]
        np.testing.assert_allclose(out[s], want)
    assert (h[ids < 0] == 0).all()
    np.testing.assert_array_equal(block.lora(c, x, a, b, ids, None, div)[0], block.lora(c, x, a, b, ids, np.ones(3), div)[0])


def test_lora_backward_by_differences():
    c, x, a, b, ids, scale, _ = _lora_case(6, 3, 2, 5, 4, 1, 2)
    dy = np.random.default_rng(3).standard_normal(c.shape)
    dx, da, db = block.lora_backward(dy, x, a, b, ids, block.lora(c, x, a, b, ids, scale)[1], scale)
    for t, d in ((x, dx), (a, da), (b, db)):
        for i in np.ndindex(*t.shape):
            old, f = t[i], []
            for e in (1e-6, -1e-6):
                t[i] = old + e
                f.append((dy * block.lora(c, x, a, b, ids, scale)[0]).sum())
            t[i] = old
            assert abs((f[0] - f[1]) / 2e-6 - d[i]) < 1e-6


def test_lora_backward_of_shared_rows():
    # two slots of one row of x: dx stays by slot, da adds them
    c, x, a, b, _, scale, _ = _lora_case(4, 2, 2, 5, 4, 2, 4)
    dy, ids = np.random.default_rng(5).standard_normal(c.shape), np.array([0, 1, 1, -1])
    h = block.lora(c, x, a, b, ids, scale, 2)[1]
    dx, da, db = block.lora_backward(dy, x, a, b, ids, h, scale, 2)
    wide = block.lora_backward(dy, x[[0, 0, 1, 1]], a, b, ids, h, scale, 1)
    for u, v in zip((dx, da, db), wide):
        np.testing.assert_allclose(u, v)
