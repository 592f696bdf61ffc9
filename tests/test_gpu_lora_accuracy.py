"""GPU tests of moe_lora and moe_lora_backward at inputs whose sums fp32 holds
exactly in any order, so that an output has one right value: the float64
result, rounded once. What is multiplied with the second matrix, h or dh, then
needs 20 bits of its 24, where two bf16 terms hold 16 or 17.

An intermediate is a sum of three products, chunks of 8 bits of an integer
below 2^20 with powers of two; the second matrix holds at most 16 entries +-1 in
a row, so its sums stay below 2^24 units.
"""

import numpy as np
import pytest
import torch

from block_helpers import f64
from helpers import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def _moe():
    import mixture_experts_grouped_moe_amd as moe
    return moe


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16).cuda()


def chunked(rng, rows, R, width):
    """(matrix [R, width], rows' values [rows, width], their products [rows, R])
    as in the docstring."""
    m = rng.integers(-(1 << 20) + 1, 1 << 20, size=(rows, R))
    mat, val = np.zeros((R, width)), rng.integers(-4, 5, size=(rows, width)).astype(np.float64)
    for j in range(3):
        mat[np.arange(R), 3 * np.arange(R) + j] = 2.0 ** (8 * j - 20)
        val[:, 3 * np.arange(R) + j] = np.sign(m) * ((np.abs(m) >> (8 * j)) & 255)
    return mat, val, m * 2.0 ** -20


def signs(rng, G, rows, R):
    """[G, rows, R] of +-1 at up to 16 places of a row."""
    out = np.zeros((G, rows, R))
    at = np.argsort(rng.random((G, rows, R)), axis=2)[:, :, :16]
    np.put_along_axis(out, at, rng.choice([-1.0, 1.0], size=at.shape), axis=2)
    return out


# every rank in the kernels (8, 16, 32, 64, 128 and between); few slots and many
CASES = [(5, 2, 8, 16), (40, 3, 16, 16), (28, 2, 32, 8), (60, 2, 64, 16), (300, 2, 128, 16), (50, 2, 40, 64),
         (2000, 3, 8, 64), (3000, 2, 16, 64), (1500, 2, 24, 64), (1500, 2, 32, 32), (1500, 2, 64, 64), (1500, 2, 128, 64)]


def case(S, G, R, bm):
    rng = np.random.default_rng(S + R)
    ids = rng.integers(0, G, size=S).astype(np.int32)
    routing = _moe().moe_align(torch.from_numpy(ids).reshape(S, 1).cuda(), G, bm)
    scale = np.array([0.5, -1.0, 2.0])[:G]
    return rng, ids, routing, scale, torch.from_numpy(scale.astype(np.float32)).cuda(), 3 * R + 512, 264


@pytest.mark.parametrize("S,G,R,bm", CASES)
def test_what_is_added_to_c(S, G, R, bm):
    rng, ids, routing, scale, s_t, wide, narrow = case(S, G, R, bm)
    a, x, h = chunked(rng, S, R, wide)
    b = signs(rng, G, narrow, R)
    delta = scale[ids][:, None] * np.einsum("snr,sr->sn", b[ids], h)
    c = bf16(-delta)                 # so that what is left of the sum shows every bit
    want = bf16(f64(c) + delta)      # (exact in fp32, rounded once)
    out, kept = _moe().moe_lora(c, bf16(x), bf16(np.stack([a] * G)), bf16(b), routing, s_t, keep_h=True)
    assert np.array_equal(f64(kept), h)
    off = (out != want).sum().item()
    assert off == 0, f"{off} of {want.numel()} elements of c"


@pytest.mark.parametrize("S,G,R,bm", CASES)
def test_what_is_added_to_dx(S, G, R, bm):
    rng, ids, routing, scale, s_t, wide, narrow = case(S, G, R, bm)
    b, dy, dh = chunked(rng, S, R, wide)
    a = signs(rng, G, narrow, R)
    delta = scale[ids][:, None] * np.einsum("skr,sr->sk", a[ids], dh)
    dx = bf16(-delta)
    want = bf16(f64(dx) + delta)
    args = bf16(np.zeros((S, narrow))), bf16(np.ascontiguousarray(a.transpose(0, 2, 1))), bf16(np.stack([b.T.copy()] * G))
    _moe().moe_lora_backward(bf16(dy), *args, routing, None, s_t, dx=dx, weights=False)
    off = (dx != want).sum().item()
    assert off == 0, f"{off} of {want.numel()} elements of dx"
