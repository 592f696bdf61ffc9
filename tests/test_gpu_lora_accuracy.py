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


# groups of one slot to a few dozen, of one segment and of several
GRADS = [(3, 3, 8, 16, 1), (9, 4, 16, 16, 1), (40, 3, 24, 16, 1), (40, 2, 64, 64, 1), (100, 5, 128, 32, 1), (64, 64, 32, 8, 1),
         (600, 20, 16, 8, 40), (300, 8, 128, 16, 40)]


@pytest.mark.parametrize("S,G,R,bm,most", GRADS)
def test_db_holds_every_bit_of_h(S, G, R, bm, most):
    """dy of +-1 and h of whole numbers below 2^18 (2^24 where a group has one
    slot, which 24 bits fill), so that up to 40 add up below 2^24."""
    moe, rng = _moe(), np.random.default_rng(S * R)
    counts = np.bincount(np.arange(S) % G, minlength=G)
    assert most == 1 or counts.max() <= most
    ids = rng.permutation(np.arange(S) % G).astype(np.int32)
    routing = moe.moe_align(torch.from_numpy(ids).reshape(S, 1).cuda(), G, bm)
    top = (1 << 24) // max(counts.max(), 1)
    h = rng.integers(-top + 1, top, size=(S, R)) * 2.0 ** -24
    N, K = 264, 136
    dy, scale = rng.choice([-1.0, 1.0], size=(S, N)), 2.0 ** rng.integers(-3, 4, size=G) * rng.choice([-1, 1], size=G)
    x, a, b = (bf16(rng.standard_normal(s)) for s in ((S, K), (G, R, K), (G, N, R)))
    h_t, s_t = (torch.from_numpy(t.astype(np.float32)).cuda() for t in (h, scale))
    assert np.array_equal(f64(h_t), h)
    _, db = moe.moe_lora_backward(bf16(dy), x, a, b, routing, h_t, s_t)
    want = np.stack([scale[g] * dy[ids == g].T @ h[ids == g] for g in range(G)])
    off = int((db.cpu().double().numpy() != want).sum())
    assert off == 0, f"{off} of {want.size}"


@pytest.mark.parametrize("S,G,R,bm,most", GRADS)
def test_da_holds_every_bit_of_dh(S, G, R, bm, most):
    """dh of 20 bits (the docstring's chunks), x of +-1 at up to 16 of a group's slots."""
    moe, rng = _moe(), np.random.default_rng(S * R + 1)
    ids = rng.permutation(np.arange(S) % G).astype(np.int32)
    routing = moe.moe_align(torch.from_numpy(ids).reshape(S, 1).cuda(), G, bm)
    N, K = 3 * R + 520, 264
    b, dy, dh = chunked(rng, S, R, N)
    x = rng.choice([-1.0, 1.0], size=(S, K))
    for g in range(G):
        at = np.flatnonzero(ids == g)
        for k in range(K):
            x[rng.permutation(at)[16:], k] = 0
    scale = 2.0 ** rng.integers(-3, 4, size=G) * rng.choice([-1, 1], size=G)
    s_t, h = torch.from_numpy(scale.astype(np.float32)).cuda(), torch.zeros((S, R), device="cuda")
    a = bf16(rng.standard_normal((G, R, K)))
    da, _ = moe.moe_lora_backward(bf16(dy), bf16(x), a, bf16(np.stack([b.T] * G)), routing, h, s_t)
    want = np.stack([scale[g] * dh[ids == g].T @ x[ids == g] for g in range(G)])
    off = int((da.cpu().double().numpy() != want).sum())
    assert off == 0, f"{off} of {want.size}"


@pytest.mark.parametrize("S,G,R,bm", [(3, 2, 8, 16), (40, 3, 16, 16), (40, 3, 32, 8), (60, 2, 64, 16), (300, 2, 128, 16),
                                      (2000, 3, 8, 64), (2000, 3, 16, 64), (1500, 2, 24, 64), (1500, 2, 128, 64)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_infinite_h_and_dh(S, G, R, bm, sign):
    """An infinite h gives infinities of the sign of scale B where a row of B has
    one sign, NaN where it has both, and reaches no other slot; dh and dx alike."""
    moe, rng = _moe(), np.random.default_rng(R)
    K, N, s = 264, 136, S // 2
    ids = rng.integers(0, G, size=S).astype(np.int32)
    g = ids[s]
    routing = moe.moe_align(torch.from_numpy(ids).reshape(S, 1).cuda(), G, bm)
    scale = torch.tensor([0.5, -2.0, 3.0])[:G].cuda()
    a, b = np.abs(rng.standard_normal((G, R, K))) + 0.1, np.abs(rng.standard_normal((G, N, R))) + 0.1
    kind = np.arange(N) % 3                       # rows of B: positive, negative, both
    b[:, kind == 1] *= -1
    b[:, kind == 2, : R // 2] *= -1
    x, c = rng.standard_normal((S, K)), bf16(rng.standard_normal((S, N)))
    args = lambda: (bf16(x), bf16(a), bf16(b), routing)  # noqa: E731
    clean = moe.moe_lora(c.clone(), *args(), scale)
    x[s, 5] = sign * np.inf
    out, h = moe.moe_lora(c.clone(), *args(), scale, keep_h=True)
    assert (f64(h)[s] == sign * np.inf).all()
    row, to = f64(out)[s], sign * np.sign(float(scale[g]))
    assert (row[kind == 0] == to * np.inf).all() and (row[kind == 1] == -to * np.inf).all() and np.isnan(row[kind == 2]).all()
    others = torch.arange(S) != s
    assert torch.equal(out[others], clean[others])
    # dh = scale B^T dy: dy infinite at a column whose entries of B are positive; dx through A, all of whose are too
    x[s, 5] = 1.0
    dy, dx = rng.standard_normal((S, N)), bf16(rng.standard_normal((S, K)))
    ref, got = dx.clone(), dx.clone()
    h0 = torch.zeros((S, R), device="cuda")
    da0, _ = moe.moe_lora_backward(bf16(dy), *args(), h0, scale, dx=ref)
    dy[s, 3] = sign * np.inf
    da, _ = moe.moe_lora_backward(bf16(dy), *args(), h0, scale, dx=got)
    assert (f64(got)[s] == to * np.inf).all() and torch.equal(got[others], ref[others])
    keep = [i for i in range(G) if i != g]
    assert torch.equal(da[keep], da0[keep])
    want = to * np.sign(f64(bf16(x))[s]) * np.inf
    with np.errstate(invalid="ignore"):
        assert np.array_equal(f64(da)[g], np.broadcast_to(want, (R, K)))
