"""GPU tests of the norm and dropout beside test_gpu_norm.py: the backward
kernels against differences of the forward kernel, with a signal well above the
rounding of its output; what lies behind strided rows; and the 8-bit outputs
taken by the GEMMs that they are for."""

import numpy as np
import pytest
import torch

import synth
from block_helpers import U, f64, normal, rng_state, strided
from helpers import need_gpu
from oracle import formats
from oracle import gemm as ogemm

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def _moe():
    import mixture_experts_grouped_moe_amd as moe
    return moe


# ------------------------------------------------------------- differences

def half_difference(v, w, dy, dv, dw):
    """(<dy, y(v + dv, w + dw) - y(v - dv, w - dw)> / 2 of the forward kernel, the
    most that its roundings can be of it: of every y half a step of bf16, 2^-8,
    its fp32 sums' (n / 2 + 8) u, and 2 u each for v + dv and w + dw)."""
    zero = torch.zeros(v.shape, dtype=torch.bfloat16, device="cuda")
    y = [f64(_moe().moe_rmsnorm(zero, w + t * dw, v + t * dv, eps=EPS)[0]) for t in (1, -1)]
    size = (np.abs(f64(dy)) * (np.abs(y[0]) + np.abs(y[1]))).sum() / 2
    return (f64(dy) * (y[0] - y[1])).sum() / 2, (1.01 * 2.0 ** -8 + (v.shape[1] / 2 + 12) * U) * size


@pytest.mark.parametrize("T,n", [(3, 256), (2, 1032), (4, 2880), (2, 8200)])
def test_gradient_of_the_rows_by_differences(T, n):
    """Along the gradient itself, and its parts in random halves of the columns.
    A row moves by 1/32 of its length. What is left of the central difference:
    with y = sqrt(n) w x / |x| and |d^k / dt^k 1 / |x + t d|| <= k! |d|^k / |x|^(k + 1),
    the third derivative of x / |x| is at most 12 (|d| / |x|)^3, a sixth of which
    counts, at an |x| of at least |v| - |d| (eps is far below)."""
    moe = _moe()
    v, dy = normal((T, n), 8, "v", "fp32", 2.0), normal((T, n), 8, "dy")
    w = 1 + 0.3 * normal((n,), 8, "w", "fp32")
    _, dres, _ = moe.moe_rmsnorm_backward(dy, v, w, eps=EPS)
    step = 1 / 32
    g = np.abs(f64(dy) * f64(w))
    left = 2 * (step / (1 - step)) ** 3 * np.sqrt(n) * np.linalg.norm(g, axis=1).sum()
    s = 1 / np.sqrt((f64(v) ** 2).mean(axis=1, keepdims=True) + EPS)
    size = s * (g + np.abs(f64(v)) * s * s * (g * np.abs(f64(v))).mean(axis=1, keepdims=True))  # of dres's terms
    for k in range(4):
        mask = torch.ones(n) if k == 0 else (torch.rand(n, generator=synth.gen(k, "m")) < 0.5).float()
        d = dres * mask.cuda()
        d = d * (step * v.norm(dim=1, keepdim=True) / d.norm(dim=1, keepdim=True))
        got, room = half_difference(v, w, dy, d, torch.zeros_like(w))
        ref = (f64(dres) * f64(d)).sum()
        room += left + (n + 16) * U * (size * np.abs(f64(d))).sum()
        assert room < abs(ref) / 4 and abs(got - ref) < room, (k, got, ref, room)


@pytest.mark.parametrize("T,n", [(3, 256), (40, 1032)])
def test_gradient_of_the_weight_by_differences(T, n):
    """y is linear in the weight."""
    moe = _moe()
    v, dy = normal((T, n), 9, "v", "fp32", 2.0), normal((T, n), 9, "dy")
    w = 1 + 0.3 * normal((n,), 9, "w", "fp32")
    _, _, dw = moe.moe_rmsnorm_backward(dy, v, w, eps=EPS)
    for k in range(3):
        mask = torch.ones(n) if k == 0 else (torch.rand(n, generator=synth.gen(k, "m")) < 0.5).float()
        d = 0.5 * dw * mask.cuda() / dw.abs().max()
        got, room = half_difference(v, w, dy, torch.zeros_like(v), d)
        ref = (f64(dw) * f64(d)).sum()
        s = 1 / np.sqrt((f64(v) ** 2).mean(axis=1, keepdims=True) + EPS)
        room += (n / 2 + 8 + T) * U * (np.abs(f64(dy) * f64(v) * s).sum(axis=0) * np.abs(f64(d))).sum()
        assert room < abs(ref) / 4 and abs(got - ref) < room, (k, got, ref, room)


# ------------------------------------------------------- behind strided rows

@pytest.mark.parametrize("T,n", [(3, 40), (129, 2880), (2000, 24)])
def test_dropout_leaves_what_lies_behind_rows(T, n):
    moe = _moe()
    x, r = normal((T, n), 5, "x"), rng_state(3, 4)
    y = moe.moe_dropout(x, 0.3, r)
    out, place = strided(torch.zeros_like(x), 8), strided(x, 24)
    assert moe.moe_dropout(strided(x, 16), 0.3, r, out=out) is out
    assert moe.moe_dropout(place, 0.3, r, out=place) is place
    for t, extra in ((out, 8), (place, 24)):
        assert torch.equal(t, y)
        behind = t.as_strided((T - 1, extra), (n + extra, 1), n)
        assert torch.isnan(behind).all()


# ------------------------------------------------- the GEMMs' 8-bit inputs

def parity(got, ref):
    """The GEMM's output in bf16 against float64 sums of the same codes."""
    assert np.abs(got - ref).max() <= 5e-3 * np.abs(ref).max()


def decodes_to(q, scale, y):
    """The decoded codes are y's values, saturated at 448 scales: half a step of
    E4M3 (2^-4 of a value, 2^-10 of the scale below the smallest normal number)
    beside y's own of bf16."""
    y = np.clip(f64(y), -448 * scale, 448 * scale)
    off = np.abs(formats.e4m3_to_f64(synth.bits(q)) * scale - y)
    assert (off <= (2.0 ** -4 + 2.0 ** -7) * np.abs(y) + 2.0 ** -10 * scale).all()


@pytest.mark.parametrize("T", [1, 9, 100, 333])
def test_mxfp8_output_through_the_grouped_gemm(T):
    moe = _moe()
    E, k, K, N = 8, 2, 256, 192
    d = synth.gemm_case(T, k, E, N, K, "e4m3", seed=8, w_std=0.5, device="cuda")
    x, res, w = normal((T, K), T, "x"), normal((T, K), T, "r", "fp32"), 1 + 0.3 * normal((K,), T, "w", "fp32")
    y, _, q, s = moe.moe_rmsnorm(x, w, res, p=0.2, rng=rng_state(1, 2), quant="mxfp8")
    routing = moe.moe_align(d["ids"], E, moe.moe_gemm_block_m("e4m3", T, moe.MOE_E4M3))
    c = moe.moe_grouped_gemm(q, d["w"], "e4m3", routing, T, k, E, k, w_scale=d["w_scale"], a_scale=s)
    h = {n: synth.bits(t) if isinstance(t, torch.Tensor) else t for n, t in d.items()}
    ref, _ = ogemm.grouped_gemm(synth.bits(q), k, h["w"], "e4m3", h["w_scale"], h["ids"], E, a_dtype="e4m3",
                                a_scale=synth.bits(s))
    parity(f64(c), ref)
    decodes_to(q, np.repeat(np.exp2(synth.bits(s).astype(np.float64) - 127), 32, axis=1), y)


@pytest.mark.parametrize("sizes", [[1], [40, 0, 70, 3], [5, 300, 0]])
def test_per_token_output_through_the_grouped_gemm(sizes):
    moe = _moe()
    K, N, T = 256, 320, sum(sizes)
    d = synth.per_token_case(sizes, N, K, 9, bias=True, device="cuda")
    x, w = normal((T, K), T, "x"), 1 + 0.3 * normal((K,), T, "w", "fp32")
    y, _, q, s = moe.moe_rmsnorm(x, w, quant="per_token")
    mapping = moe.moe_block_mapping(d["group_sizes"], T)
    c = moe.moe_grouped_gemm_per_token(q, s, d["w"], d["w_scale"], mapping, bias=d["bias"])
    h = {n: synth.bits(t) if isinstance(t, torch.Tensor) else t for n, t in d.items()}
    ref = ogemm.grouped_gemm_per_token(synth.bits(q), s.cpu().numpy(), h["w"], h["w_scale"], h["group_sizes"], bias=h["bias"])
    parity(f64(c), ref)
    decodes_to(q, f64(s)[:, None], y)
