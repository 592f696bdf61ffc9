"""GPU tests of moe_rmsnorm and moe_rmsnorm_backward at inputs whose sums and
statistics are exact in fp32, so that the outputs have one right value and no
tolerance: rows of ones and minus ones have mean v^2 = 1 and, with eps = 0,
1 / sqrt = 1.
"""

import numpy as np
import pytest
import torch

from helpers import need_gpu
from oracle import formats, quant

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def _moe():
    import mixture_experts_grouped_moe_amd as moe
    return moe


def e4m3_borders():
    """The midpoints between neighbouring E4M3 magnitudes."""
    v = formats.e4m3_to_f64(np.arange(127, dtype=np.uint8))   # 0 ... 448
    return (v[1:] + v[:-1]) / 2


# largest magnitudes: ordinary ones, scales next to the smallest and below it, and fp32's largest
TOPS = [1.0, 1.2345, 447.9, 3.3e-5, 1.7e19, 448 * 1.75 * 2.0 ** -126, 448 * 2.0 ** -126, 2.0 ** -121, 3.4e38]


@pytest.mark.parametrize("top", TOPS)
@pytest.mark.parametrize("n", [1536, 6144])   # a row in two waves and in eight
def test_per_token_codes_at_the_borders(top, n):
    """u is the weight: those next to a border between two codes, times the
    row's scale. A code is the nearest to the fp32 quotient u / scale, ties to
    even."""
    top = np.float32(top)
    scale = max(np.float32(top / np.float32(448)), np.float32(2.0 ** -126))
    at = (e4m3_borders() * np.float64(scale)).astype(np.float32)
    step = np.arange(-5, 6)[:, None]
    w = (at.view(np.int32)[None, :] + step).view(np.float32).reshape(-1)
    w = w[np.isfinite(w) & (np.abs(w) <= top)][:n - 1]
    w = np.concatenate([[top], w, np.zeros(n - 1 - w.size, np.float32)]).astype(np.float32)
    sign = np.where(np.arange(n) % 3 == 1, -1.0, 1.0)
    x = torch.from_numpy(np.stack([np.ones(n), sign])).to(torch.bfloat16).cuda()
    _, _, q, s = _moe().moe_rmsnorm(x, torch.from_numpy(w).cuda(), eps=0.0, quant="per_token", keep_y=False)
    assert (s.cpu().numpy() == scale).all()
    quotient = np.stack([w, w * sign.astype(np.float32)]) / scale
    assert quotient.dtype == np.float32
    want = formats.e4m3_to_f64(quant.e4m3_round(quotient))
    got = formats.e4m3_to_f64(q.cpu().numpy())
    off = int((got != want).sum())
    assert off == 0, f"{off} of {got.size} codes, e.g. u / scale {quotient[got != want][:4]}"


# rows that are workgroups' own (a partial row each), and one workgroup for all
# rows, whose row groups' terms it adds (16 and 4 of them). Within one of several
# workgroups rows are added in 32 bits.
@pytest.mark.parametrize("T,n", [(300, 1040), (500, 2056), (250, 16384), (16, 64), (4, 512)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dweight_of_rows_that_cancel(T, n, dtype):
    """dweight = sum of dy (v / sqrt = +-1): two rows of 2^15 cancel, one at each
    end, and what is between them is 2^-10 times whole numbers, which 32 bits
    lose beside 2^15."""
    rng = np.random.default_rng(T + n)
    sign = rng.choice([-1.0, 1.0], size=(T, n))
    dy = rng.integers(-3, 4, size=(T, n)) * 2.0 ** -10
    dy[0], dy[-1] = 2.0 ** 15, -(2.0 ** 15) * sign[0] * sign[-1]
    moe = _moe()
    to = lambda a, t: torch.from_numpy(a.astype(np.float32)).to(t).cuda()  # noqa: E731
    w = torch.ones(n, device="cuda")
    _, _, dw = moe.moe_rmsnorm_backward(to(dy, torch.bfloat16), to(sign, dtype), w, eps=0.0)
    off = int((dw.cpu().double().numpy() != (dy * sign).sum(axis=0)).sum())
    assert off == 0, f"{off} of {n}"


@pytest.mark.parametrize("power", [-74, -66, -63, 30, 55])
@pytest.mark.parametrize("n", [64, 1040, 9216])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradient_of_small_and_large_rows(power, n, dtype):
    """With eps = 0 the gradient of rows 2^power times as large is 2^-power
    times as large, and dweight is the same; rows of +-1 lose nothing to fp32's
    subnormal numbers in the sums."""
    rng, moe = np.random.default_rng(n), _moe()
    v = torch.from_numpy(rng.choice([-1.0, 1.0], size=(5, n))).to(dtype).cuda()
    dy = torch.from_numpy(rng.standard_normal((5, n))).to(torch.bfloat16).cuda()
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(n)).float().cuda()
    dx, dres, dw = moe.moe_rmsnorm_backward(dy, v, w, eps=0.0)
    got = moe.moe_rmsnorm_backward(dy, v * 2.0 ** power, w, eps=0.0)
    assert torch.isfinite(dres).all()
    for a, b in zip(got, (dx, dres, dw)):
        b = b if b is dw else (b.double() * 2.0 ** -power).to(b.dtype)
        assert int((a != b).sum()) == 0
