"""GPU tests of moe_dropout, moe_rmsnorm and moe_rmsnorm_backward against the
float64 oracle (oracle.block).

Tolerances (u = 2^-24, half a step of fp32; every one counts the roundings of
an fp32 computation, whose sums of n terms cost at most n u of the sum of
magnitudes):
* dropout: one product and a rounded scale, 2 u, before half a step of bf16.
* v = residual + drop(x): 3 u of |residual| + |drop(x)| = `size`.
* u = v r w: that, and for r half of the sum of squares' n u + its terms' 6 u
  (their v twice), the root's 2 u, two products: (n / 2 + 8) u of `size` r |w|.
* 8-bit codes: rounding is monotonic, so a code lies between those of the
  exact value moved down and up by that tolerance.
* gradient: d's terms carry (n + 16) u of their magnitudes, dweight's
  (n / 2 + 8 + rows) u of the sum of magnitudes.
"""

import numpy as np
import pytest
import torch

from block_helpers import DT, HALF, U, close, f64, normal, rng_state, strided
from helpers import need_gpu
from oracle import block as oblock
from oracle import formats, quant

pytestmark = pytest.mark.gpu

SEED, OFFSET = 0x9E3779B97F4A7C15, (7 << 32) + 5
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def _moe():
    import mixture_experts_grouped_moe_amd as moe
    return moe


# ------------------------------------------------------------------ dropout

@pytest.mark.parametrize("T,n", [(1, 8), (3, 40), (64, 256), (129, 2880), (2000, 24)])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 2.0 ** -16, 1.0])
def test_dropout(T, n, p):
    moe = _moe()
    x, r = normal((T, n), T + n, "x"), rng_state(SEED, OFFSET)
    y = moe.moe_dropout(x, p, r)
    ref = oblock.dropout(f64(x), p, SEED, OFFSET)
    assert np.array_equal(f64(y) == 0, ref == 0)
    close(f64(y), ref, (2.0 ** -8 + 2 * U) * np.abs(ref))
    z = moe.moe_dropout(strided(x, 16), p, r, out=strided(torch.empty_like(x), 8))
    assert torch.equal(z, y)
    w = strided(x, 24)
    behind = w.untyped_storage().nbytes()
    assert moe.moe_dropout(w, p, r, out=w) is w and torch.equal(w, y) and w.untyped_storage().nbytes() == behind


def test_dropout_drops_what_is_not_finite():
    x = torch.full((16, 256), float("nan"), dtype=torch.bfloat16, device="cuda")
    x[8:] = float("inf")
    y = f64(_moe().moe_dropout(x, 0.5, rng_state(1, 2)))
    keep = oblock.dropout_keep(16, 256, 0.5, 1, 2)
    assert (y[~keep] == 0).all() and np.isnan(y[:8][keep[:8]]).all() and np.isinf(y[8:][keep[8:]]).all()


def test_dropout_without_rows():
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    assert _moe().moe_dropout(x, 0.5, rng_state(1, 2)).shape == (0, 64)


def test_dropout_past_32_bits():
    """Elements whose piece number passes 2^32: the counter's second word."""
    n, T = 1 << 17, (1 << 18) + 2
    x = torch.ones((T, n), dtype=torch.bfloat16, device="cuda")  # 69 GB, in place
    _moe().moe_dropout(x, 0.5, rng_state(SEED, OFFSET), out=x)
    i = (np.arange((T - 2) * (n // 8), T * (n // 8), dtype=np.uint64))
    low = np.uint64(0xFFFFFFFF)
    c = np.stack([i & low, i >> np.uint64(32), np.full_like(i, OFFSET & 0xFFFFFFFF), np.full_like(i, OFFSET >> 32)], -1)
    w = oblock.philox4x32(c, (SEED & 0xFFFFFFFF, SEED >> 32))
    keep = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], -1).reshape(2, n) >= 32768
    assert int(i[0]) >= 1 << 32
    assert np.array_equal(f64(x[-2:]), 2.0 * keep)


# --------------------------------------------------------------------- norm

def check_norm(T, n, residual, weight, p, kind, seed=0, x=None, res=None, w=None, eps=EPS, **kw):
    moe = _moe()
    x = normal((T, n), seed + n, "x") if x is None else x
    if residual is not None and res is None:
        res = normal((T, n), seed + T, "r", residual, 2.0)
    w = (1 + 0.3 * normal((n,), seed, "w", "fp32")).to(DT[weight]) if w is None else w
    y, v, q, s = moe.moe_rmsnorm(x, w, res, eps=eps, p=p, rng=rng_state(SEED, OFFSET), quant=kind, **kw)
    d = oblock.dropout(f64(x), p, SEED, OFFSET)
    size = np.abs(d) + (np.abs(f64(res)) if res is not None else 0)
    ref_v = d + (f64(res) if res is not None else 0)
    ref = oblock.rmsnorm(ref_v, f64(w), eps)
    r = 1 / np.sqrt((ref_v ** 2).mean(axis=1, keepdims=True) + eps)
    tol = (n / 2 + 8) * U * size * r * np.abs(f64(w))
    if residual is None and p == 0:
        assert v is None
    elif v is not None:
        close(f64(v), ref_v, HALF[v.dtype] * np.abs(ref_v) + 3 * U * size, "sum")
    if y is not None:
        close(f64(y), ref, 2.0 ** -8 * np.abs(ref) + 1.01 * tol + 2.0 ** -130, "y")
    lo, hi = ref - tol, ref + tol
    if kind == "mxfp8":
        top = np.abs(ref).reshape(T, -1, 32).max(axis=2)
        room = tol.reshape(T, -1, 32).max(axis=2)
        sb = s.cpu().numpy().astype(np.int64)
        for bound, ok in ((np.maximum(top - room, 0), np.greater_equal), (top + room, np.less_equal)):
            e = np.where(bound > 0, np.frexp(np.where(bound > 0, bound, 1))[1] - 9, -127)
            assert ok(sb, np.clip(e, -127, 127) + 127).all()
        step = np.repeat(np.exp2(sb - 127.0), 32, axis=1)
        got, at = formats.e4m3_to_f64(q.cpu().numpy()), quant.e4m3_round
        assert (got >= formats.e4m3_to_f64(at(lo / step))).all() and (got <= formats.e4m3_to_f64(at(hi / step))).all()
    elif kind == "per_token":
        _, rs = oblock.quantize_per_token(ref)
        close(s.cpu().double().numpy(), rs, tol.max(axis=1) / 448 + 2 * U * rs, "scales")
        step = s.cpu().double().numpy()[:, None]
        slack = 2 * U * np.abs(ref)
        got, at = formats.e4m3_to_f64(q.cpu().numpy()), quant.e4m3_round
        assert (got >= formats.e4m3_to_f64(at((lo - slack) / step))).all()
        assert (got <= formats.e4m3_to_f64(at((hi + slack) / step))).all()
    else:
        assert q is None and s is None
    return y, v, q, s


# every row layout (up to 128, 512, 1024, 2048, 4096, 8192, 16384 columns), at its ends and inside
WIDTHS = [8, 96, 128, 136, 512, 520, 1024, 1032, 2048, 2056, 2688, 4096, 4104, 7168, 8192, 8200, 16376, 16384]


@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("residual,weight,p,kind", [
    (None, "bf16", 0.0, "per_token"), ("bf16", "fp32", 0.0, "mxfp8"), ("fp32", "bf16", 0.3, None),
    (None, "fp32", 0.2, "mxfp8"), ("bf16", "bf16", 0.5, "per_token")])
def test_norm(n, residual, weight, p, kind):
    if kind == "mxfp8":
        n = -(-n // 32) * 32
    for T in (1, 21):
        check_norm(T, n, residual, weight, p, kind, seed=T)


def test_norm_many_rows():
    check_norm(70001, 64, "fp32", "bf16", 0.25, "mxfp8")


def test_norm_what_is_left_out_and_strides():
    moe = _moe()
    T, n = 13, 544
    x, res, w = normal((T, n), 1, "x"), normal((T, n), 1, "r", "fp32"), normal((n,), 1, "w")
    r = rng_state(SEED, OFFSET)
    y, v, q, s = moe.moe_rmsnorm(x, w, res, p=0.2, rng=r, quant="mxfp8")
    only = moe.moe_rmsnorm(x, w, res, p=0.2, rng=r, quant="mxfp8", keep_y=False, keep_sum=False)
    assert only[0] is None and only[1] is None and torch.equal(only[2], q) and torch.equal(only[3], s)
    assert torch.equal(moe.moe_rmsnorm(x, w, res, p=0.2, rng=r)[0], y)
    out = [strided(torch.zeros_like(t), e) for t, e in ((y, 8), (v, 16), (q, 24), (s, 3))]
    got = moe.moe_rmsnorm(strided(x, 8), w, strided(res, 8), p=0.2, rng=r, quant="mxfp8", out=out)
    for a, b, o in zip((y, v, q, s), got, out):
        assert b is o and torch.equal(a, b)
        behind = o.as_strided((T - 1, o.stride(0) - o.shape[1]), (o.stride(0), 1), o.shape[1])
        assert (behind == 255).all() if o.dtype == torch.uint8 else torch.isnan(behind).all()  # left as it was
    stream = res.clone()  # the residual stream in place
    moe.moe_rmsnorm(x, w, stream, p=0.2, rng=r, out=(out[0], stream, None, None))
    assert torch.equal(stream, v)
    # a sum in fp32 without a residual
    wide = torch.empty((T, n), device="cuda")
    moe.moe_rmsnorm(x, w, p=0.2, rng=r, out=(out[0], wide, None, None))
    close(f64(wide), oblock.dropout(f64(x), 0.2, SEED, OFFSET), 2 * U * np.abs(f64(wide)))


def test_norm_without_rows():
    x, w = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), torch.ones(64, device="cuda")
    y, v, q, s = _moe().moe_rmsnorm(x, w, quant="mxfp8")
    assert y.shape == (0, 64) and s.shape == (0, 2)
    dx, _, dw = _moe().moe_rmsnorm_backward(x, x, w)
    assert dx.shape == (0, 64) and (dw == 0).all()


def test_fused_dropout_is_moe_dropout():
    moe = _moe()
    x, w = normal((19, 2880), 3, "x"), torch.ones(2880, dtype=torch.bfloat16, device="cuda")
    r = rng_state(5, 6)
    assert torch.equal(moe.moe_rmsnorm(x, w, p=0.3, rng=r)[1], moe.moe_dropout(x, 0.3, r))


@pytest.mark.parametrize("kind", ["mxfp8", "per_token"])
def test_norm_values_that_are_not_finite_stay_in_their_row(kind):
    moe = _moe()
    x, w = normal((6, 160), 4, "x"), torch.ones(160, device="cuda")
    clean = moe.moe_rmsnorm(x, w, quant=kind)
    x[1, 70], x[3, 5] = float("nan"), float("inf")
    y, _, q, s = moe.moe_rmsnorm(x, w, quant=kind)
    good = [0, 2, 4, 5]
    for a, b in zip((y, q, s), (clean[0], clean[2], clean[3])):
        assert torch.equal(a[good], b[good])
    # NaN: the whole row; inf: 0 elsewhere (r = 0), NaN at its place
    assert torch.isnan(y[1]).all() and torch.isnan(y[3, 5]) and (y[3].nan_to_num(0) == 0).all()
    assert (q[1] == 0x7F).all()
    if kind == "mxfp8":
        assert (s[1] == 0xFF).all() and s[3].tolist() == [0xFF, 0, 0, 0, 0] and (q[3, :32] == 0x7F).all()
        assert (q[3, 32:] == 0).all()
    else:
        assert torch.isnan(s[1]) and torch.isnan(s[3]) and (q[3] == 0x7F).all()


def test_norm_of_zeros_and_extremes():
    moe = _moe()
    x, w = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda"), torch.ones(64, device="cuda")
    x[1] = -0.0
    x[2, 7] = 2.0 ** -120
    x[3] = 2.0 ** 60
    for kind in ("mxfp8", "per_token"):
        y, _, q, s = moe.moe_rmsnorm(x, w, quant=kind)
        assert (y[:2] == 0).all() and (q[:2] == 0).all()   # a zero takes no sign
        assert (y[3] == 1).all()
        if kind == "mxfp8":
            assert (s[:2] == 0).all() and (s[3] == 127 - 8).all() and (q[3] == 0x78).all()
        else:
            assert (s[:2] == 2.0 ** -126).all() and (q[3] == 0x7E).all()
    # magnitudes around 448: saturation, and weights that make a block's largest tiny
    w = torch.full((64,), 2.0 ** -140, device="cuda")
    y, _, q, s = moe.moe_rmsnorm(x, w, quant="mxfp8")
    assert (s[3] == 0).all()                               # below 2^-127 * 448: the smallest scale
    assert (q[3].view(torch.float8_e4m3fn).float() == 0).all()   # 2^-140 / 2^-127 rounds to 0 (the smallest code is 2^-9)


@pytest.mark.parametrize("n", [64, 544, 1056, 2880, 7168, 9216])
@pytest.mark.parametrize("dtype,weight,p", [("bf16", "bf16", 0.0), ("fp32", "fp32", 0.0), ("bf16", "fp32", 0.3),
                                            ("fp32", "bf16", 0.5)])
def test_norm_backward(n, dtype, weight, p):
    moe = _moe()
    for T in (1, 37):
        v, dy, dsum = normal((T, n), T, "v", dtype, 2.0), normal((T, n), T, "dy"), normal((T, n), T, "ds", dtype)
        w = (1 + 0.3 * normal((n,), n, "w", "fp32")).to(DT[weight])
        for ds in (dsum, None):
            dx, dres, dw = moe.moe_rmsnorm_backward(dy, v, w, dsum=ds, eps=EPS, p=p, rng=rng_state(SEED, OFFSET))
            check_backward(dx, dres, dw, dy, v, w, ds, p)
    # what is left out; strides; dsum in place
    r = rng_state(SEED, OFFSET)
    dx, dres, dw = moe.moe_rmsnorm_backward(dy, v, w, dsum=dsum, eps=EPS, p=p, rng=r)
    none = moe.moe_rmsnorm_backward(dy, v, w, dsum=dsum, eps=EPS, p=p, rng=r, keep_dweight=False)
    assert none[2] is None and torch.equal(none[0], dx)
    place = strided(dsum, 8)
    ws = torch.empty(moe.moe_rmsnorm_backward_workspace_bytes(T, n), dtype=torch.uint8, device="cuda")
    got = moe.moe_rmsnorm_backward(strided(dy, 8), strided(v, 16), w, dsum=place, eps=EPS, p=p, rng=r,
                                   out=(None, place, torch.empty_like(dw)), workspace=ws)
    assert got[0] is None and torch.equal(place, dres) and torch.equal(got[2], dw)


def check_backward(dx, dres, dw, dy, v, w, dsum, p):
    T, n = v.shape
    d, ref_w = oblock.rmsnorm_backward(f64(dy), f64(v), f64(w), EPS, None if dsum is None else f64(dsum))
    s = 1 / np.sqrt((f64(v) ** 2).mean(axis=1, keepdims=True) + EPS)
    g = f64(dy) * f64(w)
    size = s * (np.abs(g) + np.abs(f64(v)) * s * s * np.abs(g * f64(v)).mean(axis=1, keepdims=True))
    size = size + (np.abs(f64(dsum)) if dsum is not None else 0)
    tol = (n + 16) * U * size
    close(f64(dres), d, HALF[dres.dtype] * (np.abs(d) + tol) + tol, "dresidual")
    ref = oblock.dropout(d, p, SEED, OFFSET)
    grow = 1 / (1 - p) if p else 1
    assert p == 0 or np.array_equal(f64(dx) == 0, ref == 0)
    close(f64(dx), ref, 2.0 ** -8 * (np.abs(ref) + grow * tol) + (grow + 0.01) * tol + 2 * U * np.abs(ref), "dx")
    close(f64(dw), ref_w, (n / 2 + 8 + T) * U * np.abs(f64(dy) * f64(v) * s).sum(axis=0), "dweight")


def test_norm_backward_many_rows_is_one_order():
    moe = _moe()
    v, dy = normal((9001, 136), 1, "v"), normal((9001, 136), 1, "dy")
    w = torch.ones(136, device="cuda")
    dx, dres, dw = moe.moe_rmsnorm_backward(dy, v, w, eps=EPS)
    check_backward(dx, dres, dw, dy, v, w, None, 0.0)
    for _ in range(3):
        assert torch.equal(moe.moe_rmsnorm_backward(dy, v, w, eps=EPS)[2], dw)


def test_norm_gradient_is_the_forward_pass_by_differences():
    """<dy, y(v + h e) - y(v - h e)> / 2h of the kernel's own forward pass along random directions e."""
    moe = _moe()
    T, n, h = 3, 256, 2.0 ** -5
    v, dy, w = normal((T, n), 8, "v", "fp32"), normal((T, n), 8, "dy"), normal((n,), 8, "w", "fp32")
    zero = torch.zeros((T, n), dtype=torch.bfloat16, device="cuda")
    _, dres, _ = moe.moe_rmsnorm_backward(dy, v, w, eps=EPS)
    for k in range(4):
        e = normal((T, n), 9 + k, "e", "fp32") / 16
        yp, ym = (moe.moe_rmsnorm(zero, w, v + t * e, eps=EPS, quant="per_token")[0] for t in (h, -h))
        # y is stored in bf16: half a step of each, and the third-order term of a step of h |e| / |v| ~ 2^-9
        num = (f64(dy) * (f64(yp) - f64(ym))).sum() / (2 * h)
        ref = (f64(dres) * f64(e)).sum()
        room = 2 * 2.0 ** -8 * np.sqrt((f64(dy) ** 2 * f64(yp) ** 2).sum()) / (2 * h) * 4  # four deviations
        assert abs(num - ref) < room + 2.0 ** -12 * abs(ref)


# ------------------------------------------------------- streams and graphs

def test_streams_and_replays():
    moe = _moe()
    T, n = 100, 2880
    x, res, w, dy = normal((T, n), 1, "x"), normal((T, n), 1, "r"), normal((n,), 1, "w"), normal((T, n), 1, "dy")
    r = rng_state(1, 0)

    def step():
        y, v, q, s = moe.moe_rmsnorm(x, w, res, p=0.2, rng=r, quant="mxfp8")
        dx, dres, dw = moe.moe_rmsnorm_backward(dy, v, w, dsum=y, p=0.2, rng=r)
        return y, v, q, s, dx, dres, dw, moe.moe_dropout(y, 0.4, r)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    eager = step()
    on = moe.moe_rmsnorm(x, w, res, p=0.2, rng=r, quant="mxfp8", stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(on, eager))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    masks = []
    for k in range(4):
        r[1] = k
        x.copy_(normal((T, n), 20 + k, "x"))
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        masks.append(want[-1] == 0)
    assert (masks[0] != masks[1]).any()
