"""GPU tests of the training entry points (moe_train.h) against the float64
oracle (oracle.train): the router with its losses and gradient, the combine
over partly routed tokens and its backward pass, the activation with an MXFP8
checkpoint, the weight gradient over MXFP8 rows, and a whole training step.

Tolerances (u = 2^-24, half a step of fp32):
* router: exp(a - m) in fp32 carries the roundings of a, of a - m and of the
  exponential's argument reduction, each up to 2u times a magnitude of at most
  D = max|a| + max(m - a) over the finite log scores a above m - 100 (below, a
  probability is under 2^-144 and only has to be tiny), plus the function's
  own error (a few u) and the sums' (one u per addition of positive terms):
  relative error below (4 D + 64 + additions) u. The gradient's terms are
  measured against the size of what is added up, with E and top_k additions.
* bf16 outputs: half a step, 2^-8 of the value, plus the fp32 error before it
  (2^-20 of the terms' size).
* dot products of N terms in fp32: N u of the sum of magnitudes.
* weight gradient: one u per slot added (twice, for the order inside an MFMA).
"""

import numpy as np
import pytest
import torch

import synth
from helpers import bf16_to_f64, need_gpu
from oracle import quant as oquant
from oracle import train as otrain

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def _moe():
    import mixture_experts_grouped_moe_amd as moe
    return moe


def f64(t):
    return t.detach().float().cpu().double().numpy()


def close(got, ref, tol, what=""):
    """|got - ref| <= tol elementwise, with equal NaN and infinity masks."""
    got, ref, tol = (np.asarray(v, dtype=np.float64) for v in (got, ref, tol))
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    # what lies past the largest float32 (and bfloat16) rounds to infinity
    ref = np.where(np.abs(ref) > 2.0 ** 128, np.copysign(np.inf, ref), ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: NaN positions differ"
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]), f"{what}: infinities differ"
    ok = ~np.isnan(ref) & ~inf
    err = np.abs(got - ref)[ok]
    bound = np.broadcast_to(tol, ref.shape)[ok]
    assert (err <= bound).all(), f"{what}: worst {np.max(err / np.maximum(bound, 1e-300)):.3g} of the tolerance"


# ------------------------------------------------------------------- router

def logits(T, E, seed, dtype="fp32", std=1.5):
    z = torch.randn((T, E), generator=synth.gen(seed, "logits"), dtype=torch.float32) * std
    return (z.to(torch.bfloat16) if dtype == "bf16" else z).cuda()


def spread(z, score):
    """D of the module's tolerance."""
    a = otrain.log_scores(z, score)
    a = np.where(np.isfinite(a), a, np.nan)
    if np.isnan(a).all():
        return 0.0
    with np.errstate(all="ignore"):
        m = np.nanmax(np.where(np.isnan(a), -np.inf, a), axis=1, keepdims=True)
        near = a > m - 100
    return float(np.max(np.where(near, np.abs(a) + (m - a), 0.0), initial=0.0))


def check_route(z, k, score="softmax", renorm=True, scale=1.0, mask=None, **kw):
    moe = _moe()
    got = moe.moe_route(z, k, score=score, renormalize=renorm, scale=scale, mask=mask, balance=True, **kw)
    torch.cuda.synchronize()
    zz, mm = f64(z), None if mask is None else mask.cpu().numpy()
    ids, w, counts, n, p, loss = otrain.route(zz, k, score, renorm, scale, mm)
    T, E = zz.shape
    assert np.array_equal(got[0].cpu().numpy(), ids)
    assert np.array_equal(got[2].cpu().numpy(), counts)
    assert int(got[3]) == n
    tol = (4 * spread(zz, score) + 64 + E) * U
    close(f64(got[1]), w, tol * np.abs(w) + 2.0 ** -120, "weights")
    with np.errstate(invalid="ignore"):
        close(f64(got[4]), p, (tol + T * U) * np.abs(p) + 2.0 ** -120, "prob_sum")
        close(f64(got[5]), loss, (2 * tol + T * U) * np.abs(loss) + 2.0 ** -120, "losses")
    # without the statistics: the same ids and weights
    ids2, w2 = moe.moe_route(z, k, score=score, renormalize=renorm, scale=scale, mask=mask)
    assert torch.equal(ids2, got[0])
    assert np.array_equal(w2.cpu().numpy(), got[1].cpu().numpy(), equal_nan=True)
    return got


def check_route_backward(z, k, fwd, score="softmax", renorm=True, scale=1.0, losses=True, seed=1, dw=None, **kw):
    moe = _moe()
    ids, _, counts, n = fwd[:4]
    T, E = z.shape
    if dw is None:
        dw = torch.randn((T, k), generator=synth.gen(seed, "dw")).cuda()
    dl = torch.tensor([0.5, -0.25], device="cuda") if losses else None
    got = moe.moe_route_backward(z, ids, dw, score=score, renormalize=renorm, scale=scale,
                                 counts=counts if losses else None, num_routed=n if losses else None, dlosses=dl, **kw)
    torch.cuda.synchronize()
    zz = f64(z)
    ref, size = otrain.route_backward(zz, ids.cpu().numpy(), dw.cpu().double().numpy(), score, renorm, scale,
                                      counts.cpu().numpy(), int(n), None if dl is None else dl.cpu().double().numpy())
    tol = (4 * spread(zz, score) + 64 + E + 2 * k) * U
    half = 2.0 ** -8 if z.dtype == torch.bfloat16 else U
    close(f64(got), ref, 2 * tol * size + half * np.abs(ref) + 2.0 ** -120, "dlogits")
    return got


SHAPES = [(1, 1, 1), (1, 8, 2), (5, 7, 7), (7, 64, 6), (33, 97, 5), (130, 128, 4), (257, 256, 8), (64, 300, 10),
          (40, 512, 8), (17, 1024, 64), (9, 1000, 1)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True),
                                          ("sigmoid", False)])
def test_route_and_gradient(T, E, k, dtype, score, renorm):
    z = logits(T, E, T * 7 + E, dtype)
    mask = (torch.rand(T, generator=synth.gen(T + E, "mask")) < 0.8).to(torch.uint8).cuda() if T > 5 else None
    fwd = check_route(z, k, score, renorm, 2.5, mask)
    check_route_backward(z, k, fwd, score, renorm, 2.5)
    check_route_backward(z, k, fwd, score, renorm, 2.5, losses=False)


@pytest.mark.parametrize("T", [0, 6001])
def test_route_no_tokens_and_many_rows_per_wave(T):
    z = logits(T, 40, 3)
    fwd = check_route(z, 3)
    check_route_backward(z, 3, fwd)


# from these lengths on a lane takes 32 logits of a row, one top_k for each list length
@pytest.mark.parametrize("T,E,k,score", [(16397, 160, 6, "softmax"), (16384, 256, 11, "sigmoid"),
                                         (8205, 500, 10, "softmax"), (8192, 300, 4, "sigmoid"),
                                         (4103, 1000, 3, "softmax"), (4096, 1024, 8, "sigmoid"),
                                         (16390, 129, 16, "softmax")])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_route_long_batches(T, E, k, score, dtype):
    z = logits(T, E, T + E, dtype)
    z[3, 5:] = float("-inf")  # five experts left, fewer than k
    z[T - 2] = float("-inf")
    z[T // 2, :] = 0.25       # all equal
    mask = (torch.rand(T, generator=synth.gen(T + E, "mask")) < 0.9).cuda()
    mask[:8] = True
    check_route(z, k, score, True, 1.5, mask)
    check_route(z, k, score, False)


# up to 256 workgroups' rows a lane takes 8 logits of a row, past them 16
@pytest.mark.parametrize("T,E,k,score", [(8193, 100, 4, "softmax"), (8192, 128, 20, "sigmoid"),
                                         (4100, 160, 6, "sigmoid"), (4096, 256, 33, "softmax"),
                                         (2049, 500, 10, "softmax"), (2048, 512, 64, "sigmoid"),
                                         (9000, 72, 10, "softmax"), (5000, 255, 17, "softmax")])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_route_gradient_of_long_batches(T, E, k, score, dtype):
    z = logits(T, E, T + E + 1, dtype)
    z[T - 1, 1:] = float("-inf")
    mask = (torch.rand(T, generator=synth.gen(T + E, "mask")) < 0.9).cuda()
    for renorm in (True, False):
        fwd = check_route(z, k, score, renorm, 0.5, mask)
        check_route_backward(z, k, fwd, score, renorm, 0.5)


def test_route_ties_take_the_lowest_expert():
    # logits of few distinct values, both zeros among them
    g = synth.gen(5, "ties")
    v = torch.tensor([-1.0, -0.0, 0.0, 0.5])
    z = v[torch.randint(0, 4, (200, 130), generator=g)].cuda()
    for zz in (z, z.to(torch.bfloat16)):
        fwd = check_route(zz, 9)
        check_route_backward(zz, 9, fwd)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True),
                                          ("sigmoid", False)])
def test_route_masked_experts_and_rows(dtype, score, renorm):
    z = torch.randn((12, 70), generator=synth.gen(6, "z"))
    low = torch.finfo(dtype).min
    z[0, 5:] = -float("inf")           # five experts left for six places
    z[1] = -float("inf")               # none
    z[2, 1:] = -float("inf")           # one
    z[3, 3:] = low                     # masked by the type's lowest value: chosen last, weight 0
    z[4] = low                         # all of them: uniform
    z[5, :] = 80.0                     # far from 0
    z[6, :] = -80.0
    z[7, 40] = 300.0
    z = z.to(dtype).cuda()
    mask = torch.ones(12, dtype=torch.bool, device="cuda")
    mask[8] = False
    z[8, 10] = float("nan")            # padding may hold anything
    z[8, 11] = float("inf")
    zz = z[:8] if score == "softmax" else z[[0, 1, 2, 5, 6, 7]]  # sigmoid of the lowest value: tested below
    got = check_route(zz, 6, score, renorm)
    check_route_backward(zz, 6, got, score, renorm, losses=False)
    m = check_route(z[8:].contiguous(), 6, score, renorm, mask=mask[8:])
    assert (m[0][0] == -1).all() and (m[1][0] == 0).all()
    d = check_route_backward(torch.where(torch.isfinite(z[8:]), z[8:], 0), 6, m, score, renorm)
    assert (d[0] == 0).all()
    moe = _moe()
    ids, w = moe.moe_route(z, 6, score=score, renormalize=renorm, mask=mask)
    dirty = moe.moe_route_backward(z, ids, torch.full_like(w, float("nan")), score=score, renormalize=renorm)
    assert (dirty[[1, 8]] == 0).all()  # nothing of a padded row's logits or weight gradients comes through


def test_route_sigmoid_of_the_lowest_value():
    # sigmoid underflows: unnormalised weights 0; renormalised, those left decide
    z = torch.full((2, 20), torch.finfo(torch.float32).min)
    z[0, :2] = torch.tensor([1.0, 2.0])
    got = check_route(z.cuda(), 4, "sigmoid", False)
    assert (got[1][0, 2:] == 0).all() and (got[1][1] == 0).all()
    got = check_route(z.cuda(), 4, "sigmoid", True)
    assert (got[1][1] == 0.25).all()


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True),
                                          ("sigmoid", False)])
def test_route_non_finite_logits_show(score, renorm):
    z = logits(6, 50, 8)
    z[2, 3] = float("nan")
    z[3] = float("nan")
    got = check_route(z, 5, score, renorm)
    assert torch.isnan(got[5][0]) and int(got[3]) == 6 and (got[0][2] >= 0).all() and (got[0][3] == -1).all()
    z = logits(6, 50, 9)
    z[1, 7] = float("inf")
    moe = _moe()
    ids, w, _, n, p, loss = moe.moe_route(z, 5, score=score, renormalize=renorm, balance=True)
    assert int(ids[1, 0]) == 7 and int(n) == 6
    assert torch.isnan(loss[0]) == (score == "softmax")
    if score == "sigmoid":
        assert torch.isfinite(w).all()


def test_route_strided_rows_and_given_outputs():
    moe = _moe()
    base = logits(30, 100, 10)
    z = base[:, 3:99]
    poison = (torch.full((30, 5), -7, dtype=torch.int32, device="cuda"),
              torch.full((30, 5), float("nan"), device="cuda"),
              torch.full((96,), -7, dtype=torch.int32, device="cuda"),
              torch.full((1,), -7, dtype=torch.int32, device="cuda"),
              torch.full((96,), float("nan"), device="cuda"), torch.full((2,), float("nan"), device="cuda"))
    ws = torch.full((moe.moe_route_workspace_bytes(30, 96),), 0xAB, dtype=torch.uint8, device="cuda")
    fwd = check_route(z, 5, out=poison, workspace=ws)
    assert fwd[0] is poison[0]
    wide = torch.full((33, 101), 9.0, device="cuda")
    check_route_backward(z, 5, fwd, out=wide[:30, 2:98])
    wide[:30, 2:98] = 9.0
    assert (wide == 9.0).all()
    b = base.to(torch.bfloat16)[:, 3:99]                    # rows on odd 2-byte addresses
    check_route_backward(b, 5, check_route(b, 5), out=wide.to(torch.bfloat16)[:30, 1:97])


def test_route_backward_skips_ids_out_of_range():
    z = logits(4, 20, 11)
    fwd = list(check_route(z, 3))
    ids = fwd[0].clone()
    ids[1, 2] = 20
    ids[2, 1] = -5
    ids[3, 0] = -1
    fwd[0] = ids
    check_route_backward(z, 3, fwd, renorm=False)
    check_route_backward(z, 3, fwd)


@pytest.mark.parametrize("E,k", [(20, 3), (300, 40)])
def test_route_backward_adds_an_expert_named_twice(E, k):
    z = logits(6, E, 13)
    fwd = list(check_route(z, k))
    ids = fwd[0].clone()
    ids[1] = ids[1, 0]              # one expert in every place
    ids[2, 1] = ids[2, 2]
    ids[4, k - 1] = ids[4, 0]
    fwd[0] = ids
    for score, renorm in (("softmax", False), ("softmax", True), ("sigmoid", False)):
        check_route_backward(z, k, fwd, score, renorm)


def test_route_repeats_bit_for_bit_on_any_stream():
    moe = _moe()
    z = logits(3000, 256, 12)
    ref = moe.moe_route(z, 8, balance=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        a = moe.moe_route(z, 8, balance=True)
        b = moe.moe_route(z, 8, balance=True, stream=side)      # both at once
        torch.cuda.synchronize()
        for x, y, r in zip(a, b, ref):
            assert torch.equal(x, r) and torch.equal(y, r)


# ------------------------------------------------------------------ combine

def _combine_case(T, k, N, E, seed, unrouted=True):
    g = synth.gen(seed, "combine")
    dy = torch.randn((T, N), generator=g).to(torch.bfloat16)
    c = torch.randn((T * k, N), generator=g).to(torch.bfloat16)
    w = torch.rand((T, k), generator=g)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    if unrouted and T > 2:
        ids[1] = -1
        ids[2, 0] = E
        c[k:2 * k] = float("nan")
        c[2 * k] = float("inf")
        w[1] = float("nan")
    return dy.cuda(), c.cuda(), w.cuda(), ids.cuda()


@pytest.mark.parametrize("T,k,N", [(1, 1, 8), (3, 2, 64), (7, 6, 1856), (50, 4, 2880), (21, 8, 7168), (5, 13, 264),
                                   (9, 10, 4104), (300, 1, 136)])
def test_combine_routed_and_backward(T, k, N):
    moe, E = _moe(), 9
    dy, c, w, ids = _combine_case(T, k, N, E, T + N)
    y = moe.moe_combine_routed(c, w, ids, E)
    dc, dw = moe.moe_combine_backward(dy, c, w, ids, E)
    torch.cuda.synchronize()
    n = ids.cpu().numpy()
    cc, ww = f64(c), w.cpu().double().numpy()
    ref = otrain.combine_routed(cc, ww, n, E)
    on = (n >= 0) & (n < E)
    size = otrain.combine_routed(np.abs(cc), np.abs(ww), n, E)
    close(f64(y), ref, 2.0 ** -8 * np.abs(ref) + k * U * size, "y")
    rc, rw, rs = otrain.combine_backward(f64(dy), cc, ww, n, E)
    close(f64(dc), rc, 2.0 ** -8 * (1 + 2.0 ** -15) * np.abs(rc), "dC")
    close(f64(dw), rw, N * U * rs, "dw")
    assert (f64(dc)[~on.reshape(-1)] == 0).all() and (f64(dw)[~on] == 0).all()
    # every slot routed: the plain combine's bits, and the same gradient without ids
    dy, c, w, ids = _combine_case(T, k, N, E, T + N, unrouted=False)
    assert torch.equal(moe.moe_combine_routed(c, w, ids, E), moe.moe_combine(c, w, k))
    a, b = moe.moe_combine_backward(dy, c, w, ids, E), moe.moe_combine_backward(dy, c, w)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_combine_backward_strides_and_rows_behind():
    moe, T, k, N = _moe(), 11, 3, 96
    dy, c, w, ids = _combine_case(T, k, N, 5, 77)
    wide = torch.full((T * k + 2, N + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    cw = torch.full((T * k, N + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    cw[:, :N] = c
    dyw = torch.cat([dy, dy], 1)[:, N:]
    dw = torch.empty((T, k), device="cuda")
    moe.moe_combine_backward(dyw, cw[:, :N], w, ids, 5, out=(wide[:, 8:N + 8], dw))
    ref = moe.moe_combine_backward(dy, c, w, ids, 5)
    torch.cuda.synchronize()
    assert torch.equal(wide[:T * k, 8:N + 8], ref[0]) and torch.equal(dw, ref[1])
    wide[:T * k, 8:N + 8] = 7.0
    assert (wide == 7.0).all()


def test_combine_over_more_than_one_launch():
    """More slots than one launch takes (2^20), and more output pieces (2^26)."""
    moe = _moe()
    g = torch.Generator(device="cuda").manual_seed(3)
    T, k, N, E = 349527, 3, 8, 5
    assert T * k > 1 << 20
    dy = torch.randn((T, N), generator=g, device="cuda").to(torch.bfloat16)
    c = torch.randn((T * k, N), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.rand((T, k), generator=g, device="cuda")
    ids = torch.randint(-1, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    on = (ids >= 0)
    dc, dw = moe.moe_combine_backward(dy, c, w, ids, E)
    ref = torch.where(on[..., None], w[..., None] * dy.float()[:, None, :], 0.0).to(torch.bfloat16)
    assert torch.equal(dc, ref.view(T * k, N))
    terms = torch.where(on[..., None], dy.double()[:, None, :] * c.double().view(T, k, N), 0.0)
    assert ((dw.double() - terms.sum(-1)).abs() <= N * U * terms.abs().sum(-1)).all()
    del dc, dw, ref, terms, dy, c
    T, N = (1 << 23) + 5, 64
    c = torch.randint(-32768, 32767, (T, N), generator=g, device="cuda", dtype=torch.int16).clamp_(-9000, 9000)
    c = (c.view(torch.int16) & 0x3FFF).view(torch.bfloat16)     # any finite bits below 2
    w = torch.rand((T, 1), generator=g, device="cuda")
    ids = torch.randint(-1, E, (T, 1), generator=g, device="cuda", dtype=torch.int32)
    y = moe.moe_combine_routed(c, w, ids, E)
    for part in (slice(0, 4096), slice(T // 2, T // 2 + 4096), slice(T - 4096, T)):
        want = torch.where(ids[part] >= 0, w[part] * c[part].float(), 0.0).to(torch.bfloat16)
        assert torch.equal(y[part], want)


def test_combine_no_tokens():
    moe = _moe()
    e = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    w, ids = torch.zeros((0, 2), device="cuda"), torch.zeros((0, 2), dtype=torch.int32, device="cuda")
    assert moe.moe_combine_routed(e, w, ids, 4).shape == (0, 64)
    assert moe.moe_combine_backward(e, e, w, ids, 4)[0].shape == (0, 64)


# --------------------------------------------------------------- activation

def _check_act(pre, dh, activation, **kw):
    moe = _moe()
    h, q, s = moe.moe_act_mxfp8(pre, activation, **kw)
    torch.cuda.synchronize()
    p = f64(pre)
    rh, rq, rs = otrain.act_mxfp8(p, activation)
    assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rs)
    close(f64(h), rh, 2.0 ** -8 * (1 + 2.0 ** -10) * np.abs(rh) + 2.0 ** -126, "h")
    q0, s0 = moe.moe_quantize_mxfp8(pre)
    assert torch.equal(q, q0) and torch.equal(s, s0)
    d, h2 = moe.moe_act_mxfp8_backward(q, s, dh, activation)
    torch.cuda.synchronize()
    rd, rh2, size = otrain.act_backward(rq, rs, f64(dh), activation)
    close(f64(d), rd, 2.0 ** -8 * np.abs(rd) + 2.0 ** -20 * size + 2.0 ** -126, "dpre")
    close(f64(h2), rh2, 2.0 ** -8 * (1 + 2.0 ** -10) * np.abs(rh2) + 2.0 ** -126, "h again")
    d1, none = moe.moe_act_mxfp8_backward(q, s, dh, activation, recompute=False)
    assert none is None and torch.equal(d1, d)
    return h, q, s


@pytest.mark.parametrize("R,N,activation", [(1, 64, "swiglu"), (1, 32, "relu2"), (42, 1856, "relu2"),
                                            (77, 5760, "swiglu"), (300, 192, "swiglu"), (129, 96, "relu2"),
                                            (1000, 448, "swiglu"), (0, 128, "swiglu"), (0, 96, "relu2")])
def test_act_checkpoint_and_backward(R, N, activation):
    g = synth.gen(R + N, "act")
    # blocks of very different magnitudes
    mag = torch.pow(2.0, torch.randint(-12, 5, (R, N // 32, 1), generator=g).float())
    pre = (torch.randn((R, N // 32, 32), generator=g) * mag).reshape(R, N).to(torch.bfloat16).cuda()
    dh = torch.randn((R, N // 2 if activation == "swiglu" else N), generator=g).to(torch.bfloat16).cuda()
    _check_act(pre, dh, activation)


def test_act_edges():
    # zeros, saturated gates on both sides, and blocks that hold a NaN or an infinity
    moe = _moe()
    pre = torch.zeros((6, 128))
    pre[1, :32] = 60.0
    pre[1, 32:64] = -60.0
    pre[1, 64:] = 3.0
    pre[2] = torch.linspace(-20, 20, 128)
    pre[3] = -1.278
    dh = torch.ones((6, 64), dtype=torch.bfloat16, device="cuda")
    _check_act(pre.to(torch.bfloat16).cuda(), dh, "swiglu")
    _check_act(pre.to(torch.bfloat16).cuda(), torch.ones((6, 128), dtype=torch.bfloat16, device="cuda"), "relu2")
    pre[4, 70] = float("inf")
    pre[5, 3] = float("nan")
    p = pre.to(torch.bfloat16).cuda()
    h, q, s = moe.moe_act_mxfp8(p, "swiglu")
    d, h2 = moe.moe_act_mxfp8_backward(q, s, dh, "swiglu")
    torch.cuda.synchronize()
    assert int(s[4, 2]) == 0xFF and int(s[5, 0]) == 0xFF and (s[:4] != 0xFF).all()
    assert torch.isnan(h[5, 3]) and torch.isfinite(h[5, 4:]).all()
    # the NaN block is 32 elements of one half; its partner half's gradient is NaN with it
    for row in (4, 5):
        assert torch.isnan(h2[row, :32]).all() and torch.isfinite(h2[row, 32:]).all()
        assert torch.isfinite(d[row, 32:64]).all() and torch.isfinite(d[row, 96:]).all()
    assert torch.isnan(d[4, :32]).all() and torch.isnan(d[5, :32]).all() and torch.isnan(d[5, 64:96]).all()


def test_act_strides_and_rows_behind():
    moe, R, N = _moe(), 13, 128
    g = synth.gen(4, "act")
    base = torch.randn((R, N + 24), generator=g).to(torch.bfloat16).cuda()
    pre = base[:, 8:8 + N]
    ref = moe.moe_act_mxfp8(pre.contiguous(), "swiglu")
    h = torch.full((R + 1, 80), 5.0, dtype=torch.bfloat16, device="cuda")
    q = torch.full((R + 1, N + 16), 0xAB, dtype=torch.uint8, device="cuda")
    s = torch.full((R + 1, 7), 0xCD, dtype=torch.uint8, device="cuda")
    moe.moe_act_mxfp8(pre, "swiglu", out=(h[:, 8:72], q[:, 16:], s[:, 3:]))
    torch.cuda.synchronize()
    assert torch.equal(h[:R, 8:72], ref[0]) and torch.equal(q[:R, 16:], ref[1]) and torch.equal(s[:R, 3:], ref[2])
    dh = torch.randn((R, 72), generator=g).to(torch.bfloat16).cuda()[:, 8:]
    want = moe.moe_act_mxfp8_backward(ref[1], ref[2], dh.contiguous(), "swiglu")
    d = torch.full((R + 1, N + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    h2 = torch.full((R + 1, 72), 5.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_act_mxfp8_backward(q[:R, 16:], s[:R, 3:], dh, "swiglu", out=(d[:, 8:], h2[:, :64]))
    torch.cuda.synchronize()
    assert torch.equal(d[:R, 8:], want[0]) and torch.equal(h2[:R, :64], want[1])
    h[:R, 8:72], q[:R, 16:], s[:R, 3:], d[:R, 8:], h2[:R, :64] = 5.0, 0xAB, 0xCD, 5.0, 5.0
    assert (h == 5).all() and (q == 0xAB).all() and (s == 0xCD).all() and (d == 5).all() and (h2 == 5).all()


# ---------------------------------------------------------- weight gradient

def _wgrad_case(T, k, E, N, K, seed):
    d = synth.config5(seed=seed, T=T, E=E, N=N, K=K, k=k, device="cuda")
    moe = _moe()
    xq, xs = moe.moe_quantize_mxfp8(d["x"])
    return xq, xs, d["grad"], d["ids"]


def _check_wgrad(xq, xs, grad, ids, E, out=None, experts=None):
    moe = _moe()
    T, k = ids.shape
    routing = moe.moe_align(ids, E, moe.moe_wgrad_block_m())
    dw = moe.moe_wgrad_mxfp8(xq, xs, grad, routing, T, k, E, out=out)
    torch.cuda.synchronize()
    n, hq, hs, hg = ids.cpu().numpy(), xq.cpu().numpy(), xs.cpu().numpy(), f64(grad)
    for e in range(E) if experts is None else experts:
        ref, size = otrain.wgrad_mxfp8_expert(hq, hs, hg, n, k, e)
        close(dw[e].cpu().double().numpy(), ref, (2 * int((n == e).sum()) + 2) * U * size, f"expert {e}")
    return dw


@pytest.mark.parametrize("T,k,E,N,K", [(300, 4, 8, 256, 384), (97, 2, 5, 160, 96), (1000, 8, 32, 64, 128),
                                       (130, 3, 7, 96, 160), (64, 6, 12, 64, 64), (1, 1, 1, 32, 32),
                                       (64, 2, 8, 512, 256), (700, 1, 2, 288, 544)])
def test_wgrad_mxfp8(T, k, E, N, K):
    case = _wgrad_case(T, k, E, N, K, T)
    dw = _check_wgrad(*case, E, out=torch.full((E, N, K), float("nan"), device="cuda"))
    # the bits of moe_wgrad on the decoded rows (exact in bf16)
    moe = _moe()
    xq, xs, grad, ids = case
    x = torch.from_numpy(oquant.mx_dequantize_e4m3(xq.cpu().numpy(), xs.cpu().numpy())).to(torch.bfloat16).cuda()
    routing = moe.moe_align(ids, E, moe.moe_wgrad_block_m())
    assert torch.equal(dw, moe.moe_wgrad(x, grad, routing, T, k, E))


def test_wgrad_mxfp8_unrouted_slots_and_empty_experts():
    xq, xs, grad, ids = _wgrad_case(200, 3, 10, 96, 128, 5)
    ids = torch.where(ids >= 7, -1, ids).contiguous()          # experts 7..9 empty, their slots routed nowhere
    ids[10:20] = -1                                            # padded tokens: rows that may hold anything
    xq[10:20], xs[10:20] = 0x7F, 0xFF
    grad[30:60] = float("nan")
    dw = _check_wgrad(xq, xs, grad, ids, 10)
    assert (dw[7:] == 0).all()


def test_wgrad_mxfp8_strides_at_the_end_of_an_allocation():
    T, k, E, N, K = 50, 2, 3, 64, 96
    xq, xs, grad, ids = _wgrad_case(T, k, E, N, K, 6)
    xw = torch.zeros((T, K + 32), dtype=torch.uint8, device="cuda")
    sw = torch.zeros((T, 8), dtype=torch.uint8, device="cuda")
    gw = torch.zeros((T * k, N + 8), dtype=torch.bfloat16, device="cuda")
    xw[:, 32:], sw[:, 5:], gw[:, 8:] = xq, xs, grad            # the last row ends with the buffer
    _check_wgrad(xw[:, 32:], sw[:, 5:], gw[:, 8:], ids, E)


def test_wgrad_strides_at_the_end_of_an_allocation():
    """The bf16 entry point: a tile wider than the rows reads nothing past the last one."""
    moe = _moe()
    T, k, E, N, K = 50, 2, 3, 64, 96
    xq, xs, grad, ids = _wgrad_case(T, k, E, N, K, 6)
    x = torch.from_numpy(oquant.mx_dequantize_e4m3(xq.cpu().numpy(), xs.cpu().numpy())).to(torch.bfloat16)
    xw = torch.zeros((T, K + 512), dtype=torch.bfloat16, device="cuda")
    gw = torch.zeros((T * k, N + 512), dtype=torch.bfloat16, device="cuda")
    xw[:, 512:], gw[:, 512:] = x.cuda(), grad
    routing = moe.moe_align(ids, E, moe.moe_wgrad_block_m())
    dw = moe.moe_wgrad(xw[:, 512:], gw[:, 512:], routing, T, k, E)
    assert torch.equal(dw, moe.moe_wgrad(x.cuda(), grad, routing, T, k, E))
    _check_wgrad(xq, xs, grad, ids, E)


def test_wgrad_mxfp8_scale_edges():
    T, k, E, N, K = 40, 1, 2, 32, 64
    xq, xs, grad, ids = _wgrad_case(T, k, E, N, K, 7)
    xs[:, 0] = 100 + torch.arange(T, device="cuda", dtype=torch.uint8)
    xq[:, 32:] = 0
    xs[:, 1] = 0
    _check_wgrad(xq, xs, grad, ids, E)
    xs[3, 1] = 0xFF                                            # a NaN block reaches its 32 columns of one expert
    moe = _moe()
    routing = moe.moe_align(ids, E, moe.moe_wgrad_block_m())
    dw = moe.moe_wgrad_mxfp8(xq, xs, grad, routing, T, k, E)
    e = int(ids[3, 0])
    assert torch.isnan(dw[e, :, 32:]).all() and torch.isfinite(dw[e, :, :32]).all() and torch.isfinite(dw[1 - e]).all()


def test_wgrad_mxfp8_no_tokens():
    moe, E, N, K = _moe(), 4, 64, 96
    ids = torch.zeros((0, 2), dtype=torch.int32, device="cuda")
    routing = moe.moe_align(ids, E, moe.moe_wgrad_block_m())
    dw = torch.full((E, N, K), float("nan"), device="cuda")
    moe.moe_wgrad_mxfp8(torch.zeros((0, K), dtype=torch.uint8, device="cuda"),
                        torch.zeros((0, K // 32), dtype=torch.uint8, device="cuda"),
                        torch.zeros((0, N), dtype=torch.bfloat16, device="cuda"), routing, 0, 2, E, out=dw)
    torch.cuda.synchronize()
    assert (dw == 0).all()


def test_wgrad_mxfp8_large_sampled():
    # ragged tiles, hundreds of blocks, many tiles per workgroup
    T, k, E, N, K = 4096, 4, 48, 1056, 2880
    case = _wgrad_case(T, k, E, N, K, 8)
    a = _check_wgrad(*case, E, experts=[0, 17, 47]).clone()
    moe = _moe()
    routing = moe.moe_align(case[3], E, moe.moe_wgrad_block_m())
    assert torch.equal(a, moe.moe_wgrad_mxfp8(*case[:3], routing, T, k, E))


# --------------------------------------------------------- the whole step

def _step(moe, d, bufs=None):
    """One forward and backward pass of a SwiGLU layer; returns its tensors."""
    T, H = d["x"].shape
    E, k, I = d["w1"].shape[0], d["k"], d["w2"].shape[2]
    xq, xs = moe.moe_quantize_mxfp8(d["x"])
    ids, w, counts, n, _, losses = moe.moe_route(d["logits"], k, mask=d["mask"], balance=True)
    routing = moe.moe_align(ids, E, moe.moe_gemm_block_m("bf16", T))
    pre = moe.moe_grouped_gemm(d["x"], d["w1"], "bf16", routing, T, k, E, k)
    h, q, s = moe.moe_act_mxfp8(pre, "swiglu")
    c = moe.moe_grouped_gemm(h, d["w2"], "bf16", routing, T, k, E, 1)
    y = moe.moe_combine_routed(c, w, ids, E)
    dc, dw = moe.moe_combine_backward(d["dy"], c, w, ids, E)
    dh = moe.moe_grouped_gemm(dc, d["w2t"], "bf16", routing, T, k, E, 1)
    dpre, h = moe.moe_act_mxfp8_backward(q, s, dh, "swiglu")
    wr = moe.moe_align(ids, E, moe.moe_wgrad_block_m())
    dw2 = moe.moe_wgrad(h, dc, wr, T * k, 1, E)
    dw1 = moe.moe_wgrad_mxfp8(xq, xs, dpre, wr, T, k, E)
    dxs = moe.moe_grouped_gemm(dpre, d["w1t"], "bf16", routing, T, k, E, 1)
    dx = moe.moe_combine_routed(dxs, d["ones"], ids, E)
    dz = moe.moe_route_backward(d["logits"], ids, dw, counts=counts, num_routed=n, dlosses=d["dlosses"])
    return {"y": y, "losses": losses, "dw1": dw1, "dw2": dw2, "dx": dx, "dz": dz, "ids": ids}


def _step_case(T=70, H=128, I=96, E=6, k=2):
    g = synth.gen(31, "step")

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g) * std
    d = {"k": k, "x": normal(T, H).to(torch.bfloat16).cuda(), "logits": normal(T, E).cuda(),
         "w1": normal(E, 2 * I, H, std=H ** -0.5).to(torch.bfloat16).cuda(),
         "w2": normal(E, H, I, std=I ** -0.5).to(torch.bfloat16).cuda(),
         "dy": normal(T, H).to(torch.bfloat16).cuda(), "mask": torch.ones(T, dtype=torch.uint8).cuda(),
         "ones": torch.ones((T, k)).cuda(), "dlosses": torch.tensor([0.3, 0.1]).cuda()}
    d["mask"][5:9] = 0
    d["x"][6] = float("nan")                        # padding may hold anything
    d["w1t"], d["w2t"] = (t.transpose(1, 2).contiguous() for t in (d["w1"], d["w2"]))
    return d


def test_training_step_against_autograd():
    moe, d = _moe(), _step_case()
    T, H = d["x"].shape
    E, k, I = 6, 2, 96
    # NaN in freed memory, so that an unwritten row that is read would show
    torch.cuda.empty_cache()
    torch.full((1 << 24,), float("nan"), device="cuda")
    got = _step(moe, d)
    torch.cuda.synchronize()
    # the same step in float64 by autograd, without any rounding
    live = torch.ones(T, dtype=torch.bool)
    live[5:9] = False
    x = torch.where(live[:, None], d["x"].double().cpu(), 0).requires_grad_()
    z = d["logits"].double().cpu().requires_grad_()
    w1, w2 = (d[n].double().cpu().requires_grad_() for n in ("w1", "w2"))
    ids = got["ids"].cpu().long()
    ix = ids.clamp(min=0)
    p = torch.softmax(z, 1)
    v = p.gather(1, ix)
    w = (v / v.sum(1, keepdim=True)) * live[:, None]
    pre = torch.einsum("th,tknh->tkn", x, w1[ix])
    h = torch.nn.functional.silu(pre[..., :I]) * pre[..., I:]
    y = (torch.einsum("tki,tkni->tkn", h, w2[ix]) * w[:, :, None]).sum(1)
    n = int(live.sum())
    f = torch.bincount(ix[live].reshape(-1), minlength=E).double() / (n * k)
    loss = torch.stack([E * (f * p[live].mean(0)).sum(), (torch.logsumexp(z[live], 1) ** 2).mean()])
    ((y * d["dy"].double().cpu()).sum() + (loss * d["dlosses"].double().cpu()).sum()).backward()
    np.testing.assert_allclose(got["losses"].cpu().numpy(), loss.detach().numpy(), rtol=1e-5)

    # relative to the largest entry. Forward: four bf16 roundings (pre, h, C,
    # y), 4 * 2^-8. Backward: those and the MXFP8 roundings of x and pre, each
    # 2^-4 of an element (2^-3 where a block's maximum saturates) whose effects
    # add up like random signs over at least 8 terms: 2 * 2^-3 / sqrt(8) + 8 * 2^-8
    for name, ref, tol in (("y", y, 2.0 ** -6), ("dz", z.grad, 0.12), ("dw1", w1.grad, 0.12), ("dw2", w2.grad, 0.12),
                           ("dx", x.grad, 0.12)):
        r, g = ref.detach().numpy(), f64(got[name])
        assert np.isfinite(g).all(), name
        err = np.abs(g - r).max() / np.abs(r).max()
        assert err <= tol, (name, err)
    assert (got["y"][5:9] == 0).all() and (got["dz"][5:9] == 0).all() and (got["dx"][5:9] == 0).all()


def test_training_step_captured_and_replayed():
    moe, d = _moe(), _step_case()
    ref = {n: t.clone() for n, t in _step(moe, d).items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(moe, d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = _step(moe, d)
    for i in range(3):
        for t in out.values():
            t.fill_(-3)
        eager = _step(moe, d)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in ref:
            assert torch.equal(out[n], ref[n]) and torch.equal(eager[n], ref[n]), (i, n)


def _far_rows(rows, width, dtype):
    """A [rows, width] view whose rows lie 2^32 + 64 bytes apart."""
    es = torch.empty((), dtype=dtype).element_size()
    ld = ((1 << 32) + 64) // es
    return torch.empty((rows - 1) * ld + width, dtype=dtype, device="cuda").as_strided((rows, width), (ld, 1))


def test_rows_more_than_32_bits_apart():
    moe = _moe()
    g = synth.gen(43, "far")
    R, k, E, N = 4, 2, 32, 128
    pre = torch.randn((R, N), generator=g).to(torch.bfloat16).cuda()
    dh = torch.randn((R, N // 2), generator=g).to(torch.bfloat16).cuda()
    z = logits(R, E, 44)
    c = torch.randn((R, N), generator=g).to(torch.bfloat16).cuda()
    dy = torch.randn((R // k, N), generator=g).to(torch.bfloat16).cuda()

    def far(t):
        return _far_rows(*t.shape, t.dtype).copy_(t)

    def like(t):
        return _far_rows(*t.shape, t.dtype)

    h, q, s = moe.moe_act_mxfp8(pre, "swiglu")
    got = moe.moe_act_mxfp8(far(pre), "swiglu", out=(like(h), like(q), like(s)))
    assert all(torch.equal(a, b) for a, b in zip(got, (h, q, s)))
    ref = moe.moe_act_mxfp8_backward(q, s, dh, "swiglu")
    got = moe.moe_act_mxfp8_backward(got[1], got[2], far(dh), "swiglu", out=tuple(like(t) for t in ref))
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    del got
    ids, w = moe.moe_route(z, k)
    zf = far(z)
    got = moe.moe_route(zf, k)
    assert torch.equal(got[0], ids) and torch.equal(got[1], w)
    ref = moe.moe_route_backward(z, ids, w)
    assert torch.equal(moe.moe_route_backward(zf, ids, w, out=like(ref)), ref)
    del zf
    ids, w = ids[:R // k].contiguous(), w[:R // k].contiguous()
    cf, dyf = far(c), far(dy)
    ref = moe.moe_combine_routed(c, w, ids, E)
    assert torch.equal(moe.moe_combine_routed(cf, w, ids, E, out=like(ref)), ref)
    dc, dw = moe.moe_combine_backward(dy, c, w, ids, E)
    got = moe.moe_combine_backward(dyf, cf, w, ids, E, out=(like(dc), torch.empty_like(dw)))
    assert torch.equal(got[0], dc) and torch.equal(got[1], dw)
    # and ld larger than a row alone says nothing of one row
    assert torch.equal(moe.moe_route(_far_rows(1, E, torch.float32).copy_(z[:1]), k)[0], moe.moe_route(z[:1], k)[0])


@pytest.mark.parametrize("T", [1, 7])
def test_router_feeds_the_decode_layer(T):
    """A decode step from logits, captured: new logits at every replay."""
    moe = _moe()
    E, k, K, N = 16, 3, 64, 96
    g = synth.gen(41, "decode")
    x = torch.randn((T, K), generator=g).to(torch.bfloat16).cuda()
    w = (torch.randn((E, N, K), generator=g) / 8).to(torch.bfloat16).cuda()
    mask = torch.ones(T, dtype=torch.bool, device="cuda")
    mask[T // 2] = T == 1              # one padded row, but for the single token
    z = torch.empty((T, E), dtype=torch.bfloat16, device="cuda")

    def step():
        ids, tw = moe.moe_route(z, k, renormalize=False, mask=mask)
        return ids, tw, moe.moe_decode_layer(x, ids, tw, w, "bf16", epilogue="relu2")

    def unfused(ids, tw):
        routing = moe.moe_align(ids, E, moe.moe_gemm_block_m("bf16", T))
        c = moe.moe_grouped_gemm(x, w, "bf16", routing, T, k, E, k, epilogue="relu2")
        return moe.moe_combine_routed(c, tw, ids, E)

    z.copy_(logits(T, E, 1, "bf16"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step()
    for i in range(4):
        z.copy_(logits(T, E, 50 + i, "bf16"))
        ids, tw, y = step()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(ids.cpu().numpy(), otrain.route(f64(z), k, "softmax", False, 1.0, mask.cpu().numpy())[0])
        assert torch.equal(out[0], ids) and torch.equal(out[1], tw) and torch.equal(out[2], y)
        assert torch.equal(y, unfused(ids, tw)) and (y[~mask] == 0).all() and (y[mask] != 0).any()


@pytest.mark.parametrize("T", [0, 1, 3, 65, 5000])
@pytest.mark.parametrize("E,k", [(1, 1), (40, 3), (256, 8), (1024, 5), (1024, 40)])
def test_route_stays_inside_its_workspace(T, E, k):
    """A workspace of exactly the stated size, and outputs of their own, inside a guarded buffer."""
    moe = _moe()
    need = moe.moe_route_workspace_bytes(T, E)
    size, guard = -(-need // 8) * 8, 16384
    buf = torch.full((guard + size + guard,), 0xAB, dtype=torch.uint8, device="cuda")
    z = logits(T, E, T + E)
    got = check_route(z, k, workspace=buf[guard:guard + need])
    assert (buf[:guard] == 0xAB).all() and (buf[guard + need:] == 0xAB).all()
    if T == 0:
        assert all((t == 0).all() for t in got[2:])


@pytest.mark.parametrize("activation", ["swiglu", "relu2"])
def test_act_in_columns_of_one_buffer(activation):
    """Input and outputs interleaved row by row, no byte shared."""
    moe, R, N = _moe(), 37, 192
    H = N // 2 if activation == "swiglu" else N
    g = synth.gen(51, "columns")
    pre = torch.randn((R, N), generator=g).to(torch.bfloat16).cuda()
    dh = torch.randn((R, H), generator=g).to(torch.bfloat16).cuda()
    ref = moe.moe_act_mxfp8(pre, activation)
    want = moe.moe_act_mxfp8_backward(ref[1], ref[2], dh, activation)

    def columns(*widths):
        """uint8 columns of these widths, each starting on 16 bytes, and the buffer."""
        at, cuts = 0, []
        for w in widths:
            cuts.append((at, at + w))
            at += -(-w // 16) * 16
        buf = torch.full((R, at + 16), 0xA5, dtype=torch.uint8, device="cuda")
        return [buf[:, a:b] for a, b in cuts], buf, cuts

    (p, h, q, s), buf, cuts = columns(2 * N, 2 * H, N, N // 32)
    p.view(torch.bfloat16).copy_(pre)
    got = moe.moe_act_mxfp8(p.view(torch.bfloat16), activation, out=(h.view(torch.bfloat16), q, s))
    assert all(torch.equal(a, b) for a, b in zip(got, ref)) and torch.equal(p.view(torch.bfloat16), pre)
    for a, b in cuts:
        buf[:, a:b] = 0xA5
    assert (buf == 0xA5).all()
    (q, s, d, dp, h), buf, cuts = columns(N, N // 32, 2 * H, 2 * N, 2 * H)
    q.copy_(ref[1]), s.copy_(ref[2]), d.view(torch.bfloat16).copy_(dh)
    got = moe.moe_act_mxfp8_backward(q, s, d.view(torch.bfloat16), activation,
                                     out=(dp.view(torch.bfloat16), h.view(torch.bfloat16)))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(q, ref[1]) and torch.equal(s, ref[2]) and torch.equal(d.view(torch.bfloat16), dh)
    for a, b in cuts:
        buf[:, a:b] = 0xA5
    assert (buf == 0xA5).all()


def test_gradients_beside_their_inputs():
    """dlogits beside logits, dC beside C: columns of one buffer."""
    moe = _moe()
    for dtype, E in (("fp32", 70), ("bf16", 70), ("fp32", 256)):
        both = torch.cat([logits(50, E, 52, dtype)] * 2, 1)
        z, keep = both[:, :E], both[:, :E].clone()
        fwd = check_route(z, 6)
        check_route_backward(z, 6, fwd, out=both[:, E:])
        check_route_backward(both[:, :E].contiguous(), 6, fwd)
        assert torch.equal(z, keep)
    T, k, N = 9, 3, 136
    dy, c, w, ids = _combine_case(T, k, N, 5, 53)
    both = torch.cat([c, c], 1)
    dw = torch.empty((T, k), device="cuda")
    ref = moe.moe_combine_backward(dy, c, w, ids, 5)
    moe.moe_combine_backward(dy, both[:, :N], w, ids, 5, out=(both[:, N:], dw))
    assert torch.equal(both[:, N:], ref[0]) and torch.equal(dw, ref[1])
    assert torch.equal(both[:, :N].contiguous().view(torch.int16), c.view(torch.int16))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("top", [-20.0, -59.0, -61.0])
@pytest.mark.parametrize("E,k", [(70, 6), (300, 20)])
def test_route_sigmoid_scores_far_below_one(dtype, top, E, k):
    """Logits spread over 70 below a largest one that lies far below 0: their shares reach down to
    e^-70, the scores themselves past the smallest float."""
    g = synth.gen(61, "low")
    z = top - 70 * torch.rand((40, E), generator=g)
    z[:, 3] = top
    z[::2, 5] = top - 29.5
    z[1, k - 1:] = float("-inf")
    z = (z.to(torch.bfloat16) if dtype == "bf16" else z).cuda()
    for renorm in (True, False):
        fwd = check_route(z, k, "sigmoid", renorm)
        check_route_backward(z, k, fwd, "sigmoid", renorm)
    check_route_backward(z, k, check_route(z, k, "softmax", False), "softmax", False)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("k", [5, 20])
def test_route_weights_beside_non_finite_logits(dtype, k):
    """Which weights a NaN or an infinite logit reaches, as moe_train.h states it."""
    moe = _moe()
    clean = logits(6, 50, 62, dtype)
    z = clean.clone()
    z[2, 3] = float("nan")
    z[4, 7] = float("inf")
    rest = clean.clone()
    rest[2, 3] = float("-inf")                         # the row without its NaN expert
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            ids, w = moe.moe_route(z, k, score=score, renormalize=renorm)
            want = moe.moe_route(rest, k, score=score, renormalize=renorm)
            assert torch.equal(ids[:4], want[0][:4]) and int(ids[4, 0]) == 7
            assert torch.equal(w[[0, 1, 3, 5]], want[1][[0, 1, 3, 5]])
            if score == "softmax" and not renorm:
                assert torch.isnan(w[2]).all()
            else:
                assert torch.equal(w[2], want[1][2])
            if score == "softmax":
                assert torch.isnan(w[4]).all()
            else:
                assert torch.isfinite(w[4]).all() and (renorm or w[4, 0] == 1.0)


def test_training_step_reads_nothing_that_it_did_not_write(monkeypatch):
    """Every output, workspace and intermediate of the step starts as one repeated byte (0xFF: NaN in
    bf16, fp32, E4M3 and E8M0); the results have the same bits whatever it is."""
    moe, d = _moe(), _step_case()
    plain, filled = {n: getattr(torch, n) for n in ("empty", "empty_strided")}, []
    byte = [0]

    def filling(name):
        def make(*args, **kw):
            t = plain[name](*args, **kw)
            if t.is_cuda:
                t.view(torch.uint8).fill_(byte[0])
                filled.append(t.numel())
            return t
        return make

    for name in plain:
        monkeypatch.setattr(torch, name, filling(name))
    runs = []
    for byte[0] in (0xFF, 0x00, 0x47):
        del filled[:]
        runs.append({n: t.clone() for n, t in _step(moe, d).items()})
        assert len(filled) > 20
    for n, t in runs[0].items():
        assert not t.is_floating_point() or torch.isfinite(t).all(), n
        for r in runs[1:]:
            assert torch.equal(r[n], t), n


def test_training_step_replayed_on_new_inputs():
    """Captured once, replayed on other logits, activations, gradients, padding and loss weights:
    every replay against an eager step on the same inputs."""
    moe, d = _moe(), _step_case()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(moe, d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = _step(moe, d)
    seen = []
    for i in range(5):
        g = synth.gen(70 + i, "replay")
        for name in ("x", "logits", "dy"):
            d[name].copy_(torch.randn(d[name].shape, generator=g).to(d[name].dtype))
        d["logits"][:, i] += 2.0                       # another favourite expert each time
        d["mask"].copy_(torch.rand(len(d["mask"]), generator=g) < (0.0 if i == 3 else 0.8))   # once all padding
        d["dlosses"].copy_(torch.rand(2, generator=g))
        for t in out.values():
            t.fill_(-3)
        eager = {n: t.clone() for n, t in _step(moe, d).items()}
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n, t in eager.items():
            assert torch.equal(out[n], t), (i, n)
        assert torch.isfinite(out["dw1"]).all() and (i != 3 or (out["dw1"] == 0).all())
        seen.append(eager["losses"])
    assert len({tuple(l.tolist()) for l in seen}) == 5


def _every_code():
    """Row t: the 256 E4M3 codes under scale byte t, and their values (float64; NaN under byte 0xFF)."""
    q = torch.arange(256, dtype=torch.uint8).repeat(256, 1)
    s = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 8)
    v = oquant.mx_dequantize_e4m3(q.numpy(), s.numpy())
    v[255] = np.nan
    return q.cuda(), s.cuda(), v


def _bf16(v):
    with np.errstate(over="ignore"):
        return torch.from_numpy(v).to(torch.bfloat16).double().numpy()


@pytest.mark.parametrize("p", [0, 60, -60])
def test_wgrad_mxfp8_decodes_every_code_under_every_scale(p):
    """One slot an expert: dW is grad times the decoded row, exact (bf16's subnormals and the
    infinities past its range with it)."""
    moe, N = _moe(), 32
    q, s, v = _every_code()
    ids = torch.arange(256, dtype=torch.int32)[:, None].cuda()
    grad = torch.full((256, N), 2.0 ** p).to(torch.bfloat16).cuda()
    routing = moe.moe_align(ids, 256, moe.moe_wgrad_block_m())
    dw = moe.moe_wgrad_mxfp8(q, s, grad, routing, 256, 1, 256)
    torch.cuda.synchronize()
    with np.errstate(over="ignore", invalid="ignore"):
        want = (_bf16(v) * 2.0 ** p).astype(np.float32)
    for n in (0, N - 1):
        got = dw[:, n].cpu().numpy()
        assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("p", [0, 50, -50])
def test_act_relu2_gradient_of_every_code_under_every_scale(p):
    """Scales up to 2^119, the largest that a finite bf16 has: the gradient is finite wherever its value is."""
    moe = _moe()
    q, s, v = (t[:247] for t in _every_code())
    dh = torch.full((247, 256), 2.0 ** p).to(torch.bfloat16).cuda()
    d, h = moe.moe_act_mxfp8_backward(q, s, dh, "relu2")
    torch.cuda.synchronize()
    with np.errstate(over="ignore", invalid="ignore"):
        assert np.array_equal(f64(d), _bf16(np.where(v > 0, 2 * v * 2.0 ** p, 0.0)))     # (NaN codes give 0)
        assert np.array_equal(f64(h), _bf16(np.where(v > 0, v * v, 0.0)))    # 8 significant bits: exact
