"""GPU tests of moe_lora and moe_lora_backward against the float64 oracle
(oracle.block).

Tolerances (u = 2^-24, half a step of fp32; the products of bf16 values are
exact). The oracle on the magnitudes gives for every output the sum of the
magnitudes of its terms, `size`; relative to it
* h: K additions, K u.
* C's addition: h's K u, its scale, the two bf16 terms (each half a step, 2^-8
  of 2^-8: 2^-16), R additions: (K + R + 4) u + 2^-16, then half a step of bf16.
* dx: the same with dh, (N + R + 4) u + 2^-16.
* da, with at most n slots in a group: dh's N u, 2^-16, n additions; db without
  the N u.
"""

import numpy as np
import pytest
import torch

import synth
from block_helpers import U, close, f64, normal, strided
from helpers import need_gpu
from oracle import block as oblock

pytestmark = pytest.mark.gpu

SPLIT = 2.0 ** -16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def _moe():
    import mixture_experts_grouped_moe_amd as moe
    return moe


class Case:
    def __init__(self, S, G, R, K, N, div=1, bm=None, seed=0, scale=True, free=0.125):
        moe = _moe()
        gen = synth.gen(seed + S + G, "ids")
        share = torch.exp(torch.randn(G, generator=gen))
        self.ids = torch.multinomial(share, max(S, 1), replacement=True, generator=gen)[:S].to(torch.int32)
        self.ids[torch.rand(S, generator=gen) < free] = -1
        self.div, self.bm = div, bm or moe.moe_lora_block_m(S, G)
        self.routing = moe.moe_align(self.ids[:, None].contiguous().cuda(), G, self.bm)
        self.c, self.x = normal((S, N), seed, "c"), normal((-(-S // div), K), seed, "x")
        self.a, self.b = normal((G, R, K), seed, "a", std=K ** -0.5), normal((G, N, R), seed, "b", std=0.1)
        self.scale = normal((G,), seed, "s", "fp32") if scale else None
        self.dy, self.dx = normal((S, N), seed, "dy", std=0.1), normal((S, K), seed, "dx", std=0.1)
        self.S, self.G, self.R, self.K, self.N = S, G, R, K, N
        # what no slot of a group may touch: rows without one hold NaN
        free = (self.ids < 0).cuda()
        if div == 1:
            self.x[free] = float("nan")
        self.c[free], self.dy[free], self.dx[free] = (float("nan"),) * 3

    def args(self):
        return self.x, self.a, self.b, self.routing

    def host(self, c):
        on = (self.ids >= 0).numpy()
        clean = lambda t: np.where(on[:, None], np.nan_to_num(f64(t)), 0)  # noqa: E731
        x = f64(self.x)
        return clean(c), np.nan_to_num(x), f64(self.a), f64(self.b), self.ids.numpy(), \
            None if self.scale is None else f64(self.scale)

    def check(self, c, h, c0):
        arg = self.host(c0)
        on = arg[4] >= 0
        ref, rh = oblock.lora(*arg, row_div=self.div)
        mag = [None if v is None else np.abs(v) for v in arg]
        zero = [np.zeros_like(mag[0])] + mag[1:4] + [arg[4], mag[5]]
        size, hsize = oblock.lora(*zero, row_div=self.div)
        tol = ((self.K + self.R + 4) * U + SPLIT) * size
        close(f64(c)[on], ref[on], (tol + 2.0 ** -8 * (np.abs(ref) + tol))[on], "c")
        assert torch.equal(c[~torch.from_numpy(on)].view(torch.int16), c0[~torch.from_numpy(on)].view(torch.int16))
        if h is not None:
            close(f64(h)[on], rh[on], (self.K * U * hsize)[on], "h")

    def check_grad(self, dx, da, db, h, dx0):
        dy, x, a, b, ids, scale = self.host(self.dy)
        on = ids >= 0
        hh = np.where(on[:, None], f64(h), 0)
        rdx, rda, rdb = oblock.lora_backward(dy, x, a, b, ids, hh, scale, self.div)
        m = np.abs
        sdx, sda, sdb = oblock.lora_backward(m(dy), m(x), m(a), m(b), ids, m(hh), None if scale is None else m(scale), self.div)
        n = max(np.bincount(ids[on], minlength=1).max(initial=0), 1)
        if dx is not None:
            ref = np.where(on[:, None], np.nan_to_num(f64(dx0)), 0) + rdx
            tol = ((self.N + self.R + 4) * U + SPLIT) * sdx
            close(f64(dx)[on], ref[on], (tol + 2.0 ** -8 * (m(ref) + tol))[on], "dx")
            off = torch.from_numpy(~on)
            assert torch.equal(dx[off].view(torch.int16), dx0[off].view(torch.int16))
        if da is not None:
            close(f64(da), rda, ((n + self.N + 4) * U + SPLIT) * sda, "da")
            close(f64(db), rdb, ((n + 4) * U + SPLIT) * sdb, "db")

    def run(self):
        moe = _moe()
        c = self.c.clone()
        out, h = moe.moe_lora(c, *self.args(), scale=self.scale, row_div=self.div, keep_h=True)
        assert out is c
        self.check(c, h, self.c)
        again = moe.moe_lora(self.c.clone(), *self.args(), scale=self.scale, row_div=self.div)
        assert torch.equal(again.view(torch.int16), c.view(torch.int16))
        dx = self.dx.clone()
        h[(self.ids < 0).cuda()] = float("nan")
        da, db = moe.moe_lora_backward(self.dy, *self.args(), h, scale=self.scale, row_div=self.div, dx=dx)
        self.check_grad(dx, da, db, h, self.dx)
        return c, h, dx, da, db


# ranks of every padded size and between; widths that end inside a step, a
# chunk and a tile; one slot; shared rows; every block size
SHAPES = [
    # S, G, R, K, N, div, bm
    (1, 1, 8, 8, 8, 1, 16), (1, 3, 16, 2048, 1856, 1, 8), (3, 2, 128, 40, 24, 2, 64), (7, 7, 16, 2688, 1856, 1, 16),
    (28, 16, 16, 2048, 1856, 1, 16), (28, 5, 64, 256, 520, 2, 8), (17, 1, 8, 264, 72, 1, 32), (64, 64, 24, 136, 264, 8, 16),
    (100, 3, 24, 264, 328, 4, 64), (333, 4, 32, 2880, 1000, 1, 64), (65, 1, 40, 72, 136, 1, 32), (200, 2, 128, 1032, 776, 1, 64),
    (129, 3, 96, 512, 248, 3, 32), (700, 1, 8, 512, 64, 7, 64), (600, 5, 56, 328, 8, 2, 16), (50, 1024, 16, 64, 48, 1, 16),
    (150, 2, 64, 1000, 1000, 1, 16), (90, 1, 128, 256, 256, 1, 8), (400, 2, 16, 8, 2056, 1, 64),
]


@pytest.mark.parametrize("S,G,R,K,N,div,bm", SHAPES)
def test_lora(S, G, R, K, N, div, bm):
    Case(S, G, R, K, N, div, bm, seed=R + K).run()


@pytest.mark.parametrize("S,G,R", [(5000, 3, 16), (3000, 200, 8), (1500, 1, 64)])
def test_lora_long_lists(S, G, R):
    """Groups of many blocks: several segments and parts of K and N."""
    Case(S, G, R, 520, 264, 1, None, seed=S, scale=False).run()


@pytest.mark.parametrize("S,G,R,K,N,bm", [(20000, 3, 16, 136, 264, None), (9000, 40, 128, 72, 136, 16),
                                          (6000, 1, 8, 264, 72, 8), (3000, 2, 32, 72, 4104, 16)])
def test_lora_segments_of_several_blocks(S, G, R, K, N, bm):
    """Lists of more blocks than the gradients have segments for."""
    Case(S, G, R, K, N, 2, bm, seed=S + R).run()


def test_lora_without_slots():
    moe = _moe()
    case = Case(0, 3, 16, 64, 48)
    c, h = moe.moe_lora(case.c, *case.args(), keep_h=True)
    assert c.shape == (0, 48) and h.shape == (0, 16)
    da, db = moe.moe_lora_backward(case.dy, *case.args(), h, dx=case.dx)
    assert (da == 0).all() and (db == 0).all()
    # slots, but none in a group
    case = Case(40, 3, 16, 64, 48, free=2.0)
    c, h, dx, da, db = case.run()
    assert (da == 0).all() and (db == 0).all() and torch.isnan(c).all()


def test_lora_strides_and_what_is_left_out():
    moe = _moe()
    case = Case(120, 4, 24, 136, 200, 2, 32, seed=5)
    c, h, dx, da, db = case.run()
    a, b = (torch.cat([t, torch.full_like(t[:, :, :8], float("nan"))], 2)[..., :t.shape[2]] for t in (case.a, case.b))
    assert a.stride(1) == 144 and b.stride(1) == 32
    c2 = strided(case.c, 16)
    ws = torch.full((moe.moe_lora_workspace_bytes(120, 4, 24, 136, 200, 32, case.routing[1].numel()),), 255,
                    dtype=torch.uint8, device="cuda")
    moe.moe_lora(c2, strided(case.x, 8), a, b, case.routing, case.scale, 2, workspace=ws)
    assert torch.equal(c2.contiguous().view(torch.int16), c.view(torch.int16))
    behind = c2.as_strided((119, 16), (216, 1), 200)
    assert torch.isnan(behind).all()
    dx2, out = strided(case.dx, 8), (torch.empty_like(da), torch.empty_like(db))
    ws = torch.full((moe.moe_lora_backward_workspace_bytes(120, 4, 24, 136, 200, 32, case.routing[1].numel()),), 255,
                    dtype=torch.uint8, device="cuda")
    got = moe.moe_lora_backward(strided(case.dy, 24), strided(case.x, 8), a, b, case.routing, h, case.scale, 2, dx=dx2,
                                out=out, workspace=ws)
    assert torch.equal(got[0], da) and torch.equal(got[1], db) and got[0] is out[0]
    assert torch.equal(dx2.contiguous().view(torch.int16), dx.view(torch.int16))
    # only dx; only the weights' gradients
    dx3 = case.dx.clone()
    assert moe.moe_lora_backward(case.dy, *case.args(), None, case.scale, 2, dx=dx3, weights=False) == (None, None)
    assert torch.equal(dx3.view(torch.int16), dx.view(torch.int16))
    got = moe.moe_lora_backward(case.dy, *case.args(), h, case.scale, 2)
    assert torch.equal(got[0], da) and torch.equal(got[1], db)


def test_lora_list_longer_than_needed_and_foreign_ids():
    """Sentinel blocks behind the list, slot ids outside [0, S) and group ids outside [0, G) name nothing."""
    moe = _moe()
    case = Case(60, 3, 16, 64, 48, 1, 16, seed=2)
    c, h, dx, da, db = case.run()
    ids, groups, post = case.routing
    more = torch.full((5 * 16,), 60, dtype=torch.int32, device="cuda")
    more[::2] = -7
    more[1::4] = 2 ** 31 - 1
    tail = torch.tensor([-1, -1, 3, 2 ** 31 - 1, -5], dtype=torch.int32, device="cuda")
    case.routing = torch.cat([ids, more]), torch.cat([groups, tail]), post
    for u, v in zip(case.run(), (c, h, dx, da, db)):
        assert torch.equal(u.nan_to_num(1.0), v.nan_to_num(1.0))


def test_lora_values_that_are_not_finite_stay_in_their_slot_and_group():
    moe = _moe()
    case = Case(90, 3, 16, 64, 72, 1, 16, seed=3, free=0.0)
    clean = case.run()
    s = int((case.ids == 1).nonzero()[0])
    g = 1
    case.x[s, 3] = float("nan")
    c, h = moe.moe_lora(case.c.clone(), *case.args(), scale=case.scale, keep_h=True)
    others = torch.arange(90) != s
    assert torch.equal(c[others], clean[0][others]) and torch.isnan(c[s]).all() and torch.isnan(h[s]).all()
    dx = case.dx.clone()
    da, db = moe.moe_lora_backward(case.dy, *case.args(), h, scale=case.scale, dx=dx)
    keep = [i for i in range(3) if i != g]
    assert torch.equal(da[keep], clean[3][keep]) and torch.equal(db[keep], clean[4][keep])
    assert torch.isnan(da[g, :, 3]).all() and torch.isnan(db[g]).all() and torch.equal(dx, clean[2])
    ok = [i for i in range(64) if i != 3]
    assert torch.equal(da[g][:, ok], clean[3][g][:, ok])
    case.x[s, 3] = float("inf")       # an infinite h: infinities of the sign of scale b
    case.a[g, :, 3] = 1.0
    c = moe.moe_lora(case.c.clone(), *case.args(), scale=case.scale)
    want = torch.sign(case.b[g].float()).sum(1)
    one_sign = want.abs() == 16
    assert torch.isinf(h[s]).sum() == 0 and not torch.isfinite(c[s]).any()
    assert torch.equal(torch.sign(c[s].float())[one_sign], torch.sign(want * case.scale[g])[one_sign])


def test_lora_rows_far_apart():
    """Rows whose offsets pass 2^32 bytes and 2^31 elements."""
    moe = _moe()
    S, K, N, G, R, ld = 4500, 64, 48, 2, 8, (1 << 20) + 8
    case = Case(S, G, R, K, N, 1, 64, seed=9)
    buf = torch.empty(S * ld, dtype=torch.bfloat16, device="cuda")   # 9.4 GB
    far = [buf.as_strided((S, w), (ld, 1), at) for w, at in ((N, 0), (K, 64), (N, 128), (K, 192))]
    for t, v in zip(far, (case.c, case.x, case.dy, case.dx)):
        t.copy_(v)
    c, h, dx, da, db = case.run()
    _, h2 = moe.moe_lora(far[0], far[1], case.a, case.b, case.routing, case.scale, keep_h=True)
    da2, db2 = moe.moe_lora_backward(far[2], far[1], case.a, case.b, case.routing, h2, case.scale, dx=far[3])
    for u, v in ((far[0], c), (far[3], dx), (da2, da), (db2, db)):
        assert torch.equal(u.contiguous().nan_to_num(1.0), v.nan_to_num(1.0))


def test_lora_shares_the_grouped_gemms_routing():
    """One adapter per expert: the GEMM's block list serves both, at its decode and its large block size."""
    moe = _moe()
    for T in (9, 200):
        E, k, K, N, R = 8, 2, 256, 192, 16
        ids = torch.stack([torch.randperm(E, generator=synth.gen(t, "r"))[:k] for t in range(T)]).to(torch.int32).cuda()
        bm = moe.moe_gemm_block_m("bf16", T)
        routing = moe.moe_align(ids, E, bm)
        x, w = normal((T, K), T, "x"), normal((E, N, K), T, "w", std=K ** -0.5)
        case = Case(T * k, E, R, K, N, k, bm, seed=T, free=0.0)
        case.ids, case.routing, case.x = ids.reshape(-1).cpu(), routing, x
        case.c = moe.moe_grouped_gemm(x, w, "bf16", routing, T, k, E, k)
        case.run()


def test_lora_streams_and_replays():
    moe = _moe()
    case = Case(300, 5, 16, 512, 264, 1, None, seed=7)
    side = torch.cuda.Stream()

    def step(c, dx):
        _, h = moe.moe_lora(c, *case.args(), scale=case.scale, keep_h=True)
        da, db = moe.moe_lora_backward(case.dy, *case.args(), h, scale=case.scale, dx=dx)
        return c, dx, da, db

    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = step(case.c.clone(), case.dx.clone())
    side.synchronize()
    eager = step(case.c.clone(), case.dx.clone())
    for u, v in zip(on_side, eager):
        assert torch.equal(u.nan_to_num(1.0), v.nan_to_num(1.0))
    c, dx = case.c.clone(), case.dx.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(c, dx)
    for k in range(4):
        case.x.copy_(normal(tuple(case.x.shape), 40 + k, "x"))
        case.scale.mul_(1.25)
        c.copy_(case.c)
        dx.copy_(case.dx)
        graph.replay()
        torch.cuda.synchronize()
        for u, v in zip(out, step(case.c.clone(), case.dx.clone())):
            assert torch.equal(u.nan_to_num(1.0), v.nan_to_num(1.0))
