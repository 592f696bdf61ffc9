"""GPU tests of the block operators together: a fine-tuning step of a layer
with adapters, norm, residual and dropout against float64 autograd, and the
layers with adapters.

The step's tensors are stored in bf16 (half a step, 2^-8 of a value) about
eight times between an input and a gradient, and the operators between are
linear maps by random matrices, which keep the relative size of an error to a
small factor: outputs are held to 8 * 2^-8 * 2 = 2^-4 of their norm. What a
mistake in the wiring does (a missing term, factor, mask or transpose) is of the
order of the norm itself.
"""

import numpy as np
import pytest
import torch

import synth
from block_helpers import f64, normal, rng_state
from helpers import bf16_to_f64, need_gpu
from oracle import block as oblock
from oracle import quant

pytestmark = pytest.mark.gpu

T, H, INNER, E, K, R = 96, 256, 192, 8, 2, 16
P1, P2, EPS = 0.2, 0.1, 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def _moe():
    import mixture_experts_grouped_moe_amd as moe
    return moe


def inputs():
    d = {"x": normal((T, H), 1, "x"), "res": normal((T, H), 1, "res", "fp32", 2.0),
         "norm": (1 + 0.3 * normal((H,), 1, "norm", "fp32")),
         "w1": normal((E, 2 * INNER, H), 1, "w1", std=H ** -0.5), "w2": normal((E, H, INNER), 1, "w2", std=INNER ** -0.5),
         "a1": normal((E, R, H), 1, "a1", std=H ** -0.5), "b1": normal((E, 2 * INNER, R), 1, "b1", std=0.2),
         "a2": normal((E, R, INNER), 1, "a2", std=INNER ** -0.5), "b2": normal((E, H, R), 1, "b2", std=0.2),
         "scale": 0.5 + torch.rand(E, generator=synth.gen(1, "s")).cuda(),
         "logits": normal((T, E), 1, "z", "fp32"), "dout": normal((T, H), 1, "dout"),
         "dnext": normal((T, H), 1, "dnext", "fp32"), "rng": rng_state(3, 5), "rng2": rng_state(4, 6)}
    d["w1_t"], d["w2_t"] = (d[n].transpose(1, 2).contiguous() for n in ("w1", "w2"))
    return d


def step(d):
    """Forward and backward of one block; the frozen weights have adapters."""
    moe = _moe()
    y, v, _, _ = moe.moe_rmsnorm(d["x"], d["norm"], d["res"], eps=EPS, p=P1, rng=d["rng"])
    ids, w = moe.moe_route(d["logits"], K)
    routing = moe.moe_align(ids, E, moe.moe_gemm_block_m("bf16", T))
    pre = moe.moe_grouped_gemm(y, d["w1"], "bf16", routing, T, K, E, K)
    yd = moe.moe_dropout(y, P2, d["rng2"])
    pre, h1 = moe.moe_lora(pre, yd, d["a1"], d["b1"], routing, d["scale"], row_div=K, keep_h=True)
    h, q, s = moe.moe_act_mxfp8(pre, "swiglu")
    c = moe.moe_grouped_gemm(h, d["w2"], "bf16", routing, T, K, E, 1)
    c, h2 = moe.moe_lora(c, h, d["a2"], d["b2"], routing, d["scale"], keep_h=True)
    out = moe.moe_combine_routed(c, w, ids, E)

    dc, _ = moe.moe_combine_backward(d["dout"], c, w, ids, E)
    dh = moe.moe_grouped_gemm(dc, d["w2_t"], "bf16", routing, T, K, E, 1)
    da2, db2 = moe.moe_lora_backward(dc, h, d["a2"], d["b2"], routing, h2, d["scale"], dx=dh)
    dpre, _ = moe.moe_act_mxfp8_backward(q, s, dh, "swiglu")
    dyd = torch.zeros((T * K, H), dtype=torch.bfloat16, device="cuda")
    da1, db1 = moe.moe_lora_backward(dpre, yd, d["a1"], d["b1"], routing, h1, d["scale"], row_div=K, dx=dyd)
    ones = torch.ones_like(w)
    dy = moe.moe_combine_routed(moe.moe_grouped_gemm(dpre, d["w1_t"], "bf16", routing, T, K, E, 1), ones, ids, E)
    dy = dy + moe.moe_dropout(moe.moe_combine_routed(dyd, ones, ids, E), P2, d["rng2"])
    dx, dres, dnorm = moe.moe_rmsnorm_backward(dy, v, d["norm"], dsum=d["dnext"], eps=EPS, p=P1, rng=d["rng"])
    return {"out": out, "v": v, "dx": dx, "dres": dres, "dnorm": dnorm, "da1": da1, "db1": db1, "da2": da2, "db2": db2}, \
        (ids, w, q, s)


class _Act(torch.autograd.Function):
    """SwiGLU whose derivative is taken at the checkpoint's values."""

    @staticmethod
    def forward(ctx, pre, kept):
        ctx.save_for_backward(kept)
        g, u = pre.chunk(2, 1)
        return g * torch.sigmoid(g) * u

    @staticmethod
    def backward(ctx, dh):
        g, u = ctx.saved_tensors[0].chunk(2, 1)
        s = torch.sigmoid(g)
        return torch.cat([dh * u * s * (1 + g * (1 - s)), dh * g * s], 1), None


def reference(d, ids, w, q, s):
    t = {k: torch.from_numpy(f64(v)) for k, v in d.items() if k not in ("rng", "rng2")}
    leaves = {k: t[k].requires_grad_() for k in ("x", "res", "norm", "a1", "b1", "a2", "b2")}
    ids, w = ids.cpu().long(), torch.from_numpy(f64(w))
    kept = torch.from_numpy(quant.mx_dequantize_e4m3(q.cpu().numpy(), s.cpu().numpy()))

    def drop(x, p, seed, offset):
        keep = torch.from_numpy(oblock.dropout_keep(T, H, p, seed, offset))
        return x * keep * (65536 / (65536 - oblock.dropout_threshold(p)))

    def lora(x, a, b):  # x by slot
        e = ids.reshape(-1)
        return t["scale"][e][:, None] * torch.stack([t[b][g] @ (t[a][g] @ r) for g, r in zip(e, x)])

    v = t["res"] + drop(t["x"], P1, 3, 5)
    y = v / torch.sqrt((v * v).mean(1, keepdim=True) + EPS) * t["norm"]
    slots = torch.arange(T * K) // K
    e = ids.reshape(-1)
    pre = torch.stack([t["w1"][g] @ r for g, r in zip(e, y[slots])]) + lora(drop(y, P2, 4, 6)[slots], "a1", "b1")
    h = _Act.apply(pre, kept)
    c = torch.stack([t["w2"][g] @ r for g, r in zip(e, h)]) + lora(h, "a2", "b2")
    out = (w[:, :, None] * c.reshape(T, K, H)).sum(1)
    ((out * t["dout"]).sum() + (v * t["dnext"]).sum()).backward()
    g = {k: v.grad.numpy() for k, v in leaves.items()}
    return {"out": out.detach().numpy(), "v": v.detach().numpy(), "dx": g["x"], "dres": g["res"], "dnorm": g["norm"],
            "da1": g["a1"], "db1": g["b1"], "da2": g["a2"], "db2": g["b2"]}


def test_fine_tuning_step():
    d = inputs()
    got, routed = step(d)
    ref = reference(d, *routed)
    for name, r in ref.items():
        off = np.linalg.norm(f64(got[name]) - r) / np.linalg.norm(r)
        assert off < 2.0 ** -4, (name, off)
    # dropped elements pass no gradient, kept ones the residual's
    keep = oblock.dropout_keep(T, H, P1, 3, 5)
    assert np.array_equal(f64(got["dx"]) != 0, keep)


def test_fine_tuning_step_captured_and_replayed():
    d = inputs()
    step(d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = step(d)
    for k in range(3):
        d["x"].copy_(normal((T, H), 10 + k, "x"))
        d["logits"].copy_(normal((T, E), 10 + k, "z", "fp32"))
        d["b1"].mul_(1.5)
        d["rng"].add_(1)
        graph.replay()
        torch.cuda.synchronize()
        want, _ = step(d)
        for name, t in want.items():
            assert torch.equal(out[name], t), name


@pytest.mark.parametrize("tokens", [9, 150])
def test_layers_with_adapters(tokens):
    moe = _moe()
    d = synth.config3(160, seed=5, bias=True, device="cuda", E=8, H=256, I=192)
    n, k = tokens, d["ids"].shape[1]
    x, ids, w = (d[t][:n].contiguous() for t in ("x", "ids", "topk_w"))
    a, b = normal((8, R, 192), 2, "a", std=192 ** -0.5), normal((8, 256, R), 2, "b", std=0.1)
    scale = torch.rand(8, generator=synth.gen(2, "s")).cuda()
    args = (x, ids, w, d["w1"], d["s1"], d["w2"], d["s2"])
    y = moe.moe_w4a16_layer(*args, b1=d["b1"], b2=d["b2"], adapter=(a, b, scale))
    routing = moe.moe_align(ids, 8, moe.moe_gemm_block_m("e2m1x2", n))
    h = moe.moe_grouped_gemm(x, d["w1"], "e2m1x2", routing, n, k, 8, k, w_scale=d["s1"], bias=d["b1"], epilogue="swiglu")
    c = moe.moe_grouped_gemm(h, d["w2"], "e2m1x2", routing, n, k, 8, 1, w_scale=d["s2"], bias=d["b2"])
    base = moe.moe_combine(c, w, k)
    assert torch.equal(moe.moe_w4a16_layer(*args, b1=d["b1"], b2=d["b2"]), base)
    delta = oblock.lora(np.zeros((n * k, 256)), bf16_to_f64(h), f64(a), f64(b), ids.cpu().numpy().reshape(-1), f64(scale))[0]
    want = (f64(w)[:, :, None] * (bf16_to_f64(c) + delta).reshape(n, k, -1)).sum(1)
    # C and y each rounded once, by half a step of bf16
    size = (np.abs(f64(w))[:, :, None] * np.abs(bf16_to_f64(c) + delta).reshape(n, k, -1)).sum(1)
    assert (np.abs(bf16_to_f64(y) - want) <= 2.0 ** -8 * (size + np.abs(want)) * 1.01 + 2.0 ** -14 * size.max()).all()
    # the squared-ReLU layer: no adapter gives the layer's bits, an adapter of zeros too
    w1, w2 = normal((8, 192, 256), 3, "w1", std=1 / 16), normal((8, 256, 192), 3, "w2", std=1 / 14)
    plain = moe.moe_relu2_layer(x, ids, w, w1, w2)
    assert torch.equal(moe.moe_relu2_layer(x, ids, w, w1, w2, adapter=(a, torch.zeros_like(b), None)), plain)
    assert not torch.equal(moe.moe_relu2_layer(x, ids, w, w1, w2, adapter=(a, b, scale)), plain)


def test_steps_side_by_side():
    # two steps on two streams at once, and their graphs replayed at once, each
    # with the workspaces that it allocated: the bits of one after the other
    ds = [inputs(), inputs()]
    ds[1]["x"] = normal((T, H), 21, "x")
    ds[1]["logits"] = normal((T, E), 21, "z", "fp32")
    want = [step(d)[0] for d in ds]
    streams, graphs, kept = [torch.cuda.Stream() for _ in ds], [], []
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = step(ds[i])[0]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(g[n], w[n]) for n in w)
    for d in ds:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            kept.append(step(d)[0])
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for g, w in zip(kept, want):
            assert all(torch.equal(g[n], w[n]) for n in w)
            for n in w:
                g[n].zero_()
