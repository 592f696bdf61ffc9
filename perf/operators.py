"""The operators of a mixture-of-experts training step beside the grouped
GEMMs, each as cases to measure: the router with its balance loss (forward and
backward), the backward pass of the top-k combine, the expert activation with
an MXFP8 checkpoint of its input (forward and backward), and the expert weight
gradient over MXFP8 activations.

`own` selects what `run` computes with: plain torch operations in 32 bits
(False) or this package's kernels (True). Both take the same state.

Notation: T tokens, E experts, k experts per token, S = T * k slots
(s = t * k + j), H the hidden width, I the expert width.
"""

import math

import torch

own = False

BLOCK = 32        # elements under one E8M0 scale
WGRAD_BLOCK = 64  # the routing block that the weight gradient reads (moe_wgrad_block_m())


# ------------------------------------------------------------------- cases

def listed():
    return [
        # a decode step of 7 tokens over 128 experts, top 6: the router alone, weights not renormalised
        {"name": "route decode", "op": "route", "T": 7, "E": 128, "k": 6, "dtype": "bf16", "score": "softmax",
         "renorm": False, "balance": False, "padded": False},
        # a training batch over 256 experts, top 8, fp32 logits, with counts and losses, padded rows among it
        {"name": "route train", "op": "route", "T": 65536, "E": 256, "k": 8, "dtype": "fp32", "score": "softmax",
         "renorm": True, "balance": True, "padded": True},
        # an ordinary micro-batch, bf16 logits over 128 experts, top 4
        {"name": "route grad", "op": "route_grad", "T": 6554, "E": 128, "k": 4, "dtype": "bf16", "score": "softmax",
         "renorm": True, "balance": True, "padded": False},
        # the large training batch with sigmoid scores
        {"name": "route grad large", "op": "route_grad", "T": 65536, "E": 256, "k": 8, "dtype": "fp32",
         "score": "sigmoid", "renorm": True, "balance": True, "padded": True},
        # a ragged fine-tuning batch of the 2880-wide layer, top 4
        {"name": "combine grad", "op": "combine_grad", "T": 333, "E": 128, "k": 4, "H": 2880, "padded": False},
        # a training batch of the 7168-wide layer, top 8, with padded rows (their slots are routed nowhere)
        {"name": "combine grad large", "op": "combine_grad", "T": 8192, "E": 256, "k": 8, "H": 7168, "padded": True},
        # the squared-ReLU layer at a decode bucket: 7 tokens, top 6, width 1856
        {"name": "act small", "op": "act", "R": 42, "N": 1856, "act": "relu2"},
        # the SwiGLU layer at 8192 tokens, top 4: gate and up of 2880 each
        {"name": "act large", "op": "act", "R": 32768, "N": 5760, "act": "swiglu"},
        # their backward passes from the checkpoint, the small one an odd row count
        {"name": "act grad", "op": "act_grad", "R": 1333, "N": 1856, "act": "relu2"},
        {"name": "act grad large", "op": "act_grad", "R": 32768, "N": 5760, "act": "swiglu"},
        # the tiny up-projection: 64 tokens, 8 experts, top 2
        {"name": "wgrad small", "op": "wgrad", "T": 64, "E": 8, "k": 2, "N": 512, "K": 256},
        # 64 experts (one rank's share of 256) with 1024 slots each on average
        {"name": "wgrad large", "op": "wgrad", "T": 8192, "E": 64, "k": 8, "N": 2048, "K": 7168},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "combine_grad", "act", "act_grad", "wgrad"])
    if op in ("route", "route_grad"):
        E = _log_int(rng, 8, 512)
        T = _log_int(rng, 1, min(65536, 65536 * 256 // E))
        return {"op": op, "T": T, "E": E, "k": rng.randint(1, min(10, E)), "dtype": rng.choice(["bf16", "fp32"]),
                "score": rng.choice(["softmax", "sigmoid"]), "renorm": rng.random() < 0.5,
                "balance": op == "route_grad" or T > 32, "padded": T > 32 and rng.random() < 0.5}
    if op == "combine_grad":
        H = 8 * _log_int(rng, 32, 896)
        k = rng.randint(1, 10)
        T = _log_int(rng, 1, 8192 * 8 * 7168 // (k * H))
        return {"op": op, "T": T, "E": 128, "k": k, "H": H, "padded": T > 32 and rng.random() < 0.5}
    if op in ("act", "act_grad"):
        act = rng.choice(["swiglu", "relu2"])
        N = 64 * _log_int(rng, 4, 90) if act == "swiglu" else 32 * _log_int(rng, 8, 90)
        return {"op": op, "R": _log_int(rng, 1, 32768 * 2880 // N), "N": N, "act": act}
    E = _log_int(rng, 4, 64)
    N, K = 32 * _log_int(rng, 4, 64), 32 * _log_int(rng, 4, 224)
    k = rng.randint(1, min(8, E))
    return {"op": op, "T": _log_int(rng, 1, 65536 // k), "E": E, "k": k, "N": N, "K": K}


# ------------------------------------------------------------------ inputs

def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _pads(g, T):
    """A token mask with about one padded row in eight."""
    return (torch.rand(T, generator=g, device="cuda") >= 0.125).to(torch.uint8)


def _routing(g, T, E, k):
    """Distinct experts per token, some experts more popular than others."""
    u = _normal(g, T, E) + 0.15 * _normal(g, E)
    return torch.sort(u, dim=1, descending=True, stable=True).indices[:, :k].to(torch.int32).contiguous()


def _checkpoint(v):
    """The MXFP8 checkpoint of float32 rows, as bytes: E4M3 codes and E8M0 scales."""
    codes, scales = _quantize(v)
    return codes.view(torch.uint8), scales.view(torch.uint8)


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    op = c["op"]
    if op in ("route", "route_grad"):
        T, E, k = c["T"], c["E"], c["k"]
        z = 1.5 * _normal(g, T, E) + 0.5 * _normal(g, E)
        c["logits"] = z.to(torch.bfloat16) if c["dtype"] == "bf16" else z
        c["mask"] = _pads(g, T) if c["padded"] else None
        c["scale"] = 1.0 if c["score"] == "softmax" else 2.5
        if op == "route_grad":  # what the forward pass left: ids, counts, the number of routed tokens
            f = _route(c["logits"], k, c["score"], c["renorm"], c["scale"], c["mask"])
            c["ids"], c["counts"], c["routed"] = f[0].contiguous(), f[2], f[3]
            c["dw"] = _normal(g, T, k) / T
            c["dlosses"] = torch.tensor([1e-2, 1e-3], device="cuda")
    elif op == "combine_grad":
        T, k, H = c["T"], c["k"], c["H"]
        c["dy"] = _normal(g, T, H).to(torch.bfloat16)
        c["c"] = _normal(g, T * k, H).to(torch.bfloat16)
        ids = _routing(g, T, c["E"], k)
        if c["padded"]:
            ids = torch.where(_pads(g, T)[:, None] != 0, ids, -1).contiguous()
        c["ids"] = ids
        c["w"] = torch.softmax(_normal(g, T, k), dim=1)
    elif op == "act":
        c["pre"] = (1.5 * _normal(g, c["R"], c["N"])).to(torch.bfloat16)
    elif op == "act_grad":
        R, N = c["R"], c["N"]
        c["q"], c["s"] = _checkpoint((1.5 * _normal(g, R, N)).to(torch.bfloat16).float())
        c["dh"] = (0.01 * _normal(g, R, N // 2 if c["act"] == "swiglu" else N)).to(torch.bfloat16)
    else:
        T, E, k, N, K = c["T"], c["E"], c["k"], c["N"], c["K"]
        c["xq"], c["xs"] = _checkpoint(_normal(g, T, K).to(torch.bfloat16).float())
        c["grad"] = (0.01 * _normal(g, T * k, N)).to(torch.bfloat16)
        ids = c["ids"] = _routing(g, T, E, k)
        # the routing that the forward pass used: each expert's slots in
        # ascending order, padded to whole blocks with S; the block's experts
        S, B = T * k, WGRAD_BLOCK
        flat = ids.reshape(-1).long()
        order = torch.sort(flat, stable=True).indices
        counts = torch.bincount(flat, minlength=E)
        blocks = (counts + B - 1) // B
        first = (torch.cumsum(blocks, 0) - blocks) * B - (torch.cumsum(counts, 0) - counts)
        most = (S + min(S, E) * (B - 1)) // B
        ids_sorted = torch.full((most * B,), S, dtype=torch.int32, device="cuda")
        ids_sorted[torch.arange(S, device="cuda") + first[flat[order]]] = order.to(torch.int32)
        experts = torch.full((most,), -1, dtype=torch.int32, device="cuda")
        used = torch.repeat_interleave(torch.arange(E, device="cuda"), blocks)
        experts[:used.numel()] = used.to(torch.int32)
        c["routing"] = (ids_sorted, experts, (blocks.sum() * B).to(torch.int32).reshape(1))
        c["cap"] = int(counts.max())  # slots of the fullest expert
    return c


# ------------------------------------------------------------- plain forms

def _log_scores(z, score):
    """a with softmax(a) the router's probabilities: the logits, or log sigmoid of them."""
    return z if score == "softmax" else torch.clamp(z, max=0) - torch.log1p(torch.exp(-z.abs()))


def _probs(a):
    m = a.amax(1, keepdim=True)
    e = torch.exp(a - m)
    s = e.sum(1, keepdim=True)
    return e / s, (m + torch.log(s)).squeeze(1)


def _chosen_weights(z, a, q, ids, score, renorm):
    """The weights of the chosen experts before the routed scale."""
    if renorm:
        v = a.gather(1, ids)
        e = torch.exp(v - v.amax(1, keepdim=True))
        return e / e.sum(1, keepdim=True)
    return q.gather(1, ids) if score == "softmax" else 1 / (1 + torch.exp(-z.gather(1, ids)))


def _route(logits, k, score, renorm, scale, mask):
    z = logits.float()
    T, E = z.shape
    live = torch.ones(T, dtype=torch.bool, device=z.device) if mask is None else mask != 0
    ids = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]  # ties: lowest expert first
    a = _log_scores(z, score)
    q, lse = _probs(a)
    w = torch.where(live[:, None], scale * _chosen_weights(z, a, q, ids, score, renorm), 0)
    counts = torch.zeros(E, dtype=torch.int32, device=z.device)
    counts.scatter_add_(0, ids.reshape(-1), live[:, None].expand(T, k).reshape(-1).to(torch.int32))
    n = live.sum(dtype=torch.int32).reshape(1)
    prob = torch.where(live[:, None], q, 0).sum(0, dtype=torch.float64)
    nd = n.double().clamp(min=1)
    balance = E * (counts.double() * prob).sum() / (k * nd * nd)
    z2 = torch.where(live, lse * lse, 0).sum(dtype=torch.float64) / nd if score == "softmax" else torch.zeros_like(nd)
    losses = torch.cat([balance.reshape(1), z2.reshape(1)]).float()
    return torch.where(live[:, None], ids, -1).to(torch.int32), w, counts, n, prob.float(), losses


def _route_grad(logits, ids, dw, counts, n, dlosses, score, renorm, scale):
    z = logits.float()
    T, E = z.shape
    k = ids.shape[1]
    live = (ids[:, :1] >= 0)
    ix = ids.long().clamp(min=0)
    a = _log_scores(z, score)
    q, lse = _probs(a)
    w = _chosen_weights(z, a, q, ix, score, renorm)
    g = scale * dw
    nf = n.float().clamp(min=1)
    cost = dlosses[0] * E / (k * nf * nf) * counts.float()
    common = cost - (q * cost).sum(1, keepdim=True)
    if score == "softmax":
        common = common + (dlosses[1] * 2 / nf) * lse[:, None]
    if renorm:
        u = w * (g - (g * w).sum(1, keepdim=True))
    else:
        u = w * g
        if score == "softmax":
            common = common - u.sum(1, keepdim=True)
    da = (q * common).scatter_add(1, ix, u)
    dz = da if score == "softmax" else da / (1 + torch.exp(z))
    return torch.where(live, dz, 0).to(logits.dtype)


def _quantize(v):
    """float32 rows -> (E4M3 values, E8M0 values) with one scale per 32: the
    shared exponent is that of the block's largest magnitude less 8."""
    R, N = v.shape
    b = v.reshape(R, N // BLOCK, BLOCK)
    top = b.abs().amax(2)
    x = torch.where(top > 0, torch.frexp(top).exponent - 9, -127).clamp(-127, 127)
    scaled = torch.ldexp(b, -x[:, :, None]).clamp(-448, 448)
    return scaled.to(torch.float8_e4m3fn).reshape(R, N), (x + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _dequantize(q, s):
    R, N = q.shape
    v = q.view(torch.float8_e4m3fn).float().reshape(R, N // BLOCK, BLOCK)
    return torch.ldexp(v, s.int()[:, :, None] - 127).reshape(R, N)


def _act(v, act):
    if act == "relu2":
        return v.clamp(min=0).square()
    g, u = v.chunk(2, dim=1)
    return g / (1 + torch.exp(-g)) * u


def _act_grad(v, dh, act):
    dh = dh.float()
    if act == "relu2":
        return 2 * v.clamp(min=0) * dh
    g, u = v.chunk(2, dim=1)
    sig = 1 / (1 + torch.exp(-g))
    return torch.cat([dh * u * sig * (1 + g * (1 - sig)), dh * g * sig], dim=1)


def _wgrad(x, grad, ids, E, cap):
    """dW[e] = sum of grad[s]^T x[s // k] over e's slots, as one batched
    product over each expert's slots padded to the fullest one's."""
    T, k = ids.shape
    flat = ids.reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E)
    place = (torch.cumsum(counts, 0) - counts)[:, None] + torch.arange(cap, device=ids.device)
    live = (torch.arange(cap, device=ids.device) < counts[:, None])[:, :, None]
    slots = order[place.clamp(max=T * k - 1)]
    left = torch.where(live, grad[slots].float(), 0).transpose(1, 2).contiguous()
    return torch.bmm(left, x[slots // k])


def run(state):
    c, op = state, state["op"]
    if own:
        import mixture_experts_grouped_moe_amd as moe
    if op == "route":
        if own:
            return moe.moe_route(c["logits"], c["k"], score=c["score"], renormalize=c["renorm"], scale=c["scale"],
                                 mask=c["mask"], balance=c["balance"])
        return _route(c["logits"], c["k"], c["score"], c["renorm"], c["scale"], c["mask"])[:6 if c["balance"] else 2]
    if op == "route_grad":
        if own:
            return moe.moe_route_backward(c["logits"], c["ids"], c["dw"], score=c["score"], renormalize=c["renorm"],
                                          scale=c["scale"], counts=c["counts"], num_routed=c["routed"],
                                          dlosses=c["dlosses"])
        return _route_grad(c["logits"], c["ids"], c["dw"], c["counts"], c["routed"], c["dlosses"], c["score"],
                           c["renorm"], c["scale"])
    if op == "combine_grad":
        if own:
            return moe.moe_combine_backward(c["dy"], c["c"], c["w"], topk_ids=c["ids"], num_experts=c["E"])
        T, k = c["w"].shape
        dy, live = c["dy"].float()[:, None, :], (c["ids"] >= 0)
        dc = torch.where(live[:, :, None], c["w"][:, :, None] * dy, 0)
        dw = torch.where(live, (c["c"].float().reshape(T, k, -1) * dy).sum(2), 0)
        return dc.to(torch.bfloat16).reshape(T * k, -1), dw
    if op == "act":
        if own:
            h, q, s = moe.moe_act_mxfp8(c["pre"], c["act"])
            return h, q.view(torch.float8_e4m3fn), s.view(torch.float8_e8m0fnu)
        v = c["pre"].float()
        return (_act(v, c["act"]).to(torch.bfloat16),) + _quantize(v)
    if op == "act_grad":
        if own:
            return moe.moe_act_mxfp8_backward(c["q"], c["s"], c["dh"], c["act"])
        v = _dequantize(c["q"], c["s"])
        return _act_grad(v, c["dh"], c["act"]).to(torch.bfloat16), _act(v, c["act"]).to(torch.bfloat16)
    if own:
        return moe.moe_wgrad_mxfp8(c["xq"], c["xs"], c["grad"], c["routing"], c["T"], c["k"], c["E"])
    return _wgrad(_dequantize(c["xq"], c["xs"]), c["grad"], c["ids"], c["E"], c["cap"])


def work(case):
    c, op = case, case["op"]
    if op in ("route", "route_grad"):
        T, E, k = c["T"], c["E"], c["k"]
        logits = T * E * (2 if c["dtype"] == "bf16" else 4)
        mask = T if c["padded"] else 0
        if op == "route":  # logits in; ids, weights and the expert sums out
            return {"bytes": logits + mask + 8 * T * k + (8 * E + 12 if c["balance"] else 0), "flops": 4 * T * E}
        return {"bytes": 2 * logits + 8 * T * k + 4 * E + 12, "flops": 8 * T * E}
    if op == "combine_grad":  # dy, C, ids and weights in; dC and dw out
        T, k, H = c["T"], c["k"], c["H"]
        return {"bytes": 2 * T * H + 4 * T * k * H + 12 * T * k, "flops": 3 * T * k * H}
    if op in ("act", "act_grad"):
        R, N = c["R"], c["N"]
        held, out = R * N + R * N // BLOCK, R * (N // 2 if c["act"] == "swiglu" else N)
        # forward: bf16 in; h and the checkpoint out. Backward: the checkpoint and dh in; dpre and h out
        return {"bytes": held + (2 * R * N + 2 * out if op == "act" else 2 * out + 2 * R * N + 2 * out),
                "flops": (6 if op == "act" else 12) * out}
    T, E, k, N, K = c["T"], c["E"], c["k"], c["N"], c["K"]
    S = T * k
    return {"bytes": T * K + T * K // BLOCK + 2 * S * N + 4 * S + 4 * E * N * K, "flops": 2 * S * N * K}


# ------------------------------------------- the definitions, in 64 bits

def _exact_scores(z, score):
    """(log of the unnormalised score, the score itself) in 64 bits."""
    if score == "softmax":
        return z, torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
    s = torch.sigmoid(z)
    return torch.log(s), s


def _exact_router(z, picked, live, k, score, renorm, scale):
    """The weights of the picked experts and both losses, differentiable in z."""
    T, E = z.shape
    _, s = _exact_scores(z, score)
    p = s / s.sum(1, keepdim=True)
    chosen = torch.take_along_dim(s, picked, 1)
    w = scale * (chosen / chosen.sum(1, keepdim=True) if renorm else chosen) * live[:, None]
    n = max(int(live.sum()), 1)
    f = torch.bincount(picked[live].reshape(-1), minlength=E).double() / (n * k)
    share = p[live].sum(0)
    z2 = torch.logsumexp(z[live], 1).pow(2).sum() / n if score == "softmax" else z.sum() * 0
    return w, f, share, torch.stack([E * (f * share / n).sum(), z2])


def _exact_checkpoint(v):
    """The nearest E4M3 multiple of the block's scale, ties to even, and the scale."""
    R, N = v.shape
    b = v.reshape(R, -1, BLOCK)
    top = b.abs().amax(2)
    e = torch.where(top > 0, torch.floor(torch.log2(top)) - 8, torch.full_like(top, -127)).clamp(-127, 127)
    r = b * torch.exp2(-e)[:, :, None]
    step = torch.exp2(torch.floor(torch.log2(r.abs().clamp(min=2.0 ** -6))) - 3)  # spacing of E4M3 at |r|
    return (torch.round(r / step) * step).clamp(-448, 448).reshape(R, N), torch.exp2(e)


def _exact_decode(codes, scales):
    """E4M3 bytes (1 sign, 4 exponent, 3 mantissa bits, bias 7) times 2^(scale - 127)."""
    b = codes.long()
    e, m = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e > 0, (1 + m / 8) * torch.exp2((e - 7).double()), m / 8 * 2.0 ** -6)
    v = torch.where(b >= 128, -mag, mag)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(BLOCK, 1)


def _exact_activation(v, act):
    if act == "relu2":
        return torch.relu(v) ** 2
    half = v.shape[1] // 2
    return v[:, :half] * torch.sigmoid(v[:, :half]) * v[:, half:]


def exact(case, seed):
    c = prepare(case, seed)
    op = c["op"]
    if op in ("route", "route_grad"):
        z = c["logits"].double()
        T, E = z.shape
        k = c["k"]
        live = torch.ones(T, dtype=torch.bool, device=z.device) if c["mask"] is None else c["mask"] == 1
        picked = torch.argsort(-z, dim=1, stable=True)[:, :k]
        z.requires_grad_(op == "route_grad")
        w, f, share, losses = _exact_router(z, picked, live, k, c["score"], c["renorm"], c["scale"])
        if op == "route_grad":
            ((w * c["dw"].double()).sum() + (losses * c["dlosses"].double()).sum()).backward()
            return z.grad
        ids = torch.where(live[:, None], picked, -1).to(torch.int32)
        n = live.sum()
        counts = torch.round(f * n * k).to(torch.int32)
        return (ids, w, counts, n.to(torch.int32).reshape(1), share, losses)[:6 if c["balance"] else 2]
    if op == "combine_grad":
        T, k = c["w"].shape
        out = c["c"].double().reshape(T, k, -1).requires_grad_()
        w = c["w"].double().requires_grad_()
        routed = (c["ids"] >= 0).double()[:, :, None]
        torch.autograd.backward((w[:, :, None] * out * routed).sum(1), c["dy"].double())
        return out.grad.reshape(T * k, -1), w.grad
    if op == "act":
        v = c["pre"].double()
        return (_exact_activation(v, c["act"]),) + _exact_checkpoint(v)
    if op == "act_grad":
        v = _exact_decode(c["q"], c["s"]).requires_grad_()
        h = _exact_activation(v, c["act"])
        h.backward(c["dh"].double())
        return v.grad, h.detach()
    x, grad, flat = _exact_decode(c["xq"], c["xs"]), c["grad"], c["ids"].reshape(-1)
    dw = torch.empty((c["E"], c["N"], c["K"]), dtype=torch.float64, device=x.device)
    for e in range(c["E"]):
        slots = torch.nonzero(flat == e).reshape(-1)
        torch.matmul(grad[slots].double().t().contiguous(), x[slots // c["k"]], out=dw[e])
    return dw
