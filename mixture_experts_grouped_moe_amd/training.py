"""Python binding of libmoe's training entry points (include/moe_train.h).

The same manner as the rest of the package: the functions have the names of
the C entry points, check shapes, dtypes and devices, and run on the current
stream of their tensors' device (or on `stream`). A whole step of a SwiGLU
layer, with x kept as MXFP8 and the first GEMM's output as a checkpoint:

    ids, w, counts, n, prob_sum, losses = moe_route(logits, top_k, balance=True)
    routing = moe_align(ids, E, moe_gemm_block_m("bf16", T))
    pre = moe_grouped_gemm(x, w1, "bf16", routing, T, k, E, k)
    h, q, s = moe_act_mxfp8(pre, "swiglu")
    c = moe_grouped_gemm(h, w2, "bf16", routing, T, k, E, 1)
    y = moe_combine_routed(c, w, ids, E)

    dc, dw = moe_combine_backward(dy, c, w, ids, E)
    dh = moe_grouped_gemm(dc, w2_t, "bf16", routing, T, k, E, 1)
    dpre, h = moe_act_mxfp8_backward(q, s, dh, "swiglu")
    dw2 = moe_wgrad(h, dc, wgrad_routing, T * k, 1, E)
    dw1 = moe_wgrad_mxfp8(xq, xs, dpre, wgrad_routing, T, k, E)
    dx = moe_combine_routed(moe_grouped_gemm(dpre, w1_t, "bf16", routing, T, k, E, 1), ones, ids, E)
    dlogits = moe_route_backward(logits, ids, dw, counts=counts, num_routed=n, dlosses=dlosses)

(w1_t, w2_t: the weights with their last two dimensions swapped; wgrad_routing
= moe_align at moe_wgrad_block_m(); xq, xs = moe_quantize_mxfp8(x).)
"""

import ctypes
import functools

import torch

from . import _ACTS, _check, _need, lib, MOE_BF16, MOE_FP32

__all__ = [
    "moe_route", "moe_route_workspace_bytes", "moe_route_backward", "moe_combine_routed", "moe_combine_backward",
    "moe_act_mxfp8", "moe_act_mxfp8_backward", "moe_wgrad_mxfp8", "MOE_SCORE_SOFTMAX", "MOE_SCORE_SIGMOID",
]

MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
_SCORES = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}
_LOGITS = {torch.float32: MOE_FP32, torch.bfloat16: MOE_BF16}


def _bind():
    i64, i32, vp, f32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float
    sig = {
        "moe_route_workspace_bytes": (i64, [i64, i32]),
        "moe_route": (i32, [vp, i32, i64, vp, i64, i32, i32, i32, i32, f32, vp, vp, i32, vp, vp, vp, vp, vp, i64, vp]),
        "moe_route_backward": (i32, [vp, i32, i64, i64, i32, i32, i32, i32, f32, vp, vp, vp, vp, vp, vp, i64, vp]),
        "moe_combine_routed": (i32, [vp, i64, vp, vp, i64, i32, i32, i64, vp, i64, vp]),
        "moe_combine_backward": (i32, [vp, i64, vp, i64, vp, vp, i64, i32, i32, i64, vp, i64, vp, vp]),
        "moe_act_mxfp8": (i32, [i32, vp, i64, i64, i64, vp, i64, vp, i64, vp, i64, vp]),
        "moe_act_mxfp8_backward": (i32, [i32, vp, i64, vp, i64, vp, i64, i64, i64, vp, i64, vp, i64, vp]),
        "moe_wgrad_mxfp8": (i32, [vp, i64, vp, i64, vp, i64, vp, vp, vp, i64, i32, i32, i64, i64, i32, i64, vp, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args


_bind()


# Calls on small inputs are bound by the host: launching takes 4.3 us, so what
# the binding adds to it is kept short (a stream object would take 2.8 us,
# torch.empty 0.4 us more than torch.empty_strided).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


@functools.lru_cache(maxsize=None)
def _one_device():
    return torch.cuda.device_count() < 2


def _on_stream(f):
    """Runs f with `stream` (default: the current stream of the first tensor's
    device) and its device current, so that what f allocates belongs to the
    stream that its kernels run on."""
    @functools.wraps(f)
    def call(*args, stream=None, **kw):
        if stream is None and _one_device():
            return f(*args, **kw)
        first = next((a for a in (*args, *kw.values()) if isinstance(a, torch.Tensor)), None)
        on_gpu = first is not None and first.is_cuda
        if stream is None:
            if not on_gpu or first.get_device() == torch.cuda.current_device():
                return f(*args, **kw)
            with torch.cuda.device(first.device):
                return f(*args, **kw)
        if on_gpu and stream.device != first.device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {first.device}")
        with torch.cuda.stream(stream):
            return f(*args, **kw)
    return call


def _stream(t):
    if _raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(t.get_device())


def _same_device(first, *others):
    dev = first.get_device()
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors on {first.device} and {t.device}")


def _new(t, rows, width, dtype):
    """An uninitialised [rows, width] on t's device."""
    return torch.empty_strided((rows, width), (width, 1), dtype=dtype, device=t.device)


def _mat(t, name, dtype, rows=None, width=None):
    """Checks a 2-d device tensor whose rows are contiguous, of at least `rows`
    rows and exactly `width` columns where given; (rows, columns, row stride).
    A single row's stride means nothing: a legal one is returned."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or not t.is_cuda or t.dim() != 2:
        _need(t, name, dtype, 2)
    (r, c), (ld, one) = t.shape, t.stride()
    if one != 1 and r * c:
        _need(t, name, dtype, 2)
    if rows is not None and (r < rows or c != width):
        raise ValueError(f"{name} must be [{rows}, {width}], got {[r, c]}")
    return r, c, ld if r > 1 else -(-c // 16) * 16


def _flat(t, name, dtype, shape):
    """Checks a contiguous device tensor of this shape."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or not t.is_cuda or t.dim() != len(shape):
        _need(t, name, dtype, len(shape))
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {list(shape)}, got {list(t.shape)}")


def _table(t, name, dtype):
    """Checks a contiguous 2-d device tensor; its shape."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or not t.is_cuda or t.dim() != 2:
        _need(t, name, dtype, 2)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.shape


def _logits(t):
    """(T, E, row stride) of the router's logits."""
    if not isinstance(t, torch.Tensor) or t.dtype not in _LOGITS:
        raise TypeError("logits must be a float32 or bfloat16 tensor")
    return _mat(t, "logits", t.dtype)


def moe_route_workspace_bytes(num_tokens, num_experts):
    """Bytes of the workspace that moe_route takes with balance=True."""
    return int(lib.moe_route_workspace_bytes(int(num_tokens), int(num_experts)))


@_on_stream
def moe_route(logits, top_k, score="softmax", renormalize=True, scale=1.0, mask=None, balance=False, out=None,
              workspace=None):
    """The router: each token's top_k experts and their weights, and with
    `balance` the statistics and losses over the routed tokens.

    logits: fp32 or bf16 [T, E] (rows may be strided); score: "softmax" or
    "sigmoid"; renormalize: divide the chosen scores by their sum; scale: a
    factor on the weights; mask: uint8 or bool [T], 0 for padding. A padded
    token, or one whose logits are all -inf, gets ids -1 and weights 0; a
    place that no expert above -inf is left for too.

    Returns (topk_ids int32 [T, top_k], topk_w fp32 [T, top_k]), followed with
    `balance` by (counts int32 [E], num_routed int32 [1], prob_sum fp32 [E],
    losses fp32 [2]): slots per expert, routed tokens, summed probabilities,
    and [balance loss, z loss] as moe_train.h defines them. `out` may give the
    two or six tensors; `workspace` a uint8 tensor of moe_route_workspace_bytes
    (calls that may run at the same time need one each).
    """
    T, E, ld = _logits(logits)
    k, dev = int(top_k), logits.device
    if out is None:
        if not 1 <= k <= E:
            raise ValueError(f"need 1 <= top_k ({k}) <= num_experts ({E})")
        out = (_new(logits, T, k, torch.int32), _new(logits, T, k, torch.float32))
        if balance:
            out += (torch.empty(E, dtype=torch.int32, device=dev), torch.empty(1, dtype=torch.int32, device=dev),
                    torch.empty(E, dtype=torch.float32, device=dev), torch.empty(2, dtype=torch.float32, device=dev))
    else:
        out = tuple(out)
        if len(out) != (6 if balance else 2):
            raise ValueError("out must hold 2 tensors, 6 with balance")
        for t, name, dtype, shape in zip(
                out, ("topk_ids", "topk_w", "counts", "num_routed", "prob_sum", "losses"),
                (torch.int32, torch.float32, torch.int32, torch.int32, torch.float32, torch.float32),
                ((T, k), (T, k), (E,), (1,), (E,), (2,))):
            _flat(t, name, dtype, shape)
        _same_device(logits, *out)
    mask_p = None
    if mask is not None:
        if not isinstance(mask, torch.Tensor) or mask.dtype not in (torch.uint8, torch.bool):
            raise TypeError("mask must be a uint8 or bool tensor")
        _flat(mask, "mask", mask.dtype, (T,))
        _same_device(logits, mask)
        mask_p = mask.data_ptr()
    stats, ws_p, ws_n = (None,) * 4, None, 0
    if balance:
        stats = [t.data_ptr() for t in out[2:]]
        if workspace is None:
            workspace = torch.empty(max(moe_route_workspace_bytes(T, E), 0), dtype=torch.uint8, device=dev)
        else:
            _need(workspace, "workspace", torch.uint8, 1)
            _same_device(logits, workspace)
        ws_p, ws_n = workspace.data_ptr(), workspace.numel()
    _check(lib.moe_route(logits.data_ptr(), _LOGITS[logits.dtype], ld, mask_p, T, E, k, _SCORES[score],
                         bool(renormalize), scale, out[0].data_ptr(), out[1].data_ptr(), bool(balance), *stats, ws_p,
                         ws_n, _stream(logits)))
    return out


@_on_stream
def moe_route_backward(logits, topk_ids, dtopk_w, score="softmax", renormalize=True, scale=1.0, counts=None,
                       num_routed=None, dlosses=None, out=None):
    """The router's gradient: dlogits [T, E] in logits' dtype, from the
    gradient dtopk_w fp32 [T, top_k] of the weights and, when given, dlosses
    fp32 [2] of the losses (with the forward pass's counts and num_routed).
    logits, topk_ids, score, renormalize and scale as in the forward pass;
    the experts chosen there are held constant."""
    T, E, ld = _logits(logits)
    rows, k = _table(topk_ids, "topk_ids", torch.int32)
    if rows != T:
        raise ValueError(f"topk_ids must be [{T}, {k}], got {[rows, k]}")
    _flat(dtopk_w, "dtopk_w", torch.float32, (T, k))
    losses = (None,) * 3
    if dlosses is not None:
        if counts is None or num_routed is None:
            raise ValueError("dlosses needs counts and num_routed")
        _flat(dlosses, "dlosses", torch.float32, (2,))
        _flat(counts, "counts", torch.int32, (E,))
        _flat(num_routed, "num_routed", torch.int32, (1,))
        _same_device(logits, dlosses, counts, num_routed)
        losses = counts.data_ptr(), num_routed.data_ptr(), dlosses.data_ptr()
    if out is None:
        out, old = _new(logits, T, E, logits.dtype), E
    else:
        old = _mat(out, "out", logits.dtype, T, E)[2]
    _same_device(logits, topk_ids, dtopk_w, out)
    _check(lib.moe_route_backward(logits.data_ptr(), _LOGITS[logits.dtype], ld, T, E, k, _SCORES[score],
                                  bool(renormalize), scale, topk_ids.data_ptr(), dtopk_w.data_ptr(), *losses,
                                  out.data_ptr(), old, _stream(logits)))
    return out


@_on_stream
def moe_combine_routed(c, topk_w, topk_ids, num_experts, out=None):
    """moe_combine over the slots whose id lies in [0, num_experts): y[t] =
    sum_j topk_w[t, j] * c[t * top_k + j] (fp32, bf16 out). The other slots'
    rows of c, which the grouped GEMM leaves as they were, are not read."""
    T, k = _table(topk_ids, "topk_ids", torch.int32)
    _flat(topk_w, "topk_w", torch.float32, (T, k))
    rows, N, cld = _mat(c, "c", torch.bfloat16)
    if rows < T * k:
        raise ValueError(f"c must hold {T * k} rows, got {rows}")
    if out is None:
        out, old = _new(c, T, N, torch.bfloat16), N
    else:
        old = _mat(out, "out", torch.bfloat16, T, N)[2]
    _same_device(c, topk_w, topk_ids, out)
    _check(lib.moe_combine_routed(c.data_ptr(), cld, topk_w.data_ptr(), topk_ids.data_ptr(), T, k, int(num_experts),
                                  N, out.data_ptr(), old, _stream(c)))
    return out


@_on_stream
def moe_combine_backward(dy, c, topk_w, topk_ids=None, num_experts=None, out=None):
    """Backward pass of the combine: dC[s] = topk_w[s] * dy[t] (bf16) and
    dtopk_w[s] = dy[t] . c[s] (fp32) for slot s = t * top_k + j.

    dy: bf16 [T, N]; c: bf16 [T * top_k, N] as combined; topk_w: fp32
    [T, top_k]; with topk_ids (int32 [T, top_k]) and num_experts, slots routed
    nowhere get zeros and their rows of c are not read. Returns (dC, dtopk_w);
    `out` may give both (not overlapping the inputs)."""
    T, k = _table(topk_w, "topk_w", torch.float32)
    rows, N, dyld = _mat(dy, "dy", torch.bfloat16)
    if rows < T:
        raise ValueError(f"dy must hold {T} rows, got {rows}")
    cld = _mat(c, "c", torch.bfloat16, T * k, N)[2]
    ids_p, E = None, 0
    if topk_ids is not None:
        if num_experts is None:
            raise ValueError("topk_ids needs num_experts")
        _flat(topk_ids, "topk_ids", torch.int32, (T, k))
        ids_p, E = topk_ids.data_ptr(), int(num_experts)
    if out is None:
        dc, dw, dcld = _new(dy, T * k, N, torch.bfloat16), _new(dy, T, k, torch.float32), N
    else:
        dc, dw = out
        dcld = _mat(dc, "dC", torch.bfloat16, T * k, N)[2]
        _flat(dw, "dtopk_w", torch.float32, (T, k))
    _same_device(dy, c, topk_w, topk_ids, dc, dw)
    _check(lib.moe_combine_backward(dy.data_ptr(), dyld, c.data_ptr(), cld, topk_w.data_ptr(), ids_p, T, k, E, N,
                                    dc.data_ptr(), dcld, dw.data_ptr(), _stream(dy)))
    return dc, dw


@_on_stream
def moe_act_mxfp8(pre, activation, out=None):
    """The expert activation, keeping its input for the backward pass as MXFP8.

    pre: bf16 [R, N], a grouped GEMM's output without epilogue; activation:
    "swiglu" (gate = first half of the columns, up = second; N % 64 == 0) or
    "relu2" (N % 32 == 0). Returns (h, q, scales): h bf16 [R, N / 2] or [R, N];
    q uint8 E4M3 codes [R, N] and scales uint8 E8M0 [R, N / 32], the bits of
    moe_quantize_mxfp8(pre). `out` may give the three."""
    act = _ACTS[activation]
    R, N, pld = _mat(pre, "pre", torch.bfloat16)
    H = N // 2 if act == 1 else N
    if out is None:
        h, hld = _new(pre, R, H, torch.bfloat16), H
        q, qld = _new(pre, R, N, torch.uint8), N
        s, sld = _new(pre, R, N // 32, torch.uint8), N // 32
    else:
        h, q, s = out
        hld = _mat(h, "h", torch.bfloat16, R, H)[2]
        qld = _mat(q, "q", torch.uint8, R, N)[2]
        sld = _mat(s, "scales", torch.uint8, R, N // 32)[2]
        _same_device(pre, h, q, s)
    _check(lib.moe_act_mxfp8(act, pre.data_ptr(), pld, R, N, h.data_ptr(), hld, q.data_ptr(), qld, s.data_ptr(), sld,
                             _stream(pre)))
    return h, q, s


@_on_stream
def moe_act_mxfp8_backward(q, scales, dh, activation, out=None, recompute=True):
    """Gradient of the expert activation from its MXFP8 checkpoint.

    q, scales: as moe_act_mxfp8 gave them; dh: bf16 [R, N / 2] or [R, N].
    Returns (dpre, h): dpre bf16 [R, N], and h bf16 recomputed from the
    checkpoint for the second weights' gradient (None with recompute=False).
    `out` may give both."""
    act = _ACTS[activation]
    R, N, qld = _mat(q, "q", torch.uint8)
    H = N // 2 if act == 1 else N
    sld = _mat(scales, "scales", torch.uint8, R, N // 32)[2]
    dhld = _mat(dh, "dh", torch.bfloat16, R, H)[2]
    if out is None:
        dpre, dld = _new(q, R, N, torch.bfloat16), N
        h, hld = (_new(q, R, H, torch.bfloat16), H) if recompute else (None, 0)
    else:
        dpre, h = out
        dld = _mat(dpre, "dpre", torch.bfloat16, R, N)[2]
        hld = _mat(h, "h", torch.bfloat16, R, H)[2] if h is not None else 0
    _same_device(q, scales, dh, dpre, h)
    _check(lib.moe_act_mxfp8_backward(act, q.data_ptr(), qld, scales.data_ptr(), sld, dh.data_ptr(), dhld, R, N,
                                      dpre.data_ptr(), dld, h.data_ptr() if h is not None else None, hld,
                                      _stream(q)))
    return dpre, h


@_on_stream
def moe_wgrad_mxfp8(xq, xs, grad, routing, num_tokens, top_k, num_experts, out=None):
    """moe_wgrad over MXFP8 activations: dW[e] = sum over slots s routed to e
    of grad[s]^T dec(xq, xs)[s // top_k], fp32 [E, N, K]. xq: uint8 E4M3 codes
    [T, K], xs: uint8 E8M0 [T, K / 32] (moe_quantize_mxfp8); grad, routing and
    out as for moe_wgrad."""
    T, k, E = int(num_tokens), int(top_k), int(num_experts)
    rows, K, xld = _mat(xq, "xq", torch.uint8)
    slots, N, gld = _mat(grad, "grad", torch.bfloat16)
    if rows < T or slots < T * k:
        raise ValueError(f"xq must hold {T} rows and grad {T * k}, got {rows} and {slots}")
    sld = _mat(xs, "xs", torch.uint8, T, K // 32)[2]
    sorted_ids, expert_ids, post_pad = routing
    for t, name in zip(routing, ("sorted_token_ids", "expert_ids", "num_tokens_post_pad")):
        _need(t, name, torch.int32, 1)
    blocks, bm = expert_ids.numel(), lib.moe_wgrad_block_m()
    if sorted_ids.numel() < blocks * bm:
        raise ValueError("routing arrays do not match moe_wgrad_block_m()")
    if out is None:
        if E < 0:
            raise ValueError(f"num_experts ({E}) is negative")
        out = torch.empty((E, N, K), dtype=torch.float32, device=xq.device)
    else:
        _flat(out, "out", torch.float32, (E, N, K))
    _same_device(xq, xs, grad, sorted_ids, expert_ids, post_pad, out)
    _check(lib.moe_wgrad_mxfp8(xq.data_ptr(), xld, xs.data_ptr(), sld, grad.data_ptr(), gld, sorted_ids.data_ptr(),
                               expert_ids.data_ptr(), post_pad.data_ptr(), T, k, E, N, K, bm, blocks, out.data_ptr(),
                               _stream(xq)))
    return out
