"""Python binding of libmoe's block entry points (include/moe_block.h): what
stands around an expert layer.

The same manner as the rest of the package. A block whose expert GEMMs read
MXFP8 activations, with dropout of the layer's output:

    y, r, q, s = moe_rmsnorm(x, weight, residual, p=p, rng=rng, quant="mxfp8")
    ... y to the router, q and s to moe_grouped_gemm(a_scale=s), r the next block's residual ...

    dx, dres, dweight = moe_rmsnorm_backward(dy, r, weight, dsum=dr, p=p, rng=rng)

Adapters of many requests beside a projection, one block list for all
projections of the batch (group = adapter; or adapter * E + expert; up to 1024
groups a list):

    routing = moe_align(adapter_of_slot, G, moe_lora_block_m(S, G))
    c = moe_grouped_gemm(...)                                  # or any shared projection
    c, h = moe_lora(c, x, a, b, routing, scale, keep_h=True)   # c += scale B (A x)

    dx = moe_grouped_gemm(dc, ...)                             # the projection's gradient
    da, db = moe_lora_backward(dc, x, a, b, routing, h, scale, dx=dx)
"""

import ctypes
import functools
import struct

import torch

from . import _check, _need, lib, MOE_BF16, MOE_FP32
from .training import _flat, _mat, _new, _on_stream, _same_device, _stream

__all__ = [
    "moe_dropout", "moe_rmsnorm", "moe_rmsnorm_backward", "moe_rmsnorm_backward_workspace_bytes",
    "moe_lora", "moe_lora_backward", "moe_lora_block_m", "moe_lora_workspace_bytes",
    "moe_lora_backward_workspace_bytes", "MOE_QUANT_NONE", "MOE_QUANT_MXFP8", "MOE_QUANT_PER_TOKEN",
]

MOE_QUANT_NONE, MOE_QUANT_MXFP8, MOE_QUANT_PER_TOKEN = 0, 1, 2
_QUANTS = {None: MOE_QUANT_NONE, "none": MOE_QUANT_NONE, "mxfp8": MOE_QUANT_MXFP8, "per_token": MOE_QUANT_PER_TOKEN}
_WIDE = {torch.float32: MOE_FP32, torch.bfloat16: MOE_BF16}

_i64, _i32, _vp, _f32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float


class MoeRmsnormArgs(ctypes.Structure):
    """ctypes mirror of moe_rmsnorm_args (include/moe_block.h)."""
    _fields_ = [
        ("rows", _i64), ("n", _i64), ("x", _vp), ("x_ld", _i64), ("p", _f32), ("rng", _vp),
        ("residual", _vp), ("residual_ld", _i64), ("residual_dtype", _i32), ("sum", _vp), ("sum_ld", _i64),
        ("weight", _vp), ("weight_dtype", _i32), ("eps", _f32), ("y", _vp), ("y_ld", _i64),
        ("quant", _i32), ("q", _vp), ("q_ld", _i64), ("scales", _vp), ("scales_ld", _i64),
    ]


class MoeRmsnormBackwardArgs(ctypes.Structure):
    """ctypes mirror of moe_rmsnorm_backward_args (include/moe_block.h)."""
    _fields_ = [
        ("rows", _i64), ("n", _i64), ("dy", _vp), ("dy_ld", _i64), ("dsum", _vp), ("dsum_ld", _i64),
        ("sum", _vp), ("sum_ld", _i64), ("sum_dtype", _i32), ("weight", _vp), ("weight_dtype", _i32), ("eps", _f32),
        ("p", _f32), ("rng", _vp), ("dresidual", _vp), ("dresidual_ld", _i64), ("dx", _vp), ("dx_ld", _i64),
        ("dweight", _vp), ("workspace", _vp), ("workspace_bytes", _i64),
    ]


_LORA = [
    ("x", _vp), ("x_ld", _i64), ("x_row_div", _i32), ("a", _vp), ("a_stride_g", _i64), ("a_ld", _i64), ("b", _vp),
    ("b_stride_g", _i64), ("b_ld", _i64), ("scale", _vp), ("sorted_slot_ids", _vp), ("group_ids", _vp),
    ("block_m", _i32), ("max_blocks", _i64),
]
_LORA_SIZES = [("num_slots", _i64), ("num_groups", _i32), ("rank", _i32), ("k", _i64), ("n", _i64)]


class MoeLoraArgs(ctypes.Structure):
    """ctypes mirror of moe_lora_args (include/moe_block.h)."""
    _fields_ = _LORA_SIZES + _LORA + [
        ("c", _vp), ("c_ld", _i64), ("h", _vp), ("workspace", _vp), ("workspace_bytes", _i64),
    ]


class MoeLoraBackwardArgs(ctypes.Structure):
    """ctypes mirror of moe_lora_backward_args (include/moe_block.h)."""
    _fields_ = _LORA_SIZES + [("dy", _vp), ("dy_ld", _i64)] + _LORA + [
        ("h", _vp), ("dx", _vp), ("dx_ld", _i64), ("da", _vp), ("db", _vp), ("workspace", _vp),
        ("workspace_bytes", _i64),
    ]


# Calls on small inputs are bound by the host: the argument structs are packed as
# bytes (a ctypes structure takes 2 us more), and sizes of workspaces are kept.
_CODES = {_i64: "q", _i32: "i", _f32: "f", _vp: "P"}


def _packer(mirror):
    """mirror(*values) as bytes, the native layout of its fields."""
    form = struct.Struct("@" + "".join(_CODES[t] for _, t in mirror._fields_))
    assert form.size <= ctypes.sizeof(mirror) < form.size + 8
    tail = bytes(ctypes.sizeof(mirror) - form.size)
    return form.pack if not tail else lambda *values: form.pack(*values) + tail


_pack_norm, _pack_norm_backward = _packer(MoeRmsnormArgs), _packer(MoeRmsnormBackwardArgs)
_pack_lora, _pack_lora_backward = _packer(MoeLoraArgs), _packer(MoeLoraBackwardArgs)


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _bind():
    args = ctypes.c_char_p
    sig = {
        "moe_dropout": (_i32, [_vp, _i64, _i64, _i64, _f32, _vp, _vp, _i64, _vp]),
        "moe_rmsnorm": (_i32, [args, _vp]),
        "moe_rmsnorm_backward": (_i32, [args, _vp]),
        "moe_rmsnorm_backward_workspace_bytes": (_i64, [_i64, _i64]),
        "moe_lora": (_i32, [args, _vp]),
        "moe_lora_backward": (_i32, [args, _vp]),
        "moe_lora_block_m": (_i32, [_i64, _i32]),
        "moe_lora_workspace_bytes": (_i64, [_i64, _i32, _i32, _i64, _i64, _i32, _i64]),
        "moe_lora_backward_workspace_bytes": (_i64, [_i64, _i32, _i32, _i64, _i64, _i32, _i64]),
    }
    for name, (res, types) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = types


_bind()

_norm_backward_bytes = functools.lru_cache(maxsize=4096)(lib.moe_rmsnorm_backward_workspace_bytes)
_lora_bytes = functools.lru_cache(maxsize=4096)(lib.moe_lora_workspace_bytes)
_lora_backward_bytes = functools.lru_cache(maxsize=4096)(lib.moe_lora_backward_workspace_bytes)


def _rng(rng):
    """The address of a dropout's {seed, offset}; 0 without one."""
    if rng is None:
        return 0
    _flat(rng, "rng", torch.int64, (2,))
    return rng.data_ptr()


def _wide(t, name):
    """The library's dtype of a matrix of the residual stream, or of the norm's weight."""
    if not isinstance(t, torch.Tensor) or t.dtype not in _WIDE:
        raise TypeError(f"{name} must be a float32 or bfloat16 tensor")
    return _WIDE[t.dtype]


def _workspace(workspace, need, like):
    """The address and size of the caller's workspace, or of a new one."""
    if workspace is None:
        if need <= 0:
            return 0, 0, None  # (the call says what is wrong with the sizes)
        workspace = torch.empty(need, dtype=torch.uint8, device=like.device)
    else:
        _need(workspace, "workspace", torch.uint8, 1)
        _same_device(like, workspace)
    return workspace.data_ptr(), workspace.numel(), workspace


@_on_stream
def moe_dropout(x, p, rng, out=None):
    """x / (1 - p) where kept and 0 elsewhere, bf16 [T, n] (rows may be strided).

    p in [0, 1], in steps of 2^-16; rng: int64 [2] on the device, {seed,
    offset} of the counter-based generator. The mask is a function of rng and
    of the element's place, so the gradient is the same call on the gradient.
    `out` may be x."""
    T, n, ld = _mat(x, "x", torch.bfloat16)
    if out is None:
        out, old = _new(x, T, n, torch.bfloat16), n
    else:
        old = _mat(out, "out", torch.bfloat16, T, n)[2]
    rng_p = _rng(rng)
    _same_device(x, rng, out)
    _check(lib.moe_dropout(x.data_ptr(), ld, T, n, p, rng_p, out.data_ptr(), old, _stream(x)))
    return out


@_on_stream
def moe_rmsnorm(x, weight, residual=None, eps=1e-6, p=0.0, rng=None, quant=None, keep_y=True, keep_sum=True, out=None):
    """The root-mean-square norm of residual + drop(x), times weight.

    x: bf16 [T, n]; weight: bf16 or fp32 [n]; residual: bf16 or fp32 [T, n];
    p, rng: dropout of x as in moe_dropout; quant: "mxfp8" (n % 32 == 0; what
    moe_grouped_gemm takes as MXFP8 activations) or "per_token" (what
    moe_grouped_gemm_per_token takes).

    Returns (y, sum, q, scales): y bf16 [T, n] (None with keep_y=False); sum =
    residual + drop(x) in the residual's dtype (None with keep_sum=False, or
    where it would be x); q uint8 E4M3 codes [T, n] with scales uint8 E8M0
    [T, n / 32] or fp32 [T] (None without quant). `out` may give the four, None
    for what is not wanted; its sum may be residual."""
    kind = _QUANTS.get(quant)
    if kind is None:
        raise ValueError(f'quant must be None, "none", "mxfp8" or "per_token", got {quant!r}')
    T, n, xld = _mat(x, "x", torch.bfloat16)
    wd = _wide(weight, "weight")
    _flat(weight, "weight", weight.dtype, (n,))
    rd, rld, res_p = MOE_BF16, 0, 0
    if residual is not None:
        rd = _wide(residual, "residual")
        rld, res_p = _mat(residual, "residual", residual.dtype, T, n)[2], residual.data_ptr()
        if residual.shape[0] != T:
            raise ValueError(f"residual must be [{T}, {n}], got {list(residual.shape)}")
    y = v = q = s = None
    yld = vld = qld = sld = 0
    if out is None:
        if keep_y:
            y, yld = _new(x, T, n, torch.bfloat16), n
        if keep_sum and (residual is not None or p > 0):
            v, vld = _new(x, T, n, torch.bfloat16 if residual is None else residual.dtype), n
        if kind:
            q, qld = _new(x, T, n, torch.uint8), n
            if kind == MOE_QUANT_MXFP8:
                s, sld = _new(x, T, n // 32, torch.uint8), n // 32
            else:
                s = torch.empty(T, dtype=torch.float32, device=x.device)
    else:
        y, v, q, s = out
        if (q is None) != (kind == 0) or (s is None) != (kind == 0):
            raise ValueError("out must give q and scales with a quant, and only then")
        if y is not None:
            yld = _mat(y, "y", torch.bfloat16, T, n)[2]
        if v is not None:
            if residual is None:
                rd = _wide(v, "sum")
            vld = _mat(v, "sum", v.dtype if residual is None else residual.dtype, T, n)[2]
        if kind:
            qld = _mat(q, "q", torch.uint8, T, n)[2]
            if kind == MOE_QUANT_MXFP8:
                sld = _mat(s, "scales", torch.uint8, T, n // 32)[2]
            else:
                _flat(s, "scales", torch.float32, (T,))
    rng_p = _rng(rng)
    _same_device(x, weight, residual, rng, y, v, q, s)
    _check(lib.moe_rmsnorm(_pack_norm(
        T, n, x.data_ptr(), xld, p, rng_p, res_p, rld, rd, _ptr(v), vld, weight.data_ptr(), wd, eps, _ptr(y), yld, kind,
        _ptr(q), qld, _ptr(s), sld), _stream(x)))
    return y, v, q, s


def moe_rmsnorm_backward_workspace_bytes(rows, n):
    """Bytes of the workspace that moe_rmsnorm_backward takes for dweight."""
    return int(lib.moe_rmsnorm_backward_workspace_bytes(int(rows), int(n)))


@_on_stream
def moe_rmsnorm_backward(dy, sum, weight, dsum=None, eps=1e-6, p=0.0, rng=None, keep_dweight=True, out=None,
                         workspace=None):
    """Gradient of moe_rmsnorm from the sum that it returned (x itself where it
    returned none).

    dy: bf16 [T, n], y's gradient; dsum: sum's gradient, in sum's dtype; weight,
    eps, p, rng as in the forward pass. Returns (dx bf16, dresidual in sum's
    dtype, dweight fp32 [n] or None); without dropout, and for a bf16 sum, dx
    and dresidual are one tensor. `out` may give the three, None for what is
    not wanted (its dresidual may be dsum); `workspace` a uint8 tensor of
    moe_rmsnorm_backward_workspace_bytes (calls that may run at the same time
    need one each)."""
    T, n, gld = _mat(dy, "dy", torch.bfloat16)
    sd, wd = _wide(sum, "sum"), _wide(weight, "weight")
    vld = _mat(sum, "sum", sum.dtype, T, n)[2]
    if sum.shape[0] != T:
        raise ValueError(f"sum must be [{T}, {n}], got {list(sum.shape)}")
    _flat(weight, "weight", weight.dtype, (n,))
    dsld = _mat(dsum, "dsum", sum.dtype, T, n)[2] if dsum is not None else 0
    dx = dres = dw = None
    dxld = drld = 0
    if out is None:
        dx, dxld = _new(dy, T, n, torch.bfloat16), n
        same = p == 0 and sd == MOE_BF16
        if not same:
            dres, drld = _new(dy, T, n, sum.dtype), n
        if keep_dweight:
            dw = torch.empty(n, dtype=torch.float32, device=dy.device)
        result = dx, dx if same else dres, dw
    else:
        dx, dres, dw = result = tuple(out)
        if dx is not None:
            dxld = _mat(dx, "dx", torch.bfloat16, T, n)[2]
        if dres is not None:
            drld = _mat(dres, "dresidual", sum.dtype, T, n)[2]
        if dw is not None:
            _flat(dw, "dweight", torch.float32, (n,))
    ws_p = ws_n = 0
    if dw is not None:
        ws_p, ws_n, workspace = _workspace(workspace, _norm_backward_bytes(T, n) if workspace is None else 0, dy)
    rng_p = _rng(rng)
    _same_device(dy, sum, weight, dsum, rng, dx, dres, dw)
    _check(lib.moe_rmsnorm_backward(_pack_norm_backward(
        T, n, dy.data_ptr(), gld, _ptr(dsum), dsld, sum.data_ptr(), vld, sd, weight.data_ptr(), wd, eps, p, rng_p,
        _ptr(dres), drld, _ptr(dx), dxld, _ptr(dw), ws_p, ws_n), _stream(dy)))
    return result


def moe_lora_block_m(num_slots, num_groups):
    """The block size to align num_slots slots over num_groups groups with."""
    return int(lib.moe_lora_block_m(int(num_slots), int(num_groups)))


def moe_lora_workspace_bytes(num_slots, num_groups, rank, k, n, block_m, max_blocks):
    """Bytes of moe_lora's workspace."""
    return int(lib.moe_lora_workspace_bytes(num_slots, num_groups, rank, k, n, block_m, max_blocks))


def moe_lora_backward_workspace_bytes(num_slots, num_groups, rank, k, n, block_m, max_blocks):
    """Bytes of moe_lora_backward's workspace."""
    return int(lib.moe_lora_backward_workspace_bytes(num_slots, num_groups, rank, k, n, block_m, max_blocks))


def _adapters(t, name):
    """(groups, rows, columns, group stride, row stride) of adapter matrices."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16 or not t.is_cuda or t.dim() != 3:
        _need(t, name, torch.bfloat16, 3)
    (G, r, c), (sg, ld, one) = t.shape, t.stride()
    if one != 1 and G * r * c:
        _need(t, name, torch.bfloat16, 3)
    if r == 1:  # (a stride that is stepped by never means nothing)
        ld = -(-c // 8) * 8
    return G, r, c, sg if G > 1 else r * ld, ld


def _lora_slots(routing, num_slots, rows, name):
    """The number of slots: num_slots, or what the list was made for (the rows
    of C or dy where it does not say), at most `rows`."""
    made = getattr(routing, "num_slots", None)
    if num_slots is None:
        return rows if made is None or made > rows else made
    S = int(num_slots)
    if S < 0 or S > rows:
        raise ValueError(f"num_slots must be in [0, {rows}], the rows of {name}, got {S}")
    if made is not None and S > made:
        raise ValueError(f"num_slots {S} exceeds the {made} slots that the routing was made for")
    return S


def _lora_args(x, a, b, routing, scale, row_div, S, N):
    """The arguments that both adapter entry points share: (sizes, fields, G, R, K)."""
    G, R, K, a_g, a_ld = _adapters(a, "a")
    G2, N2, R2, b_g, b_ld = _adapters(b, "b")
    if (G2, N2, R2) != (G, N, R):
        raise ValueError(f"b must be [{G}, {N}, {R}] beside a [{G}, {R}, {K}], got {[G2, N2, R2]}")
    div = int(row_div)
    if div < 1:
        raise ValueError(f"row_div must be >= 1, got {div}")
    x_ld = _mat(x, "x", torch.bfloat16, -(-S // div), K)[2]
    ids, groups = routing[0], routing[1]
    for t, name in ((ids, "sorted_slot_ids"), (groups, "group_ids")):
        if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or t.dim() != 1 or not t.is_contiguous():
            _need(t, name, torch.int32, 1)
    blocks = groups.numel()
    bm = ids.numel() // blocks if blocks else moe_lora_block_m(S, G)
    if bm * blocks != ids.numel():
        raise ValueError("the routing's arrays do not belong together")
    if scale is not None:
        _flat(scale, "scale", torch.float32, (G,))
    _same_device(x, a, b, ids, groups, scale)
    sizes = S, G, R, K, N
    return sizes, (x.data_ptr(), x_ld, div, a.data_ptr(), a_g, a_ld, b.data_ptr(), b_g, b_ld, _ptr(scale), ids.data_ptr(),
                   groups.data_ptr(), bm, blocks)


@_on_stream
def moe_lora(c, x, a, b, routing, scale=None, row_div=1, keep_h=False, workspace=None, num_slots=None):
    """Adds low-rank adapters to a shared projection's output, in place:
    c[s] += scale[g] * b[g] @ (a[g] @ x[s // row_div]) for the slots s of every
    group g.

    c: bf16 [at least S, N], the projection's output; x: bf16 [S / row_div, K], its
    input; a: bf16 [G, R, K], b: bf16 [G, N, R] (8 <= R <= 128, a multiple of 8;
    rows and matrices may be strided); scale: fp32 [G]; routing: moe_align's
    over the slots' group ids, at block size 8, 16, 32 or 64
    (moe_lora_block_m(S, G); with groups = experts, the grouped GEMM's own).
    Slots in no group keep their rows, and so do rows of c behind the slots. S
    is what moe_align made the routing for; num_slots takes fewer of them, or
    says it for a list of one's own, whose padding must hold no number below
    it (default: the rows of c). Returns c; with keep_h (c, h), h fp32 [S, R] =
    a @ x of the routed slots for moe_lora_backward."""
    rows, N, c_ld = _mat(c, "c", torch.bfloat16)
    S = _lora_slots(routing, num_slots, rows, "c")
    sizes, args = _lora_args(x, a, b, routing, scale, row_div, S, N)
    h = torch.empty((S, sizes[2]), dtype=torch.float32, device=c.device) if keep_h else None
    ws_p, ws_n, ws = _workspace(workspace, _lora_bytes(*sizes, *args[-2:]) if workspace is None else 0, c)
    _same_device(c, x)
    _check(lib.moe_lora(_pack_lora(*sizes, *args, c.data_ptr(), c_ld, _ptr(h), ws_p, ws_n), _stream(c)))
    return (c, h) if keep_h else c


@_on_stream
def moe_lora_backward(dy, x, a, b, routing, h, scale=None, row_div=1, dx=None, weights=True, out=None,
                      workspace=None, num_slots=None):
    """Gradients of moe_lora from dy (bf16 [at least S, N], the gradient of c
    after the addition) and the h that the forward pass kept.

    Returns (da fp32 [G, R, K], db fp32 [G, N, R]), zeros for groups without
    slots; (None, None) with weights=False. dx (bf16 [at least S, K], the shared
    projection's gradient of its input, a row per slot) gets the adapters' part
    added in place. The other arguments as in the forward pass; `out` may give
    da and db."""
    rows, N, dy_ld = _mat(dy, "dy", torch.bfloat16)
    S = _lora_slots(routing, num_slots, rows, "dy")
    sizes, args = _lora_args(x, a, b, routing, scale, row_div, S, N)
    _, G, R, K, _ = sizes
    da = db = None
    if weights:
        _flat(h, "h", torch.float32, (S, R))
        if out is None:
            da = torch.empty((G, R, K), dtype=torch.float32, device=dy.device)
            db = torch.empty((G, N, R), dtype=torch.float32, device=dy.device)
        else:
            da, db = out
            _flat(da, "da", torch.float32, (G, R, K))
            _flat(db, "db", torch.float32, (G, N, R))
    else:
        h = None
    dx_ld = _mat(dx, "dx", torch.bfloat16, S, K)[2] if dx is not None else 0
    ws_p, ws_n, ws = _workspace(workspace, _lora_backward_bytes(*sizes, *args[-2:]) if workspace is None else 0, dy)
    _same_device(dy, x, h, dx, da, db)
    _check(lib.moe_lora_backward(_pack_lora_backward(
        *sizes, dy.data_ptr(), dy_ld, *args, _ptr(h), _ptr(dx), dx_ld, _ptr(da), _ptr(db), ws_p, ws_n), _stream(dy)))
    return da, db
