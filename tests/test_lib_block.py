"""CPU tests of the block half of the C ABI (include/moe_block.h): it exports
what the header declares, and every argument check rejects bad calls before
anything reaches a GPU (all calls here are invalid on purpose)."""

import ctypes
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

moe = pytest.importorskip("mixture_experts_grouped_moe_amd")
L = moe.lib

INVALID, UNSUPPORTED = 1, 2
P = 1 << 32  # never dereferenced: every call below is rejected first
BF16, FP32 = moe.MOE_BF16, moe.MOE_FP32


@pytest.fixture
def no_device():
    if torch.cuda.is_available():
        pytest.skip("argument-rejection tests run on hosts without a GPU")


def _header():
    return re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "moe_block.h")).read(), flags=re.S)


def test_exports_every_declared_symbol():
    for name in sorted(set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", _header()))):
        assert hasattr(L, name), name
        assert name in moe.__all__ and callable(getattr(moe, name))


def test_struct_mirrors(tmp_path):
    """Field names, offsets and sizes of the ctypes mirrors are those of the header's structs."""
    structs = {m[1]: re.findall(r"(\w+);", m[0]) for m in re.findall(r"typedef struct \{(.*?)\} (\w+);", _header(), re.S)}
    mirrors = {"moe_" + re.sub(r"(?<!^)([A-Z])", r"_\1", n[3:]).lower().lstrip("_"): c for n, c in vars(moe.block).items()
               if isinstance(c, type) and issubclass(c, ctypes.Structure)}
    assert set(structs) == set(mirrors)
    lines = [f'printf("%s %zu %zu\\n", "{s}.{f}", offsetof({s}, {f}), sizeof((({s}*)0)->{f}));'
             for s, fields in structs.items() for f in fields]
    src = tmp_path / "o.c"
    src.write_text('#include <stdio.h>\n#include "moe_block.h"\nint main(void) {' + "\n".join(lines) + "return 0; }")
    subprocess.run(["gcc", "-std=c99", f"-I{ROOT}/include", str(src), "-o", str(tmp_path / "o")], check=True)
    said = subprocess.run([str(tmp_path / "o")], check=True, capture_output=True, text=True).stdout.split("\n")
    want = [f"{s}.{n} {getattr(mirrors[s], n).offset} {getattr(mirrors[s], n).size}" for s in structs
            for n, _ in mirrors[s]._fields_]
    assert [l for l in said if l] == want


def test_packed_structs_are_the_mirrors():
    """The binding packs its arguments as bytes: the mirrors' bytes."""
    for pack, mirror in ((moe.block._pack_norm, moe.block.MoeRmsnormArgs),
                         (moe.block._pack_norm_backward, moe.block.MoeRmsnormBackwardArgs),
                         (moe.block._pack_lora, moe.block.MoeLoraArgs),
                         (moe.block._pack_lora_backward, moe.block.MoeLoraBackwardArgs)):
        values = [i + 1 if t is not ctypes.c_float else i + 0.5 for i, (_, t) in enumerate(mirror._fields_)]
        assert pack(*values) == bytes(mirror(*values))


def refused(st):
    return st in (INVALID, UNSUPPORTED)


def _drop(x=P, xld=64, rows=4, n=64, p=0.5, rng=2 * P, y=3 * P, yld=64):
    return L.moe_dropout(x, xld, rows, n, p, rng, y, yld, None)


def _norm(**kw):
    d = dict(rows=4, n=64, x=P, x_ld=64, p=0.5, rng=2 * P, residual=3 * P, residual_ld=64, residual_dtype=FP32,
             sum=4 * P, sum_ld=64, weight=5 * P, weight_dtype=BF16, eps=1e-6, y=6 * P, y_ld=64, quant=1, q=7 * P,
             q_ld=64, scales=8 * P, scales_ld=2)
    return L.moe_rmsnorm(bytes(moe.block.MoeRmsnormArgs(**{**d, **kw})), None)


def _norm_bwd(**kw):
    d = dict(rows=4, n=64, dy=P, dy_ld=64, dsum=2 * P, dsum_ld=64, sum=3 * P, sum_ld=64, sum_dtype=FP32, weight=4 * P,
             weight_dtype=BF16, eps=1e-6, p=0.5, rng=5 * P, dresidual=6 * P, dresidual_ld=64, dx=7 * P, dx_ld=64,
             dweight=8 * P, workspace=9 * P, workspace_bytes=1 << 24)
    return L.moe_rmsnorm_backward(bytes(moe.block.MoeRmsnormBackwardArgs(**{**d, **kw})), None)


def test_dropout_rejects(no_device):
    assert not refused(_drop())
    assert not refused(_drop(y=P))                      # in place
    assert not refused(_drop(p=0.0, rng=None)) and not refused(_drop(p=1.0)) and not refused(_drop(rows=0, x=None, y=None))
    assert not refused(_drop(p=2.0 ** -18, rng=None))   # a threshold of 0
    for bad in (dict(rows=-1), dict(n=60), dict(n=0), dict(n=1 << 31), dict(rows=1 << 58), dict(p=-0.1), dict(p=1.1),
                dict(p=float("nan")), dict(rng=None), dict(rng=P + 4), dict(x=None), dict(y=None), dict(x=P + 8),
                dict(y=3 * P + 2), dict(xld=56), dict(yld=68), dict(y=P + 16), dict(y=P, yld=72), dict(y=2 * P),
                dict(rng=3 * P + 64), dict(rows=1 << 30, xld=1 << 40)):
        assert _drop(**bad) == INVALID, bad


def test_norm_rejects(no_device):
    assert not refused(_norm()) and L.moe_rmsnorm(None, None) == INVALID
    assert not refused(_norm(sum=3 * P))                                           # the residual in place
    assert not refused(_norm(residual=None, sum=None, p=0.0, rng=None))
    assert not refused(_norm(y=None)) and not refused(_norm(quant=0, q=None, scales=None, q_ld=0, scales_ld=0))
    assert not refused(_norm(quant=2, scales_ld=0)) and not refused(_norm(rows=0, x=None, y=None, q=None, scales=None))
    assert not refused(_norm(n=8, quant=2)) and not refused(_norm(eps=0.0))
    for bad in (dict(rows=-1), dict(rows=1 << 31), dict(n=40), dict(n=0), dict(n=60, quant=0), dict(eps=-1e-6),
                dict(eps=float("inf")), dict(eps=float("nan")), dict(p=2.0), dict(rng=None), dict(weight=None),
                dict(weight=5 * P + 8), dict(x=None), dict(x=P + 2), dict(x_ld=63), dict(x_ld=56), dict(residual=3 * P + 4),
                dict(residual_ld=60), dict(sum_ld=60), dict(sum=4 * P + 8), dict(y_ld=60), dict(y=6 * P + 8),
                dict(quant=0, y=None), dict(quant=3), dict(q=None), dict(scales=None), dict(q_ld=60), dict(q=7 * P + 4),
                dict(scales_ld=1), dict(quant=2, scales=8 * P + 2), dict(rows=1 << 30, y_ld=1 << 40)):
        assert _norm(**bad) == INVALID, bad
    assert _norm(n=16384 + 32, x_ld=1 << 15) == UNSUPPORTED
    assert _norm(residual_dtype=moe.MOE_E4M3) == UNSUPPORTED and _norm(weight_dtype=0) == UNSUPPORTED


def test_norm_backward_rejects(no_device):
    assert not refused(_norm_bwd()) and L.moe_rmsnorm_backward(None, None) == INVALID
    assert not refused(_norm_bwd(dresidual=2 * P)) and not refused(_norm_bwd(dsum=None))
    assert not refused(_norm_bwd(dweight=None, workspace=None, workspace_bytes=0))
    assert not refused(_norm_bwd(dresidual=None, dx=None))
    for bad in (dict(rows=-1), dict(n=60), dict(eps=-1.0), dict(rng=None), dict(dy=None), dict(sum=None),
                dict(weight=None), dict(dy=P + 8), dict(dsum=2 * P + 8), dict(dy_ld=60), dict(sum_ld=60),
                dict(dsum_ld=60), dict(dresidual_ld=60), dict(dx_ld=60), dict(dresidual=None, dx=None, dweight=None),
                dict(dweight=8 * P + 2), dict(workspace=None), dict(workspace=9 * P + 8),
                dict(workspace_bytes=moe.moe_rmsnorm_backward_workspace_bytes(4, 64) - 1)):
        assert _norm_bwd(**bad) == INVALID, bad
    assert _norm_bwd(n=16392, dy_ld=1 << 15) == UNSUPPORTED and _norm_bwd(sum_dtype=0) == UNSUPPORTED


def test_workspaces():
    f = moe.moe_rmsnorm_backward_workspace_bytes
    assert f(0, 64) >= 0 and f(-1, 64) == -1 and f(4, 60) == -1 and f(4, 16392) == -1 and f(4, 0) == -1
    assert f(1 << 30, 16384) == f(1 << 20, 16384) <= 256 << 20    # partial sums of workgroups, not rows


def _overlaps(call, outputs, inputs, allowed=()):
    names = outputs + inputs
    ptr = {n: (i + 20) << 32 for i, n in enumerate(names)}
    assert not refused(call(**ptr))
    for i, a in enumerate(outputs):
        for b in outputs[i + 1:] + inputs:
            st = call(**{**ptr, a: ptr[b]})
            assert refused(st) == ((a, b) not in allowed), (a, b)
            if b not in ("scale", "group_ids"):   # (of 16 bytes and less)
                assert refused(call(**{**ptr, a: ptr[b] + 16})), (a, b)


def test_overlaps_are_rejected(no_device):
    _overlaps(_drop, ["y"], ["x"], [("y", "x")])
    _overlaps(_norm, ["sum", "y", "q"], ["x", "residual", "weight"], [("sum", "residual")])
    _overlaps(_norm_bwd, ["dresidual", "dx", "dweight", "workspace"], ["dy", "dsum", "sum", "weight"],
              [("dresidual", "dsum")])
    assert _norm(scales=7 * P) == INVALID and _norm(rng=6 * P) == INVALID and _norm_bwd(rng=7 * P) == INVALID


def test_binding_rejects_before_the_library():
    x, w, r = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):            # not on a device
        moe.moe_dropout(x, 0.5, r)
    with pytest.raises(TypeError):
        moe.moe_dropout(x.float(), 0.5, r)
    with pytest.raises(ValueError):
        moe.moe_rmsnorm(x, w)
    with pytest.raises(TypeError):
        moe.moe_rmsnorm(x.half(), w)
    with pytest.raises(ValueError):
        moe.moe_rmsnorm_backward(x, x, w)


# ----------------------------------------------------------------- adapters

_LORA = dict(num_slots=20, num_groups=3, rank=16, k=64, n=48, x=20 * P, x_ld=64, x_row_div=2, a=21 * P, a_stride_g=1024,
             a_ld=64, b=22 * P, b_stride_g=768, b_ld=16, scale=23 * P, sorted_slot_ids=24 * P, group_ids=25 * P,
             block_m=16, max_blocks=4)


def _lora(**kw):
    d = dict(_LORA, c=26 * P, c_ld=48, h=27 * P, workspace=28 * P, workspace_bytes=1 << 30)
    return L.moe_lora(bytes(moe.block.MoeLoraArgs(**{**d, **kw})), None)


def _lora_bwd(**kw):
    d = dict(_LORA, dy=29 * P, dy_ld=48, h=27 * P, dx=30 * P, dx_ld=64, da=31 * P, db=32 * P, workspace=28 * P,
             workspace_bytes=1 << 30)
    return L.moe_lora_backward(bytes(moe.block.MoeLoraBackwardArgs(**{**d, **kw})), None)


def _lora_bytes(f, S=20, G=3, R=16, K=64, N=48, bm=16, mb=4):
    return f(S, G, R, K, N, bm, mb)


def test_lora_rejects(no_device):
    assert moe.moe_align_max_blocks(20, 3, 16) == 4
    assert L.moe_lora(None, None) == INVALID and L.moe_lora_backward(None, None) == INVALID
    for call in (_lora, _lora_bwd):
        assert not refused(call()) and not refused(call(scale=None)) and not refused(call(num_groups=1, a_stride_g=1024))
        assert not refused(call(rank=8, a_stride_g=512, b_ld=8, b_stride_g=384)) and not refused(call(b_ld=24, b_stride_g=2000))
        assert not refused(call(num_slots=0, max_blocks=0, x=None, sorted_slot_ids=None, group_ids=None))
        for bad in (dict(num_slots=-1), dict(num_slots=1 << 31), dict(num_groups=0), dict(rank=0), dict(rank=12),
                    dict(k=60), dict(n=44), dict(k=0), dict(k=1 << 24, x_ld=1 << 24), dict(x_row_div=0), dict(x=None),
                    dict(a=None), dict(b=None), dict(x=20 * P + 8), dict(a=21 * P + 8), dict(b=22 * P + 8), dict(x_ld=56),
                    dict(x_ld=68), dict(a_ld=60), dict(a_ld=72), dict(a_stride_g=1016), dict(b_ld=8), dict(b_stride_g=760),
                    dict(a_stride_g=1028), dict(scale=23 * P + 2), dict(sorted_slot_ids=None), dict(group_ids=None),
                    dict(group_ids=25 * P + 2), dict(block_m=24), dict(block_m=128), dict(max_blocks=3),
                    dict(max_blocks=1 << 27), dict(workspace=28 * P + 8), dict(h=27 * P + 8),
                    dict(x_ld=1 << 60), dict(a_stride_g=1 << 60)):
            assert call(**bad) == INVALID, bad
        assert call(num_groups=1025, max_blocks=30) == UNSUPPORTED
        assert call(rank=136, a_stride_g=1 << 14, b_ld=136, b_stride_g=1 << 14) == UNSUPPORTED
    assert not refused(_lora(h=None)) and not refused(_lora(workspace=None, workspace_bytes=0))   # one launch, no workspace
    wide = dict(rank=64, a_stride_g=4096, b_ld=64, b_stride_g=3200)
    assert not refused(_lora(**wide)) and _lora(**wide, workspace=None) == INVALID
    assert _lora(**wide, workspace_bytes=_lora_bytes(moe.moe_lora_workspace_bytes, R=64) - 1) == INVALID
    assert _lora(c=None) == INVALID and _lora(c_ld=40) == INVALID and _lora(c=26 * P + 8) == INVALID
    assert not refused(_lora_bwd(dx=None)) and not refused(_lora_bwd(da=None, db=None, h=None))
    for bad in (dict(workspace=None), dict(dy=None), dict(dy_ld=40), dict(dx_ld=56), dict(da=None), dict(db=None), dict(h=None),
                dict(dx=None, da=None, db=None), dict(da=31 * P + 8),
                dict(workspace_bytes=_lora_bytes(moe.moe_lora_backward_workspace_bytes) - 1)):
        assert _lora_bwd(**bad) == INVALID, bad


def test_lora_sizes():
    f, g = moe.moe_lora_workspace_bytes, moe.moe_lora_backward_workspace_bytes
    for h in (f, g):
        assert _lora_bytes(h) >= 0
        for bad in (dict(S=-1), dict(G=0), dict(G=1025), dict(R=4), dict(R=136), dict(K=4), dict(N=0), dict(bm=7), dict(mb=3)):
            assert _lora_bytes(h, **bad) == -1, bad
    m = moe.moe_lora_block_m
    assert m(0, 1) == 16 and m(31, 1) == 16 and m(32, 1) == 64 and m(1 << 30, 1024) == 64 and m(-1, 1) == -1 and m(4, 0) == -1
    # h (twice, and a part of dh per 512 columns of dy) by place; the gradients' partial sums by segments of the list
    h = 64 * (1 << 18) * 16 * 4
    assert f(1 << 24, 1, 16, 2880, 5760, 64, 1 << 18) <= 2 * h
    assert g(1 << 24, 1, 16, 2880, 5760, 64, 1 << 18) - (12 + 1) * h < 256 << 20


def test_lora_overlaps_are_rejected(no_device):
    shared = ["x", "a", "b", "scale", "sorted_slot_ids", "group_ids"]
    _overlaps(lambda **kw: _lora(rank=64, a_stride_g=4096, b_ld=64, b_stride_g=3200, **kw), ["c", "h", "workspace"], shared)
    _overlaps(_lora_bwd, ["dx", "da", "db", "workspace"], shared + ["dy", "h"])


def test_lora_binding_rejects_before_the_library():
    x, a, b = (torch.zeros(s, dtype=torch.bfloat16) for s in ((4, 64), (2, 8, 64), (2, 48, 8)))
    c, ids = torch.zeros(4, 48, dtype=torch.bfloat16), torch.zeros(16, dtype=torch.int32)
    with pytest.raises(ValueError):
        moe.moe_lora(c, x, a, b, (ids, ids, ids))
    with pytest.raises(TypeError):
        moe.moe_lora(c.float(), x, a, b, (ids, ids, ids))
    with pytest.raises(ValueError):
        moe.moe_lora_backward(c, x, a, b, (ids, ids, ids), torch.zeros(4, 8))
