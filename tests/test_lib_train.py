"""CPU tests of the training half of the C ABI (include/moe_train.h): it
exports what the header declares, and every argument check rejects bad calls
before anything reaches a GPU (all calls here are invalid on purpose)."""

import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

moe = pytest.importorskip("mixture_experts_grouped_moe_amd")
L = moe.lib

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = 0x100000  # never dereferenced: every call below is rejected first


@pytest.fixture
def no_device():
    if torch.cuda.is_available():
        pytest.skip("argument-rejection tests run on hosts without a GPU")


def test_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "moe_train.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    syms = sorted(set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", text)))
    assert len(syms) == 8, syms
    for name in syms:
        assert hasattr(L, name), name
        assert name in moe.__all__ and callable(getattr(moe, name))


def test_route_workspace():
    assert moe.moe_route_workspace_bytes(0, 8) >= 0
    assert moe.moe_route_workspace_bytes(-1, 8) == -1
    assert moe.moe_route_workspace_bytes(8, 0) == -1
    assert moe.moe_route_workspace_bytes(8, 1025) == -1
    # bounded in the number of tokens: partial sums of workgroups, not rows
    assert moe.moe_route_workspace_bytes(1 << 24, 256) == moe.moe_route_workspace_bytes(1 << 20, 256) < 8 << 20


def _route(z=P, dt=None, ld=None, mask=None, T=10, E=8, k=2, score=0, renorm=1, scale=1.0, ids=P, w=P, stats=1,
           counts=P, n=P, p=P, loss=P, ws=P, wsn=1 << 20):
    return L.moe_route(z, moe.MOE_FP32 if dt is None else dt, E if ld is None else ld, mask, T, E, k, score, renorm,
                       scale, ids, w, stats, counts, n, p, loss, ws, wsn, None)


def test_route_rejects(no_device):
    assert _route(T=-1) == INVALID
    assert _route(k=0) == INVALID
    assert _route(k=9) == INVALID
    assert _route(E=1025) == UNSUPPORTED
    assert _route(E=128, k=65) == UNSUPPORTED
    assert _route(T=2 ** 30, k=2) == INVALID
    assert _route(dt=moe.MOE_E4M3) == UNSUPPORTED
    assert _route(score=2) == INVALID
    assert _route(scale=float("inf")) == INVALID
    assert _route(scale=float("nan")) == INVALID
    assert _route(ld=7) == INVALID
    assert _route(z=None) == INVALID
    assert _route(ids=None) == INVALID
    assert _route(w=None) == INVALID
    assert _route(z=P + 2) == INVALID
    assert _route(z=P + 1, dt=moe.MOE_BF16) == INVALID
    assert _route(w=P + 2) == INVALID
    for name in ("counts", "n", "p", "loss", "ws"):
        assert _route(**{name: None}) == INVALID, name
        assert _route(**{name: P + 2}) == INVALID, name
    assert _route(ws=P + 4) == INVALID
    assert _route(wsn=moe.moe_route_workspace_bytes(10, 8) - 1) == INVALID
    assert b"workspace" in L.moe_last_error()


def _route_bwd(z=P, dt=None, ld=None, T=10, E=8, k=2, score=0, ids=2 * P, dw=3 * P, counts=4 * P, n=5 * P,
               dl=6 * P, out=7 * P, old=None):
    return L.moe_route_backward(z, moe.MOE_FP32 if dt is None else dt, E if ld is None else ld, T, E, k, score, 1,
                                1.0, ids, dw, counts, n, dl, out, E if old is None else old, None)


def test_route_backward_rejects(no_device):
    assert _route_bwd(T=-1) == INVALID
    assert _route_bwd(k=9) == INVALID
    assert _route_bwd(dt=moe.MOE_E8M0) == UNSUPPORTED
    assert _route_bwd(ld=7) == INVALID
    assert _route_bwd(old=7) == INVALID
    for name in ("z", "ids", "dw", "out"):
        assert _route_bwd(**{name: None}) == INVALID, name
    assert _route_bwd(counts=None) == INVALID
    assert _route_bwd(n=None) == INVALID
    assert _route_bwd(out=P) == INVALID           # dlogits over logits
    assert _route_bwd(out=P + 9 * 32) == INVALID  # over their last row
    assert _route_bwd(out=3 * P) == INVALID
    assert _route_bwd(out=4 * P) == INVALID
    assert b"overlap" in L.moe_last_error()


def _combine(c=P, cld=64, w=P, ids=P, T=4, k=2, E=8, n=64, y=P, yld=64):
    return L.moe_combine_routed(c, cld, w, ids, T, k, E, n, y, yld, None)


def test_combine_routed_rejects(no_device):
    assert _combine(T=-1) == INVALID
    assert _combine(k=0) == INVALID
    assert _combine(E=0) == INVALID
    assert _combine(n=60) == INVALID
    assert _combine(n=0) == INVALID
    assert _combine(cld=56) == INVALID
    assert _combine(yld=68) == INVALID
    assert _combine(T=2 ** 30, k=4) == INVALID
    for name in ("c", "w", "ids", "y"):
        assert _combine(**{name: None}) == INVALID, name
    assert _combine(c=P + 8) == INVALID
    assert _combine(ids=P + 2) == INVALID


def _combine_bwd(dy=P, dyld=64, c=2 * P, cld=64, w=P, ids=P, T=4, k=2, E=8, n=64, dc=3 * P, dcld=64, dw=4 * P):
    return L.moe_combine_backward(dy, dyld, c, cld, w, ids, T, k, E, n, dc, dcld, dw, None)


def test_combine_backward_rejects(no_device):
    assert _combine_bwd(T=-1) == INVALID
    assert _combine_bwd(k=0) == INVALID
    assert _combine_bwd(E=0) == INVALID
    assert _combine_bwd(n=4) == INVALID
    assert _combine_bwd(dyld=60) == INVALID
    assert _combine_bwd(cld=66) == INVALID
    assert _combine_bwd(dcld=0) == INVALID
    for name in ("dy", "c", "w", "dc", "dw"):
        assert _combine_bwd(**{name: None}) == INVALID, name
    assert _combine_bwd(dc=3 * P + 2) == INVALID
    assert _combine_bwd(dc=2 * P) == INVALID       # in place of C
    assert _combine_bwd(dc=P) == INVALID           # over dy
    assert _combine_bwd(dc=2 * P + 7 * 128) == INVALID


def _act(act=1, pre=P, pld=128, R=4, n=128, h=2 * P, hld=64, q=3 * P, qld=128, s=4 * P, sld=4):
    return L.moe_act_mxfp8(act, pre, pld, R, n, h, hld, q, qld, s, sld, None)


def _act_bwd(act=1, q=P, qld=128, s=2 * P, sld=4, dh=3 * P, dhld=64, R=4, n=128, dp=4 * P, dpld=128, h=5 * P, hld=64):
    return L.moe_act_mxfp8_backward(act, q, qld, s, sld, dh, dhld, R, n, dp, dpld, h, hld, None)


def test_act_rejects(no_device):
    for f in (_act, _act_bwd):
        assert f(act=0) == INVALID
        assert f(act=3) == INVALID
        assert f(R=-1) == INVALID
        assert f(n=96) == INVALID                  # SwiGLU halves of 48: not whole blocks
        assert f(act=2, n=100) == INVALID
        assert f(n=0) == INVALID
        assert f(qld=112) == INVALID
        assert f(qld=136) == INVALID
        assert f(sld=3) == INVALID
        assert f(q=None) == INVALID
        assert f(s=None) == INVALID
        assert f(q=P + 8) == INVALID
        assert f(hld=60) == INVALID
        assert f(hld=68) == INVALID
    assert _act(pre=None) == INVALID
    assert _act(h=None) == INVALID
    assert _act(pld=120) == INVALID
    assert _act(h=P) == INVALID
    assert _act(q=P) == INVALID
    assert _act(s=3 * P + 511) == INVALID          # over the codes' last byte
    assert _act_bwd(dh=None) == INVALID
    assert _act_bwd(dp=None) == INVALID
    assert _act_bwd(dhld=56) == INVALID
    assert _act_bwd(dpld=64) == INVALID
    assert _act_bwd(dp=P) == INVALID
    assert _act_bwd(h=3 * P) == INVALID            # h over dh
    assert _act_bwd(h=4 * P) == INVALID


def _wgrad(xq=P, xld=128, xs=P, xsld=4, g=P, gld=64, s=P, e=P, T=10, k=2, E=4, n=64, K=128, bm=None, mb=None, dw=P):
    bm = moe.moe_wgrad_block_m() if bm is None else bm
    mb = moe.moe_align_max_blocks(T * k, E, bm) if mb is None else mb
    return L.moe_wgrad_mxfp8(xq, xld, xs, xsld, g, gld, s, e, P, T, k, E, n, K, bm, mb, dw, None)


def test_wgrad_mxfp8_rejects(no_device):
    assert _wgrad(T=-1, mb=0) == INVALID
    assert _wgrad(k=5) == INVALID
    assert _wgrad(E=1025) == UNSUPPORTED
    assert _wgrad(n=48) == INVALID
    assert _wgrad(K=100) == INVALID
    assert _wgrad(xld=112) == INVALID
    assert _wgrad(xld=136) == INVALID
    assert _wgrad(xsld=3) == INVALID
    assert _wgrad(gld=60) == INVALID
    assert _wgrad(bm=16) == INVALID
    assert _wgrad(mb=0) == INVALID
    assert _wgrad(mb=1 << 24) == INVALID
    for name in ("xq", "xs", "g", "s", "e", "dw"):
        assert _wgrad(**{name: None}) == INVALID, name
    assert _wgrad(xq=P + 8) == INVALID
    assert _wgrad(dw=P + 4) == INVALID
    assert _wgrad(T=1 << 24, xld=128, E=4) == UNSUPPORTED   # codes of 2 GB
    assert _wgrad(n=1 << 15, K=1 << 15, xld=1 << 15, xsld=1 << 10, gld=1 << 15) == UNSUPPORTED


def _far(n):
    return [(i + 1) << 32 for i in range(n)]  # pointers far apart


def _overlaps(call, outputs, inputs):
    """Every output over every other one and over every input is refused; the call as such is not."""
    names = outputs + inputs
    ptr = dict(zip(names, _far(len(names))))
    assert call(**ptr) not in (INVALID, UNSUPPORTED), L.moe_last_error()   # (no device here)
    for i, a in enumerate(outputs):
        for b in outputs[i + 1:] + inputs:
            assert call(**{**ptr, a: ptr[b]}) == INVALID, (a, b)
            assert b"overlap" in L.moe_last_error()


def test_overlaps_are_rejected(no_device):
    _overlaps(_route, ["ids", "w", "counts", "n", "p", "loss", "ws"], ["z", "mask"])
    _overlaps(_route_bwd, ["out"], ["z", "ids", "dw", "counts", "n", "dl"])
    _overlaps(_combine, ["y"], ["c", "w", "ids"])
    _overlaps(_combine_bwd, ["dc", "dw"], ["dy", "c", "w", "ids"])
    _overlaps(_act, ["h", "q", "s"], ["pre"])
    _overlaps(_act_bwd, ["dp", "h"], ["q", "s", "dh"])
    _overlaps(_wgrad, ["dw"], ["xq", "xs", "g", "s", "e"])
    # what a call leaves out overlaps nothing
    z, ids, w = _far(3)
    assert _route(z=z, ids=ids, w=w, stats=0, counts=z, n=z, p=z, loss=z, ws=z) not in (INVALID, UNSUPPORTED)
    assert _act_bwd(q=z, s=z + 4096, dh=ids, dp=w, h=None, hld=0) not in (INVALID, UNSUPPORTED)


def test_strides_past_64_bits_are_rejected(no_device):
    big = 1 << 40
    for call, sizes in ((_route, dict(T=1 << 29, ld=big)), (_route_bwd, dict(T=1 << 29, old=big)),
                        (_combine, dict(T=1 << 29, cld=big)), (_combine_bwd, dict(T=1 << 29, dcld=big)),
                        (_act, dict(R=1 << 30, pld=big)), (_act_bwd, dict(R=1 << 30, dpld=big))):
        assert call(**sizes) == INVALID
        assert b"_ld" in L.moe_last_error()


def test_binding_rejects_before_the_library():
    z = torch.zeros(4, 8)
    ids, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    u8 = torch.zeros(4, 64, dtype=torch.uint8)
    with pytest.raises(ValueError):            # not on a device
        moe.moe_route(z, 2)
    with pytest.raises(TypeError):
        moe.moe_route(z.half(), 2)
    with pytest.raises(TypeError):
        moe.moe_route(logits=[1.0], top_k=2)
    with pytest.raises(ValueError):
        moe.moe_route_backward(z, ids, w)
    with pytest.raises(ValueError):
        moe.moe_combine_routed(x, w, ids, 8)
    with pytest.raises(ValueError):
        moe.moe_combine_backward(x, x, w)
    with pytest.raises(ValueError):
        moe.moe_act_mxfp8(x, "swiglu")
    with pytest.raises(KeyError):
        moe.moe_act_mxfp8(x, "gelu")
    with pytest.raises(ValueError):
        moe.moe_act_mxfp8_backward(u8, u8[:, :2], x[:, :32], "swiglu")
    with pytest.raises(ValueError):
        moe.moe_wgrad_mxfp8(u8, u8[:, :2], x, (ids[0], ids[0], ids[0]), 4, 1, 4)


def test_route_workspace_of_no_tokens_holds_a_row():
    # without tokens one workgroup still writes its (empty) partial row
    for E in (1, 8, 40, 127, 256, 1024):
        assert moe.moe_route_workspace_bytes(0, E) == moe.moe_route_workspace_bytes(1, E)
        assert moe.moe_route_workspace_bytes(0, E) >= 520 + 8 * (E + 1)


def _refused(status):
    return status in (INVALID, UNSUPPORTED)


def _swapped(call, a, b, **kw):
    """Whether the call is refused with the two pointers as given and exchanged (alike)."""
    first, second = _refused(call(**kw)), _refused(call(**{**kw, a: kw[b], b: kw[a]}))
    assert first == second
    return first


def test_rows_that_interleave_without_sharing_a_byte_are_accepted(no_device):
    far, base = 1 << 40, 1 << 33
    # codes and scales side by side in rows of 144 bytes, h beside pre, all in one buffer
    assert not _refused(_act(q=base, qld=144, s=base + 128, sld=144))
    assert not _refused(_act(pre=base, pld=256, h=base + 256, hld=256, q=far, s=2 * far))
    assert _refused(_act(pre=base, pld=256, h=base + 240, hld=256, q=far, s=2 * far))    # 16 bytes of pre's row
    assert _refused(_act(pre=base, pld=256, h=base + 400, hld=256, q=far, s=2 * far))    # the next row of pre
    # rows of 528 bytes: pre [0, 256), h [256, 384), codes [384, 512), scales [512, 516)
    row = dict(pld=264, hld=264, qld=528, sld=528)
    assert not _refused(_act(pre=base, h=base + 256, q=base + 384, s=base + 512, **row))
    assert not _refused(_act(pre=base, h=base + 256, q=base + 384, s=base + 524, **row))
    assert _refused(_act(pre=base, h=base + 256, q=base + 384, s=base + 511, **row))
    assert _refused(_act(pre=base, h=base + 256, q=base + 384, s=base + 525, **row))     # over pre's next row
    assert _refused(_act(pre=base + 528 * 4, h=base + 256, q=base + 384, s=base + 525, **row))   # its first row
    assert not _refused(_act(pre=base + 528 * 5, h=base + 256, q=base + 384, s=base + 525, **row))
    # dpre beside h; one row after the other matrix's last
    for kw in (dict(dp=base, dpld=192, h=base + 256, hld=192), dict(dp=base, dpld=192, h=base + 3 * 384 + 256, hld=64)):
        assert not _refused(_act_bwd(q=far, s=2 * far, dh=3 * far, **kw))
    assert _refused(_act_bwd(q=far, s=2 * far, dh=3 * far, dp=base, dpld=192, h=base + 3 * 384 + 240, hld=64))
    # dlogits beside logits, the other way round too
    assert not _swapped(_route_bwd, "z", "out", z=base, ld=16, out=base + 32, old=16)
    assert _swapped(_route_bwd, "z", "out", z=base, ld=16, out=base + 28, old=16)
    assert _swapped(_route_bwd, "z", "out", z=base, ld=15, out=base + 32, old=15)
    # a block that lies in one gap of the rows, and one that reaches the next row
    assert not _refused(_combine_bwd(dc=base, dcld=128, dw=base + 128, dy=far, c=2 * far, w=3 * far, ids=4 * far))
    assert not _refused(_combine_bwd(dc=base, dcld=128, dw=base + 224, dy=far, c=2 * far, w=3 * far, ids=4 * far))
    assert _refused(_combine_bwd(dc=base, dcld=128, dw=base + 228, dy=far, c=2 * far, w=3 * far, ids=4 * far))
    assert _refused(_combine_bwd(dc=base, dcld=128, dw=base - 28, dy=far, c=2 * far, w=3 * far, ids=4 * far))
    # rows of unequal strides have to lie apart
    assert _refused(_combine_bwd(dc=base, dcld=128, c=base + 128, cld=256, dy=far, dw=2 * far, w=3 * far, ids=4 * far))


def test_overlap_rule_is_that_of_the_bytes(no_device):
    """The dlogits / logits check against the set of bytes, at every offset around each other."""
    T, E, base = 3, 2, 1 << 33
    for ld in (2, 3, 5):
        rows = {base + 4 * (t * ld + e) for t in range(T) for e in range(E)}
        for off in range(-4 * ld, 4 * ld + 1):
            mine = {base + 4 * (off + t * ld + e) for t in range(T) for e in range(E)}
            st = _route_bwd(z=base, ld=ld, T=T, E=E, k=1, out=base + 4 * off, old=ld, ids=1 << 40, dw=1 << 41,
                            counts=1 << 42, n=1 << 43, dl=1 << 44)
            assert _refused(st) == bool(rows & mine), (ld, off)
