"""Helpers shared by the tests of the block entry points (moe_block.h)."""

import numpy as np
import torch

import synth

U = 2.0 ** -24  # half a step of fp32
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}  # half a step, relative


def f64(t):
    return t.detach().float().cpu().double().numpy()


def close(got, ref, tol, what=""):
    """|got - ref| <= tol elementwise, with equal NaN and infinity masks."""
    got, ref, tol = (np.asarray(v, dtype=np.float64) for v in (got, ref, tol))
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: NaN positions differ"
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]), f"{what}: infinities differ"
    ok = ~np.isnan(ref) & ~inf
    err, bound = np.abs(got - ref)[ok], np.broadcast_to(tol, ref.shape)[ok]
    assert (err <= bound).all(), f"{what}: worst {np.max(err / np.maximum(bound, 1e-300)):.3g} of the tolerance"


def normal(shape, seed, tag, dtype="bf16", std=1.0, device="cuda"):
    t = torch.randn(shape, generator=synth.gen(seed, tag), dtype=torch.float32) * std
    return t.to(DT[dtype]).to(device)


def rng_state(seed, offset, device="cuda"):
    wrap = lambda v: v - (1 << 64) if v >= 1 << 63 else v  # noqa: E731
    return torch.tensor([wrap(seed), wrap(offset)], dtype=torch.int64, device=device)


def strided(t, extra):
    """The same values in rows `extra` elements longer, NaN bytes behind them."""
    wide = torch.full((t.shape[0], t.shape[1] + extra), -1 if t.dtype == torch.uint8 else float("nan"),
                      dtype=torch.float32).to(t.dtype).to(t.device) if t.dtype != torch.uint8 else \
        torch.full((t.shape[0], t.shape[1] + extra), 255, dtype=torch.uint8, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]
