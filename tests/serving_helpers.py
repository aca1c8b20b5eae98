"""Inputs and error bounds shared by the serving operators' GPU tests."""

from __future__ import annotations

import numpy as np
import torch

BF16, FP16 = 2.0 ** -8, 2.0 ** -11  # half a step, relative


def randn(rng, *shape, scale=1.0) -> torch.Tensor:
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16).cuda()


def ints(a) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def assert_within(got: np.ndarray, ref: np.ndarray, tol: np.ndarray, what: str) -> None:
    """|got - ref| <= tol everywhere; infinities and NaN have to be the same."""
    fine = np.isfinite(ref)
    assert np.array_equal(np.isnan(ref), np.isnan(got)), what
    assert np.array_equal(ref[np.isinf(ref)], got[np.isinf(ref)]), what
    off = np.abs(np.where(fine, got, 0) - np.where(fine, ref, 0)) - np.where(fine, tol, 0)
    assert off.max(initial=0) <= 0, f"{what}: {off.max()} beyond the bound at {np.unravel_index(off.argmax(), off.shape)}"


def check_attention(o, lse, ref, p_round: float, what: str = "", floor: float = 0.0) -> None:
    """Outputs [..., n, H, 128] and lse [..., H, n] against the oracle's (out, lse, a, z).

    A score is a sum of 128 fp32 products and two fp32 scalings of it: off by at most 140 * 2^-24 z, z the scaled
    sum of their sizes.  exp2, the row sums over keys, warps and parts, and the division stay within 2^-17.  Both
    move the weights of numerator and denominator, hence twice; the weights' own rounding p_round and the values'
    share a = sum w |v| bound what reaches the output, which is rounded once.  floor: what weights too small for
    p_round's relative bound can add up to."""
    r, e, a, z = ref
    d = 140 * 2.0 ** -24 * z + 2.0 ** -17
    per_row = np.moveaxis(d, -2, -1)[..., None]  # [..., H, n] -> [..., n, H, 1]
    o = f64(o)
    assert_within(o, r, BF16 * np.abs(r) + a * (p_round + 2 * per_row) * (1 + BF16) + floor + 1e-30, f"output {what}")
    if lse is not None:
        assert_within(f64(lse), e, d + 2.0 ** -22 * np.abs(np.where(np.isfinite(e), e, 0)), f"lse {what}")
