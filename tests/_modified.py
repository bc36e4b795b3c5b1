"""Helpers of the modified-score and FP8 chunk attention tests: tolerance, inputs, calls."""

from __future__ import annotations

import numpy as np
import torch

# Half a step of a rounding, relative to the value.
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# A score's error: a dot product of d <= 128 terms in fp32 with sum |q k| scale <= 25 is off by at
# most 128 * 2^-24 * 25 = 2e-4; a cap adds 7e-6 of the score (the kernels' tanh), 1.8e-4 of 25; the two
# together stay below 5e-4, and a weight's relative error (numerator and sum) below twice that.
SCORE = 1e-3


def check(got: torch.Tensor, ref: np.ndarray, dev: np.ndarray, weights, keys: int, label: str = "") -> None:
    """|got - ref| <= output rounding * |ref| + weight error * dev + accumulation.

    weights: the type in which the softmax weights enter the P V product.  A relative error of at most
    e in every weight moves the output by at most e * dev (dev: the weighted mean deviation of the
    values); an fp32 sum of `keys` terms is off by at most keys * 2^-24 * sum w|v| <= .. * (|ref| + dev).
    """
    g = got.detach().double().cpu().numpy()
    assert g.shape == ref.shape, label
    assert np.isfinite(g).all(), f"{label}: non-finite output"
    acc = keys * 2.0 ** -24
    tol = (HALF[got.dtype] + acc) * np.abs(ref) + (HALF[weights] * 1.01 + SCORE + acc) * dev + 1e-7
    over = np.abs(g - ref) - tol
    assert over.size == 0 or over.max() <= 0, (
        f"{label}: off by {np.abs(g - ref).flat[over.argmax()]:.3e}, allowed {tol.flat[over.argmax()]:.3e} "
        f"({int((over > 0).sum())} of {over.size} elements)")


def slopes_of(heads: int) -> torch.Tensor:
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)], dtype=torch.float32)


def i32(values) -> torch.Tensor:
    return torch.tensor(values, dtype=torch.int32)


def cuda(x):
    return x.cuda() if isinstance(x, torch.Tensor) else x
