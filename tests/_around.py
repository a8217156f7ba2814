"""Inputs and bounds that the tests of the operators around the experts share."""
import numpy as np
import torch

from oracle import around as A
from oracle import serving as S
from tests import _serving as V

DT = {**V.DT, "fp32": torch.float32}
HALF = {**V.HALF, "fp32": 2.0 ** -24}


def held(x, dtype):
    """What the type holds of x, as float64."""
    return np.float64(np.float32(x)) if dtype == "fp32" else S.round_to(x, dtype)


def tensor(x, dtype, dev):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DT[dtype]).to(dev)


def norm_case(rng, T, D, k=1, dtype="bf16", x_type=None, r_type=None, gates=True, weight=True):
    """(x, gates, residual, weight) as their types hold them."""
    x = held(rng.standard_normal((T * k, D)) * np.exp(0.5 * rng.standard_normal((T * k, 1))), x_type or dtype)
    g = held(rng.random((T, k)) + 0.05, "fp32") if gates or k > 1 else None
    r = held(3 * rng.standard_normal((T, D)), r_type or dtype) if r_type != "none" else None
    return x, g, r, held(1 + 0.3 * rng.standard_normal(D), dtype) if weight else None


def norm_bounds(x, g, r, w, eps, k, dtype, r_type):
    """(y, how far from it 16-bit results may be, h, how far residual_out may be): a rounding of half a step each, k + 1
    roundings of 2^-24 in the sum (of fp32 numbers as they are: x and gates are given), and four in y = h * inv * w."""
    h, size = A.state(x, g, r)
    y = A.rms_norm(h, w, eps)
    dh = 2.0 ** -24 * (k + 1) * size
    mean = (h * h).mean(1, keepdims=True) + eps
    root = np.sqrt(mean)
    # the mean's error from h's, relative
    dm = (2 * np.abs(h) * dh + dh * dh).mean(1, keepdims=True) / mean
    ww = 1.0 if w is None else np.abs(w)
    dy = ww * dh / root * (1 + dm) + np.abs(y) * (dm + 5 * 2.0 ** -24)
    tiny = {"bf16": 2.0 ** -133, "fp16": 2.0 ** -24, "fp32": 2.0 ** -149}
    return (y, HALF[dtype] * np.abs(y) * 1.001 + 1.01 * dy + tiny[dtype], h,
            HALF[r_type] * np.abs(h) * 1.001 + 1.01 * dh + tiny[r_type])


def logits_case(rng, rows, vocab, dtype="fp32", spread=2.5):
    """Logits with a few likely tokens and some that are banned."""
    l = spread * rng.standard_normal((rows, vocab)) + 8 * rng.random((rows, vocab)) ** 60
    l[rng.random((rows, vocab)) < 0.01] = -np.inf
    l[:, rng.integers(vocab)] = 1.0
    return held(l, dtype)
