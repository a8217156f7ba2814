"""Inputs that the serving tests share."""
import numpy as np
import torch

from oracle import serving as S

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
HALF = {k: torch.finfo(v).eps / 2 for k, v in DT.items()}      # a rounding's largest relative error


def tensor(x, dtype, dev):
    """float64 values that the type holds exactly."""
    return torch.from_numpy(np.ascontiguousarray(x)).to(DT[dtype]).to(dev)


def array(t):
    return t.detach().double().cpu().numpy()


def i32(v, dev):
    return torch.from_numpy(np.ascontiguousarray(v, np.int32)).to(dev)


def random_cache(rng, n_blocks, heads, bs, dim, dtype, spread=0.4):
    """Records of normally distributed rows, quantised by the oracle."""
    rows = []
    for _ in range(2):
        x = rng.standard_normal((n_blocks, heads, bs, dim)) * np.exp(spread * rng.standard_normal((n_blocks, heads, bs, 1)))
        rows += S.quantise(S.round_to(x, dtype), dtype)
    return S.pages(*rows)


def shuffled_table(rng, kv_lens, bs, extra=2, spare=3):
    """(block table with -1 where nothing is held, n_blocks), blocks in random order."""
    held = [-(-n // bs) for n in kv_lens]
    n_blocks = max(sum(held) + spare, 1)
    ids = rng.permutation(n_blocks)
    table = np.full((len(kv_lens), max(held, default=0) + extra), -1, np.int32)
    at = 0
    for r, h in enumerate(held):
        table[r, :h] = ids[at:at + h]
        at += h
    return table, n_blocks


def attention_bound(ref, lse, weight, q, kmax, scale, n, dtype):
    """How far out and lse may be from 64 bits: the output's rounding and that of
    the probabilities (half a step each), scores summed in fp32 (D + 2 terms of
    at most |q||k|), exponentials and sums in fp32, and probabilities 2^-32 below
    the largest dropped."""
    h = HALF[dtype]
    D = q.shape[-1]
    ds = abs(scale) * 2.0 ** -24 * (D + 2) * np.linalg.norm(q, axis=-1) * kmax + 2.0 ** -21 * (1 + np.abs(np.where(np.isfinite(lse), lse, 0)))
    dw = h + 2 * ds + 2.0 ** -22 * np.log2(n + 2) + n * 2.0 ** -32
    tiny = 2.0 ** -25 if dtype == "fp16" else 2.0 ** -134
    return h * np.abs(ref) + 1.05 * dw[..., None] * weight + tiny, 2 * ds + 2.0 ** -21
