"""Pins of the serving oracle: the 4-bit format against its definition, and the
parts against one another."""
import numpy as np
import pytest
import torch

from oracle import serving as S


def test_round_to_is_torch_rounding_of_exact_values():
    rng = np.random.default_rng(0)
    x = rng.standard_normal(4096).astype(np.float32) * np.exp2(rng.integers(-30, 14, 4096))
    x = x.astype(np.float32)
    for name, dt in (("bf16", torch.bfloat16), ("fp16", torch.float16)):
        ref = torch.from_numpy(x).to(dt).double().numpy()
        assert np.array_equal(S.round_to(x.astype(np.float64), name), ref)
    # one rounding, not two: 1 + 2^-8 + 2^-40 is above the border of bf16's 1 and 1 + 2^-7
    assert S.round_to(1 + 2.0 ** -8 + 2.0 ** -40, "bf16") == 1 + 2.0 ** -7
    assert S.round_to(1 + 2.0 ** -8, "bf16") == 1.0


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_quantise_is_within_half_a_step(dtype):
    rng = np.random.default_rng(1)
    x = S.round_to(rng.standard_normal((512, 128)) * np.exp(3 * rng.standard_normal((512, 1))), dtype)
    codes, scales = S.quantise(x, dtype)
    v = S.values(codes, scales)
    unit = np.repeat(np.ldexp(1.0, scales.astype(int) - 127), 32, -1)
    a = np.abs(x) / unit
    step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
    assert (np.abs(v - x) <= step / 2 * unit).all()
    # the scale is the smallest at which nothing passes 7
    top = np.abs(x).reshape(512, 4, 32).max(-1)
    two = np.ldexp(1.0, scales.astype(int) - 127)
    assert (top <= 7 * two).all() and (top > 3.5 * two).all()


def test_quantise_borders_and_oddities():
    one = np.zeros(32)
    one[:16] = [7.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -5.0, 0.2500001, 6.9, -0.0, 5.0001, 4.9]
    codes, scales = S.quantise(one[None], "bf16")
    assert scales[0, 0] == 127
    assert codes[0, :16].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 8, 10, 14, 1, 7, 8, 7, 6]
    for top, s in ((7.0, 127), (7.01, 128), (3.5, 126), (3.51, 127), (0.0, 1), (2.0 ** -140, 1), (3e38, 252)):
        x = np.zeros((1, 32))
        x[0, 3] = top
        assert S.quantise(x, "bf16")[1][0, 0] == s, top
    x = np.zeros((1, 64))
    x[0, 40] = 65504.0
    assert S.quantise(x, "fp16")[1].tolist() == [[1, 140]] and S.values(*S.quantise(x, "fp16"))[0, 40] == 49152
    x[0, 3] = np.inf
    codes, scales = S.quantise(x, "bf16")
    assert scales[0, 0] == 255 and not codes[0, :32].any() and np.isnan(S.values(codes, scales)[0, :32]).all()


def test_pages_round_trip():
    rng = np.random.default_rng(2)
    kc, vc = rng.integers(0, 16, (2, 3, 2, 16, 64)).astype(np.uint8)
    ks, vs = rng.integers(0, 256, (2, 3, 2, 16, 2)).astype(np.uint8)
    data = S.pages(kc, ks, vc, vs)
    assert data.shape == (3, 2, 16 * 64 * 17 // 16)
    for got, want in zip(S.split_pages(data, 16, 64), (kc, ks, vc, vs)):
        assert np.array_equal(got, want)


def test_attention_of_one_token_is_its_value_and_gradients_of_lse():
    """One visible token: out = v, lse = s.  And d lse / d q = scale * sum p k, by differences."""
    rng = np.random.default_rng(3)
    bs, D = 16, 64
    kc, vc = rng.integers(0, 16, (2, 3, 1, bs, D)).astype(np.uint8)
    ks, vs = rng.integers(120, 128, (2, 3, 1, bs, 2)).astype(np.uint8)
    data = S.pages(kc, ks, vc, vs)
    q = rng.standard_normal((1, 1, D))
    table = np.array([[2, 0, 1]])
    out, lse, _ = S.attention(q, data, bs, table, [1], None, 0.3)
    assert np.allclose(out[0, 0], S.values(vc, vs)[2, 0, 0], rtol=1e-14)
    k = S.values(kc, ks)[table[0], 0].reshape(-1, D)
    assert np.allclose(lse, 0.3 * q[0, 0] @ k[0], rtol=1e-12)
    h = 1e-5
    e = np.zeros_like(q)
    e[0, 0, 7] = h
    up, dn = (S.attention(q + s * e, data, bs, table, [40], None, 0.3)[1][0, 0] for s in (1, -1))
    z = 0.3 * k[:40] @ q[0, 0]
    p = np.exp(z - z.max())
    assert abs((up - dn) / (2 * h) - 0.3 * (p / p.sum()) @ k[:40, 7]) < 1e-7


def test_plan_small():
    table = np.full((3, 4), -1, np.int32)
    table[0, 0], table[2, :2] = 5, (7, 8)
    t, slots, pos, req, cu, kv, left = S.plan([10, 0, 32], [8, 0, 1], [1, 2, 3, 4], table, 16, 11)
    assert t.tolist() == [[5, 4, -1, -1], [-1, -1, -1, -1], [7, 8, 3, -1]] and left == 2
    assert slots.tolist() == [90, 91, 92, 93, 94, 95, 64, 65, 48, -1, -1] and cu.tolist() == [0, 8, 8, 9]
    assert pos.tolist() == [10, 11, 12, 13, 14, 15, 16, 17, 32, 0, 0] and kv.tolist() == [18, 0, 33]
    assert req.tolist() == [0] * 8 + [2, -1, -1]
