"""Norms of queries and keys over the whole range of bf16: a norm's result is a few units whatever the size of its input."""
import numpy as np
import pytest

from oracle import serving as S
from tests import _serving as V

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("D,rot,neighbours,pad", [(64, 64, False, 0), (128, 32, True, 0), (128, 128, False, 1), (256, 256, False, 0),
                                                  (256, 0, False, 3)])
def test_sizes_whose_squares_pass_32_bits(D, rot, neighbours, pad):
    """Heads of 1e-37 to 3e38 side by side, without an eps that would hide the small ones.  pad: elements that take the heads off
    16-byte alignment."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sub_bit_moe_amd import api
    dev = torch.device("cuda:0")
    rng = np.random.default_rng(D + rot)
    T, H = 9, 7
    x = rng.standard_normal((T, H, D))
    x *= np.exp2(rng.integers(-120, 125, (T, H, 1)))
    x[0, 0] /= np.abs(x[0, 0]).max() / 3e38
    x[1, :, ::2] *= 2.0 ** -30                           # some of a head's squares pass, or vanish, others not
    x = S.round_to(x, "bf16")
    assert np.isfinite(x).all()
    w = S.round_to(1 + 0.3 * rng.standard_normal(D), "bf16")
    pos = rng.integers(0, 300, T)
    wide = torch.zeros(T, H * D + pad, dtype=torch.bfloat16, device=dev)
    wide[:, pad:] = V.tensor(x.reshape(T, -1), "bf16", dev)
    q = wide[:, pad:].unflatten(1, (H, D))
    rope = api.rope_table(300, rot, device=dev) if rot else None
    weight = V.tensor(w, "bf16", dev)
    got_q, got_k = api.qk_norm_rope(q, q, weight, weight, V.i32(pos, dev), rope, eps=0.0, neighbours=neighbours)
    rows = rope.cpu().numpy()[pos] if rot else None
    ref = S.norm_rope(x, w, rows, rot, eps=0.0, neighbours=neighbours)
    # half a step of the output's; sums and products in 32 bits: at most D / 8 + 12 roundings of values no larger than a pair's norm
    top = np.abs(S.norm_rope(x, w, None, 0, eps=0.0)).max(-1, keepdims=True) * 2 ** 0.5
    bound = V.HALF["bf16"] * np.abs(ref) + (D / 8 + 12) * 2.0 ** -24 * top
    assert (np.abs(V.array(got_q) - ref) <= bound).all()
    assert np.array_equal(V.array(got_k), S.round_to(ref, "bf16"))


def test_no_head_reaches_its_neighbours():
    """Heads of zeros, with an infinity and with a NaN beside ordinary ones, of every width."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sub_bit_moe_amd import api
    dev = torch.device("cuda:0")
    for D in (64, 128, 256):
        q = torch.randn(4, 6, D, device=dev).bfloat16()
        clean, _ = api.qk_norm_rope(q, q, None, None, None, None)
        bad = q.clone()
        bad[0, 1] = 0
        bad[1, 2, 5], bad[2, 3, D - 1], bad[3, 0, 0] = float("inf"), float("nan"), 3e38
        got, _ = api.qk_norm_rope(bad, bad, None, None, None, None)
        same = torch.ones(4, 6, dtype=torch.bool, device=dev)
        for t, h in ((0, 1), (1, 2), (2, 3), (3, 0)):
            same[t, h] = False
        assert torch.equal(got[same], clean[same])
        assert not got[0, 1].any() and torch.isnan(got[2, 3]).all()
        assert torch.isnan(got[1, 2, 5]) and not got[1, 2, :5].any() and not got[1, 2, 6:].any()
        assert got[3, 0, 0] == D ** 0.5 if D != 128 else abs(float(got[3, 0, 0]) - D ** 0.5) < 2.0 ** -8 * 16
