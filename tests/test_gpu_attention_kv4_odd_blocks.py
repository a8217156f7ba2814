"""Blocks of values that the call's type does not hold (NaN's scale, scales past the writer's for the type): what they become
reaches the rows that see their token, in their own 32 dimensions, and nothing else."""
import numpy as np
import pytest

from oracle import serving as S
from tests import _serving as V
from tests.test_gpu_attention_kv4 import _case, _run

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


@pytest.mark.parametrize("dtype,scales", [("fp16", (141, 142, 147, 200, 254, 255)), ("bf16", (253, 254, 255))])
@pytest.mark.parametrize("D,H,Hk,kv,n", [(64, 2, 1, 75, 50), (128, 3, 3, 40, 40), (256, 1, 1, 33, 30),       # few rows
                                         (64, 2, 2, 300, 200), (128, 2, 1, 260, 150), (256, 1, 1, 200, 140)])  # tiles of rows
def test_a_value_that_the_type_does_not_hold(dev, dtype, scales, D, H, Hk, kv, n):
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(D + kv)
    bs = 16
    q, data, table = _case(rng, [kv], [n], H, Hk, D, bs, dtype)
    call = lambda c: _run(api, dev, q, c, bs, table, [kv], [n], dtype, scale=0.03)      # noqa: E731
    clean, clean_lse = (V.array(a) for a in call(data))
    for at in (kv - n // 2, kv - 3, kv - n + 1):       # tokens that some rows see and some do not
        for scale in scales:
            kc, ks, vc, vs = (a.copy() for a in S.split_pages(data, bs, D))
            page, row, block = table[0, at // bs], at % bs, int(rng.integers(0, D // 32))
            dims = slice(32 * block, 32 * block + 32)
            vc[page, :, row, dims] = rng.integers(0, 16, (Hk, 32))
            vc[page, :, row, 32 * block:32 * block + 4] = [0, 8, 1, 15]
            vs[page, :, row, block] = scale
            odd = S.pages(kc, ks, vc, vs)
            out, lse = (V.array(a) for a in call(odd))
            assert np.array_equal(lse, clean_lse)
            sees = np.arange(kv - n, kv) >= at
            other = np.ones(D, bool)
            other[dims] = False
            assert np.array_equal(out[~sees], clean[~sees])
            assert np.array_equal(out[:, :, other], clean[:, :, other])
            # what the rows that see it read, its own 32 dimensions
            held = S.round_to(S.values(vc, vs)[page, :, row, dims], dtype)             # [Hk, 32]
            held = np.repeat(held, H // Hk, 0)[None].repeat(int(sees.sum()), 0)
            got = out[sees][:, :, dims]
            assert np.array_equal(np.isnan(got), np.isnan(held))
            inf = np.isinf(held)
            assert np.array_equal(got[inf], held[inf])
            with np.errstate(all="ignore"):
                ref, ref_lse, weight = S.attention(q, odd, bs, table, [kv], [0, n], 0.03)
                kmax = np.linalg.norm(S.values(kc, ks), axis=-1).max()
                bound = V.attention_bound(ref, ref_lse, weight, q, kmax, 0.03, kv, dtype)[0]
                far = np.abs(got - ref[sees][:, :, dims])[np.isfinite(held)]
                assert (far <= bound[sees][:, :, dims][np.isfinite(held)]).all()


def test_odd_blocks_of_two_tokens_meet(dev):
    """An infinity of each sign is a NaN of the rows that see both, an infinity of those that see the first."""
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(5)
    D, bs = 64, 16
    for kv, n in ((60, 60), (200, 150)):
        q, data, table = _case(rng, [kv], [n], 1, 1, D, bs, "fp16")
        kc, ks, vc, vs = (a.copy() for a in S.split_pages(data, bs, D))
        for at, code in ((kv - 30, 7), (kv - 9, 15)):
            vc[table[0, at // bs], 0, at % bs, :32], vs[table[0, at // bs], 0, at % bs, 0] = code, 160
        out, _ = _run(api, dev, q, S.pages(kc, ks, vc, vs), bs, table, [kv], [n], "fp16", scale=0.03)
        out = V.array(out)[:, 0]
        first = n - 30
        assert np.isfinite(out[:first]).all() and np.isfinite(out[:, 32:]).all()
        assert (out[first:n - 9, :32] == np.inf).all() and np.isnan(out[n - 9:, :32]).all()
