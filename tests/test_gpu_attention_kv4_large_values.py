"""Values near bf16's largest: an output is a mean of values, so it is finite wherever their sum is."""
import numpy as np
import pytest

from oracle import serving as S
from tests import _serving as V
from tests.test_gpu_attention_kv4 import _case, _check, _run

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("D,H,Hk,kv,new,scale_byte", [
    (64, 2, 1, [1, 2, 3], [1, 1, 1], 252), (128, 8, 2, [1, 7, 40], [1, 2, 30], 246), (256, 1, 1, [900], [1], 240),
    (64, 1, 1, [150], [150], 245), (128, 2, 1, [400], [200], 243), (256, 1, 1, [500, 3], [140, 1], 243)])
def test_large_values(D, H, Hk, kv, new, scale_byte):
    """Every block of values under one scale, 2^(scale_byte - 127): magnitudes up to 6 times that, and few enough of them
    that their sum stays below 2^128."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sub_bit_moe_amd import api
    assert 6 * 2.0 ** (scale_byte - 127) * (max(kv) if max(kv) > 7 else 1) < 2.0 ** 128 - 2.0 ** 104
    rng = np.random.default_rng(D + sum(kv))
    q, data, table = _case(rng, kv, new, H, Hk, D, 16, "bf16")
    kc, ks, vc, vs = S.split_pages(data, 16, D)
    data = S.pages(kc, ks, vc, np.full_like(vs, scale_byte))
    out, lse = _run(api, torch.device("cuda:0"), q, data, 16, table, kv, new, "bf16")
    _check(out, lse, q, data, 16, table, kv, new, "bf16")
