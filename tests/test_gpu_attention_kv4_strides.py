"""Strides that no address is made from."""
import numpy as np
import pytest

from tests import _serving as V
from tests.test_gpu_attention_kv4 import _case

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("T,H", [(1, 4), (3, 1), (1, 1), (150, 1)])
def test_one_token_or_one_head_of_any_stride(T, H):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sub_bit_moe_amd import api
    dev = torch.device("cuda:0")
    rng = np.random.default_rng(T + H)
    D, bs = 64, 16
    q, data, table = _case(rng, [T + 70], [T], H, 1, D, bs, "fp16")
    q = V.tensor(q, "fp16", dev)
    odd = q.as_strided((T, H, D), (H * D if T > 1 else 5, D if H > 1 else 3, 1))
    args = api.KVCache(torch.from_numpy(data).to(dev), bs, D), V.i32(table, dev), V.i32([T + 70], dev)
    cu = V.i32([0, T], dev)
    assert torch.equal(api.attention_kv4(odd, *args, cu_q=cu), api.attention_kv4(q, *args, cu_q=cu))
