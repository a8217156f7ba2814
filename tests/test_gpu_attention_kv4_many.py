"""More requests than a wave has lanes, long ones among them whose token axes are shared out, and key heads of more than 128 query
heads, against 64 bits."""
import numpy as np
import pytest

from tests import _serving as V
from tests.test_gpu_attention_kv4 import _case, _check, _run

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


@pytest.mark.parametrize("R,H,Hk,D,bs,dtype", [(70, 1, 1, 64, 16, "fp16"), (70, 2, 1, 128, 32, "bf16"), (70, 1, 1, 256, 64, "fp16"),
                                               (300, 2, 2, 64, 16, "bf16"), (300, 1, 1, 128, 16, "fp16"),
                                               (300, 1, 1, 256, 16, "bf16")])
def test_shared_axes_among_many_requests(dev, R, H, Hk, D, bs, dtype):
    """Two long single tokens and two prompts behind long contexts, in parts all of them, first, last and in the midst of requests of
    a token or none."""
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(R + D)
    new = rng.integers(0, 2, R)
    kv = new + rng.integers(0, 30, R)
    kv[rng.random(R) < 0.3] = 0
    for r, n, k in ((0, 1, 9000), (R // 2, 140, 5000), (R - 60, 1, 7001), (R - 1, 137, 4200)):
        new[r], kv[r] = n, k
    q, data, table = _case(rng, kv, list(new), H, Hk, D, bs, dtype)
    ws = api.alloc_attention_workspace(R, int(new.sum()), H, Hk, D, dev)
    first, err = None, torch.zeros(1, dtype=torch.int32, device=dev)
    for _ in range(3):                      # whoever ends last: the same bits
        out, lse = _run(api, dev, q, data, bs, table, list(kv), list(new), dtype, workspace=ws, error=err)
        assert first is None or (torch.equal(first[0], out) and torch.equal(first[1], lse))
        first = out, lse
    assert not ws[:24576].any() and int(err) == 0
    _check(out, lse, q, data, bs, table, list(kv), list(new), dtype)


@pytest.mark.parametrize("H,Hk,D,dtype", [(129, 1, 64, "fp16"), (260, 2, 128, "bf16"), (257, 1, 256, "fp16"), (128, 1, 128, "fp16")])
@pytest.mark.parametrize("kv", [[1, 0, 200, 65], [6000], [40] * 70 + [3000]])
def test_single_tokens_of_many_heads(dev, H, Hk, D, dtype, kv):
    """One token each and no cu_q, a key head's rows more than the few-row kernel takes (and just as many)."""
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(H + D + len(kv))
    q, data, table = _case(rng, kv, [1] * len(kv), H, Hk, D, 16, dtype)
    out, lse = _run(api, dev, q, data, 16, table, kv, None, dtype)
    _check(out, lse, q, data, 16, table, kv, None, dtype)
    out2, lse2 = _run(api, dev, q, data, 16, table, kv, [1] * len(kv), dtype)
    _check(out2, lse2, q, data, 16, table, kv, [1] * len(kv), dtype)
