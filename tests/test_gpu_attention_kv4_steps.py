"""Steps that hold single tokens and prompts at once, both with their token axes shared out, against 64 bits."""
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


@pytest.mark.parametrize("kv,new,H,Hk,D,bs,dtype", [
    # heads of 64: fewer tiles of rows than the chip holds at once, and more
    ([900, 2500, 40], [900, 1, 1], 64, 64, 64, 16, "bf16"),
    ([1100, 2500, 40], [1100, 1, 1], 64, 64, 64, 16, "fp16"),
    # parts of both kinds to join, in every width
    ([9900, 20000, 0, 7000, 300], [140, 1, 0, 1, 300], 1, 1, 64, 32, "fp16"),
    ([9900, 20000, 0, 7000, 300], [140, 1, 1, 2, 300], 2, 1, 128, 16, "bf16"),
    ([4000, 6000, 5, 300], [70, 1, 5, 200], 2, 1, 256, 64, "fp16")])
def test_single_tokens_beside_prompts(dev, kv, new, H, Hk, D, bs, dtype):
    """One workspace for all calls: the same bits each time, eagerly, behind a step of other requests, and replayed."""
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(kv[0] + D)
    q, data, table = _case(rng, kv, new, H, Hk, D, bs, dtype)
    ws = api.alloc_attention_workspace(len(kv), max(sum(new), 8), H, Hk, D, dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    args = (api, dev, q, data, bs, table, kv, new, dtype)
    out, lse = _run(*args, workspace=ws, error=err)
    _check(out, lse, q, data, bs, table, kv, new, dtype)
    other = _case(rng, [3000, 17], [1, 3], H, Hk, D, bs, dtype)
    for _ in range(2):
        o, s = _run(api, dev, other[0], other[1], bs, other[2], [3000, 17], [1, 3], dtype, workspace=ws)
        _check(o, s, *other[:2], bs, other[2], [3000, 17], [1, 3], dtype)
        again = _run(*args, workspace=ws, error=err)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    # recorded, with eager steps of the other requests between the replays
    cache = api.KVCache(torch.from_numpy(np.ascontiguousarray(data)).to(dev), bs, D)
    t, lens = V.i32(table, dev), V.i32(kv, dev)
    cu = V.i32(np.concatenate([[0], np.cumsum(new)]), dev)
    x = V.tensor(q, dtype, dev)
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.attention_kv4(x, cache, t, lens, cu_q=cu, out=o2, lse=l2, workspace=ws, error=err)
    for _ in range(3):
        o2.zero_(), l2.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o2, out) and torch.equal(l2, lse)
        _run(api, dev, other[0], other[1], bs, other[2], [3000, 17], [1, 3], dtype, workspace=ws)
    torch.cuda.synchronize()
    assert not ws[:24576].any() and int(err) == 0
