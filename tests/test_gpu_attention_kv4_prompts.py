"""Attention of many rows over the 4-bit cache, shared-out token axes and their joins, against 64 bits."""
import numpy as np
import pytest

from oracle import serving as S
from tests import _serving as V
from tests.test_gpu_attention_kv4 import _case, _check, _run

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D,bs,H,Hk", [(64, 16, 1, 1), (64, 64, 6, 2), (128, 16, 4, 1), (128, 128, 2, 2), (256, 16, 5, 1),
                                       (256, 64, 2, 2)])
def test_rows_around_a_workgroups(dev, dtype, D, bs, H, Hk):
    """New tokens that make 127, 128, 129 and 257 rows or so, with and without context, beside single tokens."""
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(D + bs + H)
    g = H // Hk
    new = [-(-n // g) for n in (127, 128, 129, 257)] + [1, 0, 200]
    kv = [new[0], new[1] + 70, new[2] + 1, new[3] + 333, 90, 12, 100]          # the last has more rows than tokens
    q, data, table = _case(rng, kv, new, H, Hk, D, bs, dtype)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = _run(api, dev, q, data, bs, table, kv, new, dtype, error=err)
    _check(out, lse, q, data, bs, table, kv, new, dtype)
    assert int(err) == 0


@pytest.mark.parametrize("kv,n,H,Hk,D,bs,dtype", [
    (70000, 1, 2, 1, 64, 32, "bf16"),       # several hundred parts of single tokens: joins of joins of joins
    (5000, 1, 3, 1, 256, 16, "fp16"),
    (9900, 140, 1, 1, 64, 16, "fp16"),      # rows of a prompt whose tokens are split
    (7000, 33, 4, 1, 128, 32, "bf16"),
    (2600, 67, 2, 1, 256, 16, "fp16"),
    (17000, 65, 2, 1, 256, 128, "bf16")])   # more than 64 parts
def test_shared_token_axes(dev, kv, n, H, Hk, D, bs, dtype):
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(kv)
    q, data, table = _case(rng, [kv], [n], H, Hk, D, bs, dtype)
    ws = api.alloc_attention_workspace(1, n, H, Hk, D, dev)
    first, err = None, torch.zeros(1, dtype=torch.int32, device=dev)
    for _ in range(3):                      # whoever ends last: the same bits
        out, lse = _run(api, dev, q, data, bs, table, [kv], [n], dtype, workspace=ws, error=err)
        assert first is None or (torch.equal(first[0], out) and torch.equal(first[1], lse))
        first = out, lse
    assert not ws[:24576].any() and int(err) == 0             # ready for the next call
    _check(out, lse, q, data, bs, table, [kv], [n], dtype)


def test_many_requests_with_prompts(dev):
    """More requests than a wave has lanes, and than a workgroup, single tokens and prompts in turn."""
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(8)
    for R in (63, 64, 65, 300):
        new = np.where(rng.random(R) < 0.08, rng.integers(65, 150, R), rng.integers(0, 3, R))
        kv = new + rng.integers(0, 40, R)
        q, data, table = _case(rng, kv, list(new), 2, 1, 64, 16, "fp16")
        out, lse = _run(api, dev, q, data, 16, table, list(kv), list(new), "fp16")
        _check(out, lse, q, data, 16, table, list(kv), list(new), "fp16")


@pytest.mark.parametrize("D", [64, 128, 256])
def test_hidden_tokens_of_prompts_may_hold_anything(dev, D):
    """As for single tokens: what a row does not see takes no part, in tiles that some rows see whole, others in part."""
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(D)
    kv, new, H, Hk, bs = [700, 300, 150], [200, 300, 150], 1, 1, 16
    q, data, table = _case(rng, kv, new, H, Hk, D, bs, "bf16")
    kc, ks, vc, vs = (a.copy() for a in S.split_pages(data, bs, D))
    free = sorted(set(range(data.shape[0])) - set(table[table >= 0].tolist()))
    ks[free], vs[free] = 255, 255
    ks[table[0, 43], :, 12:], vs[table[0, 43], :, 12:] = 255, 255      # behind request 0's 700 tokens
    vs[table[1, 6], 0, 4, 1] = 255                                     # request 1, token 100: a value
    ks[table[1, 12], 0, 8, 0] = 255                                    # request 1, token 200: a key
    table = table.copy()
    table[0, 3], table[2, 0] = 10 ** 6, -5                             # 16 tokens that no row sees
    data = S.pages(kc, ks, vc, vs)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = _run(api, dev, q, data, bs, table, kv, new, "bf16", error=err)
    assert int(err) == 1
    _check(out, lse, q, data, bs, table, kv, new, "bf16")
    got = V.array(out)[200:500, 0]
    assert not np.isnan(got[:100]).any() and np.isnan(got[100:, 32:64]).all() and not np.isnan(got[100:200, :32]).any()
    assert np.isnan(got[200:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_queries_of_every_size(dev, dtype):
    """Rows that differ by powers of two, with outliers, of zeros, and rows with an infinity or a NaN, which stay alone."""
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(3)
    for D, n in ((64, 150), (128, 150), (128, 3), (256, 131)):
        kv, H, Hk, bs = n + 90, 1, 1, 32
        q, data, table = _case(rng, [kv], [n], H, Hk, D, bs, dtype)
        small = 2.0 ** -9
        q = q * np.exp2(rng.integers(-6, 3, (n, 1, 1)))
        q[1::7, :, 5] *= 64
        q[2] = 0
        q[1] *= small
        q = S.round_to(q, dtype)
        out, lse = _run(api, dev, q, data, bs, table, [kv], [n], dtype)
        _check(out, lse, q, data, bs, table, [kv], [n], dtype)
        bad = q.copy()
        bad[0, 0, D - 1], bad[n - 1, 0, 3] = np.inf, np.nan
        out2, lse2 = _run(api, dev, bad, data, bs, table, [kv], [n], dtype)
        for at in (0, n - 1):
            assert torch.isnan(out2[at]).all() and torch.isnan(lse2[at]).all()
        assert torch.equal(out2[1:n - 1], out[1:n - 1]) and torch.equal(lse2[1:n - 1], lse[1:n - 1])


def test_scales(dev):
    """A scale of zero (every seen token alike, the hidden ones not), below zero, and one that makes scores huge."""
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(4)
    kv, new, H, Hk, D, bs = [260, 40], [150, 1], 1, 1, 128, 16
    for dtype, scale in (("bf16", 0.0), ("fp16", 0.0), ("bf16", -0.7), ("fp16", 25.0)):
        q, data, table = _case(rng, kv, new, H, Hk, D, bs, dtype)
        out, lse = _run(api, dev, q, data, bs, table, kv, new, dtype, scale=scale)
        _check(out, lse, q, data, bs, table, kv, new, dtype, scale=scale)


def test_overlapping_requests_leave_the_workspace_ready(dev):
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(5)
    kv, new, H, Hk, D, bs = [3000, 2000, 2500], [150, 140, 160], 1, 1, 64, 16
    q, data, table = _case(rng, kv, new, H, Hk, D, bs, "fp16")
    cache, ws = api.KVCache(torch.from_numpy(data).to(dev), bs, D), api.alloc_attention_workspace(3, 450, H, Hk, D, dev)
    args = V.tensor(q, "fp16", dev), cache, V.i32(table, dev), V.i32(kv, dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    api.attention_kv4(*args, cu_q=V.i32([0, 400, 10, 450], dev), workspace=ws, error=err)
    assert int(err) == 4 and not ws[:24576].any()
    out, lse = api.attention_kv4(*args, cu_q=V.i32([0, 150, 290, 450], dev), workspace=ws, return_lse=True)
    _check(out, lse, q, data, bs, table, kv, new, "fp16")


def test_capture_with_prompts(dev):
    """A graph of a step with prompts, replayed over other lengths, eager calls between."""
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(6)
    kv, new, H, Hk, D, bs = [2700, 300, 60], [140, 200, 1], 2, 1, 128, 16
    q, data, table = _case(rng, kv, new, H, Hk, D, bs, "bf16")
    cache = api.KVCache(torch.from_numpy(data).to(dev), bs, D)
    tt, n, qt = V.i32(table, dev), V.i32(kv, dev), V.tensor(q, "bf16", dev)
    cu = V.i32(np.concatenate([[0], np.cumsum(new)]), dev)
    ws = api.alloc_attention_workspace(3, sum(new), H, Hk, D, dev)
    out, lse = torch.empty_like(qt), torch.empty(sum(new), H, device=dev)
    call = lambda **k: api.attention_kv4(qt, cache, tt, n, cu_q=cu, workspace=ws, **k)      # noqa: E731
    call(out=out, lse=lse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out=out, lse=lse)
    for less in (0, 40, 59, 0):
        now = [k - less for k in kv]
        n.copy_(V.i32(now, dev))
        g.replay()
        e = call(return_lse=True)
        torch.cuda.synchronize()
        assert torch.equal(e[0], out) and torch.equal(e[1], lse)
        _check(out, lse, q, data, bs, table, now, new, "bf16")


def test_a_cache_past_32_bits(dev):
    """Blocks beyond 4 GiB: written, read back and attended to by both kernels."""
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(7)
    H, Hk, D, bs, n_blocks = 1, 1, 256, 256, 66000
    cache = api.alloc_kv_cache(n_blocks, Hk, D, bs, dev)
    assert cache.data.numel() > 1 << 32
    kv, new = [700, 300], [1, 150]
    small = V.random_cache(rng, 5, Hk, bs, D, "bf16")
    at = [n_blocks - 1, 61681, n_blocks - 7, 65000, 64000]
    cache.data[at] = torch.from_numpy(small).to(dev)
    table = np.array([[at[0], at[1], at[2]], [at[3], at[4], -1]])
    local = np.array([[0, 1, 2], [3, 4, -1]])
    q = S.round_to(rng.standard_normal((151, H, D)), "bf16")
    cu = [0, 1, 151]
    out, lse = api.attention_kv4(V.tensor(q, "bf16", dev), cache, V.i32(table, dev), V.i32(kv, dev), cu_q=V.i32(cu, dev),
                                 return_lse=True)
    _check(out, lse, q, small, bs, local, kv, new, "bf16")
    x = V.tensor(S.round_to(rng.standard_normal((4, 1, D)), "bf16"), "bf16", dev)
    slots = V.i32([at[0] * bs + 255, at[1] * bs, 3, at[3] * bs + 17], dev)
    api.qk_norm_rope_store(x, x, x, None, None, None, None, slots, cache)
    _, v = api.kv_load(cache, slots, dtype=torch.bfloat16)
    assert np.array_equal(V.array(v), S.values(*S.quantise(V.array(x), "bf16")))
