"""Attention over the 4-bit cache against 64 bits."""
import numpy as np
import pytest

from oracle import serving as S
from tests import _serving as V

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _case(rng, kv, new, H, Hk, D, bs, dtype):
    table, n_blocks = V.shuffled_table(rng, kv, bs)
    data = V.random_cache(rng, n_blocks, Hk, bs, D, dtype)
    q = S.round_to(1.5 * rng.standard_normal((sum(new), H, D)), dtype)
    return q, data, table


def _run(api, dev, q, data, bs, table, kv, new, dtype, scale=None, **kw):
    cache = api.KVCache(torch.from_numpy(data).to(dev), bs, q.shape[-1])
    cu = None if new is None else V.i32(np.concatenate([[0], np.cumsum(new)]), dev)
    return api.attention_kv4(V.tensor(q, dtype, dev), cache, V.i32(table, dev), V.i32(kv, dev), cu_q=cu, scale=scale,
                             return_lse=True, **kw)


def _check(out, lse, q, data, bs, table, kv, new, dtype, scale=None, rows=slice(None)):
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    cu = None if new is None else np.concatenate([[0], np.cumsum(new)])
    ref, ref_lse, weight = S.attention(q, data, bs, table, kv, cu, scale)
    k = S.values(*S.split_pages(data, bs, q.shape[-1])[:2])
    kmax = np.nanmax(np.linalg.norm(k, axis=-1))
    b_out, b_lse = V.attention_bound(ref, ref_lse, weight, q, kmax, scale, max(kv, default=0), dtype)
    got, got_lse = V.array(out), V.array(lse)
    empty = np.isneginf(ref_lse)
    assert (got[empty] == 0).all() and np.isneginf(got_lse[empty]).all()
    assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.array_equal(np.isnan(got_lse), np.isnan(ref_lse))
    with np.errstate(invalid="ignore"):
        far = np.abs(got - ref) / b_out
        far_lse = np.abs(np.where(empty, 0, got_lse - np.where(empty, 0, ref_lse))) / b_lse
    assert np.nanmax(far, initial=0) <= 1 and np.nanmax(far_lse, initial=0) <= 1, (np.nanmax(far), np.nanmax(far_lse))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D,bs,H,Hk", [(64, 16, 4, 4), (64, 128, 6, 2), (128, 16, 8, 2), (128, 32, 5, 1), (128, 64, 3, 3),
                                       (256, 16, 2, 1), (256, 256, 4, 4), (128, 16, 40, 1), (64, 16, 17, 1)])
def test_single_tokens(dev, dtype, D, bs, H, Hk):
    """Lengths at every border: nothing, one token, tiles and blocks that end inside and at their ends."""
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(D + bs + H)
    kv = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 500, 0, 1023]
    q, data, table = _case(rng, kv, [1] * len(kv), H, Hk, D, bs, dtype)
    out, lse = _run(api, dev, q, data, bs, table, kv, None, dtype)
    _check(out, lse, q, data, bs, table, kv, None, dtype)
    # given as cu_q: the same bits
    out2, lse2 = _run(api, dev, q, data, bs, table, kv, [1] * len(kv), dtype)
    _check(out2, lse2, q, data, bs, table, kv, [1] * len(kv), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D,bs,H,Hk", [(64, 16, 3, 1), (128, 16, 4, 2), (128, 64, 7, 1), (256, 32, 2, 2)])
def test_prompts_and_pieces(dev, dtype, D, bs, H, Hk):
    """Ragged new tokens: none, one, prompts without context, pieces behind one, and
    requests that hold fewer tokens than they have rows (the first rows see nothing)."""
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(D + bs + H + 1)
    kv = [5, 40, 0, 70, 33, 200, 16, 4, 129]
    new = [5, 0, 0, 1, 33, 21, 16, 9, 130]
    q, data, table = _case(rng, kv, new, H, Hk, D, bs, dtype)
    out, lse = _run(api, dev, q, data, bs, table, kv, new, dtype)
    _check(out, lse, q, data, bs, table, kv, new, dtype)


@pytest.mark.parametrize("kv,new,H,Hk,D,bs", [([3000], [1], 8, 1, 128, 16), ([5, 9001, 700], [1, 1, 1], 4, 2, 64, 32),
                                              ([2500, 30], [3, 1], 32, 2, 128, 16), ([4100], [70], 4, 2, 256, 64),
                                              ([1500, 1200], [300, 1], 8, 2, 128, 32)])
def test_long_axes(dev, kv, new, H, Hk, D, bs):
    """Long caches and few rows (the token axis is shared out), and the reverse."""
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(sum(kv))
    q, data, table = _case(rng, kv, new, H, Hk, D, bs, "bf16")
    out, lse = _run(api, dev, q, data, bs, table, kv, new, "bf16", scale=0.2)
    _check(out, lse, q, data, bs, table, kv, new, "bf16", scale=0.2)


def test_many_requests(dev):
    """More requests than a scan's round, with and without tokens."""
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(31)
    kv = rng.integers(0, 60, 700)
    new = np.minimum(rng.integers(0, 3, 700), kv)
    q, data, table = _case(rng, kv, list(new), 2, 1, 64, 16, "fp16")
    out, lse = _run(api, dev, q, data, 16, table, list(kv), list(new), "fp16")
    _check(out, lse, q, data, 16, table, list(kv), list(new), "fp16")


def test_hidden_tokens_may_hold_anything(dev):
    """Rows behind a length, blocks outside the cache, and later tokens of the same
    prompt take no part, NaN among them; a NaN that a row sees is a NaN of that
    row: in every dimension for a key, in its 32 for a value."""
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(12)
    for D in (64, 128, 256):
        kv, new, H, Hk, bs = [37, 50, 20, 64], [1, 50, 20, 2], 2, 1, 16
        q, data, table = _case(rng, kv, new, H, Hk, D, bs, "bf16")
        kc, ks, vc, vs = (a.copy() for a in S.split_pages(data, bs, D))
        free = sorted(set(range(data.shape[0])) - set(table[table >= 0].tolist()))
        ks[free], vs[free] = 255, 255
        last = table[0, 2]
        ks[last, :, 5:], vs[last, :, 5:] = 255, 255               # behind request 0's 37 tokens
        vs[table[1, 1], 0, 4, D // 32 - 1] = 255                  # request 1, token 20: a value
        ks[table[1, 2], 0, 9, 0] = 255                            # request 1, token 41: a key
        table = table.copy()
        table[2, 0] = 10 ** 6                                     # request 2's first 16 tokens
        table[3, 1] = -3
        data = S.pages(kc, ks, vc, vs)
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        out, lse = _run(api, dev, q, data, bs, table, kv, new, "bf16", error=err)
        assert int(err) == 1
        _check(out, lse, q, data, bs, table, kv, new, "bf16")
        got = V.array(out)[1:51]
        assert not np.isnan(got[:20]).any() and np.isnan(got[20:, :, D - 32:]).all()
        assert not np.isnan(got[20:41, :, :D - 32]).any() and np.isnan(got[41:]).all()


def test_extreme_scores(dev):
    """Scores that rise and fall by far more than an exponential holds, alike scores, and a scale of zero or below."""
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(14)
    kv, H, Hk, D, bs = [300, 33], 4, 2, 64, 16
    for dtype, scale in (("bf16", 40.0), ("fp16", -9.0), ("fp16", 0.0)):
        q, data, table = _case(rng, kv, [1, 1], H, Hk, D, bs, dtype)
        out, lse = _run(api, dev, q, data, bs, table, kv, None, dtype, scale=scale)
        _check(out, lse, q, data, bs, table, kv, None, dtype, scale=scale)


def test_lengths_outside_are_cut_and_counted(dev):
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(15)
    kv, H, Hk, D, bs = [48, 20], 2, 1, 64, 16
    q, data, table = _case(rng, kv, [1, 1], H, Hk, D, bs, "fp16")
    table = table[:, :3].copy()
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = _run(api, dev, q, data, bs, table, [2 ** 31 - 1, -5], None, "fp16", error=err)
    assert int(err) == 2
    _check(out, lse, q, data, bs, table, [48, 0], None, "fp16")
    # tokens of no request get nothing; a cu_q that falls or passes q is reported
    cache = api.KVCache(torch.from_numpy(data).to(dev), bs, D)
    qt = V.tensor(np.concatenate([q, q, q]), "fp16", dev)
    out, lse = api.attention_kv4(qt, cache, V.i32(table, dev), V.i32(kv, dev), cu_q=V.i32([1, 2, 4], dev), return_lse=True)
    assert not out[[0, 4, 5]].any() and torch.isneginf(lse[[0, 4, 5]]).all() and torch.isfinite(lse[1:4]).all()
    for cu in ([0, 3, 2], [0, 1, 7], [-1, 1, 2]):
        err.zero_()
        api.attention_kv4(qt, cache, V.i32(table, dev), V.i32(kv, dev), cu_q=V.i32(cu, dev), error=err)
        assert int(err) & 4, cu


def test_strided_queries_streams_and_workspaces(dev):
    """q as a slice of a wider tensor, a kept workspace over calls of other sizes, another stream: the same bits."""
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(16)
    kv, H, Hk, D, bs = [700, 3, 1200], 8, 2, 128, 32
    q, data, table = _case(rng, kv, [1] * 3, H, Hk, D, bs, "bf16")
    cache = api.KVCache(torch.from_numpy(data).to(dev), bs, D)
    args = cache, V.i32(table, dev), V.i32(kv, dev)
    qt = V.tensor(q, "bf16", dev)
    out, lse = api.attention_kv4(qt, *args, return_lse=True)
    _check(out, lse, q, data, bs, table, kv, None, "bf16")
    wide = torch.zeros(3, 2 * H + 1, D + 8, dtype=torch.bfloat16, device=dev)
    wide[:, :2 * H:2, :D] = qt
    ws = api.alloc_attention_workspace(3, 40, H, Hk, D, dev)
    for _ in range(3):
        assert torch.equal(api.attention_kv4(wide[:, :2 * H:2, :D], *args, workspace=ws), out)
        few = api.attention_kv4(qt[:1], cache, args[1][:1], args[2][:1], workspace=ws)
        assert few.shape == (1, H, D)
        many = qt[:1].expand(40, H, D).contiguous()
        api.attention_kv4(many, cache, args[1][:1], args[2][:1], cu_q=V.i32([0, 40], dev), workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    there = api.attention_kv4(qt, *args, workspace=ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(there, out)


def test_capture(dev):
    """A graph over lengths on the GPU: replayed as the requests grow, eager calls between."""
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(17)
    kv, H, Hk, D, bs = [40, 900, 0], 4, 2, 64, 16
    q, data, table = _case(rng, [60, 960, 60], [1] * 3, H, Hk, D, bs, "fp16")
    cache = api.KVCache(torch.from_numpy(data).to(dev), bs, D)
    tt, n, qt = V.i32(table, dev), V.i32(kv, dev), V.tensor(q, "fp16", dev)
    ws = api.alloc_attention_workspace(3, 3, H, Hk, D, dev)
    out, lse = torch.empty_like(qt), torch.empty(3, H, device=dev)
    api.attention_kv4(qt, cache, tt, n, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.attention_kv4(qt, cache, tt, n, out=out, lse=lse, workspace=ws)
    for grow in (0, 1, 17, 40):
        now = [k + grow for k in kv]
        n.copy_(V.i32(now, dev))
        g.replay()
        e = api.attention_kv4(qt, cache, tt, n, return_lse=True, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(e[0], out) and torch.equal(e[1], lse)
        _check(out, lse, q, data, bs, table, now, None, "fp16")
