"""Queries one of whose dimensions is far beyond the others, where keys are small: their scores are sums in 32 bits as all scores
are, however many rows a request has."""
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


def _outliers(q, data, bs, D, size, rows):
    """q with dimension 32 i + 7 + i at `size` on the given rows; keys with zeros there."""
    q = q.copy()
    kc, ks, vc, vs = (a.copy() for a in S.split_pages(data, bs, D))
    for i in range(D // 32):
        q[rows, :, 33 * i + 7] = size * np.sign(q[rows, :, 33 * i + 7])
        kc[..., 33 * i + 7] = 0
    return q, S.pages(kc, ks, vc, vs)


def _check(out, lse, q, data, bs, table, kv, new, dtype, scale):
    """attention_bound, with what a sum in 32 bits is off by in place of its |q||k|: (D + 2) roundings of terms of at most
    sum |q_i k_i|."""
    D = q.shape[-1]
    cu = np.concatenate([[0], np.cumsum(new)])
    ref, ref_lse, weight = S.attention(q, data, bs, table, kv, cu, scale)
    k = np.abs(S.values(*S.split_pages(data, bs, D)[:2])).reshape(-1, D)
    most = (np.abs(q).reshape(-1, D) @ k.T).max(-1).reshape(q.shape[:2])
    b_out, b_lse = V.attention_bound(ref, ref_lse, weight, most[..., None], 1.0, scale * (D + 2) / 3, max(kv), dtype)
    got, got_lse = V.array(out), V.array(lse)
    empty = np.isneginf(ref_lse)
    assert (got[empty] == 0).all() and np.isneginf(got_lse[empty]).all()
    far = np.abs(got - ref) / b_out
    far_lse = np.abs(np.where(empty, 0, got_lse) - np.where(empty, 0, ref_lse)) / b_lse
    assert far.max() <= 1 and far_lse.max() <= 1, (far.max(), far_lse.max())


@pytest.mark.parametrize("dtype,size", [("fp16", 2048.0), ("fp16", 30000.0), ("bf16", 2.0 ** 14), ("bf16", 2.0 ** 40)])
@pytest.mark.parametrize("kv,new,H,Hk,D,bs", [
    ([260, 90], [150, 1], 2, 2, 64, 16), ([150, 400], [150, 131], 1, 1, 128, 32), ([230], [70], 4, 2, 256, 16),
    ([9900], [140], 1, 1, 64, 16), ([7000], [133], 1, 1, 128, 32), ([2600], [67], 2, 1, 256, 16),      # in parts
    ([100], [200], 1, 1, 128, 16)])                                                                   # rows that see nothing
def test_scores_are_sums_in_32_bits(dev, dtype, size, kv, new, H, Hk, D, bs):
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(D + kv[0])
    q, data, table = _case(rng, kv, new, H, Hk, D, bs, dtype)
    q, data = _outliers(q, data, bs, D, size, slice(None))
    ws = api.alloc_attention_workspace(len(kv), sum(new), H, Hk, D, dev)
    first, err = None, torch.zeros(1, dtype=torch.int32, device=dev)
    for _ in range(2):
        out, lse = _run(api, dev, q, data, bs, table, kv, new, dtype, scale=0.1, workspace=ws, error=err)
        assert first is None or (torch.equal(first[0], out) and torch.equal(first[1], lse))
        first = out, lse
    assert not ws[:24576].any() and int(err) == 0
    _check(out, lse, q, data, bs, table, kv, new, dtype, 0.1)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_one_such_row_among_others(dev, D):
    """A single row of many, blocks that are not there and a NaN among the values: the other rows are held to the usual bound."""
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(D)
    kv, new, bs, dtype = [700, 300], [300, 300], 16, "fp16"
    q, data, table = _case(rng, kv, new, 1, 1, D, bs, dtype)
    q, data = _outliers(q, data, bs, D, 8192.0, [5, 420])
    kc, ks, vc, vs = (a.copy() for a in S.split_pages(data, bs, D))
    vs[table[1, 9], 0, 3, 1] = 255                             # request 1's token 147
    data, table = S.pages(kc, ks, vc, vs), table.copy()
    table[0, 3], table[1, 1] = 10 ** 6, -4
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = _run(api, dev, q, data, bs, table, kv, new, dtype, scale=0.1, error=err)
    assert int(err) == 1
    out, sees = V.array(out), np.zeros((600, 1, D), bool)
    sees[300 + 147:, :, 32:64] = True
    assert np.array_equal(np.isnan(out), sees)
    vs[table[1, 9], 0, 3, 1] = 127
    clean = S.pages(kc, ks, vc, vs)
    cu = [0, 300, 600]
    ref, ref_lse, weight = S.attention(q, clean, bs, table, kv, cu, 0.1)
    kmax = np.linalg.norm(S.values(kc, ks), axis=-1).max()
    b_out, b_lse = V.attention_bound(ref, ref_lse, weight, q, kmax, 0.1, 700, dtype)
    assert (np.abs(out - ref) <= b_out)[~sees].all()
    seen = np.isfinite(ref_lse)
    assert (np.abs(V.array(lse) - ref_lse) <= b_lse)[seen].all()
