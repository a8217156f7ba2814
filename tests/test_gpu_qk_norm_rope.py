"""Norm, rotation and the 4-bit cache's writer and reader against 64 bits."""
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


def _inputs(rng, T, H, Hk, D, rot, dtype, rows=5000):
    x = rng.standard_normal((T, H + 2 * Hk, D)) * np.exp(rng.standard_normal((T, H + 2 * Hk, 1)))
    x = S.round_to(x, dtype)
    w = S.round_to(1 + 0.3 * rng.standard_normal((2, D)), dtype)
    pos = rng.integers(0, rows, T)
    pos[:1] = rows - 1
    return x, w, pos


def _q_bound(x, w, ref, dtype):
    """Half a step, and fp32's sums and products: at most D / 8 + 12 roundings of
    values no larger than a pair's norm."""
    y = S.norm_rope(x, w, None, 0)
    top = np.abs(y).max(-1, keepdims=True) * 2 ** 0.5
    return V.HALF[dtype] * np.abs(ref) + (x.shape[-1] / 8 + 12) * 2.0 ** -24 * top + (2.0 ** -25 if dtype == "fp16" else 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D,rot,neighbours", [(64, 64, False), (64, 32, True), (128, 128, False), (128, 128, True),
                                              (128, 16, False), (256, 64, False), (256, 256, True), (128, 0, False)])
def test_norm_rope_and_store(dev, dtype, D, rot, neighbours):
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(D + rot)
    for T, H, Hk in ((1, 1, 1), (7, 6, 2), (65, 5, 5)):
        x, w, pos = _inputs(rng, T, H, Hk, D, rot, dtype)
        t = V.tensor(x.reshape(T, -1), dtype, dev)                # a joint projection: strided views
        q, k, v = t[:, :H * D].view(T, H, D), t[:, H * D:(H + Hk) * D].view(T, Hk, D), t[:, (H + Hk) * D:].view(T, Hk, D)
        qw, kw = V.tensor(w[0], dtype, dev), V.tensor(w[1], dtype, dev)
        rope = api.rope_table(5000, rot, 10000.0, dev) if rot else None
        rows = rope.cpu().numpy()[pos] if rot else None
        p = V.i32(pos, dev)
        qo, ko = api.qk_norm_rope(q, k, qw, kw, p, rope, neighbours=neighbours)
        ref_q = S.norm_rope(x[:, :H], w[0], rows, rot, neighbours=neighbours)
        ref_k = S.round_to(S.norm_rope(x[:, H:H + Hk], w[1], rows, rot, neighbours=neighbours), dtype)
        assert (np.abs(V.array(qo) - ref_q) <= _q_bound(x[:, :H], w[0], ref_q, dtype)).all()
        assert np.array_equal(V.array(ko), ref_k)
        # the same with the cache: its bytes are the quantised keys and values, the rest stays
        bs = 16 if T < 60 else 32
        nb = -(-T // bs) + 3
        slots = rng.permutation(nb * bs)[:T]
        slots[T // 2] = -1 if T > 1 else slots[0]
        before = rng.integers(0, 256, (nb, Hk, bs * D * 17 // 16)).astype(np.uint8)
        cache = api.KVCache(torch.from_numpy(before.copy()).to(dev), bs, D)
        ko2 = torch.empty_like(ko)
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        qo2 = api.qk_norm_rope_store(q, k, v, qw, kw, p, rope, V.i32(slots, dev), cache, neighbours=neighbours, k_out=ko2,
                                     error=err)
        assert torch.equal(qo2, qo) and torch.equal(ko2, ko) and int(err) == 0
        parts = [a.copy() for a in S.split_pages(before, bs, D)]
        for n, rounded in ((0, ref_k), (2, x[:, H + Hk:])):
            codes, scales = S.quantise(rounded, dtype)
            for i, s in enumerate(slots):
                if s >= 0:
                    parts[n][s // bs, :, s % bs], parts[n + 1][s // bs, :, s % bs] = codes[i], scales[i]
        assert np.array_equal(cache.data.cpu().numpy(), S.pages(*parts))
        kl, vl = api.kv_load(cache, V.i32(slots, dev), dtype=V.DT[dtype])
        for got, rounded in ((kl, ref_k), (vl, x[:, H + Hk:])):
            want = S.values(*S.quantise(rounded, dtype)) * (slots >= 0)[:, None, None]
            assert np.array_equal(V.array(got), want)


def test_cached_codes_do_not_depend_on_the_call(dev):
    """A prompt in one call, token by token, in place, on another stream, and without 16-byte alignment: the same bytes."""
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(5)
    T, H, Hk, D, bs = 40, 4, 2, 128, 16
    x, w, pos = _inputs(rng, T, H, Hk, D, D, "bf16")
    rope = api.rope_table(5000, D, 10000.0, dev)
    qw, kw = V.tensor(w[0], "bf16", dev), V.tensor(w[1], "bf16", dev)
    slots, p = V.i32(rng.permutation(64)[:T], dev), V.i32(pos, dev)

    def parts(pad):
        flat = torch.zeros(T, (H + 2 * Hk) * D + pad, dtype=torch.bfloat16, device=dev)
        flat[:, pad:] = V.tensor(x.reshape(T, -1), "bf16", dev)
        f = flat[:, pad:]
        return f[:, :H * D].unflatten(1, (H, D)), f[:, H * D:(H + Hk) * D].unflatten(1, (Hk, D)), f[:, (H + Hk) * D:].unflatten(1, (Hk, D))

    q, k, v = parts(0)
    one = api.alloc_kv_cache(4, Hk, D, bs, dev)
    q1 = api.qk_norm_rope_store(q, k, v, qw, kw, p, rope, slots, one)
    many = api.alloc_kv_cache(4, Hk, D, bs, dev)
    for t in range(T):
        a = slice(t, t + 1)
        qt = api.qk_norm_rope_store(q[a], k[a], v[a], qw, kw, p[a], rope, slots[a], many)
        assert torch.equal(qt, q1[a])
    assert torch.equal(one.data, many.data)
    for pad in (1, 4):                                           # 2- and 8-byte aligned heads
        qo, ko, vo = parts(pad)
        odd = api.alloc_kv_cache(4, Hk, D, bs, dev)
        assert torch.equal(api.qk_norm_rope_store(qo, ko, vo, qw, kw, p, rope, slots, odd), q1)
        assert torch.equal(one.data, odd.data)
    q, k, v = parts(0)
    side, there = torch.cuda.Stream(), api.alloc_kv_cache(4, Hk, D, bs, dev)
    side.wait_stream(torch.cuda.current_stream())
    api.qk_norm_rope_store(q, k, v, qw, kw, p, rope, slots, there, q_out=q, k_out=k, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(q, q1) and torch.equal(one.data, there.data)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_every_16_bit_value_is_cached_as_the_oracle_does(dev, dtype):
    """V takes every bit pattern, alone beside zeros and among its neighbours (infinities and NaN included)."""
    from sub_bit_moe_amd import api
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(V.DT[dtype])
    x = every.double().numpy()
    alone = np.zeros((2048, 1, 1024))
    alone.reshape(-1, 32)[np.arange(65536), np.arange(65536) % 32] = x
    beside = x.reshape(-1, 64)[np.random.default_rng(0).permutation(1024)]
    for rows, D in ((alone.reshape(-1, 1, 64), 64), (beside.reshape(-1, 1, 64), 64), (x.reshape(-1, 1, 256), 256)):
        T = rows.shape[0]
        cache = api.alloc_kv_cache(-(-T // 16), 1, D, 16, dev)
        v = V.tensor(rows, dtype, dev)
        slots = torch.arange(T, dtype=torch.int32, device=dev)
        zero = torch.zeros_like(v)
        api.qk_norm_rope_store(zero, zero, v, None, None, None, None, slots, cache)
        codes, scales = S.quantise(rows, dtype)
        _, _, vc, vs = S.split_pages(cache.data.cpu().numpy(), 16, D)
        vc, vs = vc[:, 0].reshape(-1, D)[:T], vs[:, 0].reshape(-1, D // 32)[:T]
        assert np.array_equal(vs, scales[:, 0])
        neg_zero = (codes[:, 0] & 7) == 0                        # the sign of a NaN or a zero is free
        assert np.array_equal(np.where(neg_zero, 0, vc), np.where(neg_zero, 0, codes[:, 0]))
        _, got = api.kv_load(cache, slots, dtype=V.DT[dtype])
        assert np.array_equal(V.array(got), S.values(codes, scales), equal_nan=True)


def test_values_by_every_code_and_scale(dev):
    """kv_load of each of the 16 codes at each scale byte, rounded to the type."""
    from sub_bit_moe_amd import api
    codes = np.tile(np.arange(16, dtype=np.uint8), (256, 4))[:, None, None]          # [block, 1, 1, 64] per scale
    codes = np.repeat(codes, 16, 2)
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None, None, None], 16, 2).repeat(2, 3)
    cache = api.KVCache(torch.from_numpy(S.pages(codes, scales, codes[::-1], scales[::-1])).to(dev), 16, 64)
    slots = torch.arange(0, 4096, 16, dtype=torch.int32, device=dev)
    for dtype in ("bf16", "fp16"):
        k, v = api.kv_load(cache, slots, dtype=V.DT[dtype])
        want = S.round_to(S.values(codes, scales)[:, :, 0], dtype)
        assert np.array_equal(V.array(k), want, equal_nan=True)
        assert np.array_equal(V.array(v), want[::-1], equal_nan=True)


def test_positions_and_slots_outside_are_left_out_and_counted(dev):
    from sub_bit_moe_amd import api
    T, H, Hk, D = 6, 2, 1, 64
    rng = np.random.default_rng(8)
    x, w, _ = _inputs(rng, T, H, Hk, D, D, "fp16")
    t = V.tensor(x, "fp16", dev)
    rope = api.rope_table(10, D, 10000.0, dev)
    pos, slots = V.i32([0, 10, 3, -1, 9, 2 ** 31 - 1], dev), V.i32([0, 1, 64, 2, -9, 3], dev)
    cache = api.alloc_kv_cache(4, Hk, D, 16, dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    q_out = torch.full((T, H, D), 7.0, dtype=torch.float16, device=dev)
    api.qk_norm_rope_store(t[:, :2], t[:, 2:3], t[:, 3:], None, None, pos, rope, slots, cache, q_out=q_out, error=err)
    assert int(err) == 4                                          # three positions, one slot
    assert (q_out[[1, 3, 5]] == 7).all() and (q_out[[0, 2, 4]] != 7).any(-1).all()
    written = cache.data.cpu().numpy()
    k, _ = api.kv_load(cache, V.i32([0, 1, 2, 3, 64, -1], dev), error=err)
    assert int(err) == 5 and k[0].abs().sum() > 0 and not k[1:].any()
    assert not written[1:].any()


def test_capture(dev):
    """Recorded once and replayed with other inputs, eager work between."""
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(9)
    T, H, Hk, D = 9, 4, 2, 128
    rope = api.rope_table(5000, D, 10000.0, dev)
    x, w, pos = _inputs(rng, T, H, Hk, D, D, "bf16")
    t, p = V.tensor(x, "bf16", dev), V.i32(pos, dev)
    slots = V.i32(rng.permutation(32)[:T], dev)
    cache, q_out = api.alloc_kv_cache(2, Hk, D, 16, dev), torch.empty(T, H, D, dtype=torch.bfloat16, device=dev)
    kv = [torch.empty(T, Hk, D, dtype=torch.bfloat16, device=dev) for _ in range(2)]

    def go(c, q, k, v):
        api.qk_norm_rope_store(t[:, :H], t[:, H:H + Hk], t[:, H + Hk:], None, None, p, rope, slots, c, q_out=q)
        api.kv_load(c, slots, k=k, v=v)

    go(cache, q_out, *kv)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go(cache, q_out, *kv)
    for _ in range(3):
        x, _, pos = _inputs(rng, T, H, Hk, D, D, "bf16")
        t.copy_(V.tensor(x, "bf16", dev))
        p.copy_(V.i32(pos, dev))
        g.replay()
        other = api.alloc_kv_cache(2, Hk, D, 16, dev)
        e = [torch.empty_like(a) for a in (q_out, *kv)]
        go(other, *e)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(e, (q_out, *kv))) and torch.equal(other.data, cache.data)
