"""What the serving entry points refuse, before anything is launched (no GPU needed)."""
import ctypes as C

import pytest

from sub_bit_moe_amd import _native as N
from sub_bit_moe_amd import api

EINVAL, ERANGE, ENOSPACE = -1, -5, -6
A = 4096                                   # an aligned address that nothing reads


def _heads(data=A, ts=512, hs=64):
    return C.byref(N.Heads(data, ts, hs))


PLAN = dict(ctx=A, new=A, R=2, free=A, cap=8, n_free=A, table=A, width=4, n_blocks=8, bs=16, most=10, slots=A, pos=A,
            req=A, cu=A, kv=A + 64, out=A + 128, err=0, stream=0)
QK = dict(q=_heads(), k=_heads(), v=_heads(), qw=0, kw=0, pos=A, rope=A, rows=9, rot=64, eps=1e-6, T=2, H=4, Hk=2, D=64,
          qo=_heads(), ko=None, slots=A, cache=A, n_blocks=4, bs=16, flags=0, err=0, stream=0)
LOAD = dict(cache=A, n_blocks=4, Hk=2, bs=16, D=64, slots=A, T=3, k=A, v=A, flags=0, err=0, stream=0)
ATT = dict(q=_heads(), cache=A, n_blocks=4, bs=16, table=A, width=4, kv=A, cu=0, R=2, T=2, H=4, Hk=2, D=64, scale=1.0,
           out=A, lse=0, flags=0, ws=A, ws_bytes=1 << 40, err=0, stream=0)


@pytest.mark.parametrize("change,status", [
    (dict(R=-1), EINVAL), (dict(R=4097), EINVAL), (dict(bs=24), EINVAL), (dict(bs=8), EINVAL), (dict(bs=8192), EINVAL),
    (dict(cap=-1), EINVAL), (dict(width=-1), EINVAL), (dict(most=-1), EINVAL), (dict(most=2 ** 30 + 1), EINVAL),
    (dict(n_blocks=-1), EINVAL), (dict(n_blocks=2 ** 27), ERANGE), (dict(ctx=0), EINVAL), (dict(new=0), EINVAL),
    (dict(n_free=0), EINVAL), (dict(table=0), EINVAL), (dict(free=0), EINVAL), (dict(slots=0), EINVAL),
    (dict(pos=0), EINVAL), (dict(req=0), EINVAL), (dict(cu=0), EINVAL), (dict(kv=0), EINVAL), (dict(out=0), EINVAL),
    (dict(out=A), EINVAL), (dict(kv=A), EINVAL)])
def test_plan(change, status):
    assert N.lib().sbm_kv_plan(*{**PLAN, **change}.values()) == status
    assert N.lib().sbm_last_error()


@pytest.mark.parametrize("change,status", [
    (dict(flags=1), EINVAL), (dict(T=-1), EINVAL), (dict(H=0), EINVAL), (dict(Hk=0), EINVAL), (dict(H=65537), EINVAL),
    (dict(D=96), EINVAL), (dict(rot=72), EINVAL), (dict(rot=128), EINVAL), (dict(rot=-16), EINVAL),
    (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL), (dict(rows=-1), EINVAL), (dict(bs=48), EINVAL),
    (dict(n_blocks=0), EINVAL), (dict(n_blocks=2 ** 28), ERANGE), (dict(cache=A + 8), EINVAL), (dict(T=2 ** 29), ERANGE),
    (dict(q=None), EINVAL), (dict(q=_heads(0)), EINVAL), (dict(k=None), EINVAL), (dict(v=None), EINVAL),
    (dict(slots=0), EINVAL), (dict(pos=0), EINVAL), (dict(rope=0), EINVAL), (dict(qo=None), EINVAL),
    (dict(cache=0), EINVAL), (dict(q=_heads(A + 1)), EINVAL)])
def test_norm_rope(change, status):
    assert N.lib().sbm_qk_norm_rope(*{**QK, **change}.values()) == status


@pytest.mark.parametrize("change,status", [
    (dict(flags=4), EINVAL), (dict(T=-1), EINVAL), (dict(Hk=0), EINVAL), (dict(n_blocks=0), EINVAL), (dict(bs=17), EINVAL),
    (dict(D=32), EINVAL), (dict(T=2 ** 30), ERANGE), (dict(n_blocks=2 ** 28), ERANGE), (dict(cache=0), EINVAL),
    (dict(slots=0), EINVAL), (dict(k=A + 2), EINVAL), (dict(v=A + 8), EINVAL)])
def test_load(change, status):
    assert N.lib().sbm_kv_load(*{**LOAD, **change}.values()) == status


@pytest.mark.parametrize("change,status", [
    (dict(flags=2), EINVAL), (dict(R=-1), EINVAL), (dict(R=4097), EINVAL), (dict(T=-1), EINVAL), (dict(H=0), EINVAL),
    (dict(Hk=3), EINVAL), (dict(Hk=0), EINVAL), (dict(n_blocks=0), EINVAL), (dict(width=-1), EINVAL), (dict(bs=20), EINVAL),
    (dict(D=80), EINVAL), (dict(width=2 ** 27), ERANGE), (dict(T=3), EINVAL), (dict(R=0, cu=A), EINVAL), (dict(q=None), EINVAL),
    (dict(cache=0), EINVAL), (dict(table=0), EINVAL), (dict(kv=0), EINVAL), (dict(out=0), EINVAL), (dict(ws=0), EINVAL),
    (dict(q=_heads(A + 8)), EINVAL), (dict(q=_heads(A, 12)), EINVAL), (dict(q=_heads(A, 512, 68)), EINVAL),
    (dict(out=A + 4), EINVAL), (dict(ws=A + 8), EINVAL), (dict(cache=A + 1), EINVAL), (dict(ws_bytes=0), ENOSPACE),
    (dict(T=2 ** 30, H=64, Hk=1, cu=A), ERANGE)])
def test_attention(change, status):
    assert N.lib().sbm_attention_kv4(*{**ATT, **change}.values()) == status


def test_nothing_to_do_is_no_error():
    assert N.lib().sbm_qk_norm_rope(*{**QK, "T": 0, "q": None}.values()) == 0
    assert N.lib().sbm_kv_load(*{**LOAD, "T": 0, "slots": 0}.values()) == 0
    assert N.lib().sbm_attention_kv4(*{**ATT, "T": 0, "R": 0, "q": None}.values()) == 0


def test_sizes():
    assert N.lib().sbm_kv_cache_bytes(3, 2, 16, 128) == 3 * 2 * 16 * 136
    for bad in ((0, 2, 16, 128), (3, 0, 16, 128), (3, 2, 12, 128), (3, 2, 16, 100)):
        assert N.lib().sbm_kv_cache_bytes(*bad) == 0
    assert api.attention_workspace_bytes(3, 3, 8, 2, 128) > 0
    for bad in ((-1, 3, 8, 2, 128), (3, -1, 8, 2, 128), (3, 3, 8, 3, 128), (3, 3, 8, 2, 96)):
        assert api.attention_workspace_bytes(*bad) == 0


def test_front_end():
    torch = pytest.importorskip("torch")
    q = torch.zeros(2, 4, 64, dtype=torch.float16)
    cache = api.KVCache(torch.zeros(3, 2, 16 * 68, dtype=torch.uint8), 16, 64)
    n = torch.ones(2, dtype=torch.int32)
    table = torch.zeros(2, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="on the GPU"):
        api.attention_kv4(q, cache, table, n, workspace=torch.zeros(16, dtype=torch.uint8))
    with pytest.raises(ValueError):
        api.alloc_kv_cache(3, 2, 96)
    with pytest.raises(ValueError, match="holds 2 heads of 64"):
        api.attention_kv4(torch.zeros(2, 3, 64, dtype=torch.float16), cache, table, n)
    with pytest.raises(ValueError, match="same requests"):
        api.attention_kv4(q, cache, table[:1], n)
    with pytest.raises(ValueError, match="neighbouring"):
        api.qk_norm_rope(q[..., ::2], q, None, None, n, None)
    with pytest.raises(TypeError):
        api.qk_norm_rope(q.float(), q.float(), None, None, n, None)
    with pytest.raises(ValueError, match="one row for each request"):
        api.kv_plan(n, n[:1], n, n[:1], table, 4, 16, 8)
