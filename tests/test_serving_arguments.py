"""What the serving calls accept and refuse of their tensors (no GPU needed: addresses and devices are stand-ins)."""
import pytest

from sub_bit_moe_amd import _native as N
from sub_bit_moe_amd import api
from tests.test_serving_refusals import ATT, EINVAL, _heads

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("shape,ts,hs", [((1, 4), 12, 64), ((1, 4), 1, 64), ((2, 1), 64, 4), ((1, 1), 3, 5), ((1, 1), 0, 0)])
def test_strides_that_no_address_is_made_from_do_not_matter(shape, ts, hs):
    """One token's token stride and one head's head stride; the call goes on to its next check."""
    T, H = shape
    call = {**ATT, "R": T, "T": T, "H": H, "Hk": 1, "q": _heads(4096, ts, hs), "ws_bytes": 0}
    assert N.lib().sbm_attention_kv4(*call.values()) == -6             # the workspace is too small


@pytest.mark.parametrize("shape,ts,hs", [((2, 4), 12, 64), ((1, 4), 256, 12), ((2, 1), 4, 64)])
def test_strides_that_addresses_are_made_from_are_refused(shape, ts, hs):
    T, H = shape
    call = {**ATT, "R": T, "T": T, "H": H, "Hk": 1, "q": _heads(4096, ts, hs), "ws_bytes": 0}
    assert N.lib().sbm_attention_kv4(*call.values()) == EINVAL


class _There:
    """A CPU tensor that says it is on the GPU."""

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return 0


def _rows(*shape):
    return _There(torch.zeros(shape, dtype=torch.float16))


def _ints(*shape):
    return _There(torch.zeros(shape, dtype=torch.int32))


def test_missing_arguments_are_named():
    q, k = _rows(2, 4, 64), _rows(2, 2, 64)
    rope = _There(torch.zeros(9, 64))
    cache = api.KVCache(_There(torch.zeros(3, 2, 16 * 68, dtype=torch.uint8)), 16, 64)
    with pytest.raises(ValueError, match="positions"):
        api.qk_norm_rope(q, k, None, None, None, rope)
    with pytest.raises(ValueError, match="slots"):
        api.qk_norm_rope_store(q, k, k, None, None, None, None, None, cache)
    with pytest.raises(ValueError, match="v "):
        api.qk_norm_rope_store(q, k, None, None, None, None, None, _ints(2), cache)
    with pytest.raises(ValueError, match="rope"):
        api.qk_norm_rope(q, k, None, None, _ints(2), _There(torch.zeros(9)))
    with pytest.raises(ValueError, match="q must be"):
        api.qk_norm_rope(_rows(2, 64), k, None, None, None, None)
    with pytest.raises(ValueError, match="k must be"):
        api.qk_norm_rope(q, _rows(2 * 64), None, None, None, None)
    with pytest.raises(ValueError, match="q must be"):
        api.attention_kv4(_rows(2, 64), cache, _ints(2, 3), _ints(2))


def test_tensors_of_another_device_than_the_stream_are_refused(monkeypatch):
    """A launch goes to the device of its stream, which is the current one where none is given."""
    class Stream:
        device_index, cuda_stream = 1, 7

    monkeypatch.setattr(api, "_current_stream", (lambda d: 40 + d, lambda: 1))
    monkeypatch.setattr(api, "_made_on", lambda stream, make, *a, **k: _There(torch.zeros(2, 4, 64)))
    monkeypatch.setattr(api, "check", lambda status: pytest.fail("launched"))
    q = _rows(2, 4, 64)
    cache = api.KVCache(_There(torch.zeros(3, 4, 16 * 68, dtype=torch.uint8)), 16, 64)
    plan = api.KVPlan(_ints(8), _ints(8), _ints(8), _ints(3), _ints(2), _ints(1), _ints(1), None)
    for kw in ({}, {"stream": Stream()}):
        for call in (lambda: api.qk_norm_rope(q, q, None, None, None, None, **kw),
                     lambda: api.kv_load(cache, _ints(2), k=_rows(2, 4, 64), v=_rows(2, 4, 64), **kw),
                     lambda: api.attention_kv4(q, cache, _ints(2, 3), _ints(2), out=_rows(2, 4, 64),
                                               workspace=_There(torch.zeros(64, dtype=torch.uint8)), **kw),
                     lambda: api.kv_plan(_ints(2), _ints(2), _ints(4), _ints(1), _ints(2, 3), 4, 16, 8, plan=plan, **kw)):
            with pytest.raises(ValueError, match="on device 0"):
                call()
    assert api._stream(None, 1) == 41 and api._stream(Stream(), 1) == 7 and api._stream() == 41
