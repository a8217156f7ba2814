"""What the serving calls accept and refuse of their tensors (no GPU needed: addresses and devices are stand-ins)."""
import pytest

from sub_bit_moe_amd import _native as N
from tests.test_serving_refusals import ATT, EINVAL, _heads


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
