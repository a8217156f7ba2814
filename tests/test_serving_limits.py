"""The serving entry points' size limits: what an index of 32 bits would not hold is refused, before anything is launched (no GPU
needed; what is refused is refused before a pointer is read)."""
import pytest

from sub_bit_moe_amd import _native as N
from tests.test_serving_refusals import ATT, EINVAL, ERANGE, PLAN


@pytest.mark.parametrize("bs,width", [(16, (2 ** 31 - 256) // 16), (256, (2 ** 31 - 256) // 256), (16, (2 ** 31 - 4096) // 16 + 1),
                                      (4096, 2 ** 19)])
def test_attention_refuses_requests_whose_positions_would_wrap(bs, width):
    """Reads run up to 512 positions ahead of a request's last token."""
    assert N.lib().sbm_attention_kv4(*{**ATT, "bs": bs, "width": width}.values()) == ERANGE
    assert b"in one request" in N.lib().sbm_last_error()


def test_plan_refuses_tokens_that_could_pass_31_bits():
    """A context of 2^30 tokens, the most that a plan takes, and as many new ones would be 2^31."""
    assert N.lib().sbm_kv_plan(*{**PLAN, "most": 2 ** 30}.values()) == EINVAL
    assert b"max_tokens" in N.lib().sbm_last_error()


# 6 requests, each array in a page of its own
APART = {**PLAN, "R": 6, "ctx": 0x10000, "new": 0x20000, "free": 0x30000, "n_free": 0x40000, "table": 0x50000, "slots": 0x60000,
         "pos": 0x70000, "req": 0x80000, "cu": 0x90000, "kv": 0xA0000, "out": 0xB0000}


@pytest.mark.parametrize("change", [
    dict(kv=0x10004), dict(kv=0x10000 - 20), dict(kv=0x20004), dict(ctx=0xA0004),      # the lengths of fewer requests, for one
    dict(cu=0x10000 + 20), dict(cu=0x20000 - 24), dict(slots=0x30000 + 28), dict(pos=0x10004), dict(req=0x20000 - 36),
    dict(out=0x10004), dict(n_free=0xA0008), dict(table=0x10000 - 92), dict(table=0x30000 + 4), dict(err=0x10000),
    dict(pos=0x60000 + 36), dict(kv=0x50004), dict(cu=0xA0000), dict(out=0x90018), dict(err=0xB0000)])
def test_plan_refuses_arrays_that_overlap(change):
    """Its workgroups read the lengths while others write the results."""
    assert N.lib().sbm_kv_plan(*{**APART, **change}.values()) == EINVAL
    assert b"overlap" in N.lib().sbm_last_error()
