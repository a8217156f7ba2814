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
