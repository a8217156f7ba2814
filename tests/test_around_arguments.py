"""What the front end of the operators around the experts says of its arguments, before the library is asked (no GPU needed)."""
import pytest

from sub_bit_moe_amd import api

torch = pytest.importorskip("torch")


def _x():
    return torch.zeros(4, 8, dtype=torch.float16)


@pytest.mark.parametrize("call", [api.add_rms_norm, api.add_rms_norm_fp8])
@pytest.mark.parametrize("repeat", [0, -1])
def test_no_rows_of_a_token_are_refused_by_name(call, repeat):
    with pytest.raises(ValueError, match="repeat"):
        call(_x(), repeat=repeat)


def test_missing_arguments_are_named():
    for call, what in ((lambda: api.add_rms_norm(None), "x must"), (lambda: api.add_rms_norm_fp8(None), "x must"),
                       (lambda: api.moe_route(None, 1), "logits must"),
                       (lambda: api.sample(None, torch.zeros(4)), "logits must")):
        with pytest.raises(ValueError, match=what + " be given"):
            call()


@pytest.mark.parametrize("k", [0, -1])
def test_no_experts_of_a_token_are_refused_by_name(k):
    with pytest.raises(ValueError, match="k must"):
        api.moe_route(torch.zeros(4, 8), k)
