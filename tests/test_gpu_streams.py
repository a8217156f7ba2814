"""Calls with stream=: what they make is that stream's own, in the allocator's books too."""
import pytest

from tests import _parity as P
from tests import _serving as V

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _stream_of(t):
    """The stream whose memory t is in."""
    at = t.data_ptr()
    for segment in torch.cuda.memory_snapshot():
        if segment["address"] <= at < segment["address"] + segment["total_size"]:
            return segment["stream"]
    raise AssertionError("not the allocator's")


@pytest.fixture
def side():
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    yield s
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()


def _owned(side, *made):
    for t in made:
        assert _stream_of(t) == side.cuda_stream


def test_serving_calls(dev, side):
    from sub_bit_moe_amd import api
    T, H, Hk, D = 5, 4, 2, 64
    x = torch.randn(T, H + 2 * Hk, D, device=dev).half()
    q, k, v = x[:, :H], x[:, H:H + Hk], x[:, H + Hk:]
    cache = api.alloc_kv_cache(8, Hk, D, 16, dev)
    lens, new = V.i32([2, 0], dev), V.i32([3, 2], dev)
    table = V.i32([[0, -1], [-1, -1]], dev)
    free, n_free = V.i32([5, 6, 7], dev), V.i32([3], dev)
    side.wait_stream(torch.cuda.current_stream())
    plan = api.kv_plan(lens, new, free, n_free, table, 8, 16, T, stream=side)
    _owned(side, plan.slots, plan.error)
    _owned(side, *api.qk_norm_rope(q, k, None, None, None, None, stream=side))
    _owned(side, api.qk_norm_rope_store(q, k, v, None, None, None, None, plan.slots, cache, stream=side))
    _owned(side, *api.kv_load(cache, plan.slots, stream=side))
    out, lse = api.attention_kv4(q, cache, table, plan.kv_lens, cu_q=plan.cu_q, return_lse=True, stream=side)
    _owned(side, out, lse)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, api.attention_kv4(q, cache, table, plan.kv_lens, cu_q=plan.cu_q)) and int(plan.error) == 0


def test_expert_calls(dev, side):
    from sub_bit_moe_amd import api
    words, _ = api.build_dictionary(0.885)
    image = api.device_image(words, dev)
    d, f = 512, 768
    up, down = (api.ExpertStack.from_symbols([m for m, _ in e], [s for _, s in e], words, dev)
                for e in (P.host_experts(2, f, d, 0.886, 1), P.host_experts(2, d, f, 0.886, 2)))
    x = torch.randn(3, d, device=dev).half()
    ids = V.i32([0, 1, 0], dev)
    side.wait_stream(torch.cuda.current_stream())
    _owned(side, *api.decode_dense(up, 0, image, stream=side))
    _owned(side, api.moe_fused_decode_matvec(up, image, x, ids, stream=side))
    _owned(side, *api.moe_fused_ffn(up, down, image, x, ids, stream=side))
    _owned(side, *api.moe_fused_layers([up], [down], image, x, ids[None], stream=side))
    _owned(side, api.rms_glue(x, stream=side))


def test_calls_of_several_steps(dev, side):
    """The generator, which reads sizes back between its passes, and decode + library products: all on one stream."""
    from sub_bit_moe_amd import api, hybrid, synth
    words, checksum = api.build_dictionary(0.885)
    trie = torch.from_numpy(api.build_trie(words)).to(dev)
    table = torch.from_numpy(synth.scale_table().view("int16")).to(dev)
    image = api.device_image(words, dev)
    made = lambda **k: [api.generate_stack(7, 0, 2, m, *s, 0.885, trie, table, dict_checksum=checksum, **k)    # noqa: E731
                        for m, s in ((0, (768, 512)), (1, (512, 768)))]
    here = made()
    side.wait_stream(torch.cuda.current_stream())
    there = made(stream=side)
    for a, b in zip(here, there):
        _owned(side, b.codes, b.scales)
        assert bytes(a.host_desc[0]) + bytes(a.host_desc[1]) == bytes(b.host_desc[0]) + bytes(b.host_desc[1])
        for d in a.host_desc:
            part = slice(d.code_base, d.code_base + d.n_codes)
            assert torch.equal(a.codes[part], b.codes[part])
        assert torch.equal(a.scales, b.scales)
    x = torch.randn(3, 512, device=dev).half()
    side.wait_stream(torch.cuda.current_stream())
    y, h = hybrid.expert_ffn(*there, 1, image, x, stream=side)
    _owned(side, y, h)
    torch.cuda.current_stream().wait_stream(side)
    want = hybrid.expert_ffn(*here, 1, image, x)
    assert torch.equal(y, want[0]) and torch.equal(h, want[1])
