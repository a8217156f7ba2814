"""The choice of the next token against 64 bits: the same tokens, probabilities to a few roundings of fp32."""
import numpy as np
import pytest

from oracle import around as A
from tests import _around as R
from tests import _serving as V

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
# logprobs in fp32 from 64 bits: half a step, and weights that are whole multiples of 2^-42
CLOSE = dict(rtol=2.0 ** -23, atol=1e-9)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _check(dev, l, u, dtype="fp32", place=None, **how):
    """how: temperature, top_k, top_p, min_p of each row."""
    from sub_bit_moe_amd import api
    tl = place(l) if place else R.tensor(l, dtype, dev)
    how = {n: np.broadcast_to(v, u.shape) for n, v in how.items()}
    f = {n: V.i32(v, dev) if n == "top_k" else R.tensor(np.array(v, np.float64), "fp32", dev) for n, v in how.items()}
    error = torch.zeros(1, dtype=torch.int32, device=dev)
    tokens, logprobs = api.sample(tl, R.tensor(u, "fp32", dev), return_logprobs=True, error=error, **f)
    want = [A.sample(l[r], float(np.float32(u[r])), **{n: int(v[r]) if n == "top_k" else float(np.float32(v[r])) for n, v in how.items()})
            for r in range(len(u))]
    got = tokens.cpu().numpy()
    assert tokens.dtype == torch.int32 and got.tolist() == [t for t, _ in want]
    np.testing.assert_allclose(V.array(logprobs), [p for _, p in want], **CLOSE)
    assert int(error) == sum(t < 0 for t, _ in want)
    return tokens, logprobs


def _mixed(rng, n):
    return dict(temperature=rng.choice([0.0, 0.3, 0.7, 1.0, 1.3, 5.0], n), top_k=rng.choice([0, 0, 1, 2, 20, 50, 1000], n),
                top_p=rng.choice([1.0, 1.0, 0.0, 0.1, 0.5, 0.9, 0.95, 0.999], n), min_p=rng.choice([0.0, 0.0, 0.01, 0.1, 1.0], n))


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("vocab", [1, 2, 3, 63, 64, 65, 255, 1000, 1023, 1024, 1025, 4097, 8191, 32000, 32769, 50021, 131072, 262144 + 3])
def test_sizes(dev, vocab, dtype):
    rng = np.random.default_rng(vocab)
    n = 40 if vocab < 10000 else 12
    l = R.logits_case(rng, n, vocab, dtype)
    _check(dev, l, rng.random(n), dtype)
    for _ in range(3):
        _check(dev, l, rng.random(n), dtype, **_mixed(rng, n))


@pytest.mark.parametrize("rows", [1, 2, 3, 7, 16, 33, 100, 257, 600])
def test_rows(dev, rows):
    rng = np.random.default_rng(rows)
    l = R.logits_case(rng, rows, 5000, "bf16")
    _check(dev, l, rng.random(rows), "bf16", **_mixed(rng, rows))


def test_the_largest_vocabulary(dev):
    rng = np.random.default_rng(1)
    l = R.logits_case(rng, 4, 1 << 20, "fp32")
    _check(dev, l, rng.random(4), temperature=[1.0, 1.0, 0.0, 2.0], top_p=[1.0, 0.9, 1.0, 0.99], top_k=[0, 0, 0, 100000])
    l[:] = 0.0                                                            # 2^20 weights of one
    tokens, logprobs = _check(dev, l, np.array([0.0, 0.25, 0.5, 1.0]), top_p=[1.0, 0.5, 0.5, 0.25])
    assert tokens.tolist() == [0, 1 << 17, 1 << 18, (1 << 18) - 1]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_equal_logits(dev, dtype):
    """Few values, each many times: filters end inside a run of equal ones, which the lower index wins."""
    rng = np.random.default_rng(2)
    for vocab, values in ((100, 2), (5000, 3), (40000, 5), (40000, 1), (131072, 20)):
        l = np.float64(rng.integers(0, values, (8, vocab)))
        l[1, : vocab // 2] = -np.inf
        l[2] *= -0.0
        _check(dev, l, rng.random(8), dtype)
        _check(dev, l, rng.random(8), dtype, top_k=[1, 3, 17, 50, vocab // 2, vocab - 1, vocab, vocab + 5])
        _check(dev, l, rng.random(8), dtype, top_p=[0.0, 0.1, 0.123, 0.3, 0.51, 0.77, 0.9, 0.99], temperature=0.8)
        _check(dev, l, rng.random(8), dtype, top_p=0.6, top_k=[vocab // 3] * 8, min_p=[0, 0.1, 0.3, 0.4, 0.5, 0.9, 1.0, 2.0], temperature=1.7)


def test_draws_at_the_ends(dev):
    rng = np.random.default_rng(3)
    l = R.logits_case(rng, 10, 3000)
    u = np.array([0.0, -0.0, -1.0, 1.0, 2.0, 1 - 2.0 ** -24, 2.0 ** -149, np.inf, -np.inf, 0.5])
    _check(dev, l, u)
    _check(dev, l, u, top_k=1)
    _check(dev, l, u, top_p=0.7, top_k=30)


def test_rows_without_a_distribution(dev):
    rng = np.random.default_rng(4)
    n = 14
    l = R.logits_case(rng, n, 700)
    l[0, 699] = np.nan
    l[1, 0] = np.inf
    l[2] = -np.inf
    l[3, 1:] = -np.inf
    l[4] = -np.inf
    l[4, 350] = -3.4e38
    u, t, k, p, m = rng.random(n), np.ones(n), np.zeros(n), np.ones(n), np.zeros(n)
    u[5] = t[6] = p[7] = m[8] = np.nan
    t[9] = -1.0
    t[10] = np.inf
    p[11], m[12], k[13] = -3.0, -3.0, -5
    tokens, _ = _check(dev, l, u, temperature=t, top_k=k, top_p=p, min_p=m)
    assert tokens.tolist()[3:5] == [0, 350]


def test_far_logits_and_extreme_temperatures(dev):
    rng = np.random.default_rng(5)
    n = 8
    l = np.float64(np.float32(rng.standard_normal((n, 2000)) * np.array([[1e-3, 1, 1e2, 1e4, 1e30, 1e-30, 1e37, 3]]).T))
    u = rng.random(n)
    _check(dev, l, u)
    _check(dev, l, u, temperature=[1e-3, 1e-2, 1e2, 1e4, 1e30, 1e-30, 1e37, 1e-38], top_p=0.9)
    _check(dev, l, u, temperature=[1e-38, 1e38, 1e-6, 1e6, 1e-3, 1e3, 1e-2, 1e2], top_k=700)
    l = np.tile(np.float64(np.float32(np.linspace(-40, 40, 3001))), (n, 1))         # a slope: every bin has its share
    _check(dev, l, u, temperature=[0.1, 0.5, 1, 2, 5, 10, 40, 100], top_p=0.999)
    _check(dev, l, u, temperature=[0.1, 0.5, 1, 2, 5, 10, 40, 100], top_k=[2500, 3000, 1500, 3001, 2, 1000, 2999, 77])


def test_wide_filters(dev):
    """Filters that keep tens of thousands of tokens."""
    rng = np.random.default_rng(6)
    n, vocab = 10, 100003
    l = R.held(rng.standard_normal((n, vocab)), "fp32")
    _check(dev, l, rng.random(n), top_p=np.linspace(0.5, 0.9999, n))
    _check(dev, l, rng.random(n), top_k=np.linspace(20000, 99999, n), top_p=0.97)
    _check(dev, l, rng.random(n), top_k=30000, min_p=0.05, temperature=2.5, top_p=np.linspace(0.3, 0.99, n))
    l = R.held(l, "bf16")
    _check(dev, l, rng.random(n), "bf16", top_p=np.linspace(0.5, 0.9999, n), top_k=70000)


def test_frequencies_are_the_probabilities(dev):
    """Evenly spaced numbers give each token its share, to one draw."""
    from sub_bit_moe_amd import api
    p = np.array([0.4, 0.05, 0.25, 0.0, 0.3])
    with np.errstate(divide="ignore"):
        l = torch.from_numpy(np.log(p)).float().to(dev)
    n = 4096
    got = torch.bincount(api.sample(l.expand(n, 5), (torch.arange(n, device=dev) + 0.5) / n).long(), minlength=5)
    assert np.abs(got.cpu().numpy() - n * p).max() <= 1.001


def test_strides_and_buffers(dev):
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(7)
    for dtype in ("fp32", "bf16"):
        l = R.logits_case(rng, 9, 1001, dtype)
        wide = torch.full((9, 1500), float("nan"), dtype=R.DT[dtype], device=dev)
        wide[:, 3:1004] = R.tensor(l, dtype, dev)
        _check(dev, l, rng.random(9), dtype, place=lambda _: wide[:, 3:1004], top_k=40)
    u = torch.rand(9, device=dev)
    tokens, logprobs = torch.full((10,), -7, dtype=torch.int32, device=dev), torch.full((10,), -7.0, device=dev)
    got = api.sample(wide[:, 3:1004], u, tokens=tokens[:9], logprobs=logprobs[:9])
    assert got[0].data_ptr() == tokens.data_ptr() and int(tokens[9]) == -7 and float(logprobs[9]) == -7
    assert torch.equal(api.sample(wide[:, 3:1004], u), tokens[:9])
    assert api.sample(wide[:0, 3:1004], u[:0]).shape == (0,)


def test_workspace_of_anything_is_used_again(dev):
    """Calls of other sizes and types one after the other in one workspace, whatever it held."""
    from sub_bit_moe_amd import api
    ws = torch.full((max(api.sample_workspace_bytes(r, v) for r, v in ((2, 200000), (70, 9000), (300, 100))),), 0xA5, dtype=torch.uint8, device=dev)
    for rows, vocab, dtype in ((1, 200000, torch.float32), (70, 9000, torch.bfloat16), (300, 100, torch.float16), (2, 200000, torch.bfloat16)):
        l, u = (3 * torch.randn(rows, vocab, device=dev)).to(dtype), torch.rand(rows, device=dev)
        p = torch.full((rows,), 0.9, device=dev)
        want = api.sample(l, u, top_p=p)
        for _ in range(3):
            assert torch.equal(api.sample(l, u, top_p=p, workspace=ws), want)
        ws.random_(0, 255)


def test_a_workspace_serves_smaller_calls(dev):
    """One made for the most rows and tokens, for every step of a batch that shrinks."""
    from sub_bit_moe_amd import api
    ws = api.alloc_sample_workspace(600, 70000, dev)
    for rows, vocab in ((600, 70000), (300, 70000), (256, 70000), (255, 40000), (100, 33000), (3, 70000), (1, 50)):
        l, u = 3 * torch.randn(rows, vocab, device=dev), torch.rand(rows, device=dev)
        k = torch.full((rows,), 300, dtype=torch.int32, device=dev)
        assert torch.equal(api.sample(l, u, top_k=k, workspace=ws), api.sample(l, u, top_k=k))


def test_offsets_past_32_bits(dev):
    from sub_bit_moe_amd import api
    l = torch.zeros(9000, 250000, dtype=torch.bfloat16, device=dev)          # 4.5 GB
    l[-1] = (3 * torch.randn(250000, device=dev)).bfloat16()
    u = torch.full((9000,), 0.5, device=dev)
    got = api.sample(l, u)
    assert torch.equal(got[-1:], api.sample(l[-1:].clone(), u[-1:])) and (got[:-1] == 125000).all()


def test_more_rows_than_a_launch_has(dev):
    from sub_bit_moe_amd import api
    n = (1 << 22) + 5
    l = torch.zeros(n, 2, device=dev)
    l[::3, 1] = 50.0
    got = api.sample(l, torch.full((n,), 0.5, device=dev))              # a tie's second half; the likely one
    assert (got == 1).all()
    l[::3, 0] = 100.0
    got = api.sample(l, torch.full((n,), 0.5, device=dev))
    assert (got[::3] == 0).all() and (got[1::3] == 1).all() and (got[2::3] == 1).all()


def test_captured_on_a_stream_of_its_own_and_replayed(dev):
    from sub_bit_moe_amd import api
    for rows, vocab in ((3, 70000), (40, 3000)):
        l, u = torch.randn(rows, vocab, device=dev), torch.rand(rows, device=dev)
        p, k = torch.full((rows,), 0.8, device=dev), torch.full((rows,), 500, dtype=torch.int32, device=dev)
        call = lambda **o: api.sample(l, u, top_p=p, top_k=k, return_logprobs=True, **o)         # noqa: E731
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = call()
        for i in range(3):
            l.copy_(2 * torch.randn_like(l))
            want = call()
            torch.cuda.synchronize()
            graph.replay()
            there = call(stream=side)
            torch.cuda.synchronize()
            for a, b, c in zip(got, want, there):
                assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("vocab", [3, 700, 5000, 40000, 100003])
def test_filters_that_end_near_the_types_lowest(dev, vocab):
    """Logits from -3.4e38 to -3.05e38 and temperatures at which their weights differ: a filter's end lies among them."""
    rng = np.random.default_rng(vocab)
    n = 12
    l = np.float64(np.float32(-3.05e38 - 0.35e38 * rng.random((n, vocab))))
    l[:, :3] = np.float64(np.float32([-3.05e38, -3.1e38, -3.3e38]))
    l[3, 3:] = -np.inf
    l[4, 1:] = np.float64(np.float32(-3.4028234e38))
    u = rng.random(n)
    u[0] = 0.9
    for t in (1e38, 3e37, 3e36):
        for how in (dict(), dict(min_p=0.9), dict(min_p=0.3), dict(top_p=0.4), dict(top_p=0.9), dict(top_p=0.9, min_p=0.8), dict(top_k=2),
                    dict(top_k=max(vocab // 2, 1)), dict(top_k=max(vocab // 3, 1), top_p=0.7, min_p=0.75)):
            _check(dev, l, u, temperature=t, **how)
            _check(dev, R.held(l, "bf16"), u, "bf16", temperature=t, **how)


@pytest.mark.parametrize("vocab", [32768, 32769, 47104, 48128, 48129, 49151, 49152, 49153, 65536])
def test_rows_of_one_and_of_several_workgroups(dev, vocab):
    """Around the lengths from which a row no longer stays in registers, and from which workgroups share it."""
    rng = np.random.default_rng(vocab)
    for rows in (1, 5, 130):
        l = R.logits_case(rng, rows, vocab, "bf16")
        _check(dev, l, rng.random(rows), "bf16", **_mixed(rng, rows))
