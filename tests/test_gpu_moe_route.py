"""Routing to experts against 64 bits: the same experts in the same order, gates to a few roundings of fp32."""
import numpy as np
import pytest

from oracle import around as A
from tests import _around as R
from tests import _serving as V

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
# gates in fp32: an exponential and a sum of at most 4096 of them in 32 bits or more, a division, a product, a rounding
CLOSE = dict(rtol=2.0 ** -19, atol=1e-38)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _check(dev, l, k, bias=None, requests=None, dtype="fp32", place=None, **how):
    from sub_bit_moe_amd import api
    tl = place(l) if place else R.tensor(l, dtype, dev)
    error = torch.zeros(1, dtype=torch.int32, device=dev)
    ids, gates = api.moe_route(tl, k, bias=None if bias is None else R.tensor(bias, "fp32", dev),
                               requests=None if requests is None else V.i32(requests, dev), error=error, **how)
    want, g, refused = A.route(l, k, bias, requests=requests, **how)
    assert ids.dtype == torch.int32 and np.array_equal(ids.cpu().numpy(), want)
    assert gates.dtype == torch.float32
    np.testing.assert_allclose(V.array(gates), g, **CLOSE)
    assert int(error) == refused
    return ids, gates


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("E", [1, 2, 7, 8, 31, 60, 64, 65, 100, 128, 129, 255, 256, 257, 512, 513, 1000, 1024, 1025, 2048, 2049, 4095, 4096])
def test_sizes(dev, E, dtype):
    rng = np.random.default_rng(E)
    l = R.held(rng.standard_normal((5, E)), dtype)
    for k in {1, min(E, 3), min(E, 32)}:
        for sigmoid in (False, True):
            bias = R.held(0.1 * rng.standard_normal(E), "fp32")
            _check(dev, l, k, dtype=dtype, sigmoid=sigmoid)
            _check(dev, l, k, bias, dtype=dtype, sigmoid=sigmoid, renormalise=True, scale=2.5)


@pytest.mark.parametrize("E,groups,top,k", [(256, 8, 4, 8), (160, 8, 3, 6), (64, 64, 5, 5), (30, 10, 10, 30), (2048, 16, 2, 4), (4096, 64, 64, 32),
                                            (72, 9, 1, 8), (24, 3, 2, 1)])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_groups(dev, E, groups, top, k, best, sigmoid):
    rng = np.random.default_rng(E + k)
    l = R.held(1.5 * rng.standard_normal((33, E)), "fp32")
    l[4:9][rng.random((5, E)) < 0.6] = -np.inf
    for bias in (None, R.held(0.2 * rng.standard_normal(E), "fp32")):
        _check(dev, l, k, bias, sigmoid=sigmoid, n_groups=groups, top_groups=top, group_best=best, renormalise=True)


@pytest.mark.parametrize("T", [1, 3, 4, 5, 63, 1000])
def test_many_tokens(dev, T):
    rng = np.random.default_rng(T)
    l = R.held(rng.standard_normal((T, 96)), "bf16")
    _check(dev, l, 4, dtype="bf16")
    _check(dev, l, 4, R.held(0.02 * rng.standard_normal(96), "fp32"), dtype="bf16", n_groups=4, top_groups=2)


@pytest.mark.parametrize("E", [8, 64, 300, 2048])
def test_equal_scores_go_to_the_lowest_expert(dev, E):
    rng = np.random.default_rng(E)
    l = rng.choice([-2.0, 0.0, 1.0], (12, E))             # no two sums of two scores, biased or not, are equal
    l[0] = 0.0
    l[1, ::2] = -0.0
    l[1, 1::2] = 0.0
    bias = np.float64(rng.integers(0, 2, E)) / 4
    for sigmoid in (False, True):
        _check(dev, l, min(E, 8), sigmoid=sigmoid)
        _check(dev, l, min(E, 8), bias, sigmoid=sigmoid)
        _check(dev, l, min(E // 2, 8), bias, sigmoid=sigmoid, n_groups=4, top_groups=2, renormalise=True)


def test_masked_experts_padding_and_rows_without_a_distribution(dev):
    rng = np.random.default_rng(3)
    E = 40
    l = R.held(rng.standard_normal((12, E)), "fp32")
    l[0, 3:] = -np.inf                   # three left
    l[1] = -np.inf                       # nothing
    l[2, 7] = np.nan
    l[3, 39] = np.inf
    l[4, 1:] = -np.inf
    l[5] = 3.4e38
    l[6] = -3.4e38
    l[6, 5] = 3.4e38
    bias = R.held(0.1 * rng.standard_normal(E), "fp32")
    bias[9] = -np.inf
    requests = np.arange(12)
    requests[[8, 11]] = -1
    for b in (None, bias):
        for sigmoid in (False, True):
            for more in ({}, dict(renormalise=True), dict(n_groups=5, top_groups=2), dict(n_groups=20, top_groups=20, group_best=1)):
                k = 4
                _check(dev, l, k, b, requests, sigmoid=sigmoid, **more)
    bias[9] = np.nan
    ids, gates = _check(dev, l, 2, bias, requests)
    held = (ids >= 0).any(1).nonzero().flatten().tolist()
    assert held == [0, 4]                # whose logits leave that expert out


def test_scores_that_vanish(dev):
    """Sigmoid scores of 0 in 64 bits: gates stay 0, also divided by their sum."""
    l = np.full((3, 16), -1e4)
    l[1, 4] = 0.0
    _check(dev, l, 3, sigmoid=True, renormalise=True)
    _check(dev, l, 3, np.arange(16) / 64.0, sigmoid=True, renormalise=True)
    l = np.float64(np.float32([[60, 50.5, 50, 0, -700, -800, 40, 41]]))
    _check(dev, l, 8, sigmoid=True)
    _check(dev, l, 8)


def test_near_ties(dev):
    """Logits and biases of fp32's last bits: the order is that of 64 bits."""
    rng = np.random.default_rng(4)
    for E in (32, 256, 2048):
        base = R.held(rng.standard_normal((200, 1)) + 1.0, "fp32")
        l = np.float64(np.float32(base * (1 + 2.0 ** -23 * rng.integers(-3, 4, (200, E)))))
        _check(dev, l, 8)
        bias = R.held(1e-9 * rng.standard_normal(E), "fp32")
        for sigmoid in (False, True):
            _check(dev, l, 8, bias, sigmoid=sigmoid)
            _check(dev, l, 8, bias, sigmoid=sigmoid, n_groups=8, top_groups=3)


def test_strides_buffers_and_no_tokens(dev):
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(5)
    for dtype in ("fp32", "bf16"):
        l = R.held(rng.standard_normal((11, 70)), dtype)
        wide = torch.full((11, 200), float("nan"), dtype=R.DT[dtype], device=dev)
        wide[:, 5:75] = R.tensor(l, dtype, dev)
        _check(dev, l, 3, dtype=dtype, place=lambda _: wide[:, 5:75])
    ids = torch.full((12, 3), -7, dtype=torch.int32, device=dev)
    gates = torch.full((12, 3), -7.0, dtype=torch.float32, device=dev)
    got = api.moe_route(R.tensor(l, "fp32", dev), 3, ids=ids[:11], gates=gates[:11])
    assert got[0].data_ptr() == ids.data_ptr() and (ids[11] == -7).all() and (gates[11] == -7).all()
    assert api.moe_route(torch.empty(0, 9, device=dev), 2)[0].shape == (0, 2)


def test_offsets_past_32_bits(dev):
    from sub_bit_moe_amd import api
    l = torch.zeros(600000, 2048, device=dev)                              # 4.9 GB
    l[-1] = torch.randn(2048, device=dev)
    ids, gates = api.moe_route(l, 4)
    a, b = api.moe_route(l[-1:].clone(), 4)
    assert torch.equal(ids[-1:], a) and torch.equal(gates[-1:], b)
    assert torch.equal(ids[:-1], torch.arange(4, device=dev, dtype=torch.int32).expand(599999, 4))


def test_captured_on_a_stream_of_its_own_and_replayed(dev):
    from sub_bit_moe_amd import api
    l, bias = torch.randn(64, 2048, device=dev), 1e-3 * torch.randn(2048, device=dev)
    call = lambda **k: (*api.moe_route(l, 2, renormalise=True, **k), *api.moe_route(l, 6, bias=bias, sigmoid=True, n_groups=8, top_groups=3, **k))  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for i in range(3):
        l.copy_(torch.randn_like(l))
        want = call()
        torch.cuda.synchronize()
        graph.replay()
        there = call(stream=side)
        torch.cuda.synchronize()
        for a, b, c in zip(got, want, there):
            assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("E", [1, 40, 100, 128, 200, 256, 500, 1000, 2048, 4096])
@pytest.mark.parametrize("others", ["finite", "masked", "some"])
def test_no_number_at_any_place(dev, E, others):
    """A NaN or +inf at each of the places that a lane has, beside finite logits, beside -inf alone, and beside both."""
    rng = np.random.default_rng(E)
    at = sorted({0, E - 1, *(p for p in range(0, E, 64)), *(int(p) for p in rng.integers(0, E, 12)),
                 *(p + j for p in range(0, E, 256) for j in range(1, 4) if p + j < E)})
    l = R.held(rng.standard_normal((2 * len(at) + 2, E)), "fp32")
    if others == "masked":
        l[:] = -np.inf
    elif others == "some":
        l[rng.random(l.shape) < 0.9] = -np.inf
    for i, p in enumerate(at):
        l[2 * i, p], l[2 * i + 1, p] = np.nan, np.inf
    bias = R.held(0.1 * rng.standard_normal(E), "fp32")
    groups = next(g for g in (4, 5, 3, 1) if E % g == 0)
    k = min(3, E // groups)
    for b in (None, bias):
        for sigmoid in (False, True):
            for renormalise in (False, True):
                _check(dev, l, k, b, sigmoid=sigmoid, renormalise=renormalise)
                _check(dev, l, k, b, sigmoid=sigmoid, renormalise=renormalise, n_groups=groups, top_groups=max(1, groups // 2))
    _check(dev, l, k, requests=np.full(l.shape[0], -1))                # padding is not counted


def test_scores_far_below_the_largest(dev):
    """Softmax scores that 64 bits hold as denormals or not at all: the choice, the groups and the gates are those of 64 bits."""
    l = np.zeros((1, 16))
    l[0, 0], l[0, 3] = 1000.0, 100.0
    bias = np.zeros(16)
    bias[0] = -np.inf
    for k in (1, 2, 5):
        ids, gates = _check(dev, l, k, bias, renormalise=True)           # nothing is left of any score: gates stay 0
        assert not gates.any()
    l[0] = 0.0
    l[0, [0, 3, 7, 9]] = 1000.0, 300.0, 270.0, 330.0
    _check(dev, l, 4, bias, renormalise=True)
    _check(dev, l, 4, bias)
    l = np.float64([[0, -800, -720, -720, -700, -700], [0, -800, -700, -720, -720, -700], [-690, -690, -700, -680, 0, -1e5]])
    for best in (1, 2):
        ids, _ = _check(dev, l, 4, n_groups=3, top_groups=2, group_best=best)
        _check(dev, l, 4, n_groups=3, top_groups=2, group_best=best, renormalise=True)
        _check(dev, l, 4, np.float64([0, 0, 0, 0, 0, 0]), n_groups=3, top_groups=2, group_best=best, renormalise=True)
    assert ids[0].tolist() == [0, 4, 5, 1]


def test_sigmoid_scores_far_below_one(dev):
    """As far down as 64 bits hold 1 / (1 + e^-l)."""
    l = np.float64([[-500, -500, -501, -700, -5000, -5000], [-486, -485, -484, -490, -495, -600], [-708, -708.5, -709.5, -712, -745, -3e38],
                    [-712, -720, -745, -800, -1e4, -3e38]])
    l = np.float64(np.float32(l))
    for b in (None, np.zeros(6)):
        _check(dev, l, 2, b, sigmoid=True, renormalise=True)
        _check(dev, l, 4, b, sigmoid=True, renormalise=True, scale=2.5)
        _check(dev, l, 2, b, sigmoid=True, renormalise=True, n_groups=3, top_groups=1)
        _check(dev, l, 2, b, sigmoid=True, renormalise=True, n_groups=2, top_groups=1)


@pytest.mark.parametrize("E,groups", [(128, 64), (256, 32), (2048, 64), (60, 20)])
@pytest.mark.parametrize("size", [20.0, 1e3, 1e6])
def test_groups_whose_largest_cancel(dev, E, groups, size):
    """Biases of both signs, far larger than the scores: a group's value is what their sum leaves of them."""
    rng = np.random.default_rng(E + int(size))
    T, per = 400, E // groups
    l = R.held(rng.standard_normal((T, E)), "fp32")
    bias = np.full((groups, per), -2 * size)
    bias[:, 0], bias[:, 1] = size, -size
    bias = np.float64(np.float32(bias.reshape(-1)))
    for sigmoid in (False, True):
        _check(dev, l, 5, bias, sigmoid=sigmoid, n_groups=groups, top_groups=5, renormalise=True)


@pytest.mark.parametrize("lowest", [-3.4028234663852886e38, -3e38, -1.8e38, 1.8e38, 3.4028234663852886e38])
def test_groups_of_the_types_lowest_and_largest_biases(dev, lowest):
    """Experts kept back by the type's lowest value are experts still: their groups are chosen where there are no others."""
    rng = np.random.default_rng(6)
    for E, groups in ((12, 3), (256, 8), (2048, 16)):
        l = R.held(rng.standard_normal((9, E)), "fp32")
        per = E // groups
        bias = np.zeros((groups, per))
        bias[1:] = lowest
        bias[-1, 0] = 0.25
        bias = np.float64(np.float32(bias.reshape(-1)))
        for sigmoid in (False, True):
            for best in (1, 2):
                for top in (1, 2, groups):
                    k = min(per * top, 32)
                    ids, _ = _check(dev, l, k, bias, sigmoid=sigmoid, n_groups=groups, top_groups=top, group_best=best)
                    assert (ids >= 0).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("E", [1, 8, 60, 64, 128, 200, 256, 512, 1000, 1024, 2048, 4096])
def test_gates_to_what_is_claimed(dev, E, dtype):
    """Gates are of 64 bits (weights to 4e-14) and rounded to fp32: half a step, 2^-24.  A softmax that is not renormalised divides by a
    sum of fp32 exponentials, which adds, in units of 2^-24: 4 for an exponential, 2 for the additions of fours in 32 bits (the rest are in
    64), and for the exponent -t, whose difference and product are rounded once each to 2^-24 of t, 2 ln 2 times t: on the sum's
    average."""
    rng = np.random.default_rng(E + 1)
    l = 2 * rng.standard_normal((24, E))
    l[0] *= 20
    l = R.held(l, dtype)
    l[1:5][rng.random((4, E)) < 0.5] = -np.inf
    l[5] = 0.75
    t = np.where(l > -np.inf, (l.max(1, keepdims=True).clip(-1e30) - l) / np.log(2), 0.0)
    p = np.where(l > -np.inf, np.exp2(-t), 0.0)
    sums = 6 + 2 * np.log(2) * (p * t).sum(1, keepdims=True) / p.sum(1, keepdims=True).clip(1)
    bias = R.held(0.1 * rng.standard_normal(E), "fp32")
    groups = 4 if E % 4 == 0 else 1
    for k in {1, min(E // groups, 6)}:
        for b in (None, bias):
            for sigmoid in (False, True):
                for how in (dict(), dict(renormalise=True, scale=2.5), dict(n_groups=groups, top_groups=max(1, groups // 2)), dict(scale=0.1)):
                    how = {**how, "scale": float(np.float32(how.get("scale", 1.0)))}
                    _, gates = _check(dev, l, k, b, dtype=dtype, sigmoid=sigmoid, **how)
                    want = A.route(l, k, b, sigmoid=sigmoid, **how)[1]
                    units = 1 + (0 if sigmoid or how.get("renormalise") else sums)
                    assert (np.abs(V.array(gates) - want) <= (2.0 ** -24 * units + 1e-12) * want + 2.0 ** -149).all()
