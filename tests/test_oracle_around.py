"""Pins of the oracle of the operators around the experts, against their definitions by other ways."""
import numpy as np
import pytest
import torch

from oracle import around as A


def test_e4m3_is_torchs():
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn)
    assert np.array_equal(A.E4M3, codes.double().numpy())
    rng = np.random.default_rng(0)
    a = (rng.standard_normal(4096) * np.exp2(rng.integers(-12, 8, 4096))).astype(np.float32)
    a = a[np.abs(a) <= 448]
    assert np.array_equal(A.to_e4m3(a.astype(np.float64)), torch.from_numpy(a).to(torch.float8_e4m3fn).double().numpy())
    # halves to the even code, above and below the least normal number
    for x, y in ((1.0625, 1.0), (1.1875, 1.25), (2.0 ** -10, 0.0), (1.5 * 2.0 ** -9, 2.0 ** -8), (500.0, 448.0), (-464.0, -448.0)):
        assert A.to_e4m3(np.array([x]))[0] == y


@pytest.mark.parametrize("block", [0, 32, 128])
def test_fp8_is_within_half_a_step_and_fills_its_range(block):
    rng = np.random.default_rng(1)
    y = rng.standard_normal((40, 300)) * np.exp(4 * rng.standard_normal((40, 1)))
    v, scales, powers = A.fp8(y, block)
    unit = np.repeat(scales, block or 300, 1)[:, :300]
    a = np.abs(y) / unit
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(a, 1e-30))), -6) - 3)
    assert (np.abs(v - y) <= step / 2 * unit * (1 + 1e-12) + (a > 448) * 1e-4 * unit).all()
    top = np.stack([a[:, d:d + (block or 300)].max(1) for d in range(0, 300, block or 300)], 1)
    assert (top <= 448 * (1 + 2.0 ** -23)).all() and (top > (224 if block == 32 else 447.99)).all()
    assert powers is None or np.array_equal(np.exp2(powers - 127.0), scales)


def test_norm_of_known_rows():
    h, size = A.state([[3.0, 4.0], [np.nan, 1.0]], [[0.5, 0.0]], [[1.5, 3.0]])
    assert h.tolist() == [[3.0, 5.0]] and size.tolist() == [[3.0, 5.0]]
    assert np.allclose(A.rms_norm(np.array([[3.0, 4.0]]), eps=0.0), np.array([[3, 4]]) / np.sqrt(12.5))


def test_route_is_softmax_and_topk():
    rng = np.random.default_rng(2)
    l = rng.standard_normal((20, 24))
    ids, gates, refused = A.route(l, 3)
    p, i = torch.from_numpy(l).softmax(1).topk(3)
    assert refused == 0 and np.array_equal(ids, i.numpy()) and np.allclose(gates, p.numpy(), rtol=1e-13)
    ids, gates, _ = A.route(l, 3, renormalise=True, scale=2.0)
    assert np.allclose(gates.sum(1), 2.0)
    # groups: only the best group's experts, by its two largest
    l[:] = 0
    l[:, [1, 5, 6]] = [3.0, 2.0, 2.0]
    ids, _, _ = A.route(l, 2, n_groups=6, sigmoid=True)
    assert (ids == [5, 6]).all()
    ids, _, _ = A.route(l, 2, n_groups=6, sigmoid=True, group_best=1)
    assert (ids == [1, 0]).all()


def test_kept_and_sample_by_hand():
    l = np.log([0.5, 0.2, 0.2, 0.1])
    keep = lambda **k: A.kept(l, **k)[0].tolist()                            # noqa: E731
    assert keep() == [0, 1, 2, 3] and keep(top_k=2) == [0, 1] and keep(min_p=0.3) == [0, 1, 2] and keep(top_p=0.6) == [0, 1]
    assert keep(top_p=0.0) == [0] and keep(top_k=3, top_p=0.75) == [0, 1] and keep(top_k=3, top_p=0.8) == [0, 1, 2]
    assert keep(temperature=0.0, top_k=3) == [0]
    assert [A.sample(l, u)[0] for u in (0.0, 0.499, 0.51, 0.69, 0.71, 0.95, 1.0)] == [0, 0, 1, 1, 2, 3, 3]
    assert abs(A.sample(l, 0.6, top_k=2)[1] - np.log(0.5 / 0.7)) < 1e-12 or A.sample(l, 0.6, top_k=2)[0] == 0
    assert A.sample([-np.inf, -np.inf], 0.5)[0] == A.sample([0.0, np.nan], 0.5)[0] == A.sample([0.0, np.inf], 0.5)[0] == -1


def test_choice_near_the_types_lowest():
    l = [-3.05e38, -3.1e38, -3.3e38]
    assert A.kept(l, temperature=1e38, min_p=0.9)[0].tolist() == [0, 1] and A.kept(l, temperature=1e38, top_p=0.5)[0].tolist() == [0, 1]
    assert A.kept(l, temperature=1e38, top_p=0.3)[0].tolist() == [0] and A.kept(l, temperature=1e38)[0].tolist() == [0, 1, 2]
    assert A.sample(l, 0.9, temperature=1e38, min_p=0.9)[0] == 1


def test_a_row_of_masks_with_no_number_is_refused():
    for bad in (np.nan, np.inf):
        for at in (0, 1, 100, 127):
            l = np.full((1, 128), -np.inf)
            l[0, at] = bad
            for how in (dict(), dict(bias=np.zeros(128)), dict(n_groups=4), dict(sigmoid=True), dict(renormalise=True)):
                ids, gates, refused = A.route(l, 2, **how)
                assert refused == 1 and (ids == -1).all() and not gates.any()
    assert A.route(np.full((1, 128), -np.inf), 2)[2] == 0


def test_scores_far_below_the_largest():
    l, bias = np.zeros((1, 16)), np.zeros(16)
    l[0, 0], l[0, 3], bias[0] = 1000.0, 100.0, -np.inf
    ids, gates, _ = A.route(l, 2, bias, renormalise=True)
    assert ids.tolist() == [[1, 2]] and gates.tolist() == [[0.0, 0.0]]
    ids, _, _ = A.route([[0, -800, -720, -720, -700, -700]], 4, n_groups=3, top_groups=2)
    assert ids.tolist() == [[0, 4, 5, 1]]
    ids, gates, _ = A.route([[-500.0, -500.0, -700.0]], 2, sigmoid=True, renormalise=True)
    assert ids.tolist() == [[0, 1]] and gates.tolist() == [[0.5, 0.5]]


def test_groups_by_what_cancels_and_by_the_types_lowest():
    # scores 1/4 each: values 0.5, 0.5 + 0.125 and the lowest
    ids, _, _ = A.route([[0.0] * 4], 1, [1e6, -1e6, 1e6, -1e6 + 0.125], n_groups=2)
    assert ids.tolist() == [[2]]
    ids, _, _ = A.route([[0.0] * 4], 3, [0.0, 0.0, -3.4028234663852886e38, -3.4028234663852886e38], n_groups=2, top_groups=2)
    assert ids.tolist() == [[0, 1, 2]]


def test_scales_of_results_past_32_bits():
    y = np.zeros((3, 32))
    y[0, 0], y[1, 3], y[2, 5] = 1e39, 2.0 ** 128, 6.1e40
    v, scales, powers = A.fp8(y, 32)
    assert powers[:, 0].tolist() == [248, 247, 254]
    assert v[1, 3] == 2.0 ** 128 and abs(v[0, 0] / 1e39 - 1) < 2.0 ** -4 and np.isfinite(v).all()
