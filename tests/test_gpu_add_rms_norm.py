"""Norm with the residual's addition and the sum over a token's experts, 16- and 8-bit results, against 64 bits."""
import numpy as np
import pytest

from oracle import around as A
from tests import _around as R
from tests import _serving as V

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
EPS = 1e-6


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _check(dev, x, g, r, w, dtype="bf16", x_type=None, r_type=None, eps=EPS, repeat=1, block=None, place=None):
    """One call against the oracle; place: makes a tensor of values (for strides)."""
    from sub_bit_moe_amd import api
    place = place or (lambda v, t: R.tensor(v, t, dev))
    x_type, r_type = x_type or dtype, r_type or dtype
    k = 1 if g is None else g.shape[1]
    tx = place(x, x_type)
    tg = None if g is None else R.tensor(g, "fp32", dev)
    tr = None if r is None else place(r, r_type)
    tw = None if w is None else R.tensor(w, dtype, dev)
    how = dict(weight=tw, residual=tr, gates=tg, eps=eps, repeat=repeat, dtype=R.DT[dtype])
    y, dy, h, dh = R.norm_bounds(x, g, r, w, eps, k, dtype, r_type)
    if block is None:
        out, res = api.add_rms_norm(tx, **how)
        got = V.array(out)
        assert out.dtype == R.DT[dtype] and got.shape == (y.shape[0] * repeat, y.shape[1])
        assert (np.abs(got - y.repeat(repeat, 0)) <= dy.repeat(repeat, 0)).all()
    else:
        codes, scales, res = api.add_rms_norm_fp8(tx, scale_block=block, **how)
        want, unit, powers = A.fp8(y, block)
        n = block or y.shape[1]
        s = scales.cpu().numpy() if powers is None else np.exp2(scales.cpu().numpy() - 127.0)
        assert np.array_equal(s, unit.repeat(repeat, 0)) and (powers is None or np.array_equal(scales.cpu().numpy(), powers.repeat(repeat, 0)))
        got = codes.double().cpu().numpy() * np.repeat(s.astype(np.float64), n, 1)[:, :y.shape[1]]
        assert np.array_equal(got, want.repeat(repeat, 0))
    if r is None:
        assert res is None
    else:
        assert res.dtype == R.DT[r_type] and (np.abs(V.array(res) - h) <= dh).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [1, 2, 7, 8, 9, 63, 64, 65, 100, 511, 512, 513, 1000, 2080, 4099, 8192, 8200, 16384, 16391, 32767, 32768])
def test_widths(dev, D, dtype):
    rng = np.random.default_rng(D)
    _check(dev, *R.norm_case(rng, 3, D, dtype=dtype, gates=False), dtype=dtype)


@pytest.mark.parametrize("dtype,x_type,r_type", [("bf16", "bf16", "fp32"), ("fp16", "fp32", "fp16"), ("bf16", "fp32", "fp32"), ("fp16", "fp16", "fp32"),
                                                 ("fp16", "fp32", "fp32"), ("bf16", "fp32", "bf16")])
@pytest.mark.parametrize("T,D,k,repeat", [(5, 2080, 1, 1), (17, 768, 2, 2), (3, 333, 8, 3), (64, 130, 4, 1), (2, 20001, 3, 2)])
@pytest.mark.parametrize("block", [None, 0, 32])
def test_types_experts_and_repeats(dev, T, D, k, repeat, dtype, x_type, r_type, block):
    rng = np.random.default_rng(T * D + k)
    _check(dev, *R.norm_case(rng, T, D, k, dtype, x_type, r_type), dtype=dtype, x_type=x_type, r_type=r_type, repeat=repeat, block=block)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("block", [0, 32, 128])
@pytest.mark.parametrize("D", [1, 31, 32, 33, 127, 128, 129, 512, 520, 2080, 8192, 12000, 32768])
def test_eight_bits(dev, D, block, dtype):
    rng = np.random.default_rng(D + block)
    _check(dev, *R.norm_case(rng, 7, D, dtype=dtype, gates=False), dtype=dtype, block=block)


def test_every_code_and_border(dev):
    """Rows whose results are e4m3 numbers, borders between two, and what is beside those."""
    from sub_bit_moe_amd import api
    D = 32
    borders = np.concatenate([A.E4M3, (A.E4M3[1:] + A.E4M3[:-1]) / 2])
    a = np.concatenate([borders * s for s in (1, 1 + 2.0 ** -22, 1 - 2.0 ** -22)])
    a = np.concatenate([a, -a, np.zeros(-2 * a.size % (D - 1))]).reshape(-1, D - 1)
    x = np.concatenate([np.full((a.shape[0], 1), 448.0), a], 1)
    x = np.float64(np.float32(x))
    # an eps beside which the mean is nothing: the norm divides by 2^60
    want, unit, powers = A.fp8(A.rms_norm(x, None, 2.0 ** 120), 32)
    codes, scales, _ = api.add_rms_norm_fp8(R.tensor(x, "fp32", dev), eps=2.0 ** 120, scale_block=32, dtype=torch.bfloat16)
    assert np.array_equal(scales.cpu().numpy(), powers)
    assert np.array_equal(codes.double().cpu().numpy() * unit, want)


@pytest.mark.parametrize("block", [None, 0, 32])
def test_strides_and_odd_addresses(dev, block):
    """Columns of a joint array, from any element on; rows behind one another are read as they stand."""
    rng = np.random.default_rng(5)
    T, D = 9, 261

    def place(v, t):
        wide = torch.full((v.shape[0], 3 * D + 5), float("nan"), dtype=R.DT[t], device=dev)
        wide[:, 3:3 + D] = R.tensor(v, t, dev)
        return wide[:, 3:3 + D]

    _check(dev, *R.norm_case(rng, T, D, 2, "fp16"), dtype="fp16", place=place, repeat=2, block=block)
    # one row for all tokens
    x, g, r, w = R.norm_case(rng, T, D, gates=False)
    r[:] = r[0]
    _check(dev, x, g, r, w, place=lambda v, t: R.tensor(v[:1], t, dev).expand(T, D) if v is r else R.tensor(v, t, dev), block=block)


def test_results_in_place_and_into_slices(dev):
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(6)
    T, D = 21, 900
    x, _, r, w = R.norm_case(rng, T, D, gates=False)
    y, dy, h, dh = R.norm_bounds(x, None, r, w, EPS, 1, "bf16", "bf16")
    tx, tr, tw = (R.tensor(v, "bf16", dev) for v in (x, r, w))
    joint = torch.zeros(T, 2 * D + 3, dtype=torch.bfloat16, device=dev)
    out, res = api.add_rms_norm(tx, tw, tr, out=joint[:, 1:1 + D], residual_out=joint[:, D + 2:2 * D + 2])
    assert (np.abs(V.array(out) - y) <= dy).all() and (np.abs(V.array(res) - h) <= dh).all()
    assert not joint[:, 0].any() and not joint[:, D + 1].any() and not joint[:, -1].any()
    first = out.clone(), res.clone()
    out, res = api.add_rms_norm(tx, tw, tr, out=tx, residual_out=tr)
    assert out is tx and res is tr and torch.equal(tx, first[0]) and torch.equal(tr, first[1])
    # and the sum alone in a buffer, without a residual before
    tx, buf = R.tensor(x, "bf16", dev), torch.empty(T, D, dtype=torch.float32, device=dev)
    _, res = api.add_rms_norm(tx, tw, residual_out=buf)
    assert res is buf and torch.equal(buf, tx.float())


def test_a_gate_of_zero_takes_no_part(dev):
    rng = np.random.default_rng(7)
    x, g, r, w = R.norm_case(rng, 6, 300, 3, "fp16", "fp32")
    g[0] = 0.0
    g[1, 1] = g[2, 0] = -0.0
    x[0:3] = np.nan
    x[4] = np.inf
    x[6] = np.nan
    _check(dev, x, g, r, w, dtype="fp16", x_type="fp32")
    _check(dev, x, g, r, w, dtype="fp16", x_type="fp32", block=128)


@pytest.mark.parametrize("block", [None, 0, 32, 128])
def test_rows_of_zeros_infinities_and_nan(dev, block):
    from sub_bit_moe_amd import api
    x = np.random.default_rng(8).standard_normal((5, 200))
    x[0] = 0
    x[1, 150] = np.nan
    x[2, 3] = np.inf
    x[3, 3] = -np.inf
    x = R.held(x, "bf16")
    tx = R.tensor(x, "bf16", dev)
    y = A.rms_norm(x)
    if block is None:
        got = V.array(api.add_rms_norm(tx)[0])
        assert np.array_equal(np.isnan(got), np.isnan(y)) and not got[0].any() and not np.nan_to_num(got[2:4]).any()
        return
    codes, scales, _ = api.add_rms_norm_fp8(tx, scale_block=block)
    want, unit, powers = A.fp8(y, block)
    if powers is None:
        assert np.array_equal(scales.cpu().numpy(), unit, equal_nan=True)
    else:
        assert np.array_equal(scales.cpu().numpy(), powers)
    got = codes.double().cpu().numpy() * np.repeat(unit, block or 200, 1)[:, :200]
    assert np.array_equal(got, want, equal_nan=True)
    assert not codes.view(torch.uint8)[torch.from_numpy(np.isnan(want)).to(dev)].any()


@pytest.mark.parametrize("size,eps", [(1e36, 1e-6), (1e19, 0.0), (1e-20, 0.0), (1e-36, 0.0), (1e-30, 1e-6)])
@pytest.mark.parametrize("block", [None, 32])
def test_rows_whose_squares_32_bits_do_not_hold(dev, size, eps, block):
    rng = np.random.default_rng(9)
    x, _, _, w = R.norm_case(rng, 3, 1000, gates=False)
    _check(dev, R.held(x * size, "bf16"), None, None, w, eps=eps, block=block)


def test_no_rows_and_many_rows(dev):
    from sub_bit_moe_amd import api
    e = torch.empty(0, 64, dtype=torch.float16, device=dev)
    out, res = api.add_rms_norm(e, residual=e)
    assert out.shape == res.shape == (0, 64)
    out, _ = api.add_rms_norm(e, gates=torch.empty(0, 2, dtype=torch.float32, device=dev), repeat=2)
    assert out.shape == (0, 64)
    rng = np.random.default_rng(10)
    _check(dev, *R.norm_case(rng, 70001, 16, dtype="fp16", gates=False), dtype="fp16")


def test_more_rows_than_a_launch_has(dev):
    from sub_bit_moe_amd import api
    for n, D in (((1 << 21) + 3, 512), ((1 << 26) + 37, 8)):            # a row to a workgroup; 32 to one
        x = torch.ones(n, D, dtype=torch.float16, device=dev)
        x[n // 2:] = -2.0
        out, _ = api.add_rms_norm(x, eps=0.0)
        assert (out[:n // 2] == 1).all() and (out[n // 2:] == -1).all()


def test_offsets_past_32_bits(dev):
    from sub_bit_moe_amd import api
    x = torch.zeros(140000, 16400, dtype=torch.bfloat16, device=dev)          # 4.6 GB
    x[-1] = torch.randn(16400, device=dev).bfloat16()
    out, _ = api.add_rms_norm(x)
    assert torch.equal(out[-1:], api.add_rms_norm(x[-1:].clone())[0]) and not out[:-1].any()


def test_captured_on_a_stream_of_its_own_and_replayed(dev):
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(11)
    x, g, r, w = R.norm_case(rng, 32, 2080, 2, "fp16", "fp32", "fp32")
    tx, tg, tr, tw = R.tensor(x, "fp32", dev), R.tensor(g, "fp32", dev), R.tensor(r, "fp32", dev), R.tensor(w, "fp16", dev)
    call = lambda **k: (*api.add_rms_norm(tx, tw, tr, gates=tg, repeat=2, **k),                  # noqa: E731
                        *api.add_rms_norm_fp8(tx, tw, tr, gates=tg, scale_block=32, **k))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for i in range(3):
        tx.copy_(torch.randn_like(tx))
        want = call()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        there = call(stream=side)
        torch.cuda.synchronize()
        for a, b in zip(there, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("block", [0, 32, 128])
@pytest.mark.parametrize("dtype,r_type", [("bf16", "bf16"), ("bf16", "fp32")])
@pytest.mark.parametrize("D", [32, 100, 256, 2080, 8200, 32768])
def test_eight_bits_of_results_past_32_bits(dev, D, block, dtype, r_type):
    """bf16 weights up to the type's largest: finite results from 2^128 on have scales and codes as the smaller ones do."""
    rng = np.random.default_rng(D + block)
    x, g, r, w = R.norm_case(rng, 6, D, dtype=dtype, x_type="fp32", r_type=r_type, gates=False)
    w = R.held(np.where(rng.random(D) < 0.5, 3.3e38, 1e38) * rng.uniform(0.5, 1.0, D), "bf16")
    x[0] = r[0] = x[4] = r[4] = 0.0
    x[0, D // 2], x[4, 0] = 7.0, -1e-3                        # alone in their rows: sqrt(D) times their weights
    x[1] *= 1e-3
    x = R.held(x, "fp32")
    w[0], w[D // 2] = R.held([3.3e38, 3.3895e38], "bf16")
    _check(dev, x, None, r, w, dtype=dtype, x_type="fp32", r_type=r_type, block=block)
    w[:] = R.held([3.3895e38], "bf16")
    _check(dev, x, None, r, w, dtype=dtype, x_type="fp32", r_type=r_type, block=block)
    x[2, D - 1], x[3, 1] = np.nan, np.inf                      # which are still no numbers
    _check_bad(dev, x, w, block)


def _check_bad(dev, x, w, block):
    from sub_bit_moe_amd import api
    codes, scales, _ = api.add_rms_norm_fp8(R.tensor(x, "fp32", dev), R.tensor(w, "bf16", dev), scale_block=block)
    want, unit, powers = A.fp8(A.rms_norm(x, w), block)
    assert np.array_equal(scales.cpu().numpy(), unit if powers is None else powers, equal_nan=True)
    got = codes.double().cpu().numpy() * np.repeat(unit, block or x.shape[1], 1)[:, :x.shape[1]]
    assert np.array_equal(got, want, equal_nan=True)


def test_every_code_and_border_of_the_smallest_scale(dev):
    """Results below the least normal number of 32 bits: e4m3 numbers, borders between two, and what is beside those."""
    from sub_bit_moe_amd import api
    D = 32
    borders = np.concatenate([A.E4M3, (A.E4M3[1:] + A.E4M3[:-1]) / 2])
    a = np.concatenate([borders * s for s in (1, 1 + 2.0 ** -22, 1 - 2.0 ** -22)])
    a = np.concatenate([a, -a, np.zeros(-2 * a.size % D)])
    a = a[np.argsort(np.abs(a), kind="stable")].reshape(-1, D)             # rows of like sizes
    for power in (-126, -127, -130):
        x = np.float64(np.float32(a * 2.0 ** (power + 60)))
        # an eps beside which the mean is nothing: the norm divides by 2^60
        y = A.rms_norm(x, None, 2.0 ** 120)
        for block in (32, 0, 128):
            want, unit, powers = A.fp8(y, block)
            codes, scales, _ = api.add_rms_norm_fp8(R.tensor(x, "fp32", dev), eps=2.0 ** 120, scale_block=block, dtype=torch.bfloat16)
            assert np.array_equal(scales.cpu().numpy(), unit if powers is None else powers)
            assert np.array_equal(codes.double().cpu().numpy() * unit, want)


@pytest.mark.parametrize("block", [0, 128])
def test_borders_with_scales_that_are_no_powers_of_two(dev, block):
    """Results that are a scale times a border between two codes go to the even one, whatever the scale's reciprocal rounds to."""
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(12)
    borders = (A.E4M3[1:] + A.E4M3[:-1]) / 2
    unit = 1 + rng.integers(0, 1 << 18, 400) / 2.0 ** 18                   # 448 and borders times these are fp32 numbers
    x = np.concatenate([448 * unit[:, None], unit[:, None] * borders[None]], 1)[:, :127]
    assert np.array_equal(x, np.float64(np.float32(x)))
    want, scale, _ = A.fp8(A.rms_norm(x, None, 2.0 ** 120), block)         # the norm divides by 2^60
    codes, scales, _ = api.add_rms_norm_fp8(R.tensor(x, "fp32", dev), eps=2.0 ** 120, scale_block=block, dtype=torch.bfloat16)
    assert np.array_equal(scales.cpu().numpy(), scale)
    assert np.array_equal(codes.double().cpu().numpy() * scale, want)


@pytest.mark.parametrize("block", [0, 32])
def test_the_sum_beside_8_bit_results_is_rounded_once(dev, block):
    """bf16 residuals below the least normal number: between two, with something beside the middle."""
    m = np.arange(1, 128)
    D = m.size
    x = np.stack([(2 * m + 1) * 2.0 ** -133, np.full(D, 2.0 ** -126), (2 * m + 1) * 2.0 ** -133, np.full(D, -2.0 ** -126),
                  (2 * m + 1) * 2.0 ** -133, np.zeros(D)])
    x = R.held(x, "fp32")
    g = np.float64([[0.5, 2.0 ** -30], [-0.5, 2.0 ** -30], [0.5, 1.0]])
    from sub_bit_moe_amd import api
    r = np.zeros((3, D))
    _, _, res = api.add_rms_norm_fp8(R.tensor(x, "fp32", dev), None, R.tensor(r, "bf16", dev), gates=R.tensor(g, "fp32", dev), scale_block=block)
    want = np.stack([m + 1, -(m + 1), np.where(m % 2, m + 1, m)]) * 2.0 ** -133
    assert np.array_equal(V.array(res), want)
