"""sbm_kv_plan against the oracle's step, exactly; refusals change nothing."""
import numpy as np
import pytest

from oracle import serving as S
from tests import _serving as V

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _case(rng, R, bs, ctx_most, new_most):
    ctx = rng.integers(0, ctx_most + 1, R)
    new = rng.integers(0, new_most + 1, R) * (rng.random(R) < 0.7)
    edge = rng.random(R) < 0.5                     # contexts at a block's border
    ctx = np.where(edge, ctx // bs * bs, ctx)
    held = -(-ctx // bs)
    need = int((-(-(ctx + new) // bs) - held).sum())
    n_blocks = int(held.sum()) + need + 6
    ids = rng.permutation(n_blocks)
    width = int((-(-(ctx + new) // bs)).max(initial=0)) + 1
    table = np.full((R, width), -7, np.int32)
    at = 0
    for i in range(R):
        table[i, :held[i]] = ids[at:at + held[i]]
        at += held[i]
    return ctx, new, ids[at:], table, n_blocks


def _run(api, dev, ctx, new, free, table, n_blocks, bs, max_tokens, n_free=None, stream=None):
    t = V.i32(table, dev)
    args = (V.i32(ctx, dev), V.i32(new, dev), V.i32(free, dev), V.i32([len(free) if n_free is None else n_free], dev), t)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    p = api.kv_plan(*args, n_blocks, bs, max_tokens, stream=stream)
    if stream is not None:
        torch.cuda.current_stream().wait_stream(stream)
    return p, args


def _check(p, ref):
    got = (p.block_table, p.slots, p.positions, p.requests, p.cu_q, p.kv_lens, p.n_free)
    for name, g, w in zip("table slots positions requests cu_q kv_lens n_free".split(), got, ref):
        assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1)), name


@pytest.mark.parametrize("R,bs,ctx,new", [(1, 16, 0, 1), (1, 16, 40, 300), (3, 32, 100, 5), (64, 16, 500, 1),
                                          (255, 16, 60, 40), (256, 64, 300, 3), (257, 128, 4000, 700), (1000, 16, 90, 2),
                                          (4096, 16, 40, 30)])
def test_plan_is_the_oracles(dev, R, bs, ctx, new):
    from sub_bit_moe_amd import api
    rng = np.random.default_rng(R + bs)
    c, n, free, table, n_blocks = _case(rng, R, bs, ctx, new)
    max_tokens = int(n.sum()) + 9
    p, args = _run(api, dev, c, n, free, table, n_blocks, bs, max_tokens)
    ref = S.plan(c, n, free, table, bs, max_tokens)
    _check(p, ref)
    assert int(p.error) == 0
    # again, on what the first call left (its table has the new columns): the same
    p2 = api.kv_plan(*args, n_blocks, bs, max_tokens, plan=p)
    _check(p2, ref)
    # exactly as many places as tokens, and another stream
    p3, _ = _run(api, dev, c, n, free, table, n_blocks, bs, int(n.sum()), stream=torch.cuda.Stream())
    _check(p3, S.plan(c, n, free, table, bs, int(n.sum())))


def test_plan_without_requests_or_tokens(dev):
    from sub_bit_moe_amd import api
    p, _ = _run(api, dev, [], [], [3], np.zeros((0, 2)), 4, 16, 5)
    assert p.slots.tolist() == [-1] * 5 and p.cu_q.tolist() == [0] and p.n_free.tolist() == [1]
    p, _ = _run(api, dev, [5, 0], [0, 0], [3], [[2, -1], [-1, -1]], 4, 16, 0)
    assert p.cu_q.tolist() == [0, 0, 0] and p.kv_lens.tolist() == [5, 0] and int(p.error) == 0


@pytest.mark.parametrize("what", ["pool", "n_free below zero", "n_free past the list", "width", "context below zero",
                                  "new below zero", "context too long", "tokens", "one request's tokens"])
def test_refused_plan_changes_nothing(dev, what):
    from sub_bit_moe_amd import _native as N
    from sub_bit_moe_amd import api
    ctx, new, free = [20, 3, 0], [30, 1, 17], [9, 8, 7, 6, 5]
    table = [[1, 2, -1, -1], [3, -1, -1, -1], [-1] * 4]
    bs, n_free, max_tokens, bit = 16, None, 60, None
    if what == "pool":
        free, bit = [9, 8, 7], N.SBM_PLAN_EPOOL
    elif what == "n_free below zero":
        n_free, bit = -1, N.SBM_PLAN_EPOOL
    elif what == "n_free past the list":
        n_free, bit = 6, N.SBM_PLAN_EPOOL
    elif what == "width":
        new, bit = [45, 1, 17], N.SBM_PLAN_EWIDTH
    elif what == "context below zero":
        ctx, bit = [20, -3, 0], N.SBM_PLAN_ELENGTH
    elif what == "new below zero":
        new, bit = [30, -1, 17], N.SBM_PLAN_ELENGTH
    elif what == "context too long":
        ctx, bit = [20, 2 ** 30 + 1, 0], N.SBM_PLAN_ELENGTH
    elif what == "tokens":
        max_tokens, bit = 47, N.SBM_PLAN_ETOKENS
    else:
        new, bit = [2 ** 31 - 1, 1, 17], N.SBM_PLAN_ETOKENS
    p, args = _run(api, dev, ctx, new, free, table, 10, bs, max_tokens, n_free)
    assert int(p.error) & bit
    assert p.block_table.tolist() == table and p.n_free.tolist() == args[3].tolist()
    assert p.slots.tolist() == [-1] * max_tokens and p.cu_q.tolist() == [0] * 4
    assert p.kv_lens.tolist() == [max(c, 0) for c in ctx]
    assert p.requests.tolist() == [-1] * max_tokens and p.positions.tolist() == [0] * max_tokens


def test_blocks_outside_the_cache_get_no_slot(dev):
    from sub_bit_moe_amd import _native as N
    from sub_bit_moe_amd import api
    # request 0's last held block and the second block popped are outside
    p, _ = _run(api, dev, [20, 0], [14, 20], [4, 99, 5], [[1, -5, -1], [-1] * 3], 10, 16, 40)
    assert int(p.error) == N.SBM_PLAN_EBLOCK
    assert p.slots.tolist()[:14] == [-1] * 12 + [80, 81]
    assert p.slots.tolist()[14:34] == [-1] * 16 + [64, 65, 66, 67]
