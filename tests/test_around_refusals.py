"""What the operators around the experts refuse, before anything is launched (no GPU needed)."""
import ctypes as C

import pytest

from sub_bit_moe_amd import _native as N
from sub_bit_moe_amd import api

EINVAL, ENOSPACE = -1, -6
A = 1 << 20                                # aligned addresses that nothing reads, apart
NORM = dict(x=A, xs=64, gates=0, k=1, res=2 * A, rs=64, w=3 * A, eps=1e-6, T=3, D=64, ro=4 * A, ros=64, out=5 * A, os=64, repeat=1, scales=0, block=0,
            flags=0)
FP8 = {**NORM, "flags": N.SBM_F_OUT_FP8, "scales": 6 * A, "block": 32}
ROUTE = dict(l=A, ls=64, bias=0, req=0, T=3, E=64, k=2, G=1, top=1, best=2, scale=1.0, ids=2 * A, gates=3 * A, flags=0, err=0)
SAMPLE = dict(l=A, ls=100, R=3, V=100, u=2 * A, t=0, tk=0, tp=0, mp=0, tok=3 * A, lp=0, flags=0, ws=4 * A, n=1 << 30, err=0, reserved=0)


def _norm(x, xs, gates, k, res, rs, w, eps, T, D, ro, ros, out, os, repeat, scales, block, flags):
    a = N.NormArgs(x, xs, gates, res, rs, w, ro, ros, out, os, scales, eps, T, D, k, repeat, block, flags)
    return N.lib().sbm_add_rms_norm(C.byref(a), None)


def _route(l, ls, bias, req, T, E, k, G, top, best, scale, ids, gates, flags, err):
    return N.lib().sbm_moe_route(C.byref(N.RouteArgs(l, ls, bias, req, ids, gates, err, scale, T, E, k, G, top, best, flags)), None)


def _sample(l, ls, R, V, u, t, tk, tp, mp, tok, lp, flags, ws, n, err, reserved):
    a = N.SampleArgs(l, ls, u, t, tk, tp, mp, tok, lp, ws, n, err, R, V, flags, reserved)
    return N.lib().sbm_sample(C.byref(a), None)


@pytest.mark.parametrize("change", [
    dict(T=-1), dict(D=0), dict(D=32769), dict(k=0), dict(k=65, gates=7 * A), dict(k=2), dict(repeat=0), dict(repeat=65), dict(eps=-1.0),
    dict(eps=float("nan")), dict(flags=1), dict(block=32), dict(xs=-1), dict(rs=-1), dict(ros=-1), dict(os=-64), dict(os=63), dict(ros=63),
    dict(repeat=2, T=1, os=0), dict(x=0), dict(out=0), dict(x=A + 1), dict(res=2 * A + 1), dict(w=3 * A + 1), dict(ro=4 * A + 1), dict(out=5 * A + 1),
    dict(gates=7 * A + 2), dict(flags=N.SBM_F_IN_F32, x=A + 2), dict(flags=N.SBM_F_RESIDUAL_F32, res=2 * A + 2),
    # outputs over inputs and each other
    dict(out=A + 2), dict(out=A - 2), dict(out=A, repeat=2), dict(out=A, k=2, gates=7 * A), dict(out=A, os=65), dict(out=A, flags=N.SBM_F_IN_F32),
    dict(out=2 * A), dict(out=3 * A + 126), dict(out=4 * A), dict(out=4 * A + 382), dict(ro=2 * A + 2), dict(ro=2 * A, ros=65), dict(ro=A),
    dict(gates=5 * A + 380), dict(ro=3 * A)])
def test_norm(change):
    assert _norm(**{**NORM, **change}) == EINVAL
    assert N.lib().sbm_last_error()


@pytest.mark.parametrize("change", [dict(block=64), dict(block=-1), dict(scales=0), dict(scales=5 * A + 100), dict(scales=A), dict(block=0, scales=6 * A + 2),
                                    dict(out=A), dict(scales=4 * A + 300)])
def test_norm_in_8_bits(change):
    assert _norm(**{**FP8, **change}) == EINVAL


@pytest.mark.parametrize("change", [
    dict(T=-1), dict(E=0), dict(E=4097), dict(k=0), dict(k=33), dict(k=65), dict(G=0), dict(G=65), dict(G=5), dict(G=4, top=5), dict(G=4, top=0),
    dict(G=32, top=1, k=3), dict(best=0), dict(best=3), dict(ls=-1), dict(scale=float("inf")), dict(scale=float("nan")), dict(flags=1),
    dict(flags=N.SBM_F_IN_BF16 | N.SBM_F_IN_F32), dict(l=0), dict(ids=0), dict(gates=0), dict(l=A + 1), dict(l=A + 2, flags=N.SBM_F_IN_F32),
    dict(bias=5 * A + 2), dict(req=5 * A + 1), dict(ids=2 * A + 2), dict(gates=3 * A + 2), dict(err=6 * A + 2), dict(ids=A), dict(gates=A + 380),
    dict(gates=2 * A + 20), dict(req=2 * A), dict(bias=3 * A), dict(err=A + 4), dict(err=2 * A + 20)])
def test_route(change):
    assert _route(**{**ROUTE, **change}) == EINVAL
    assert N.lib().sbm_last_error()


@pytest.mark.parametrize("change,status", [
    (dict(R=-1), EINVAL), (dict(V=0), EINVAL), (dict(V=(1 << 20) + 1), EINVAL), (dict(ls=-1), EINVAL), (dict(flags=2), EINVAL),
    (dict(flags=N.SBM_F_IN_BF16 | N.SBM_F_IN_F32), EINVAL), (dict(l=0), EINVAL), (dict(u=0), EINVAL), (dict(tok=0), EINVAL), (dict(ws=0), EINVAL),
    (dict(l=A + 1), EINVAL), (dict(l=A + 2, flags=N.SBM_F_IN_F32), EINVAL), (dict(u=2 * A + 2), EINVAL), (dict(t=6 * A + 1), EINVAL),
    (dict(tk=6 * A + 2), EINVAL), (dict(tp=6 * A + 2), EINVAL), (dict(mp=6 * A + 2), EINVAL), (dict(tok=3 * A + 2), EINVAL), (dict(lp=6 * A + 2), EINVAL),
    (dict(err=6 * A + 1), EINVAL), (dict(ws=4 * A + 8), EINVAL), (dict(n=0), ENOSPACE), (dict(tok=A), EINVAL), (dict(tok=2 * A + 8), EINVAL),
    (dict(lp=3 * A + 8), EINVAL), (dict(ws=A), EINVAL), (dict(err=3 * A + 8), EINVAL), (dict(tk=3 * A), EINVAL), (dict(lp=4 * A), EINVAL),
    (dict(reserved=1), EINVAL)])
def test_sample(change, status):
    assert _sample(**{**SAMPLE, **change}) == status
    assert N.lib().sbm_last_error()


def test_nothing_to_do_is_no_error():
    assert _norm(**{**NORM, "T": 0, "x": 0}) == 0
    assert _route(**{**ROUTE, "T": 0, "l": 0}) == 0
    assert _sample(**{**SAMPLE, "R": 0, "l": 0}) == 0


def test_no_arguments():
    assert N.lib().sbm_add_rms_norm(None, None) == N.lib().sbm_moe_route(None, None) == N.lib().sbm_sample(None, None) == EINVAL


def test_packed_arguments_are_the_structures():
    for pack, kind in ((api._pack_norm, N.NormArgs), (api._pack_route, N.RouteArgs), (api._pack_sample, N.SampleArgs)):
        v = [0.5 if t in (C.c_double, C.c_float) else 3 + i for i, (_, t) in enumerate(kind._fields_)]
        assert pack(*v) == bytes(kind(*v))


def test_sizes():
    assert api.sample_workspace_bytes(3, 100) > 0
    for bad in ((-1, 100), (3, 0), (3, (1 << 20) + 1)):
        assert api.sample_workspace_bytes(*bad) == 0


def test_front_end():
    torch = pytest.importorskip("torch")
    x, f = torch.zeros(4, 8, dtype=torch.float16), torch.zeros(4, 8)
    one, i = torch.zeros(4), torch.zeros(4, dtype=torch.int32)
    for call, kind, text in (
            (lambda: api.add_rms_norm(x), ValueError, "on the GPU"),
            (lambda: api.add_rms_norm(x[0]), ValueError, "tokens"),
            (lambda: api.add_rms_norm(f), ValueError, "dtype must be given"),
            (lambda: api.add_rms_norm(x.double()), TypeError, "float16 or bfloat16"),
            (lambda: api.add_rms_norm(x, gates=torch.zeros(3, 2)), ValueError, "gates"),
            (lambda: api.add_rms_norm(x, repeat=0), ValueError, "on the GPU|repeat"),
            (lambda: api.moe_route(f[0], 1), ValueError, "logits"),
            (lambda: api.moe_route(f.double(), 1), TypeError, "float32"),
            (lambda: api.moe_route(f, 1), ValueError, "on the GPU"),
            (lambda: api.sample(f, one), ValueError, "on the GPU"),
            (lambda: api.sample(i.view(2, 2), one), TypeError, "float32")):
        with pytest.raises(kind, match=text):
            call()
