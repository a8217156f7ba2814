"""Norms, routing, experts and sampling as a decoder step runs them: one mixture layer against 64 bits, padding among its tokens; and
the whole in a captured graph, replayed beside eager calls."""
import numpy as np
import pytest

from oracle import around as A
from oracle import codec as OC
from tests import _around as R
from tests import _parity as P
from tests import _serving as V

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
D, F, E, VOCAB = 512, 768, 6, 1500


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


@pytest.fixture(scope="module")
def layer(dev):
    from sub_bit_moe_amd import api
    words, _ = api.build_dictionary(0.885)
    host = [P.host_experts(E, F, D, 0.886, 1), P.host_experts(E, D, F, 0.886, 2)]
    up, down = (api.ExpertStack.from_symbols([m for m, _ in e], [s for _, s in e], words, dev) for e in host)
    dense = [[OC.dequantize(m, s) for m, s in e] for e in host]
    rng = np.random.default_rng(3)
    router, unembed = rng.standard_normal((D, E)) * D ** -0.5, rng.standard_normal((D, VOCAB)) * 3 * D ** -0.5
    return dict(up=up, down=down, image=api.device_image(words, dev), dense=dense, router=R.tensor(router, "fp32", dev),
                unembed=R.tensor(unembed, "fp32", dev), weight=R.tensor(1 + 0.2 * rng.standard_normal(D), "fp16", dev))


def _step(layer, x, residual, requests, u, k, ws=None):
    """norm, router, experts, norm of their sum, logits, tokens: everything that is made on the way."""
    from sub_bit_moe_amd import api
    T = x.shape[0]
    h, r1 = api.add_rms_norm(x, layer["weight"], residual, repeat=k)
    logits = torch.matmul(h[::k].float(), layer["router"])
    ids, gates = api.moe_route(logits, k, renormalise=True, scale=0.05, requests=requests)
    y, _ = api.moe_fused_ffn(layer["up"], layer["down"], layer["image"], h, ids.view(-1), out_f32=True,
                             workspace=ws and ws["ffn"], y=ws and ws["y"])
    out, r2 = api.add_rms_norm(y, layer["weight"], r1, gates=gates)
    codes, scales, r3 = api.add_rms_norm_fp8(y, layer["weight"], r1, gates=gates, scale_block=32)
    vocab = torch.matmul(out.float(), layer["unembed"])
    token, logprob = api.sample(vocab, u, temperature=torch.full((T,), 0.7, device=x.device), top_p=torch.full((T,), 0.9, device=x.device),
                                top_k=torch.full((T,), 40, dtype=torch.int32, device=x.device), return_logprobs=True)
    return dict(h=h, r1=r1, logits=logits, ids=ids, gates=gates, y=y, out=out, r2=r2, codes=codes, scales=scales, r3=r3, vocab=vocab,
                token=token, logprob=logprob)


def _inputs(dev, T, seed, padded=0):
    rng = np.random.default_rng(seed)
    x, _, r, _ = R.norm_case(rng, T, D, dtype="fp16", gates=False)
    requests = np.arange(T)
    requests[T - padded:] = -1
    return R.tensor(x, "fp16", dev), R.tensor(r, "fp16", dev), V.i32(requests, dev), R.tensor(rng.random(T), "fp32", dev)


@pytest.mark.parametrize("T,k,padded", [(1, 1, 0), (1, 3, 0), (13, 2, 4), (150, 2, 5)])
def test_a_layer(dev, layer, T, k, padded):
    x, residual, requests, u = _inputs(dev, T, 10 * T + k, padded)
    y = torch.full((T * k, D), float("nan"), device=dev)              # rows of padding are left as they are
    s = {n: t.cpu() for n, t in _step(layer, x, residual, requests, u, k, dict(ffn=None, y=y)).items()}
    w = V.array(layer["weight"])
    # each part from what the part before made
    want, dy, h, dh = R.norm_bounds(V.array(x), None, V.array(residual), w, 1e-6, 1, "fp16", "fp16")
    assert (np.abs(V.array(s["h"]) - want.repeat(k, 0)) <= dy.repeat(k, 0)).all() and (np.abs(V.array(s["r1"]) - h) <= dh).all()
    ids, gates, _ = A.route(V.array(s["logits"]), k, renormalise=True, scale=0.05, requests=requests.cpu().numpy())
    assert np.array_equal(s["ids"].numpy(), ids)
    np.testing.assert_allclose(V.array(s["gates"]), gates, rtol=2.0 ** -19)
    rows = V.array(s["h"])
    for i in range(T * k):
        e = ids.reshape(-1)[i]
        got = V.array(s["y"][i])
        if e < 0:
            assert np.isnan(got).all()
            continue
        up, down = layer["dense"][0][e], layer["dense"][1][e]
        P.assert_close(got, down @ np.maximum(up @ rows[i], 0), rl2=2e-3, mr=1e-2, what=f"row {i}")
    want, dy, h, dh = R.norm_bounds(V.array(s["y"]), V.array(s["gates"]), V.array(s["r1"]), w, 1e-6, k, "fp16", "fp16")
    assert (np.abs(V.array(s["out"]) - want) <= dy).all() and (np.abs(V.array(s["r2"]) - h) <= dh).all()
    assert (np.abs(V.array(s["r3"]) - h) <= dh).all()                 # rounded from 64 bits, not from 32
    values, unit, powers = A.fp8(want, 32)
    assert np.array_equal(s["scales"].numpy(), powers)
    assert np.array_equal(s["codes"].double().numpy() * np.repeat(unit, 32, 1), values)
    for t in range(T):
        token, logprob = A.sample(V.array(s["vocab"][t]), float(u[t]), temperature=float(np.float32(0.7)),
                                  top_k=40, top_p=float(np.float32(0.9)))
        assert int(s["token"][t]) == token and abs(float(s["logprob"][t]) - logprob) <= 1e-6


def test_captured_and_replayed_beside_eager_steps(dev, layer):
    """Two graphs and eager calls share a workspace, one after the other."""
    from sub_bit_moe_amd import api
    T, k = 24, 2
    ws = dict(ffn=api.alloc_ffn_workspace(E, T * k, dev), y=torch.zeros(T * k, D, device=dev))
    x, residual, requests, u = _inputs(dev, T, 99, 3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(layer, x, residual, requests, u, k, ws)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            made = _step(layer, x, residual, requests, u, k, ws)
        graphs.append((g, made))
    for i in range(3):
        new = _inputs(dev, T, 200 + i, i)
        for a, b in zip((x, residual, requests, u), new):
            a.copy_(b)
        ws["y"].zero_()
        want = {n: t.clone() for n, t in _step(layer, x, residual, requests, u, k, ws).items()}
        torch.cuda.synchronize()
        for g, made in graphs:
            g.replay()
            torch.cuda.synchronize()
            # the experts' row sums depend on the order of their atomics; everything that follows depends on them
            for n in ("h", "r1", "logits", "ids", "gates"):
                assert torch.equal(made[n], want[n]), n
            got = V.array(made["out"])
            assert np.linalg.norm(got - V.array(want["out"])) <= 2e-3 * np.linalg.norm(got)
            assert ((made["token"] >= 0) & (made["token"] < VOCAB)).all() and torch.isfinite(made["logprob"]).all()
            # and what was made from this replay's own rows is what an eager call makes of them
            out, r2 = api.add_rms_norm(made["y"], layer["weight"], made["r1"], gates=made["gates"])
            assert torch.equal(out, made["out"]) and torch.equal(r2, made["r2"])
            how = dict(temperature=torch.full((T,), 0.7, device=dev), top_p=torch.full((T,), 0.9, device=dev),
                       top_k=torch.full((T,), 40, dtype=torch.int32, device=dev))
            assert torch.equal(api.sample(made["vocab"], u, **how), made["token"])


def test_the_example_routes_and_samples(dev):
    """A decoder with a router and a vocabulary, padding among its tokens."""
    import importlib.util
    import os
    spec = importlib.util.spec_from_file_location("serve_example", os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                                                                "examples", "serve.py"))
    serve = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(serve)
    d = serve.Decoder(2, 3, 40, 64, n_experts=8, top_k=2, vocab=900)
    p = d.plan(V.i32([9, 0, 20], dev), 31)                              # two tokens of padding
    assert int(p.error) == 0
    y = d(torch.randn(31, d.d, device=dev, dtype=torch.float16), p)
    assert torch.isfinite(y[:29]).all()
    t = d.next_tokens(y, p, torch.tensor([0.1, 0.5, 0.9], device=dev), top_k=V.i32([1, 5, 0], dev))
    assert ((t >= 0) & (t < 900)).all()
