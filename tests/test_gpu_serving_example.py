"""The serving example: a prompt in one step, in pieces and token by token gives the same cache and hidden states."""
import importlib.util
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve.py")


def test_pieces_give_what_the_prompt_gives():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("serve_example", PATH)
    serve = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(serve)
    n, R = 150, 2
    g = torch.Generator(device="cuda").manual_seed(2)
    got = []
    x = [torch.randn(n, 2080, generator=g, device="cuda", dtype=torch.float16) for _ in range(R)]
    for pieces in ((n,), (100, 30) + (1,) * 20):
        d = serve.Decoder(1, R, n + 10, 2 * n, n_experts=8)
        ys, at = [[], []], 0
        for m in pieces:
            p = d.plan(torch.full((R,), m, dtype=torch.int32, device="cuda"), R * m)
            assert int(p.error) == 0
            y = d(torch.cat([t[at:at + m] for t in x]), p)
            for r in range(R):
                ys[r].append(y[r * m:(r + 1) * m])
            at += m
        assert d.context.tolist() == [n, n] and int(d.n_free) == d.n_blocks - R * -(-n // serve.BLOCK)
        got.append(torch.stack([torch.cat(t) for t in ys]).float())
    # products of other shapes round their sums to fp16 differently, which a 4-bit code may turn into its neighbour
    assert (got[0] - got[1]).norm() <= 0.02 * got[0].norm()


def test_the_example_runs():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    out = subprocess.run([sys.executable, PATH, "--layers", "1", "--requests", "3", "--prompt", "70", "--steps", "4"],
                         capture_output=True, text=True, timeout=110)
    assert out.returncode == 0, out.stderr[-2000:]
    assert "tokens/s" in out.stdout
