"""A decoder of compressed experts served in running batches: per step one plan of the paged cache, and in each layer the
norm and rotation of queries and keys with the 4-bit cache's writer, attention over the cache, and the layer's expert.

    python examples/serve.py [--layers 4] [--requests 32] [--prompt 700] [--steps 32]

Weights are random and experts are picked by the token's position: the example is about the calls.  Lengths, tables and the
free list stay on the GPU; the steps of single tokens are one captured graph.
"""
import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from sub_bit_moe_amd import api, stack  # noqa: E402

HEADS, KV_HEADS, DIM, BLOCK = 16, 4, 128, 32


class Decoder:
    def __init__(self, n_layers: int, n_requests: int, most_tokens: int, max_new: int, n_experts: int = 24, device="cuda",
                 seed: int = 5):
        """most_tokens: of a request; max_new: new tokens of one step."""
        self.experts = stack.build(stack.StackConfig(n_layers=n_layers, n_experts=n_experts, seed=seed, n_tokens=1), device)
        self.n_experts, self.d = n_experts, self.experts.cfg.d_model
        g = torch.Generator(device=device).manual_seed(seed)
        half = dict(dtype=torch.float16, device=device)
        rand = lambda *s: torch.randn(*s, generator=g, **half)                                   # noqa: E731
        self.qkv = [rand(self.d, (HEADS + 2 * KV_HEADS) * DIM) * self.d ** -0.5 for _ in range(n_layers)]
        self.out = [rand(HEADS * DIM, self.d) * (HEADS * DIM) ** -0.5 for _ in range(n_layers)]
        self.q_weight, self.k_weight = torch.ones(DIM, **half), torch.ones(DIM, **half)
        self.width = -(-most_tokens // BLOCK)
        self.n_blocks = n_requests * self.width
        self.caches = [api.alloc_kv_cache(self.n_blocks, KV_HEADS, DIM, BLOCK, device) for _ in range(n_layers)]
        self.rope = api.rope_table(most_tokens, DIM, device=device)
        # kept for all layers and steps
        self.attention_ws = api.alloc_attention_workspace(n_requests, max_new, HEADS, KV_HEADS, DIM, device)
        self.expert_ws = api.alloc_ffn_workspace(n_experts, max_new, device)
        ints = dict(dtype=torch.int32, device=device)
        self.free, self.n_free = torch.arange(self.n_blocks, **ints), torch.full((1,), self.n_blocks, **ints)
        self.table = torch.full((n_requests, self.width), -1, **ints)
        self.context = torch.zeros(n_requests, **ints)

    def plan(self, new_lens, max_tokens: int, plan=None):
        """Blocks for the step's new tokens; afterwards the requests hold them."""
        p = api.kv_plan(self.context, new_lens, self.free, self.n_free, self.table, self.n_blocks, BLOCK, max_tokens, plan=plan)
        self.context.copy_(p.kv_lens)
        self.n_free.copy_(p.n_free)
        return p

    def __call__(self, x, plan):
        """x [tokens, d] of the plan's tokens in order (past the last one: anything); returns the last layer's, fp16."""
        T = x.shape[0]
        experts = (plan.positions * 7 + plan.requests.clamp(min=0)) % self.n_experts
        for i, cache in enumerate(self.caches):
            qkv = torch.matmul(unit(x), self.qkv[i]).view(T, HEADS + 2 * KV_HEADS, DIM)
            q, k, v = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV_HEADS], qkv[:, HEADS + KV_HEADS:]
            q = api.qk_norm_rope_store(q, k, v, self.q_weight, self.k_weight, plan.positions, self.rope, plan.slots, cache)
            a = api.attention_kv4(q, cache, self.table, plan.kv_lens, cu_q=plan.cu_q, workspace=self.attention_ws)
            x = x + torch.matmul(a.view(T, HEADS * DIM), self.out[i])
            y, _ = api.moe_fused_ffn(self.experts.up[i], self.experts.down[i], self.experts.image, unit(x), experts,
                                     workspace=self.expert_ws, out_f32=True)
            x = x + unit(y).to(x.dtype)
        return x


def unit(x):
    """Rows at unit RMS."""
    f = x.float()
    return (f * torch.rsqrt((f * f).mean(-1, keepdim=True) + 1e-6)).to(torch.float16)


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--layers", type=int, default=4)
    p.add_argument("--requests", type=int, default=32)
    p.add_argument("--prompt", type=int, default=700)
    p.add_argument("--steps", type=int, default=32)
    a = p.parse_args()
    d = Decoder(a.layers, a.requests, a.prompt + a.steps + 8, max(a.requests, 2 * a.prompt))
    g = torch.Generator(device="cuda").manual_seed(1)
    # prompts, two requests at a time
    torch.cuda.synchronize()
    start = time.perf_counter()
    for r in range(0, a.requests, 2):
        new = torch.zeros(a.requests, dtype=torch.int32, device="cuda")
        new[r:r + 2] = a.prompt
        n = a.prompt * min(2, a.requests - r)
        d(torch.randn(n, d.d, generator=g, device="cuda", dtype=torch.float16), d.plan(new, n))
    torch.cuda.synchronize()
    print(f"prompts: {a.requests * a.prompt / (time.perf_counter() - start):.0f} tokens/s")
    # single tokens: each step's output is the next one's input
    one = torch.ones(a.requests, dtype=torch.int32, device="cuda")
    x = torch.randn(a.requests, d.d, generator=g, device="cuda", dtype=torch.float16)
    plan = api.alloc_kv_plan(a.requests, a.requests, d.table)

    def step():
        x.copy_(unit(d(x, d.plan(one, a.requests, plan))))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(a.steps):
        graph.replay()
    torch.cuda.synchronize()
    took = time.perf_counter() - start
    assert int(plan.error) == 0 and torch.isfinite(x).all()
    print(f"single tokens: {took / a.steps * 1e3:.3f} ms a step of {a.requests} requests, {a.requests * a.steps / took:.0f} tokens/s")


if __name__ == "__main__":
    main()
