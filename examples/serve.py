"""A decoder of compressed experts served in running batches: per step one plan of the paged cache, and in each layer the
norm and rotation of queries and keys with the 4-bit cache's writer, attention over the cache, the routing, and the experts;
the norms between them add what came before to the residual stream, and each step ends with the choice of the next tokens.

    python examples/serve.py [--layers 4] [--requests 32] [--prompt 700] [--steps 32] [--top-k 2] [--vocab 32000]

Weights are random: the example is about the calls.  Lengths, tables, the free list and the tokens stay on the GPU; the steps of
single tokens are one captured graph.
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
                 seed: int = 5, top_k: int = 0, vocab: int = 0):
        """most_tokens: of a request; max_new: new tokens of one step; top_k: experts of a token, chosen by a router (0: one, picked
        by the token's position)."""
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
        self.expert_ws = api.alloc_ffn_workspace(n_experts, max_new * max(top_k, 1), device)
        self.top_k = top_k
        if top_k:
            self.router = [rand(self.d, n_experts) * self.d ** -0.5 for _ in range(n_layers)]
        if vocab:
            self.embedding, self.unembed = rand(vocab, self.d), rand(self.d, vocab) * 3 * self.d ** -0.5
            self.sample_ws = api.alloc_sample_workspace(n_requests, vocab, device)
        ints = dict(dtype=torch.int32, device=device)
        self.free, self.n_free = torch.arange(self.n_blocks, **ints), torch.full((1,), self.n_blocks, **ints)
        self.table = torch.full((n_requests, self.width), -1, **ints)
        self.context = torch.zeros(n_requests, **ints)
        # random experts' results at unit size
        n = min(8, max_new)
        h, _ = api.add_rms_norm(rand(n, self.d))
        y, _ = self.ffn(0, h, torch.arange(n, **ints) % n_experts)
        self.gain = float(y.square().mean()) ** -0.5

    def ffn(self, i: int, h, ids):
        e = self.experts
        return api.moe_fused_ffn(e.up[i], e.down[i], e.image, h, ids, workspace=self.expert_ws, out_f32=True)

    def plan(self, new_lens, max_tokens: int, plan=None):
        """Blocks for the step's new tokens; afterwards the requests hold them."""
        p = api.kv_plan(self.context, new_lens, self.free, self.n_free, self.table, self.n_blocks, BLOCK, max_tokens, plan=plan)
        self.context.copy_(p.kv_lens)
        self.n_free.copy_(p.n_free)
        return p

    def __call__(self, x, plan):
        """x [tokens, d] of the plan's tokens in order (past the last one: anything); returns the residual stream, fp16."""
        T, k = x.shape[0], max(self.top_k, 1)
        rows = gates = None                        # the experts' results that are still to be added
        for i, cache in enumerate(self.caches):
            if rows is None:
                h, _ = api.add_rms_norm(x)
            else:
                h, x = api.add_rms_norm(rows, residual=x, gates=gates)
            qkv = torch.matmul(h, self.qkv[i]).view(T, HEADS + 2 * KV_HEADS, DIM)
            q, key, v = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV_HEADS], qkv[:, HEADS + KV_HEADS:]
            q = api.qk_norm_rope_store(q, key, v, self.q_weight, self.k_weight, plan.positions, self.rope, plan.slots, cache)
            a = api.attention_kv4(q, cache, self.table, plan.kv_lens, cu_q=plan.cu_q, workspace=self.attention_ws)
            a = torch.matmul(a.view(T, HEADS * DIM), self.out[i])
            # a row for each of a token's experts
            h, x = api.add_rms_norm(a, residual=x, repeat=k)
            if self.top_k:
                ids, gates = api.moe_route(torch.matmul(h[::k], self.router[i]), k, renormalise=True, scale=self.gain,
                                           requests=plan.requests)
            else:
                ids = (plan.positions * 7 + plan.requests.clamp(min=0)) % self.n_experts
                gates = torch.full((T, 1), self.gain, device=x.device)
            rows, _ = self.ffn(i, h, ids.view(-1))
        return api.add_rms_norm(rows, residual=x, gates=gates)[1]

    def next_tokens(self, x, plan, u, **how):
        """Of each request's last new token: x as __call__ gives it; u, how: api.sample's numbers."""
        h, _ = api.add_rms_norm(x[(plan.cu_q[1:] - 1).clamp(min=0).long()])
        return api.sample(torch.matmul(h, self.unembed), u, workspace=self.sample_ws, **how)


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--layers", type=int, default=4)
    p.add_argument("--requests", type=int, default=32)
    p.add_argument("--prompt", type=int, default=700)
    p.add_argument("--steps", type=int, default=32)
    p.add_argument("--top-k", type=int, default=2)
    p.add_argument("--vocab", type=int, default=32000)
    a = p.parse_args()
    d = Decoder(a.layers, a.requests, a.prompt + a.steps + 8, max(a.requests, 2 * a.prompt), top_k=a.top_k, vocab=a.vocab)
    g = torch.Generator(device="cuda").manual_seed(1)
    token = torch.zeros(a.requests, dtype=torch.int32, device="cuda")
    # every request's wishes
    how = dict(temperature=torch.full((a.requests,), 0.8, device="cuda"), top_p=torch.full((a.requests,), 0.95, device="cuda"),
               top_k=torch.full((a.requests,), 50, dtype=torch.int32, device="cuda"))
    # prompts, two requests at a time
    torch.cuda.synchronize()
    start = time.perf_counter()
    for r in range(0, a.requests, 2):
        new = torch.zeros(a.requests, dtype=torch.int32, device="cuda")
        new[r:r + 2] = a.prompt
        n = a.prompt * min(2, a.requests - r)
        ids = torch.randint(0, a.vocab, (n,), generator=g, device="cuda")
        p = d.plan(new, n)
        first = d.next_tokens(d(d.embedding[ids], p), p, torch.rand(a.requests, generator=g, device="cuda"), **how)
        token[r:r + 2] = first[r:r + 2]
    torch.cuda.synchronize()
    print(f"prompts: {a.requests * a.prompt / (time.perf_counter() - start):.0f} tokens/s")
    # single tokens: each step's are the next one's input
    one = torch.ones(a.requests, dtype=torch.int32, device="cuda")
    plan = api.alloc_kv_plan(a.requests, a.requests, d.table)
    u = torch.rand(a.requests, generator=g, device="cuda")

    def step():
        p = d.plan(one, a.requests, plan)
        token.copy_(d.next_tokens(d(d.embedding[token.long()], p), p, u, **how))

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
        u.uniform_(generator=g)
        graph.replay()
    torch.cuda.synchronize()
    took = time.perf_counter() - start
    assert int(plan.error) == 0 and bool(((token >= 0) & (token < a.vocab)).all())
    print(f"single tokens: {took / a.steps * 1e3:.3f} ms a step of {a.requests} requests, {a.requests * a.steps / took:.0f} tokens/s")


if __name__ == "__main__":
    main()
