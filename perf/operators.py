"""What is measured of the serving operators around the compressed experts: step plans of a paged cache, norms and
rotation of queries and keys, the 4-bit cache's writer and reader, and attention over that cache.

With own = False run() computes each operator from elementary torch operations; with own = True it makes the
package's calls.  Lengths are a ramp fixed by the case and shuffled by the seed, so a case's work is the same for
every seed.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
LIMIT = 131072          # positions in the rotation table
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)

# ------------------------------------------------------------------ cases


def _plan(name, requests, ctx_lo, ctx_hi, prompts, chunk, block):
    return {"name": name, "kind": "plan", "requests": requests, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi,
            "prompts": prompts, "chunk": chunk, "block": block}


def _qk(name, kind, tokens, heads, kv_heads, dim, rot, pairs, dtype, block=16):
    return {"name": name, "kind": kind, "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "rot": rot, "pairs": pairs, "dtype": dtype, "block": block}


def _att(name, requests, ctx_lo, ctx_hi, prompts, chunk, padded, heads, kv_heads, dim, block, dtype):
    return {"name": name, "kind": "attention", "requests": requests, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi,
            "prompts": prompts, "chunk": chunk, "padded": padded, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "block": block, "dtype": dtype}


def listed():
    return [
        # one decode step of 64 running requests
        _plan("plan decode 64", 64, 1, 9000, 0, 1, 16),
        # a step that admits 200 prompts of 301 tokens beside 312 running requests
        _plan("plan mixed 512", 512, 1, 4000, 200, 301, 32),
        # a prompt's queries and keys, kept dense (no cache)
        _qk("norm prompt 4096", "dense", 4096, 32, 8, 128, 128, "halves", "bf16"),
        # a few tokens, half of each head rotated, neighbouring pairs
        _qk("norm few 37", "dense", 37, 12, 4, 64, 32, "neighbours", "fp16"),
        # one decode step's queries, keys and values, into the cache and back
        _qk("store decode 64", "store", 64, 32, 8, 128, 128, "halves", "bf16"),
        # a long prompt written to the cache and read back
        _qk("store prompt 8191", "store", 8191, 40, 8, 128, 128, "halves", "fp16", 32),
        # one request, short: what one interactive user waits for
        _att("decode 1 x 1000", 1, 1000, 1000, 0, 1, 0, 16, 16, 64, 16, "fp16"),
        # a running batch with ragged lengths, padded to a captured batch size by requests without tokens
        _att("decode 64 x 16000", 64, 500, 16000, 0, 1, 3, 32, 8, 128, 16, "bf16"),
        # two very long documents
        _att("decode 2 x 250000", 2, 199001, 250001, 0, 1, 0, 64, 8, 128, 64, "bf16"),
        # new prompts without context
        _att("prompt 2 x 4000", 2, 0, 0, 2, 4000, 0, 32, 8, 128, 32, "bf16"),
        # pieces of prompts beside running requests in one step
        _att("mixed 24", 24, 300, 6000, 4, 511, 0, 24, 3, 128, 16, "fp16"),
        # wide heads, later piece of one long prompt
        _att("piece 1024 of 20000", 1, 19000, 19000, 1, 1024, 0, 16, 4, 256, 64, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["plan", "dense", "store", "attention", "attention", "attention"])
    block = rng.choice([16, 32, 64, 128])
    if kind == "plan":
        r = _log(rng, 1, 700)
        prompts = rng.choice([0, rng.randint(0, r)])
        c = _plan("", r, rng.randint(0, 50), _log(rng, 60, 9000), prompts, _log(rng, 1, min(4000, 60000 // r + 1)), block)
    else:
        dim = rng.choice([64, 128, 128, 256])
        kv_heads = rng.choice([1, 2, 3, 4, 8, 16])
        group = rng.choice([1, 2, 4, 5, 8]) if kv_heads <= 8 else rng.choice([1, 2])
        dtype = rng.choice(["bf16", "fp16"])
        if kind in ("dense", "store"):
            tokens = _log(rng, 1, min(8000, 40 * 8192 * 128 // (kv_heads * (group + 1) * dim)))
            rot = rng.choice([dim, dim, dim // 2])
            c = _qk("", kind, tokens, kv_heads * group, kv_heads, dim, rot, rng.choice(["halves", "halves", "neighbours"]),
                    dtype, block)
        elif rng.random() < 0.6:       # single tokens
            r = _log(rng, 1, 100)
            hi = _log(rng, 20, max(40, min(200000, 60_000_000 // (r * kv_heads * dim // 16))))
            c = _att("", r, rng.randint(1, hi), hi, 0, 1, rng.choice([0, 0, rng.randint(0, r - 1)]), kv_heads * group,
                     kv_heads, dim, block, dtype)
        else:                           # prompts, or pieces of prompts beside single tokens
            r = rng.randint(1, 12)
            hi = _log(rng, 1, 6000)
            c = _att("", r, rng.randint(0, hi), hi, rng.randint(1, min(r, 4)), _log(rng, 2, 1500), 0, kv_heads * group,
                     kv_heads, dim, block, dtype)
            while work(c)["flops"] > 2.5e11:        # below the largest listed
                c["chunk"] = c["chunk"] * 3 // 4
    del c["name"]
    return c


def _ramp(lo, hi, n):
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _lengths(c):
    """(context, new) tokens of each request, in the case's own order."""
    ctx = _ramp(c["ctx_lo"], c["ctx_hi"], c["requests"])
    step = c["requests"] / max(1, c["prompts"])
    prompts = {int(i * step) for i in range(c["prompts"])}
    return ctx, [c["chunk"] if i in prompts else 1 for i in range(c["requests"])]


def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float16


def work(c):
    if c["kind"] == "plan":
        ctx, new = _lengths(c)
        blocks = sum(-(-(a + b) // c["block"]) - -(-a // c["block"]) for a, b in zip(ctx, new))
        return {"bytes": 16 * len(ctx) + 12 * sum(new) + 8 * blocks, "flops": 2 * sum(new)}
    if c["kind"] in ("dense", "store"):
        q, k = c["tokens"] * c["heads"] * c["dim"], c["tokens"] * c["kv_heads"] * c["dim"]
        bytes_ = 4 * q + c["tokens"] * (4 + 4 * c["rot"]) + 2 * c["dim"] * 2
        bytes_ += 4 * k if c["kind"] == "dense" else 2 * (2 * k + 2 * (17 * k // 32) + 2 * k) + 4 * c["tokens"]
        return {"bytes": bytes_, "flops": 8 * (q + k)}
    ctx, new = _lengths(c)
    kv = sum(a + b for a, b in zip(ctx[c["padded"]:], new[c["padded"]:]))
    pairs = sum(b * a + b * (b + 1) // 2 for a, b in zip(ctx[c["padded"]:], new[c["padded"]:]))
    return {"bytes": kv * c["kv_heads"] * c["dim"] * 17 // 16 + sum(new) * c["heads"] * (4 * c["dim"] + 4) + 4 * kv // c["block"],
            "flops": 4 * pairs * c["heads"] * c["dim"]}

# ------------------------------------------------------------------ inputs


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    if c["kind"] == "plan":
        return _prepare_plan(c, g)
    if c["kind"] == "attention":
        return _prepare_attention(c, g)
    return _prepare_qk(c, g)


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device=DEV)


def _shuffled(c, g):
    ctx, new = _lengths(c)
    order = torch.randperm(c["requests"], generator=g, device=DEV).tolist()
    return [ctx[i] for i in order], [new[i] for i in order], order


def _prepare_plan(c, g):
    """A pool whose blocks are in random order; each request holds those of its context; 5 tokens of padding."""
    ctx, new, _ = _shuffled(c, g)
    bs = c["block"]
    width = -(-(c["ctx_hi"] + c["chunk"]) // bs) + 3
    held = [-(-a // bs) for a in ctx]
    need = sum(-(-(a + b) // bs) for a, b in zip(ctx, new)) - sum(held)
    n_blocks = sum(held) + need + 17
    ids = torch.randperm(n_blocks, generator=g, device=DEV).to(torch.int32)
    col = torch.arange(width, device=DEV)[None]
    has = _ints(held, torch.int64)
    first = torch.cumsum(has, 0) - has
    table = torch.where(col < has[:, None], ids[(first[:, None] + col).clamp(max=n_blocks - 1)], -1).contiguous()
    free = ids[sum(held):].contiguous()
    return {"kind": "plan", "ctx": _ints(ctx), "new": _ints(new), "table": table, "free": free,
            "n_free": _ints([free.numel()]), "n_blocks": n_blocks, "block": bs, "max_tokens": sum(new) + 5}


def _rope(rot):
    """cos and sin of position * 10000^(-2i/rot), from angles in 64 bits."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    angle = torch.arange(LIMIT, dtype=torch.float64, device=DEV)[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)


def _prepare_qk(c, g):
    """One product's q, k and v side by side, as a projection leaves them; positions from anywhere; distinct slots."""
    t, h, kvh, d, dt = c["tokens"], c["heads"], c["kv_heads"], c["dim"], _dtype(c)
    qkv = torch.randn(t, (h + 2 * kvh) * d, generator=g, device=DEV)
    qkv *= torch.exp(0.5 * torch.randn(t, h + 2 * kvh, generator=g, device=DEV)).repeat_interleave(d, 1)
    qkv = qkv.to(dt)
    n_blocks = -(-t // c["block"]) + 9
    return {"kind": c["kind"], "q": qkv[:, :h * d].view(t, h, d), "k": qkv[:, h * d:(h + kvh) * d].view(t, kvh, d),
            "v": qkv[:, (h + kvh) * d:].view(t, kvh, d),
            "qw": (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(dt),
            "kw": (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(dt),
            "pos": torch.randint(0, LIMIT, (t,), generator=g, device=DEV, dtype=torch.int32),
            "slots": torch.randperm(n_blocks * c["block"], generator=g, device=DEV)[:t].sort()[0].to(torch.int32),
            "rope": _rope(c["rot"]), "neighbours": c["pairs"] == "neighbours", "block": c["block"],
            "cache": torch.zeros(n_blocks, kvh, c["block"] * d * 17 // 16, dtype=torch.uint8, device=DEV)}


def _prepare_attention(c, g):
    """A cache of normally distributed keys and values, its blocks in random order; queries of unit size."""
    ctx, new, order = _shuffled(c, g)
    bs, d, kvh, dt = c["block"], c["dim"], c["kv_heads"], _dtype(c)
    kv = [0 if i < c["padded"] else a + b for a, b, i in zip(ctx, new, order)]
    held = [-(-n // bs) for n in kv]
    n_blocks = sum(held) + 5
    cache = torch.empty(n_blocks, kvh, bs * d * 17 // 16, dtype=torch.uint8, device=DEV)
    for at in range(0, n_blocks, max(1, (1 << 27) // (kvh * bs * d))):
        piece = cache[at:at + max(1, (1 << 27) // (kvh * bs * d))]
        x = torch.randn(2, piece.shape[0], kvh, bs, d, generator=g, device=DEV)
        x *= torch.exp(0.3 * torch.randn(2, piece.shape[0], kvh, bs, 1, generator=g, device=DEV))
        codes, scales = _quantise(x, 140)
        piece.copy_(torch.cat([codes[0].flatten(2), codes[1].flatten(2), scales[0].flatten(2), scales[1].flatten(2)], 2))
    ids = torch.randperm(n_blocks, generator=g, device=DEV).to(torch.int32)
    width = max(held) + 2
    has = _ints(held, torch.int64)
    first = torch.cumsum(has, 0) - has
    col = torch.arange(width, device=DEV)[None]
    table = torch.where(col < has[:, None], ids[(first[:, None] + col).clamp(max=n_blocks - 1)], -1).contiguous()
    starts = [0]
    for b in new:
        starts.append(starts[-1] + b)
    q = torch.randn(starts[-1], c["heads"], d, generator=g, device=DEV).to(dt)
    return {"kind": "attention", "q": q, "cache": cache, "table": table, "kv": _ints(kv), "block": bs,
            "kv_heads": kvh, "cu_q": None if max(new) == 1 else _ints(starts), "most_kv": max(kv), "most_q": max(new),
            "scale": 1.5 / math.sqrt(d)}

# ------------------------------------------------------------------ plain forms


def run(s):
    if own:
        return _own(s)
    if s["kind"] == "plan":
        return _plain_plan(s)
    if s["kind"] == "attention":
        return _plain_attention(s)
    return _plain_qk(s)


def _plain_plan(s):
    bs, ctx, new, table = s["block"], s["ctx"].long(), s["new"].long(), s["table"]
    old, total = (ctx + bs - 1) // bs, (ctx + new + bs - 1) // bs
    upto = torch.cumsum(total - old, 0)
    cu = torch.cat([torch.zeros_like(ctx[:1]), torch.cumsum(new, 0)])
    # new blocks, from the end of the free ones; the place behind the table takes what there are not
    f = torch.arange(s["free"].numel(), device=DEV)
    owner = torch.searchsorted(upto, f, right=True).clamp(max=ctx.numel() - 1)
    at = owner * table.shape[1] + old[owner] + f - (upto - total + old)[owner]
    flat = torch.cat([table.reshape(-1), table.new_zeros(1)])
    flat[torch.where(f < upto[-1], at, table.numel())] = s["free"][(s["n_free"].long() - 1 - f) % s["free"].numel()]
    table = flat[:-1].view(table.shape)
    t = torch.arange(s["max_tokens"], device=DEV)
    real = t < cu[-1]
    request = torch.searchsorted(cu[1:], t, right=True).clamp(max=ctx.numel() - 1)
    pos = ctx[request] + t - cu[request]
    slot = table[request, torch.where(real, pos // bs, 0)].long() * bs + pos % bs
    return {"block_table": table, "slots": torch.where(real, slot, -1).int(), "positions": torch.where(real, pos, 0).int(),
            "requests": torch.where(real, request, -1).int(), "cu_q": cu.int(), "kv_lens": (ctx + new).int(),
            "n_free": (s["n_free"] - upto[-1]).int()}


def _norm_rope(x, w, s):
    rope = s["rope"][s["pos"].long()][:, None].to(x.dtype)
    half = rope.shape[-1] // 2
    cos, sin = rope[..., :half], rope[..., half:]
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.to(x.dtype)
    turned, rest = y[..., :2 * half], y[..., 2 * half:]
    if s["neighbours"]:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = turned[..., :half], turned[..., half:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, rest], -1)


def _once(x, dtype):
    """64 bits to 16 in one rounding: the bits below those of 32 are first gathered in the lowest that 32 keep."""
    b = x.view(torch.int64)
    low = (1 << 29) - 1
    b = torch.where((b & low) != 0, (b & ~low) | (1 << 29), b)
    return b.view(torch.float64).to(torch.float32).to(dtype)


def _quantise(x, most):
    """x [..., D] in 32 bits to (codes uint8 [..., D/2], scales uint8 [..., D/32])."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    bits = b.abs().amax(-1).view(torch.int32)
    scale = ((bits >> 23) - 2 + ((bits & 0x7FFFFF) > 0x600000).int()).clamp(1, most)
    a = (b / torch.exp2((scale - 127).float())[..., None]).abs()
    code = ((a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)
            + 8 * torch.signbit(b).byte()).view(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.byte()


def _values(codes, scales):
    """The values of codes uint8 [..., D/2] and scales uint8 [..., D/32], in 32 bits."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
    x = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    x = table[x.int()].view(*scales.shape, 32)
    return (x * torch.exp2(scales.float() - 127)[..., None]).flatten(-2)


def _fields(page, bs, d):
    """Pages uint8 [..., bs * D * 17 / 16] as (K codes, V codes, K scales, V scales), each [..., bs, :]."""
    n, m = bs * d // 2, bs * d // 32
    return (page[..., :n].unflatten(-1, (bs, -1)), page[..., n:2 * n].unflatten(-1, (bs, -1)),
            page[..., 2 * n:2 * n + m].unflatten(-1, (bs, -1)), page[..., 2 * n + m:].unflatten(-1, (bs, -1)))


def _plain_qk(s):
    dt = s["q"].dtype
    q = _norm_rope(s["q"].float(), s["qw"], s).to(dt)
    # K in 64 bits: its values are beside the borders of 4-bit codes
    k = _once(_norm_rope(s["k"].double(), s["kw"], s), dt)
    if s["kind"] == "dense":
        return {"q": q, "k": k}
    bs, d, most = s["block"], q.shape[-1], 140 if dt == torch.float16 else 252
    slots = s["slots"].long()
    block, row = slots // bs, slots % bs
    kc, vc, ks, vs = _fields(s["cache"], bs, d)
    kc[block, :, row], ks[block, :, row] = _quantise(k.float(), most)
    vc[block, :, row], vs[block, :, row] = _quantise(s["v"].float(), most)
    return {"q": q, "k": _values(kc[block, :, row], ks[block, :, row]).to(dt),
            "v": _values(vc[block, :, row], vs[block, :, row]).to(dt)}


def _plain_attention(s):
    q, bs, kvh = s["q"], s["block"], s["kv_heads"]
    d, heads, r = q.shape[-1], q.shape[1], s["kv"].numel()
    group, most = heads // kvh, s["most_q"]
    kv = s["kv"].long()
    cu = torch.arange(r + 1, device=DEV) if s["cu_q"] is None else s["cu_q"].long()
    new = cu[1:] - cu[:-1]
    pages = -(-s["most_kv"] // bs)
    kc, vc, ks, vs = _fields(s["cache"][s["table"][:, :pages].long().clamp(min=0)].transpose(1, 2), bs, d)
    k = _values(kc, ks).flatten(2, 3)                                     # [r, kvh, pages * bs, d]
    v = _values(vc, vs).flatten(2, 3)
    i = torch.arange(most, device=DEV)
    at = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)                       # [r, most]
    x = q[at].float().view(r, most, kvh, group, d).permute(0, 2, 3, 1, 4).reshape(r, kvh, group * most, d)
    score = torch.matmul(x, k.transpose(2, 3)).mul_(s["scale"]).view(r, kvh, group, most, -1)
    col = torch.arange(k.shape[2], device=DEV)
    last = kv[:, None] - new[:, None] + i                                     # the last token that a row sees
    seen = (col <= last[..., None]) & (i < new[:, None])[..., None]
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0, top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(r, kvh, group * most, -1), v).view(r, kvh, group, most, d)
    out = torch.where(total > 0, out / total, 0)
    lse = (top + total.log()).squeeze(-1)
    t = torch.arange(q.shape[0], device=DEV)
    request = torch.searchsorted(cu[1:], t, right=True)
    out, lse = out.permute(0, 3, 1, 2, 4).flatten(2, 3), lse.permute(0, 3, 1, 2).flatten(2)
    return {"out": out[request, t - cu[request]].to(q.dtype), "lse": lse[request, t - cu[request]]}

# ------------------------------------------------------------------ the package's calls


def _own(s):
    from sub_bit_moe_amd import api
    if s["kind"] == "plan":
        p = api.kv_plan(s["ctx"], s["new"], s["free"], s["n_free"], s["table"], s["n_blocks"], s["block"], s["max_tokens"])
        return {"block_table": p.block_table, "slots": p.slots, "positions": p.positions, "requests": p.requests,
                "cu_q": p.cu_q, "kv_lens": p.kv_lens, "n_free": p.n_free}
    if s["kind"] == "dense":
        q, k = api.qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["pos"], s["rope"], eps=EPS, neighbours=s["neighbours"])
        return {"q": q, "k": k}
    cache = api.KVCache(s["cache"], s["block"], s["q"].shape[-1])
    if s["kind"] == "store":
        q = api.qk_norm_rope_store(s["q"], s["k"], s["v"], s["qw"], s["kw"], s["pos"], s["rope"], s["slots"], cache,
                                   eps=EPS, neighbours=s["neighbours"])
        k, v = api.kv_load(cache, s["slots"], dtype=q.dtype)
        return {"q": q, "k": k, "v": v}
    if "workspace" not in s:            # kept by a program for all its layers and steps
        s["workspace"] = api.alloc_attention_workspace(s["kv"].numel(), s["q"].shape[0], s["q"].shape[1], s["kv_heads"],
                                                       s["q"].shape[2])
    out, lse = api.attention_kv4(s["q"], cache, s["table"], s["kv"], cu_q=s["cu_q"], scale=s["scale"], return_lse=True,
                                 workspace=s["workspace"])
    return {"out": out, "lse": lse}

# ------------------------------------------------------------------ the definition in 64 bits


def exact(c, seed):
    s = prepare(c, seed)
    if c["kind"] == "plan":
        return None
    return _exact_attention(s) if c["kind"] == "attention" else _exact_qk(s)


def _nearest(x, bits, floor):
    """x in 64 bits rounded to `bits` significant ones, halves to even, with nothing finer than 2^floor."""
    quantum = torch.exp2((torch.frexp(x)[1] - bits).clamp(min=floor).double())
    return (x / quantum).round() * quantum


def _held(x, most):
    """What the 4-bit cache holds of x: the nearest of the sixteen values in each block of 32."""
    b = x.unflatten(-1, (-1, 32))
    # the smallest power of two at which nothing passes 7
    size = torch.full_like(b[..., 0], -126.0)
    top = b.abs().amax(-1)
    for e in range(-126, most - 126):
        size = torch.where(top > 7 * 2.0 ** e, size.clamp(min=e + 1.0), size)
    unit = torch.exp2(size.clamp(max=most - 127.0))[..., None]
    got = torch.zeros_like(b)
    off = b.abs().clone()
    for n, value in enumerate(E2M1[1:], 1):
        far = (b.abs() - value * unit).abs()
        better = (far < off) | ((far == off) & (n % 2 == 0))
        got, off = torch.where(better, value * unit, got), torch.where(better, far, off)
    return (got * torch.where(b < 0, -1.0, 1.0)).flatten(-2)


def _exact_qk(s):
    half = s["neighbours"] is False
    rope = s["rope"][s["pos"].long()].double()
    n = rope.shape[1] // 2
    by = torch.complex(rope[:, :n], rope[:, n:])[:, None]

    def turned(x, w):
        x = x.double()
        y = w.double() * x / ((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
        pair = y[..., :2 * n].unflatten(-1, (2, n) if half else (n, 2))
        z = by * (torch.complex(pair[..., 0, :], pair[..., 1, :]) if half else torch.complex(pair[..., 0], pair[..., 1]))
        z = torch.stack([z.real, z.imag], -2 if half else -1).flatten(-2)
        return torch.cat([z, y[..., 2 * n:]], -1)

    q, k = turned(s["q"], s["qw"]), turned(s["k"], s["kw"])
    if s["kind"] == "dense":
        return {"q": q, "k": k}
    fp16 = s["q"].dtype == torch.float16
    most = 140 if fp16 else 252
    return {"q": q, "k": _held(_nearest(k, 11 if fp16 else 8, -24 if fp16 else -133), most),
            "v": _held(s["v"].double(), most)}


def _exact_attention(s):
    q, bs = s["q"].double(), s["block"]
    d, kvh = q.shape[-1], s["kv_heads"]
    out, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    kv = s["kv"].tolist()
    cu = list(range(len(kv) + 1)) if s["cu_q"] is None else s["cu_q"].tolist()

    def read(codes, scales):
        even, odd = codes.to(torch.int64) % 16, codes.to(torch.int64) // 16
        n = torch.stack([even, odd], -1).flatten(-2)
        e, m = n // 2 % 4, (n % 2).double()
        size = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e.double() - 1)) * torch.where(n > 7, -1.0, 1.0)
        return size * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)

    for r, n in enumerate(kv):
        a, b = cu[r], cu[r + 1]
        if n == 0 or a == b:
            continue
        page = s["cache"][s["table"][r, :-(-n // bs)].long()]                 # [pages, kvh, bytes]
        cut = [0, bs * d // 2, bs * d, bs * d + bs * d // 32, page.shape[-1]]
        part = [page[:, :, x:y].reshape(page.shape[0], kvh, bs, -1) for x, y in zip(cut, cut[1:])]
        for h in range(kvh):
            k = read(part[0][:, h], part[2][:, h]).flatten(0, 1)[:n]
            v = read(part[1][:, h], part[3][:, h]).flatten(0, 1)[:n]
            group = q.shape[1] // kvh
            for j in range(h * group, (h + 1) * group):
                z = s["scale"] * (q[a:b, j] @ k.T)
                z = z.masked_fill(torch.arange(n, device=DEV)[None] > torch.arange(n - (b - a), n, device=DEV)[:, None], -math.inf)
                lse[a:b, j] = torch.logsumexp(z, -1)
                out[a:b, j] = torch.softmax(z, -1) @ v
    return {"out": out, "lse": lse}
