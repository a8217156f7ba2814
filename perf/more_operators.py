"""What is measured of the operators that a decoder step has around its experts and its attention: the norm with the
residual's addition and the sum over a token's experts, the routing to experts, and the choice of the next token.

With own = False run() computes each operator from elementary torch operations; with own = True it makes the
package's calls.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}

# ------------------------------------------------------------------ cases


def _norm(name, tokens, dim, dtype, x, residual, k, repeat, block=-1):
    """block: -1 for 16-bit results; 0, 128, 32: 8 bits with a scale for the row or so many elements."""
    return {"name": name, "kind": "norm", "tokens": tokens, "dim": dim, "dtype": dtype, "x": x, "residual": residual, "k": k,
            "repeat": repeat, "block": block}


def _route(name, tokens, experts, k, dtype, sigmoid, bias, groups, top_groups, renormalise, padded=0):
    return {"name": name, "kind": "route", "tokens": tokens, "experts": experts, "k": k, "dtype": dtype, "sigmoid": sigmoid,
            "bias": bias, "groups": groups, "top_groups": top_groups, "renormalise": renormalise, "padded": padded}


def _sample(name, rows, vocab, dtype, filters):
    return {"name": name, "kind": "sample", "rows": rows, "vocab": vocab, "dtype": dtype, "filters": filters}


def listed():
    return [
        # one interactive user's token, after an expert of the c2048 width
        _norm("norm one token", 1, 2080, "fp16", "fp32", "fp16", 1, 1),
        # a decode step: two experts' rows joined, and the next experts' input twice
        _norm("norm decode 64 of 2", 64, 2080, "fp16", "fp32", "fp32", 2, 2),
        # a prompt between attention and experts
        _norm("norm prompt 8191", 8191, 4096, "bf16", "bf16", "bf16", 1, 1),
        # a prompt of a wide model in front of an 8-bit product
        _norm("norm prompt 4096 in 8 bits", 4096, 8192, "bf16", "bf16", "bf16", 1, 1, 32),
        # one step of the c2048 stack: one of 2048 experts each, padded to a captured batch size
        _route("route decode 64 of 2048", 64, 2048, 1, "fp32", False, False, 1, 1, False, 5),
        # a few tokens of a small mixture
        _route("route few 7 of 60", 7, 60, 4, "bf16", False, False, 1, 1, True),
        # a prompt with balanced, grouped experts
        _route("route prompt 8192 of 256", 8192, 256, 8, "fp32", True, True, 8, 4, True),
        # all tokens of a step of long prompts over the c2048 stack's experts
        _route("route prompt 16384 of 2048", 16384, 2048, 2, "fp32", False, True, 1, 1, True),
        # one interactive user's next token
        _sample("sample one of 32000", 1, 32000, "fp16", "all"),
        # a running batch whose users asked for different things
        _sample("sample 64 of 131072", 64, 131072, "bf16", "mixed"),
        # many short answers, temperature alone
        _sample("sample 200 of 50021", 200, 50021, "fp32", "none"),
        # a large batch with nucleus sampling
        _sample("sample 256 of 150001", 256, 150001, "fp32", "top_p"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "route", "sample"])
    if kind == "norm":
        dim = rng.choice([_log(rng, 64, 16384), 64 * _log(rng, 1, 256), 2080, 2048])
        k = rng.choice([1, 1, 2, 4, 8])
        repeat = rng.choice([1, 1, k])
        dtype = rng.choice(["bf16", "fp16"])
        tokens = _log(rng, 1, max(1, min(8192, (3 << 25) // (dim * (2 + 2 * k + 2 * repeat)))))
        c = _norm("", tokens, dim, dtype, rng.choice([dtype, "fp32"]), rng.choice([dtype, dtype, "fp32"]), k, repeat,
                  rng.choice([-1, -1, 0, 128, 32]))
    elif kind == "route":
        groups = rng.choice([1, 1, 1, 2, 4, 8])
        experts = groups * max(1, _log(rng, 8, 2048) // groups)
        top_groups = rng.randint((groups + 1) // 2, groups)
        k = min(rng.choice([1, 2, 4, 6, 8]), experts // groups * top_groups)
        c = _route("", _log(rng, 1, min(16384, (1 << 25) // experts)), experts, k, rng.choice(["fp32", "fp32", "bf16", "fp16"]),
                   rng.random() < 0.4, rng.random() < 0.5, groups, top_groups, rng.random() < 0.5, rng.choice([0, 0, 3]))
    else:
        vocab = _log(rng, 1000, 200000)
        c = _sample("", _log(rng, 1, min(400, 38_000_000 // vocab)), vocab, rng.choice(["fp32", "bf16", "fp16"]),
                    rng.choice(["all", "mixed", "mixed", "none", "top_p"]))
    del c["name"]
    return c


def _size(dtype):
    return 4 if dtype == "fp32" else 2


def work(c):
    if c["kind"] == "norm":
        n = c["tokens"] * c["dim"]
        out = 2 * n if c["block"] < 0 else n + (4 * c["tokens"] if c["block"] == 0 else
                                                (4 if c["block"] == 128 else 1) * c["tokens"] * -(-c["dim"] // c["block"]))
        bytes_ = c["k"] * n * _size(c["x"]) + 2 * n * _size(c["residual"]) + c["repeat"] * out + 2 * c["dim"]
        return {"bytes": bytes_ + 4 * c["k"] * c["tokens"], "flops": (2 * c["k"] + 4) * n}
    if c["kind"] == "route":
        n = c["tokens"] * c["experts"]
        return {"bytes": n * _size(c["dtype"]) + 8 * c["tokens"] * c["k"] + 4 * c["experts"] * c["bias"], "flops": 4 * n}
    n = c["rows"] * c["vocab"]
    return {"bytes": n * _size(c["dtype"]) + 28 * c["rows"], "flops": 4 * n}

# ------------------------------------------------------------------ inputs


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return {"norm": _prepare_norm, "route": _prepare_route, "sample": _prepare_sample}[c["kind"]](c, g)


def _prepare_norm(c, g):
    """Experts' or attention's rows of differing sizes, a residual stream with a few large dimensions, gates that sum to 1."""
    t, d, k, dt = c["tokens"], c["dim"], c["k"], DT[c["dtype"]]
    x = torch.randn(t * k, d, generator=g, device=DEV) * torch.exp(0.5 * torch.randn(t * k, 1, generator=g, device=DEV))
    residual = 2 * torch.randn(t, d, generator=g, device=DEV)
    residual[:, torch.randint(0, d, (3,), generator=g, device=DEV)] *= 30
    gates = torch.rand(t, k, generator=g, device=DEV) + 0.05
    return {"kind": "norm", "x": x.to(DT[c["x"]]), "residual": residual.to(DT[c["residual"]]),
            "weight": (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(dt),
            "gates": gates / gates.sum(1, keepdim=True) if k > 1 or c["x"] == "fp32" else None,
            "dtype": dt, "k": k, "repeat": c["repeat"], "block": c["block"]}


def _prepare_route(c, g):
    t, e = c["tokens"], c["experts"]
    logits = torch.randn(t, e, generator=g, device=DEV) + 0.5 * torch.randn(e, generator=g, device=DEV)
    requests = torch.arange(t, device=DEV, dtype=torch.int32)
    if c["padded"]:
        requests[max(0, t - c["padded"]):] = -1
    # a bias for balance: of the size of the chosen scores' differences
    size = 0.05 if c["sigmoid"] else 0.5 / e
    return {"kind": "route", "logits": logits.to(DT[c["dtype"]]), "k": c["k"], "sigmoid": c["sigmoid"],
            "bias": size * torch.randn(e, generator=g, device=DEV) if c["bias"] else None, "groups": c["groups"],
            "top_groups": c["top_groups"], "renormalise": c["renormalise"], "requests": requests if c["padded"] else None,
            "scale": 2.5 if c["sigmoid"] else 1.0}


def _prepare_sample(c, g):
    """Logits of a vocabulary whose likely tokens are few, some of them banned; every user's wishes."""
    r, v = c["rows"], c["vocab"]
    logits = torch.empty(r, v, dtype=DT[c["dtype"]], device=DEV)
    for at in range(0, r, 32):
        part = logits[at:at + 32]
        x = 2.2 * torch.randn(part.shape, generator=g, device=DEV)
        x += 9 * torch.rand(part.shape, generator=g, device=DEV) ** 40
        x.masked_fill_(torch.rand(part.shape, generator=g, device=DEV) < 0.001, -math.inf)
        part.copy_(x)

    def one_of(*values):
        at = torch.randint(0, len(values), (r,), generator=g, device=DEV)
        return torch.tensor(values, device=DEV)[at]

    s = {"kind": "sample", "logits": logits, "u": torch.rand(r, generator=g, device=DEV),
         "temperature": 0.6 + 0.7 * torch.rand(r, generator=g, device=DEV), "top_k": None, "top_p": None, "min_p": None}
    if c["filters"] == "mixed":
        s["temperature"] *= one_of(0.0, 1.0, 1.0, 1.0, 1.0)
        s["top_k"] = one_of(0, 0, 20, 50, 1000).int()
        s["top_p"] = one_of(1.0, 0.5, 0.9, 0.95)
        s["min_p"] = one_of(0.0, 0.0, 0.01, 0.1)
    elif c["filters"] == "all":
        s["top_k"], s["top_p"], s["min_p"] = one_of(50, 64).int(), one_of(0.9, 0.95), one_of(0.01, 0.02)
    elif c["filters"] == "top_p":
        s["top_p"] = one_of(0.8, 0.9, 0.95)
    return s

# ------------------------------------------------------------------ plain forms


def run(s):
    if own:
        return _own(s)
    return {"norm": _plain_norm, "route": _plain_route, "sample": _plain_sample}[s["kind"]](s)


def _once(x, dtype):
    """64 bits to 16 in one rounding: the bits below those of 32 are first gathered in the lowest that 32 keep."""
    if dtype == torch.float32:
        return x.float()
    b = x.view(torch.int64)
    low = (1 << 29) - 1
    b = torch.where((b & low) != 0, (b & ~low) | (1 << 29), b)
    return b.view(torch.float64).to(torch.float32).to(dtype)


def _plain_norm(s):
    # 8-bit results are beside the borders of their codes: in 64 bits
    wide = torch.float32 if s["block"] < 0 else torch.float64
    h = s["residual"].to(wide)
    x = s["x"].to(wide).view(h.shape[0], s["k"], -1)
    h = h + (x[:, 0] if s["gates"] is None else (x * s["gates"].to(wide)[..., None]).sum(1))
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["weight"].to(wide)
    y = y.repeat_interleave(s["repeat"], 0)
    if s["block"] < 0:
        return {"out": y.to(s["dtype"]), "residual": h.to(s["residual"].dtype)}
    block = s["block"] or y.shape[1]
    b = torch.nn.functional.pad(y, (0, -y.shape[1] % block)).unflatten(1, (-1, block))
    top = b.abs().amax(-1)
    if s["block"] == 32:
        m, e = torch.frexp(top / 448)
        scale = torch.exp2((e - (m == 0.5).int()).clamp(-126, 127).double())
    else:
        scale = (top / 448).float().clamp(min=2.0 ** -126).double()
    a = b / scale[..., None]
    # e4m3: four significant bits, nothing finer than 2^-9
    step = torch.exp2((torch.frexp(a)[1] - 4).clamp(min=-9).double())
    a = (torch.round(a / step) * step).clamp(-448, 448)
    value = (a * scale[..., None]).flatten(1)[:, :y.shape[1]]
    return {"out": value.to(s["dtype"]), "scale": scale.float(), "residual": _once(h, s["residual"].dtype)}


def _plain_route(s):
    logits, k, groups = s["logits"].double(), s["k"], s["groups"]          # scores beside one another's values: in 64 bits
    if s["sigmoid"]:
        score = 1 / (1 + torch.exp(-logits))
    else:
        score = torch.exp(logits - logits.amax(1, keepdim=True))
        score = score / score.sum(1, keepdim=True)
    choice = logits if s["bias"] is None else score + s["bias"].double()
    if groups > 1:
        value = (score if s["bias"] is None else choice).unflatten(1, (groups, -1)).sort(dim=2, descending=True)[0][..., :2].sum(2)
        best = value.sort(dim=1, descending=True, stable=True)[1][:, :s["top_groups"]]
        stays = torch.zeros_like(value, dtype=torch.bool).scatter_(1, best, True)
        choice = choice.masked_fill(~stays.repeat_interleave(choice.shape[1] // groups, 1), -math.inf)
    ids = choice.sort(dim=1, descending=True, stable=True)[1][:, :k]
    gates = score.gather(1, ids)
    if s["renormalise"]:
        gates = gates / gates.sum(1, keepdim=True)
    gates = (s["scale"] * gates).float()
    if s["requests"] is not None:
        pad = (s["requests"] < 0)[:, None]
        ids, gates = ids.masked_fill(pad, -1), gates.masked_fill(pad, 0)
    return {"ids": ids.int(), "gates": gates}


def _plain_sample(s):
    logits, t = s["logits"].float(), s["temperature"].double()[:, None]
    level, index = logits.sort(dim=1, descending=True, stable=True)
    rank = torch.arange(logits.shape[1], device=DEV)
    z = level.double() - level[:, :1].double()
    z = torch.where(t > 0, z / t, torch.where(rank == 0, 0, -math.inf))
    w = torch.exp(z)                                      # running sums beside others' borders: in 64 bits
    if s["top_k"] is not None:
        w = torch.where((s["top_k"][:, None] > 0) & (rank >= s["top_k"][:, None]), 0, w)
    if s["min_p"] is not None:
        w = torch.where(w >= s["min_p"].double()[:, None], w, 0)
    if s["top_p"] is not None:
        upto = w.cumsum(1)
        before = torch.nn.functional.pad(upto[:, :-1], (1, 0))
        p = s["top_p"].double()[:, None]
        w = torch.where((p < 1) & (before >= p * upto[:, -1:]), 0, w)
    w = torch.zeros_like(w).scatter_(1, index, w)
    upto = w.cumsum(1)
    total = upto[:, -1:]
    token = (upto <= s["u"].double()[:, None] * total).sum(1, keepdim=True)
    return {"token": token[:, 0].int(), "logprob": (w.gather(1, token) / total).log()[:, 0].float()}

# ------------------------------------------------------------------ the package's calls


def _own(s):
    from sub_bit_moe_amd import api
    if s["kind"] == "norm":
        if s["block"] < 0:
            out, residual = api.add_rms_norm(s["x"], s["weight"], s["residual"], gates=s["gates"], eps=EPS, repeat=s["repeat"])
            return {"out": out, "residual": residual}
        codes, scales, residual = api.add_rms_norm_fp8(s["x"], s["weight"], s["residual"], gates=s["gates"], eps=EPS,
                                                       repeat=s["repeat"], scale_block=s["block"])
        # what the codes stand for; a code times a power of two is a bf16 number
        block, wide = s["block"] or codes.shape[1], s["dtype"] if (s["block"], s["dtype"]) == (32, torch.bfloat16) else torch.float32
        scale = torch.exp2(scales.float() - 127) if s["block"] == 32 else scales
        by = scale.to(wide)
        if codes.shape[1] % block:
            out = codes.to(wide).mul_(by.repeat_interleave(block, 1)[:, :codes.shape[1]])
        else:
            out = codes.to(wide).unflatten(1, (-1, block)).mul_(by[..., None]).flatten(1)
        return {"out": out.to(s["dtype"]), "scale": scale, "residual": residual}
    if s["kind"] == "route":
        ids, gates = api.moe_route(s["logits"], s["k"], bias=s["bias"], sigmoid=s["sigmoid"], n_groups=s["groups"],
                                   top_groups=s["top_groups"], renormalise=s["renormalise"], scale=s["scale"],
                                   requests=s["requests"])
        return {"ids": ids, "gates": gates}
    if "workspace" not in s:            # kept by a program for all its steps
        s["workspace"] = api.alloc_sample_workspace(*s["logits"].shape)
    token, logprob = api.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                                min_p=s["min_p"], return_logprobs=True, workspace=s["workspace"])
    return {"token": token, "logprob": logprob}

# ------------------------------------------------------------------ the definition in 64 bits


def exact(c, seed):
    s = prepare(c, seed)
    return {"norm": _exact_norm, "route": _exact_route, "sample": _exact_sample}[c["kind"]](s)


def _exact_norm(s):
    k, rows = s["k"], s["residual"].shape[0]
    h = s["residual"].double()
    for j in range(k):
        part = s["x"][j::k].double()
        h = h + (part if s["gates"] is None else s["gates"][:, j:j + 1].double() * part)
    size = torch.sqrt(torch.linalg.vector_norm(h, dim=1) ** 2 / h.shape[1] + EPS)
    y = s["weight"].double() * (h / size[:, None])
    if s["block"] < 0:
        return {"out": y[torch.arange(rows * s["repeat"], device=DEV) // s["repeat"]], "residual": h}
    # every number that e4m3 has, and the borders between them
    held = torch.tensor([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)][:-1],
                        dtype=torch.float64, device=DEV)
    border = (held[1:] + held[:-1]) / 2
    width = s["block"] or y.shape[1]
    out, scales = [], []
    for at in range(0, y.shape[1], width):
        part = y[:, at:at + width]
        need = part.abs().max(1)[0] / held[-1]
        if s["block"] == 32:
            power = torch.ceil(torch.log2(need)).clamp(-126, 127)
            power = torch.where(need > torch.exp2(power), power + 1, power)
            power = torch.where(need <= torch.exp2(power - 1), power - 1, power).clamp(-126, 127)
            unit = torch.exp2(power)
        else:
            unit = torch.clamp(need.to(torch.float32), min=2.0 ** -126).double()
        a = (part / unit[:, None]).abs()
        low, high = torch.searchsorted(border, a), torch.searchsorted(border, a, right=True)
        code = torch.where(low != high, low + low % 2, low)          # on a border: the even one
        out.append(torch.sign(part) * held[code] * unit[:, None])
        scales.append(unit)
    again = torch.arange(rows, device=DEV).repeat_interleave(s["repeat"])
    return {"out": torch.cat(out, 1)[again], "scale": torch.stack(scales, 1)[again], "residual": h}


def _exact_route(s):
    logits = s["logits"].double().cpu().numpy()
    if logits.size > 1 << 23:
        return None
    bias = None if s["bias"] is None else s["bias"].double().cpu().numpy()
    t, e = logits.shape
    gates = np.zeros((t, s["k"]))
    skip = np.zeros(t, bool) if s["requests"] is None else s["requests"].cpu().numpy() < 0
    for i in range(t):
        if skip[i]:
            continue
        l = logits[i]
        score = 1 / (1 + np.exp(-l)) if s["sigmoid"] else np.exp(l - np.logaddexp.reduce(l))
        by = l if bias is None else score + bias
        ok = np.ones(e, bool)
        if s["groups"] > 1:
            n = e // s["groups"]
            value = [np.sort((score if bias is None else by)[j * n:(j + 1) * n])[-2:].sum() for j in range(s["groups"])]
            for j in np.argsort(-np.array(value), kind="stable")[s["top_groups"]:]:
                ok[j * n:(j + 1) * n] = False
        ids = np.flatnonzero(ok)
        ids = ids[np.argsort(-by[ids], kind="stable")][:s["k"]]
        gates[i] = s["scale"] * score[ids] / (score[ids].sum() if s["renormalise"] else 1.0)
    return {"ids": None, "gates": torch.from_numpy(gates)}


def _exact_sample(s):
    def host(x, off):
        return np.full(s["logits"].shape[0], off, np.float64) if x is None else x.double().cpu().numpy()

    rows = zip(s["logits"].cpu(), host(s["u"], 0), host(s["temperature"], 1), host(s["top_k"], 0), host(s["top_p"], 1),
               host(s["min_p"], 0))
    logprob = []
    for row, u, t, top_k, top_p, min_p in rows:
        l = row.double().numpy()
        if t == 0:
            logprob.append(0.0)
            continue
        likely = np.flatnonzero(l > -np.inf)
        likely = likely[np.argsort(-l[likely], kind="stable")]
        if top_k > 0:
            likely = likely[:int(top_k)]
        w = np.exp((l[likely] - l.max()) / t)
        likely, w = likely[w >= min_p], w[w >= min_p]
        if top_p < 1:
            n = 1 + int(np.searchsorted(np.cumsum(w), top_p * w.sum()))
            likely, w = likely[:n], w[:n]
        order = np.argsort(likely)
        at = order[min(int(np.searchsorted(np.cumsum(w[order]), u * w.sum(), side="right")), w.size - 1)]
        logprob.append(math.log(w[at] / w.sum()))
    return {"token": None, "logprob": torch.tensor(logprob, dtype=torch.float64)}
