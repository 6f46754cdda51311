"""The operators around a quantized layer that its users train, serve and
score with: low-rank adapters of many requests beside the shared projection
(forward and gradients), and the log probabilities of given tokens with
entropy and top alternatives (forward and gradient).

``run`` computes them in plain torch operations in fp32, or, where ``own`` is
true, through the library's entry points; ``exact`` is the definition in
64 bits, one adapter or one block of rows at a time.
"""
import math

import torch

own = False


# ------------------------------------------------------------------ cases

def listed():
    return [
        # Decode: one request through a 4096 x 4096 attention projection, the
        # quantized product's fp32 output; latency counts.
        dict(name="adapter_decode_1", op="adapter", T=1, n=4096, m=4096, r=16, L=8, x="bf16", w="bf16", y="f32",
             runs=1),
        # Decode: a batch of 64 requests through the MLP up projection, each
        # with its own choice among 32 adapters.
        dict(name="adapter_decode_64", op="adapter", T=64, n=4096, m=11008, r=16, L=32, x="bf16", w="bf16", y="f32",
             runs=64),
        # fp32 activations and adapters, odd sizes (a layer whose output side
        # is 4096 - 1 wide, a ragged number of tokens).
        dict(name="adapter_f32_odd", op="adapter", T=777, n=2731, m=4095, r=12, L=5, x="f32", w="f32", y="f32",
             runs=9),
        # Prefill: twelve requests of different lengths through the widest
        # layer (28672 x 8192), eight adapters of rank 64.
        dict(name="adapter_prefill", op="adapter", T=4096, n=8192, m=28672, r=64, L=8, x="bf16", w="bf16", y="bf16",
             runs=12),
        # A small fine-tuning step through one 4096 x 4096 projection.
        dict(name="adapter_grad_small", op="adapter_grad", T=96, n=4096, m=4096, r=16, L=4, x="bf16", w="bf16",
             y="bf16", runs=6),
        # A fine-tuning step: 8192 calibration tokens through the MLP up
        # projection, eight adapters of rank 32.
        dict(name="adapter_grad", op="adapter_grad", T=8192, n=4096, m=11008, r=32, L=8, x="bf16", w="bf16",
             y="bf16", runs=24),
        # Decode: the next token's log probabilities for one request.
        dict(name="logprobs_1", op="logprobs", T=1, V=32000, k=8, x="f32"),
        # Decode: a batch of 64 over a large vocabulary.
        dict(name="logprobs_64", op="logprobs", T=64, V=128000, k=20, x="bf16"),
        # Perplexity of one 2048-token segment, odd vocabulary, fp32 logits.
        dict(name="logprobs_odd", op="logprobs", T=2047, V=50257, k=1, x="f32"),
        # Perplexity of two 2048-token segments with five alternatives each.
        dict(name="logprobs_4096", op="logprobs", T=4096, V=32000, k=5, x="bf16"),
        # The gradient of a small batch's loss.
        dict(name="logprobs_grad_small", op="logprobs_grad", T=64, V=32000, x="f32"),
        # The gradient of a fine-tuning step's loss.
        dict(name="logprobs_grad", op="logprobs_grad", T=4096, V=32000, x="bf16"),
    ]


def _log(rng, a, b):
    return max(a, min(b, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))


def _width(rng, a, b):
    """A layer's width: mostly a multiple of 64 or 16, at times any number."""
    v = _log(rng, a, b)
    step = rng.choice((64, 64, 16, 1))
    return max(step, v // step * step)


def draw(rng):
    op = rng.choice(("adapter", "adapter", "adapter_grad", "logprobs", "logprobs", "logprobs_grad"))
    if op in ("adapter", "adapter_grad"):
        n, m = _width(rng, 64, 8192), _width(rng, 64, 11008)
        r = rng.choice((1, 4, 8, 8, 16, 16, 16, 24, 32, 32, 64, 64, 96, 128))
        most = (1 << (33 if op == "adapter" else 31)) // (r * (n + m))      # no more than the listed ones' products
        T = _log(rng, 1, min(4096, most))
        x = rng.choice(("bf16", "bf16", "f32"))
        w = "f32" if x == "f32" and rng.random() < 0.5 else "bf16"
        y = "f32" if x == "f32" else rng.choice(("bf16", "f32")) if op == "adapter" else "bf16"
        return dict(op=op, T=T, n=n, m=m, r=r, L=_log(rng, 1, min(32, 512 // r)), x=x, w=w, y=y,
                    runs=_log(rng, 1, T))
    T, V = _log(rng, 1, 2048), _log(rng, 100, 50000)
    case = dict(op=op, T=T, V=V, x=rng.choice(("bf16", "f32")))
    if op == "logprobs":
        case["k"] = rng.choice((0, 1, 2, 5, 8, 20, 32))
    return case


# ------------------------------------------------------------------ inputs

_TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    f32 = dict(dtype=torch.float32, device="cuda")

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, **f32) * std).to(dtype)

    op, T, xt = case["op"], case["T"], _TYPE[case["x"]]
    s = dict(case=case)
    if op in ("adapter", "adapter_grad"):
        n, m, r, L = (case[k] for k in ("n", "m", "r", "L"))
        wt, yt = _TYPE[case["w"]], _TYPE[case["y"]]
        # `runs` requests of random lengths, each with one of the adapters or none
        cuts = torch.randint(0, T, (max(case["runs"] - 1, 0),), generator=g, device="cuda")
        request = torch.bucketize(torch.arange(T, device="cuda"), cuts.sort().values, right=True)
        choice = torch.randint(-1 if case["runs"] > 1 else 0, L, (case["runs"],), generator=g, device="cuda")
        s["ids"] = choice[request].to(torch.int32)
        s["x"] = normal(T, n, dtype=xt)
        s["down"] = normal(L, r, n, std=n ** -0.5, dtype=wt)
        s["up"] = normal(L, r, m, std=r ** -0.5, dtype=wt)
        s["scale"] = torch.rand(L, generator=g, **f32) + 0.5
        if op == "adapter":
            s["base"] = normal(T, m, dtype=yt)                # the shared projection's output
            s["y"] = torch.empty(T, m, dtype=yt, device="cuda")
            s["h"] = torch.empty(T, r, **f32)
        else:
            s["dy"] = normal(T, m, dtype=yt)
            s["h"] = _hidden(s["x"].float(), s["ids"], s["down"].float()).sum(1)
            s["dx_base"] = normal(T, n, dtype=xt)             # the shared projection's part of dx
            s["dx"] = torch.empty(T, n, dtype=xt, device="cuda")
            s["d_down"] = torch.empty(L, r, n, **f32)
            s["d_up"] = torch.empty(L, r, m, **f32)
        return s
    V = case["V"]
    x = normal(T, V, std=2.5)
    # some tokens are barred (logit -inf), as a sampler's mask leaves them
    x.masked_fill_(torch.rand(V, generator=g, **f32) < 0.01, float("-inf"))
    x[:, 0].nan_to_num_(neginf=0.0)                           # at least one token is left
    s["logits"] = x.to(xt)
    s["tokens"] = torch.randint(0, V, (T,), generator=g, device="cuda").to(torch.int32)
    s["tokens"][torch.rand(T, generator=g, **f32) < 0.05] = -1  # padding: no token is given
    if op == "logprobs":
        k = case["k"]
        for name in ("logprob", "entropy", "lse"):
            s[name] = torch.empty(T, **f32)
        s["top_values"] = torch.empty(T, k, **f32)
        s["top_ids"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
    else:
        s["lse"], _, s["entropy"] = _softmax(s["logits"].float())
        s["g_logprob"], s["g_entropy"] = normal(T, std=-1.0 / T), normal(T, std=0.1 / T)
        s["d_logits"] = torch.empty(T, V, dtype=xt, device="cuda")
    return s


# ------------------------------------------------------------------ the operators

def run(s):
    op = s["case"]["op"]
    if own:
        import post_weight_quantization_09_b200 as Q
        if op == "adapter":
            Q.quip_adapter_apply(s["x"], s["ids"], s["down"], s["up"], s["scale"], s["y"], base=s["base"], h=s["h"])
            return s["y"], s["h"]
        if op == "adapter_grad":
            Q.quip_adapter_backward(s["x"], s["dy"], s["ids"], s["down"], s["up"], s["scale"], s["h"], dx=s["dx"],
                                    dx_base=s["dx_base"], d_down=s["d_down"], d_up=s["d_up"])
            return s["dx"], s["d_down"], s["d_up"]
        if op == "logprobs":
            Q.quip_logprobs(s["logits"], s["tokens"], s["logprob"], entropy=s["entropy"], lse=s["lse"],
                            top_values=s["top_values"], top_ids=s["top_ids"])
            return s["logprob"], s["entropy"], s["lse"], s["top_values"], s["top_ids"]
        Q.quip_logprobs_backward(s["logits"], s["tokens"], s["lse"], s["d_logits"], g_logprob=s["g_logprob"],
                                 g_entropy=s["g_entropy"], entropy=s["entropy"])
        return s["d_logits"]
    return {"adapter": _adapter, "adapter_grad": _adapter_grad, "logprobs": _logprobs,
            "logprobs_grad": _logprobs_grad}[op](s)


def _hidden(x, ids, down):
    """T x L x r: down_l x_t where adapter l is token t's, 0 elsewhere."""
    L, r, n = down.shape
    h = (x @ down.reshape(L * r, n).t()).reshape(-1, L, r)
    return torch.where((ids[:, None] == torch.arange(L, device=x.device))[:, :, None], h, 0.0)


def _adapter(s):
    """y = base + scale up (down x) for the token's adapter; h = down x."""
    L, r, m = s["up"].shape
    h = _hidden(s["x"].float(), s["ids"], s["down"].float())
    delta = (h * s["scale"][:, None]).reshape(-1, L * r) @ s["up"].float().reshape(L * r, m)
    return (s["base"].float() + delta).to(s["base"].dtype), h.sum(1)


def _adapter_grad(s):
    L, r, m = s["up"].shape
    n = s["down"].shape[2]
    x, dy = s["x"].float(), s["dy"].float()
    mine = (s["ids"][:, None] == torch.arange(L, device=x.device))[:, :, None]
    dh = _hidden(dy, s["ids"], s["up"].float()) * s["scale"][:, None]
    dx = s["dx_base"].float() + dh.reshape(-1, L * r) @ s["down"].float().reshape(L * r, n)
    d_down = (dh.reshape(-1, L * r).t() @ x).reshape(L, r, n)
    h = torch.where(mine, s["h"][:, None, :], 0.0) * s["scale"][:, None]
    d_up = (h.reshape(-1, L * r).t() @ dy).reshape(L, r, m)
    return dx.to(s["dx_base"].dtype), d_down, d_up


def _softmax(x):
    """(lse, p, entropy) of the rows of x; a barred entry counts nothing."""
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - top)
    z = e.sum(1, keepdim=True)
    lse = (top + z.log())[:, 0]
    p = e / z
    entropy = torch.where(p > 0, p * (lse[:, None] - x), 0.0).sum(1)
    return lse, p, entropy


def _logprobs(s):
    x, tokens, k = s["logits"].float(), s["tokens"].long(), s["case"]["k"]
    lse, _, entropy = _softmax(x)
    given = x.gather(1, tokens.clamp(min=0)[:, None])[:, 0] - lse
    logprob = torch.where(tokens >= 0, given, 0.0)
    values, ids = torch.sort(x, dim=1, descending=True, stable=True)   # ties: the lowest index first
    return logprob, entropy, lse, values[:, :k] - lse[:, None], ids[:, :k].to(torch.int32)


def _logprobs_grad(s):
    x, tokens = s["logits"].float(), s["tokens"].long()
    logp = x - s["lse"][:, None]
    p = torch.exp(logp)
    given = (tokens >= 0).float()
    g = s["g_logprob"] * given
    d = -g[:, None] * p - s["g_entropy"][:, None] * torch.where(p > 0, p * (logp + s["entropy"][:, None]), 0.0)
    d.scatter_add_(1, tokens.clamp(min=0)[:, None], g[:, None])
    return d.to(s["logits"].dtype)


# ------------------------------------------------------------------ what a pass cannot do without

_SIZE = {"bf16": 2, "f32": 4}


def work(case):
    T, x = case["T"], _SIZE[case["x"]]
    if case["op"] in ("adapter", "adapter_grad"):
        n, m, r = case["n"], case["m"], case["r"]
        used = min(case["L"], case["runs"])                   # adapters that some request names, at most
        w = used * r * (n + m)
        if case["op"] == "adapter":
            return {"bytes": T * (n * x + 2 * m * _SIZE[case["y"]] + 4 + 4 * r) + w * _SIZE[case["w"]],
                    "flops": 2 * T * r * (n + m)}
        return {"bytes": T * (3 * n * x + m * _SIZE[case["y"]] + 4 + 4 * r) + w * _SIZE[case["w"]]
                + 4 * case["L"] * r * (n + m),
                "flops": 4 * T * r * (n + m)}
    V = case["V"]
    if case["op"] == "logprobs":
        return {"bytes": T * (V * x + 16 + 8 * case["k"]), "flops": 6 * T * V}
    return {"bytes": T * (2 * V * x + 20), "flops": 8 * T * V}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("adapter", "adapter_grad"):
        x, down, up, ids = s["x"].double(), s["down"].double(), s["up"].double(), s["ids"]
        scale = s["scale"].double()
        out = (s["base"] if case["op"] == "adapter" else s["dx_base"]).double()
        if case["op"] == "adapter":
            h = torch.zeros(case["T"], case["r"], dtype=torch.float64, device="cuda")
            for a in range(case["L"]):
                t = (ids == a).nonzero()[:, 0]
                h[t] = x[t] @ down[a].T
                out[t] += scale[a] * (h[t] @ up[a])
            return out, h
        d_down, d_up = torch.zeros_like(down), torch.zeros_like(up)
        for a in range(case["L"]):
            t = (ids == a).nonzero()[:, 0]
            dy = s["dy"][t].double()
            dh = scale[a] * (dy @ up[a].T)
            out[t] += dh @ down[a]
            d_down[a] = dh.T @ x[t]
            d_up[a] = scale[a] * (s["h"][t].double().T @ dy)
        return out, d_down, d_up
    T, V, step = case["T"], case["V"], 256
    pieces = []
    for t in range(0, T, step):
        x, tokens = s["logits"][t:t + step].double(), s["tokens"][t:t + step].long()
        rows = torch.arange(x.shape[0], device="cuda")
        given = tokens >= 0
        if case["op"] == "logprobs":
            logp = torch.log_softmax(x, 1)
            p = torch.softmax(x, 1)
            logprob = logp[rows, tokens.clamp(min=0)].masked_fill(~given, 0.0)
            entropy = -(p * logp.masked_fill(p == 0, 0.0)).sum(1)
            # a stable order by falling value: equal values by rising index
            ids = torch.argsort(-x, dim=1, stable=True)[:, :case["k"]]
            pieces.append((logprob, entropy, torch.logsumexp(x, 1), logp.gather(1, ids), ids.to(torch.int32)))
        else:
            logp = x - s["lse"][t:t + step].double()[:, None]
            p = logp.exp()
            g = s["g_logprob"][t:t + step].double().masked_fill(~given, 0.0)
            ge = s["g_entropy"][t:t + step].double()
            d = -p * (g[:, None] + ge[:, None] * (logp.masked_fill(p == 0, 0.0)
                                                  + s["entropy"][t:t + step].double()[:, None]))
            d[rows, tokens.clamp(min=0)] += g
            pieces.append((d,))
    whole = tuple(torch.cat(c) for c in zip(*pieces))
    return whole if case["op"] == "logprobs" else whole[0]
