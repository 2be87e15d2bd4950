"""The token log-probability and 4-bit head operators as workloads: inputs, plain forms, 64-bit values.

Three ways a language-model head is used next to its training loss:

score   log-probability of given tokens, entropy and the best alternatives of every position, from hidden
        states x [N, D] and the head's weight [V, D] (bf16 or fp32), or from the head in 4 bits;
train   log-probability and entropy with the gradients of x, weight and bias for given upstream gradients;
linear  the logits themselves from the head in 4 bits.

With z = s (x W^T + b):  lse = log sum_v exp z_v,  logprob = z_y - lse (0 where the token is ignored),
entropy = lse - sum_v p_v z_v,  alternatives = the k largest z by value, then by lowest index.
A 4-bit weight is two's complement nibbles q (element 2i in byte i's low half) times one bf16 scale for
each run of `group` elements of a row.
"""
import math

import torch

own = False

IGNORE = -100
DEV = "cuda"


def listed():
    return [
        # one block of a block-diffusion decoder (4 masked tokens): confidence, entropy and the token to place
        {"name": "score-block4", "kind": "score", "dtype": "bf16", "N": 4, "D": 2560, "V": 151936, "k": 1, "sigma": 0.05,
         "scale": 1.0, "bias": False, "ignored": 0.0},
        # the smallest call: one token with its 8 best alternatives from a mid-size head
        {"name": "score-1-mid", "kind": "score", "dtype": "bf16", "N": 1, "D": 2048, "V": 32000, "k": 8, "sigma": 0.06,
         "scale": 1.0, "bias": False, "ignored": 0.0},
        # scoring a whole batch of sequences for evaluation
        {"name": "score-4096", "kind": "score", "dtype": "bf16", "N": 4096, "D": 2560, "V": 151936, "k": 8, "sigma": 0.04,
         "scale": 1.0, "bias": False, "ignored": 0.5},
        # odd vocabulary, logit scale, a bias that rules entries out with -inf, and 20 alternatives
        {"name": "score-ragged", "kind": "score", "dtype": "bf16", "N": 1001, "D": 4096, "V": 128257, "k": 20, "sigma": 0.06,
         "scale": 0.5, "bias": True, "ignored": 0.3},
        # a policy-gradient step over two sequences of 2048 tokens
        {"name": "train-4096", "kind": "train", "dtype": "bf16", "N": 4096, "D": 2560, "V": 151936, "k": 0, "sigma": 0.04,
         "scale": 1.0, "bias": False, "ignored": 0.5},
        # the same on a mid-size head with a bias and a ragged batch
        {"name": "train-mid", "kind": "train", "dtype": "bf16", "N": 1001, "D": 2048, "V": 32000, "k": 0, "sigma": 0.04,
         "scale": 1.0, "bias": True, "ignored": 0.2},
        # odd vocabulary with a logit scale
        {"name": "train-ragged", "kind": "train", "dtype": "bf16", "N": 517, "D": 4096, "V": 128257, "k": 0, "sigma": 0.04,
         "scale": 0.5, "bias": False, "ignored": 0.3},
        # the fp32 element type, where launches are what it costs
        {"name": "train-fp32-tiny", "kind": "train", "dtype": "fp32", "N": 64, "D": 64, "V": 512, "k": 0, "sigma": 0.2,
         "scale": 1.0, "bias": True, "ignored": 0.5},
        # logits of one decoded token from a 4-bit head
        {"name": "linear-w4-1", "kind": "linear", "dtype": "w4", "N": 1, "D": 2560, "V": 151936, "group": 128,
         "sigma": 0.05, "out": "fp32", "bias": False},
        # logits of 24 concurrent sequences, small groups, odd vocabulary, 16-bit logits
        {"name": "linear-w4-24", "kind": "linear", "dtype": "w4", "N": 24, "D": 4096, "V": 128257, "group": 64,
         "sigma": 0.04, "out": "bf16", "bias": True},
        # one block of the decoder from the 4-bit head
        {"name": "score-w4-block4", "kind": "score", "dtype": "w4", "N": 4, "D": 2560, "V": 151936, "k": 1, "group": 128,
         "sigma": 0.05, "scale": 1.0, "bias": False, "ignored": 0.0},
        # eleven positions of a mid-size 4-bit head with alternatives
        {"name": "score-w4-11-mid", "kind": "score", "dtype": "w4", "N": 11, "D": 2048, "V": 32000, "k": 8, "group": 32,
         "sigma": 0.06, "scale": 1.0, "bias": True, "ignored": 0.2},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["score", "score", "train", "train", "linear", "score-w4"])
    c = {"kind": kind, "sigma": rng.choice([0.02, 0.04, 0.06]), "bias": rng.random() < 0.4}
    if kind == "linear" or kind == "score-w4":
        D = 32 * _spread(rng, 2, 160)
        c.update(dtype="w4", N=_spread(rng, 1, 64), D=D, V=_spread(rng, 500, 160000), group=rng.choice([32, 64, 128]))
        if kind == "linear":
            c["out"] = rng.choice(["fp32", "bf16"])
            return c
        c.update(kind="score", k=rng.choice([0, 1, 4, 8, 20]), scale=rng.choice([1.0, 0.5]), ignored=rng.choice([0.0, 0.4]))
        return c
    c.update(k=0 if kind == "train" else rng.choice([0, 1, 4, 8, 20]), scale=rng.choice([1.0, 1.0, 0.5, 0.8]),
             ignored=rng.choice([0.0, 0.2, 0.5]))
    if rng.random() < 0.2:
        c.update(dtype="fp32", N=_spread(rng, 1, 300), D=8 * _spread(rng, 2, 40), V=_spread(rng, 300, 6000), sigma=0.2)
        return c
    D, V = 8 * _spread(rng, 8, 600), _spread(rng, 500, 160000)
    # no more work than the largest listed case of its kind
    most = min(4096, 4096 * 2560 * 151936 // (D * V))
    c.update(dtype="bf16", N=_spread(rng, 1, max(2, most)), D=D, V=V)
    return c


def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def prepare(case, seed):
    g = _generator(seed)
    N, D, V, kind = case["N"], case["D"], case["V"], case["kind"]
    dt = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
    s = {"case": case, "x": torch.randn(N, D, device=DEV, generator=g).to(dt), "bias": None}
    if case["dtype"] == "w4":
        # a symmetric round-to-nearest quantisation of a normal weight: integers of spread 2.2 in -7..7
        n = -(-D // case["group"])
        s["packed"] = _nibbles(torch.randn(V, D, device=DEV, generator=g).mul_(2.2).round_().clamp_(-7, 7).to(torch.int8))
        step = torch.rand(V, n, device=DEV, generator=g) * 0.4 + 0.8
        s["scales"] = (step * (case["sigma"] / 2.2)).to(torch.bfloat16)
    else:
        s["weight"] = torch.randn(V, D, device=DEV, generator=g).mul_(case["sigma"]).to(dt)
    if case["bias"]:
        b = torch.randn(V, device=DEV, generator=g) * 0.5
        if kind == "score":
            b[torch.rand(V, device=DEV, generator=g) < 0.1] = -math.inf  # entries that may not be chosen
        s["bias"] = b.to(dt)
    if kind != "linear":
        t = torch.randint(0, V, (N,), device=DEV, generator=g)
        s["token"] = torch.where(torch.rand(N, device=DEV, generator=g) < case["ignored"], IGNORE, t)
    if kind == "train":
        s["dlogprob"] = torch.randn(N, device=DEV, generator=g) / N  # advantages over the batch
        s["dentropy"] = torch.full((N,), 0.01 / N, device=DEV)       # an entropy bonus
        s["x"].requires_grad_()
        s["weight"].requires_grad_()
        if s["bias"] is not None:
            s["bias"].requires_grad_()
    return s


def _nibbles(q):
    u = q & 15
    return (u[:, 0::2] | (u[:, 1::2] << 4)).view(torch.uint8)


def _unpack(packed, scales, group, D, dtype):
    """The 4-bit weight's values [V, D]."""
    q = torch.stack((packed & 15, packed >> 4), 2).view(packed.shape[0], D).view(torch.int8)
    q = ((q ^ 8) - 8).to(dtype)
    return q * scales.to(dtype).repeat_interleave(group, 1)[:, :D]


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- the framework's operators
def _own(st):
    from linear_diffusion_cross_b200.logprob import fused_linear_logprobs
    from linear_diffusion_cross_b200.w4 import W4Weight, linear_w4
    c = st["case"]
    w = W4Weight(st["packed"], st["scales"], c["group"]) if c["dtype"] == "w4" else st["weight"]
    if c["kind"] == "linear":
        return linear_w4(st["x"], w, st["bias"], out_dtype=torch.float32 if c["out"] == "fp32" else torch.bfloat16)
    r = fused_linear_logprobs(st["x"], st["token"], w, st["bias"], top_k=c["k"], logit_scale=c["scale"], ignore_index=IGNORE)
    out = [r.logprob, r.entropy]
    if c["kind"] == "train":
        leaves = [st["x"], st["weight"]] + ([] if st["bias"] is None else [st["bias"]])
        return out + list(torch.autograd.grad(out, leaves, [st["dlogprob"], st["dentropy"]]))
    return out + [r.lse] + ([r.top_ids, r.top_logprobs] if c["k"] else [])


# ---------------------------------------------------------------- the plain form, in 32 bits
@torch.no_grad()
def _plain(st):
    c = st["case"]
    D = c["D"]
    if c["dtype"] == "w4":
        w = _unpack(st["packed"], st["scales"], c["group"], D, torch.float32)
    else:
        w = st["weight"].float()
    x = st["x"].float()
    z = x @ w.T
    if st["bias"] is not None:
        z += st["bias"].float()
    if c["kind"] == "linear":
        return z if c["out"] == "fp32" else z.to(torch.bfloat16)
    z *= c["scale"]
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    l = e.sum(1, keepdim=True)
    lse = m + torch.log(l)
    p = e / l
    logp = z - lse
    entropy = -torch.where(p > 0, p * logp, 0).sum(1, keepdim=True)
    valid = st["token"] != IGNORE
    y = torch.where(valid, st["token"], 0)[:, None]
    logprob = torch.where(valid, logp.gather(1, y)[:, 0], 0)
    out = [logprob, entropy[:, 0]]
    if c["kind"] == "train":
        a, de = torch.where(valid, st["dlogprob"], 0)[:, None], st["dentropy"][:, None]
        G = -p * (a + de * (logp + entropy))
        G.scatter_add_(1, y, a)
        G *= c["scale"]
        grads = [G @ w, G.T @ x] + ([] if st["bias"] is None else [G.sum(0)])
        return out + [d.to(st["x"].dtype) for d in grads]
    out.append(lse[:, 0])
    if c["k"]:
        ids, top = _best(z, x, w, st["bias"], c)
        out += [ids.int(), (top - lse).float()]
    return out


def _best(z, x, w, bias, c):
    """The k largest logits: candidates in 32 bits, their order in 64 (neighbours may be closer than 32 bits tell)."""
    ids = z.topk(min(c["k"] + 8, c["V"]), 1).indices.sort(1).values
    t = (x.double()[:, None, :] * w[ids].double()).sum(2)
    if bias is not None:
        t = t + bias[ids].double()
    top, at = (t * c["scale"]).sort(dim=1, descending=True, stable=True)
    return ids.gather(1, at)[:, : c["k"]], top[:, : c["k"]]


# ---------------------------------------------------------------- 64 bits, from the definitions
@torch.no_grad()
def exact(case, seed):
    st = prepare(case, seed)
    N, D, V, s = case["N"], case["D"], case["V"], case.get("scale", 1.0)
    if case["dtype"] == "w4":
        w = _unpack(st["packed"], st["scales"], case["group"], D, torch.float64)
    else:
        w = st["weight"].double()
    b = torch.zeros((), device=DEV, dtype=torch.float64) if st["bias"] is None else st["bias"].double()
    rows = max(1, min(N, int(2e8 // V)))  # tokens at a time
    parts, dx = [], []
    dw, db = torch.zeros(0), torch.zeros(0)
    if case["kind"] == "train":
        dw, db = torch.zeros(V, D, device=DEV, dtype=torch.float64), torch.zeros(V, device=DEV, dtype=torch.float64)
    for i in range(0, N, rows):
        x = st["x"][i:i + rows].double()
        z = s * (x @ w.T + b)
        if case["kind"] == "linear":
            parts.append([z])
            continue
        lse = torch.logsumexp(z, 1)
        p = torch.softmax(z, 1)
        surprise = torch.where(p > 0, lse[:, None] - z, 0.0)
        ent = (p * surprise).sum(1)
        tok = st["token"][i:i + rows]
        n = torch.arange(len(tok), device=DEV)
        lp = torch.zeros_like(lse)
        lp[tok != IGNORE] = (z[n, tok.clamp_min(0)] - lse)[tok != IGNORE]
        if case["kind"] == "train":
            parts.append([lp, ent])
            a = st["dlogprob"][i:i + rows].double() * (tok != IGNORE)
            q = st["dentropy"][i:i + rows].double()[:, None] * (surprise - ent[:, None])
            gz = p * (q - a[:, None])
            gz[n, tok.clamp_min(0)] += a
            gz *= s
            dx.append(gz @ w)
            dw += gz.T @ x
            db += gz.sum(0)
            continue
        k = case["k"]
        if not k:
            parts.append([lp, ent, lse])
            continue
        best = torch.sort(z, dim=1, descending=True, stable=True)
        parts.append([lp, ent, lse, best.indices[:, :k].int(), best.values[:, :k] - lse[:, None]])
    out = [torch.cat(t) for t in zip(*parts)]
    if case["kind"] == "train":
        out += [torch.cat(dx), dw] + ([] if st["bias"] is None else [db])
    return out[0] if case["kind"] == "linear" else out


def work(case):
    """Each input read once, each output written once; the products that the results cannot do without."""
    N, D, V, kind = case["N"], case["D"], case["V"], case["kind"]
    e = 4 if case["dtype"] == "fp32" else 2
    if case["dtype"] == "w4":
        weight = V * D // 2 + V * -(-D // case["group"]) * 2
    else:
        weight = V * D * e
    b = weight + N * D * e + (V * e if case["bias"] else 0)
    if kind == "linear":
        return {"bytes": b + N * V * (4 if case["out"] == "fp32" else 2), "flops": 2 * N * D * V}
    if kind == "train":
        return {"bytes": 2 * b + N * (8 + 8 + 8), "flops": 6 * N * D * V}
    return {"bytes": b + N * (8 + 12 + 8 * case["k"]), "flops": 2 * N * D * V}
