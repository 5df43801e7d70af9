"""The operators that train and serve adapters on a packed model, as calls to be timed and compared.

A packed weight ("Sherry": 3:4 ternary, 5 bits per block of 4 weights, scales alpha) is frozen; what a user
trains or swaps per request are low-rank adapters beside it, and what they read off the end of the model are the
log probabilities of tokens.  Four operators:

  lora           Y = X (T alpha)^T + s_a (X A_a^T) B_a^T, adapter a = ids[m] of every token (none: -1)
  lora_backward  dX = dY (T alpha) + P A_a with P = s_a dY B_a;  dA_a = P^T X;  dB_a = dY^T U with
                 U = s_a X A_a^T kept from the forward pass (sums over the tokens of adapter a)
  logprobs       of every row of logits: log p(target), entropy, the `top` likeliest tokens (ties: lowest id)
  logprobs_backward  dlogits = g (onehot(target) - p) - h p (log p + H) for d logp = g, d entropy = h

`run` computes them with elementary torch operations in fp32 where `own` is false, and with the framework's
entry points where it is true, on the same inputs.
"""
import math

import torch

own = False

BF16 = torch.bfloat16
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token of one request: a decode step's projection, where latency is everything
        {"name": "lora_decode_1", "op": "lora", "M": 1, "N": 2048, "K": 2048, "R": 16, "adapters": 8,
         "gran": "group", "group": 128, "out": "bf16", "mixed": True, "none": 0.0, "keep": False},
        # sixteen requests, each with an adapter of its own: a batched decode step
        {"name": "lora_decode_16", "op": "lora", "M": 16, "N": 8192, "K": 2048, "R": 16, "adapters": 16,
         "gran": "group", "group": 128, "out": "f32", "mixed": True, "none": 0.0, "keep": False},
        # prompts of several requests put together, some without an adapter; odd sizes, row scales
        {"name": "lora_ragged_331", "op": "lora", "M": 331, "N": 2050, "K": 8192, "R": 8, "adapters": 5,
         "gran": "channel", "group": 0, "out": "bf16", "mixed": False, "none": 0.2, "keep": False},
        # a training batch over four adapters, or a long prefill: the forward pass that keeps U
        {"name": "lora_prefill_4096", "op": "lora", "M": 4096, "N": 8192, "K": 2048, "R": 64, "adapters": 4,
         "gran": "group", "group": 128, "out": "bf16", "mixed": False, "none": 0.0, "keep": True},
        # the smallest training step: few tokens, a narrow projection
        {"name": "lora_backward_64", "op": "lora_backward", "M": 64, "N": 512, "K": 2048, "R": 8, "adapters": 2,
         "gran": "group", "group": 128, "out": "bf16", "mixed": False, "none": 0.0},
        # a ragged batch of three adapters with tokens of none between them, gradients accumulated in fp32
        {"name": "lora_backward_1000", "op": "lora_backward", "M": 1000, "N": 2048, "K": 8192, "R": 16, "adapters": 3,
         "gran": "channel", "group": 0, "out": "f32", "mixed": True, "none": 0.1},
        # an ordinary training batch on the widest projection
        {"name": "lora_backward_4096", "op": "lora_backward", "M": 4096, "N": 8192, "K": 2048, "R": 32, "adapters": 4,
         "gran": "group", "group": 128, "out": "bf16", "mixed": False, "none": 0.0},
        # the token just sampled, with its alternatives: one row of a large vocabulary
        {"name": "logprobs_1", "op": "logprobs", "M": 1, "V": 128256, "type": "bf16", "top": 20, "pad": 0, "banned": 0.0},
        # scoring a short text: an odd vocabulary in fp32, rows of a padded buffer, some tokens banned
        {"name": "logprobs_77_odd", "op": "logprobs", "M": 77, "V": 50257, "type": "f32", "top": 5, "pad": 47,
         "banned": 0.01},
        # scoring a batch
        {"name": "logprobs_2048", "op": "logprobs", "M": 2048, "V": 128256, "type": "bf16", "top": 8, "pad": 0,
         "banned": 0.0},
        # the gradient of a short odd batch in fp32
        {"name": "logprobs_backward_77_odd", "op": "logprobs_backward", "M": 77, "V": 50257, "type": "f32", "pad": 47,
         "banned": 0.01},
        # the gradient of a training batch
        {"name": "logprobs_backward_2048", "op": "logprobs_backward", "M": 2048, "V": 128256, "type": "bf16", "pad": 0,
         "banned": 0.0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lora", "lora", "lora_backward", "lora_backward", "logprobs", "logprobs_backward"])
    if op in ("lora", "lora_backward"):
        M = _log_int(rng, 1, 4096)
        N = _log_int(rng, 64, 8192)
        K = 128 * _log_int(rng, 2, 64)
        while M * N * K > 4096 * 8192 * 2048:
            M = (M + 1) // 2
        gran = rng.choice(["group", "group", "channel", "tensor"])
        case = {"op": op, "M": M, "N": N, "K": K, "R": rng.choice([8, 16, 24, 32, 64]),
                "adapters": _log_int(rng, 1, 32), "gran": gran, "group": rng.choice([64, 128]) if gran == "group" else 0,
                "out": rng.choice(["bf16", "f32"]), "mixed": rng.random() < 0.5, "none": rng.choice([0.0, 0.0, 0.3])}
        if op == "lora":
            case["keep"] = rng.random() < 0.5
        return case
    V = _log_int(rng, 1000, 128256)
    M = _log_int(rng, 1, 4096)
    while M * V > 2048 * 128256:
        M = (M + 1) // 2
    case = {"op": op, "M": M, "V": V, "type": rng.choice(["bf16", "f32"]), "pad": rng.choice([0, 0, 3, 64]),
            "banned": rng.choice([0.0, 0.01])}
    if case["type"] == "f32" and M * V > 1024 * 128256:
        case["M"] = (M + 1) // 2
    if op == "logprobs":
        case["top"] = rng.choice([0, 1, 5, 20])
    return case


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = "cuda"

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=dev)

    s = dict(case)
    M = case["M"]
    if case["op"] in ("lora", "lora_backward"):
        N, K, R, n = case["N"], case["K"], case["R"], case["adapters"]
        # packed planes: every nibble and sign bit is a valid code, so random bits are a random ternary weight
        s["idx"] = torch.randint(-2 ** 31, 2 ** 31, (N, K // 32), generator=g, device=dev, dtype=torch.int64).to(torch.int32)
        s["sgn"] = torch.randint(0, 256, (N, K // 32), generator=g, device=dev, dtype=torch.int64).to(torch.uint8)
        scales = {"group": N * (K // case["group"]) if case["group"] else 0, "channel": N, "tensor": 1}[case["gran"]]
        # the mean |w| of the kept weights of a layer with std 0.02: near 0.02, a little different from group to group
        s["scales"] = 0.02 * (1.0 + 0.08 * normal(scales)).clamp(0.5, 2.0)
        s["X"] = normal(M, K).to(BF16)
        s["A"] = (normal(n, R, K) / math.sqrt(K)).to(BF16)
        s["B"] = (0.05 * normal(n, N, R)).to(BF16)
        s["scaling"] = 0.5 + 1.5 * uniform(n)
        ids = torch.randint(0, n, (M,), generator=g, device=dev)
        if not case["mixed"]:
            ids = ids.sort().values  # the tokens of a request stand together
        ids = torch.where(uniform(M) < case["none"], -torch.ones_like(ids), ids)
        s["ids"] = ids.to(torch.int32)
        if case["op"] == "lora_backward":
            s["dY"] = (normal(M, N) / N).to(BF16)
            # U of the forward pass, which a training program keeps
            u = torch.einsum("mk,ark->mar", s["X"].double(), s["A"].double())
            pick = (ids[:, None] == torch.arange(n, device=dev)) * s["scaling"].double()
            s["U"] = torch.einsum("mar,ma->mr", u, pick).float()
        return s
    V = case["V"]
    # logits as a head gives them: a spread of a few units, one token that leads; rows of a padded buffer
    z = 2.5 * torch.randn((M, V + case["pad"]), generator=g, device=dev, dtype=torch.float32)
    lead = torch.randint(0, V, (M, 1), generator=g, device=dev)
    z.scatter_add_(1, lead, 6.0 + 4.0 * uniform(M, 1))
    if case["banned"]:
        z = z.masked_fill(torch.rand(z.shape, generator=g, device=dev) < case["banned"], -math.inf)
    s["logits"] = z.to(TYPES[case["type"]])[:, :V]
    del z
    # the targets: mostly the leading token, others anywhere, one in sixteen left out (-1)
    t = torch.where(uniform(M) < 0.6, lead[:, 0], torch.randint(0, V, (M,), generator=g, device=dev))
    s["targets"] = torch.where(uniform(M) < 1 / 16, -torch.ones_like(t), t).to(torch.int32)
    if case["op"] == "logprobs_backward":
        s["dlogp"] = normal(M) / M
        s["dentropy"] = 0.01 * normal(M) / M
        # the row statistics that the forward pass keeps: the largest logit, log of the sum of exp(z - largest), entropy
        top = s["logits"].max(1).values.double()
        lsum = torch.empty(M, dtype=torch.float64, device=dev)
        ent = torch.empty(M, dtype=torch.float64, device=dev)
        for i in range(0, M, 256):
            d = s["logits"][i:i + 256].double() - top[i:i + 256, None]
            e = d.exp()
            total = e.sum(1)
            lsum[i:i + 256] = total.log()
            ent[i:i + 256] = total.log() - torch.where(e > 0, e * d, 0.0).sum(1) / total
        s["stats"] = torch.stack([top, lsum], 1).float()
        s["entropy"] = ent.float()
    return s


# ---- the framework's calls ---------------------------------------------------------------------------------

def _framework(s):
    import sparse_ternary_weight_b200 as sw
    if s["op"] in ("lora", "lora_backward"):
        gran = {"group": sw.PER_GROUP, "channel": sw.PER_CHANNEL, "tensor": sw.PER_TENSOR}[s["gran"]]
        P = sw.PackedWeight(s["idx"], s["sgn"], s["scales"], s["N"], s["K"], gran, s["group"])
        dt = TYPES[s["out"]]
        if s["op"] == "lora":
            return sw.linear_lora(s["X"], P, s["A"], s["B"], s["ids"], s["scaling"], out_dtype=dt, return_u=s["keep"])
        return sw.linear_lora_backward(s["dY"], s["X"], P, s["A"], s["B"], s["ids"], s["U"], s["scaling"], grad_dtype=dt)
    if s["op"] == "logprobs":
        r = sw.token_logprobs(s["logits"], s["targets"], top=s["top"])
        out = [r.logp, r.entropy, r.stats]
        return out + [r.top_logp, r.top_ids] if s["top"] else out
    return sw.token_logprobs_backward(s["logits"], s["targets"], s["stats"], s["entropy"], s["dlogp"], s["dentropy"])


# ---- the plain forms ---------------------------------------------------------------------------------------

def _dense(s):
    """T alpha [N, K] in fp32 from the packed planes."""
    N, K = s["N"], s["K"]
    shift = torch.arange(8, device="cuda", dtype=torch.int32)
    nib = ((s["idx"][:, :, None] >> (4 * shift)) & 15).reshape(N, K // 4, 1)
    neg = ((s["sgn"].to(torch.int32)[:, :, None] >> shift) & 1).reshape(N, K // 4, 1)
    zero = nib >> 2
    first = 1.0 - 2.0 * neg
    signs = torch.cat([first, first * (1 - (nib & 2)), first * (1 - 2 * (nib & 1))], 2)
    pos = torch.arange(4, device="cuda", dtype=torch.int32)
    place = (pos - (pos > zero).to(torch.int32)).clamp(max=2).to(torch.int64)
    t = torch.where(pos == zero, 0.0, signs.gather(2, place)).reshape(N, K)
    if s["gran"] == "tensor":
        return t * s["scales"]
    return (t.reshape(-1, s["group"] or K) * s["scales"][:, None]).reshape(N, K)


def _pick(s):
    """[M, adapters]: the scaling of the token's adapter in its column, 0 elsewhere."""
    return (s["ids"][:, None] == torch.arange(s["adapters"], device="cuda")) * s["scaling"]


def _plain_lora(s):
    X, A, B = s["X"].float(), s["A"].float(), s["B"].float()
    n, R = s["adapters"], s["R"]
    each = (X @ A.reshape(n * R, -1).T).reshape(-1, n, R) * _pick(s)[:, :, None]
    Y = X @ _dense(s).T + each.reshape(-1, n * R) @ B.transpose(1, 2).reshape(n * R, -1)
    Y = Y.to(TYPES[s["out"]])
    return (Y, each.sum(1)) if s["keep"] else Y


def _plain_lora_backward(s):
    G, X, A, B = s["dY"].float(), s["X"].float(), s["A"].float(), s["B"].float()
    n, R, dt = s["adapters"], s["R"], TYPES[s["out"]]
    pick = _pick(s)
    each = (G @ B.transpose(1, 2).reshape(n * R, -1).T).reshape(-1, n, R) * pick[:, :, None]
    dX = G @ _dense(s) + each.reshape(-1, n * R) @ A.reshape(n * R, -1)
    dA = (each.reshape(-1, n * R).T @ X).reshape(A.shape)
    u = s["U"][:, None, :] * (s["ids"][:, None] == torch.arange(n, device="cuda"))[:, :, None]
    dB = (u.reshape(-1, n * R).T @ G).reshape(n, R, -1).transpose(1, 2).contiguous()
    return dX.to(BF16), dA.to(dt), dB.to(dt)


def _plain_logprobs(s):
    z = s["logits"].float()
    largest = z.max(1, keepdim=True).values
    d = z - largest
    e = d.exp()
    total = e.sum(1)
    lsum = total.log()
    entropy = lsum - torch.where(e > 0, e * d, 0.0).sum(1) / total
    del e
    t = s["targets"].long()
    logp = torch.where(t < 0, 0.0, d.gather(1, t.clamp(min=0)[:, None])[:, 0] - lsum)
    stats = torch.cat([largest, lsum[:, None]], 1)
    if not s["top"]:
        return [logp, entropy, stats]
    top, ids = z.sort(dim=1, descending=True, stable=True)
    best = d.gather(1, ids[:, :s["top"]]) - lsum[:, None]
    return [logp, entropy, stats, best, ids[:, :s["top"]].to(torch.int32)]


def _plain_logprobs_backward(s):
    lp = s["logits"].float() - s["stats"][:, :1] - s["stats"][:, 1:]
    p = lp.exp()
    w = torch.where(p > 0, s["dlogp"].mul(s["targets"] >= 0)[:, None] + s["dentropy"][:, None] * (lp + s["entropy"][:, None]), 0.0)
    out = -p * w
    t = s["targets"].long()
    out.scatter_add_(1, t.clamp(min=0)[:, None], (s["dlogp"] * (t >= 0))[:, None])
    return out.to(s["logits"].dtype)


def run(state):
    if own:
        return _framework(state)
    return {"lora": _plain_lora, "lora_backward": _plain_lora_backward, "logprobs": _plain_logprobs,
            "logprobs_backward": _plain_logprobs_backward}[state["op"]](state)


def work(case):
    M = case["M"]
    if case["op"] in ("lora", "lora_backward"):
        N, K, R, n = case["N"], case["K"], case["R"], case["adapters"]
        scales = {"group": N * (K // case["group"]) if case["group"] else 0, "channel": N, "tensor": 1}[case["gran"]]
        weight = N * K * 5 // 32 + 4 * scales
        used = min(n, M)
        size = 2 if case["out"] == "bf16" else 4
        if case["op"] == "lora":
            return {"bytes": weight + 2 * M * K + 2 * used * R * (K + N) + 4 * M + size * M * N
                    + (4 * M * R if case["keep"] else 0),
                    "flops": 2 * M * N * K + 2 * M * R * (K + N)}
        return {"bytes": weight + 2 * M * (N + K) + 2 * used * R * (K + N) + 4 * M * R + 4 * M + 2 * M * K
                + size * n * R * (K + N),
                "flops": 2 * M * N * K + 4 * M * R * (K + N)}
    V = case["V"]
    size = 2 if case["type"] == "bf16" else 4
    if case["op"] == "logprobs":
        return {"bytes": M * V * size + 20 * M + 8 * M * case["top"], "flops": 6 * M * V}
    return {"bytes": 2 * M * V * size + 24 * M, "flops": 6 * M * V}


# ---- the definitions, in 64 bits ---------------------------------------------------------------------------

def _exact_weight(s):
    table = torch.zeros(32, 4, dtype=torch.float64)
    for code in range(32):
        kept = [p for p in range(4) if p != (code >> 2 & 3)]
        lead = -1.0 if code & 16 else 1.0
        table[code, kept[0]] = lead
        table[code, kept[1]] = -lead if code & 2 else lead
        table[code, kept[2]] = -lead if code & 1 else lead
    table = table.cuda()
    N, K = s["N"], s["K"]
    W = torch.empty(N, K // 32, 8, 4, dtype=torch.float64, device="cuda")
    for j in range(8):
        code = torch.bitwise_and(torch.bitwise_right_shift(s["idx"], 4 * j), 15)
        code = code + 16 * torch.bitwise_and(torch.bitwise_right_shift(s["sgn"], j), 1).to(torch.int32)
        W[:, :, j] = table[code.long()]
    W = W.reshape(N, K)
    a = s["scales"].double()
    if s["gran"] == "tensor":
        return W.mul_(a[0])
    if s["gran"] == "channel":
        return W.mul_(a.view(N, 1))
    return W.view(N, K // s["group"], s["group"]).mul_(a.view(N, -1, 1)).view(N, K)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "lora":
        X = s["X"].double()
        Y = torch.matmul(X, _exact_weight(s).t())
        U = torch.zeros(case["M"], case["R"], dtype=torch.float64, device="cuda")
        for a in range(case["adapters"]):
            at = (s["ids"] == a).nonzero()[:, 0]
            u = s["scaling"][a].double() * torch.matmul(X[at], s["A"][a].double().t())
            U[at] = u
            Y[at] += torch.matmul(u, s["B"][a].double().t())
        return (Y, U) if case["keep"] else Y
    if case["op"] == "lora_backward":
        X, G = s["X"].double(), s["dY"].double()
        dX = torch.matmul(G, _exact_weight(s))
        dA = torch.zeros(s["A"].shape, dtype=torch.float64, device="cuda")
        dB = torch.zeros(s["B"].shape, dtype=torch.float64, device="cuda")
        for a in range(case["adapters"]):
            at = (s["ids"] == a).nonzero()[:, 0]
            P = s["scaling"][a].double() * torch.matmul(G[at], s["B"][a].double())
            dX[at] += torch.matmul(P, s["A"][a].double())
            dA[a] = torch.matmul(P.t(), X[at])
            dB[a] = torch.matmul(G[at].t(), s["U"][at].double())
        return dX, dA, dB
    M, V = case["M"], case["V"]
    target = s["targets"].long()
    if case["op"] == "logprobs":
        logp = torch.zeros(M, dtype=torch.float64, device="cuda")
        entropy = torch.zeros(M, dtype=torch.float64, device="cuda")
        best = torch.zeros(M, case["top"], dtype=torch.float64, device="cuda")
        ids = torch.zeros(M, case["top"], dtype=torch.int32, device="cuda")
        stats = torch.zeros(M, 2, dtype=torch.float64, device="cuda")
        for i in range(0, M, 128):
            z = s["logits"][i:i + 128].double()
            stats[i:i + 128, 0] = z.amax(1)
            stats[i:i + 128, 1] = z.logsumexp(1) - z.amax(1)
            lp = torch.log_softmax(z, 1)
            p = lp.exp()
            entropy[i:i + 128] = -(p * lp.clamp(min=-1e300)).sum(1)
            t = target[i:i + 128]
            logp[i:i + 128] = torch.where(t >= 0, lp.gather(1, t.clamp(min=0).view(-1, 1)).view(-1), 0.0)
            for j in range(case["top"]):
                value = lp.max(1, keepdim=True).values
                first = torch.where(lp == value, torch.arange(V, device="cuda"), V).min(1).values
                best[i:i + 128, j] = value[:, 0]
                ids[i:i + 128, j] = first.to(torch.int32)
                lp.scatter_(1, first.view(-1, 1), -math.inf)
        return [logp, entropy, stats] + ([best, ids] if case["top"] else [])
    out = torch.empty(M, V, dtype=torch.float64, device="cuda")
    g, h = s["dlogp"].double(), s["dentropy"].double()
    for i in range(0, M, 128):
        z = s["logits"][i:i + 128].double()
        lp = torch.log_softmax(z, 1)
        p = lp.exp()
        H = -(p * lp.clamp(min=-1e300)).sum(1, keepdim=True)
        t = target[i:i + 128]
        hot = torch.zeros_like(p)
        hot.scatter_(1, t.clamp(min=0).view(-1, 1), 1.0)
        d = g[i:i + 128].view(-1, 1) * (t >= 0).view(-1, 1) * (hot - p)
        out[i:i + 128] = d - h[i:i + 128].view(-1, 1) * p * (lp.clamp(min=-1e300) + H)
    return out
