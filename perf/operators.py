"""The training-step operators beside the embedding gradient: what they compute in plain
torch, what a user's call of each looks like, and the sizes they are measured at.

Three operators:

* ``token_logprobs``: per row of logits, the log probability of the row's token, the
  entropy of the row's distribution and its most likely alternatives;
* ``token_logprobs_backward``: the gradient of those log probabilities and entropies with
  respect to the logits;
* ``orthogonalize_update``: five Newton-Schulz steps towards the nearest orthogonal matrix
  of an update, as the Muon optimiser takes them.

With ``own`` false, ``run`` computes them with elementary torch operations in 32 bits;
with ``own`` true it calls ``embedding_weight_grad_gb300``.
"""
import math

import torch

own = False

COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5
LARGEST_LOGITS = 8192 * 129280      # elements of the largest logits drawn
LARGEST_UPDATE = 7168 * 7168        # elements of the largest update drawn
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # serving: one sequence's next token over a large vocabulary, 20 alternatives
        {"name": "logprobs decode 1x129280", "op": "logprobs", "rows": 1, "vocab": 129280, "dtype": "bf16",
         "top": 20, "scale": 1.25, "padding": 0.0, "allowed": 1.0, "row_pad": 0},
        # serving: constrained decoding of a small batch; nine tenths of the vocabulary is
        # masked with -inf, and the last row has nothing left
        {"name": "logprobs masked 16x256000", "op": "logprobs", "rows": 16, "vocab": 256000, "dtype": "fp32",
         "top": 5, "scale": 1.0, "padding": 0.0, "allowed": 0.1, "row_pad": 0},
        # training: GPT-2-like vocabulary, whose odd width leaves the rows unaligned; padding tokens
        {"name": "logprobs train 8192x50257", "op": "logprobs", "rows": 8192, "vocab": 50257, "dtype": "bf16",
         "top": 0, "scale": 1.0, "padding": 0.05, "allowed": 1.0, "row_pad": 0},
        # training on rewards: a large vocabulary with alternatives, at a sampling temperature of 0.8
        {"name": "logprobs train 8192x129280", "op": "logprobs", "rows": 8192, "vocab": 129280, "dtype": "bf16",
         "top": 8, "scale": 1.25, "padding": 0.05, "allowed": 1.0, "row_pad": 0},
        # the gradient of a small model's loss
        {"name": "backward 4096x1024", "op": "backward", "rows": 4096, "vocab": 1024, "dtype": "fp32",
         "entropy": False, "scale": 1.0, "padding": 0.05, "allowed": 1.0, "row_pad": 0},
        # the gradient at the GPT-2-like vocabulary: unaligned rows
        {"name": "backward 8192x50257", "op": "backward", "rows": 8192, "vocab": 50257, "dtype": "bf16",
         "entropy": False, "scale": 1.0, "padding": 0.05, "allowed": 1.0, "row_pad": 0},
        # policy gradient with an entropy bonus over a large vocabulary
        {"name": "backward 8192x129280 entropy", "op": "backward", "rows": 8192, "vocab": 129280, "dtype": "bf16",
         "entropy": True, "scale": 1.25, "padding": 0.05, "allowed": 1.0, "row_pad": 0},
        # one small matrix: latency counts
        {"name": "orthogonalize 256x256", "op": "orthogonalize", "batch": 1, "rows": 256, "cols": 256, "dtype": "fp32"},
        # odd sizes, more rows than columns
        {"name": "orthogonalize 4097x1001", "op": "orthogonalize", "batch": 1, "rows": 4097, "cols": 1001, "dtype": "fp32"},
        # the square matrices of 24 layers of hidden size 1024 in one call
        {"name": "orthogonalize 24x1024x1024", "op": "orthogonalize", "batch": 24, "rows": 1024, "cols": 1024, "dtype": "bf16"},
        # a wide projection of a hidden size of 7168
        {"name": "orthogonalize 2048x7168", "op": "orthogonalize", "batch": 1, "rows": 2048, "cols": 7168, "dtype": "bf16"},
        # the largest: a square projection of a hidden size of 7168
        {"name": "orthogonalize 7168x7168", "op": "orthogonalize", "batch": 1, "rows": 7168, "cols": 7168, "dtype": "fp32"},
    ]


def _log_uniform(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, n + (n == 3072)))


def draw(rng):
    op = rng.choice(["logprobs", "backward", "orthogonalize"])
    dtype = rng.choice(["bf16", "fp32"])
    if op == "orthogonalize":
        rows, cols = _log_uniform(rng, 8, 7168), _log_uniform(rng, 8, 7168)
        most = min(LARGEST_UPDATE // (rows * cols), int(7168 ** 3 / (rows * cols * min(rows, cols))), 32)
        return {"op": op, "batch": _log_uniform(rng, 1, max(1, most)), "rows": rows, "cols": cols, "dtype": dtype}
    vocab = _log_uniform(rng, 64, 256000)
    elements = LARGEST_LOGITS if dtype == "bf16" else LARGEST_LOGITS // 2
    case = {"op": op, "rows": _log_uniform(rng, 1, min(131072, elements // vocab)), "vocab": vocab, "dtype": dtype,
            "scale": rng.choice([1.0, 1.25, 0.5]), "padding": rng.choice([0.0, 0.05, 0.3]),
            "allowed": rng.choice([1.0, 1.0, 0.1]), "row_pad": rng.choice([0, 0, 3, 64])}
    if op == "logprobs":
        case["top"] = rng.choice([0, 1, 5, 8, 20])
    else:
        case["entropy"] = rng.random() < 0.5
    return case


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _logits(case, g):
    """Logits of a model that is often, not always, sure of the token; -inf where a token
    is not allowed.  Rows of a wider buffer where row_pad is not 0."""
    n, V = case["rows"], case["vocab"]
    z = torch.empty(n, V + case["row_pad"], dtype=DTYPES[case["dtype"]], device="cuda")[:, :V]
    targets = torch.randint(V, (n,), generator=g, device="cuda")
    lift = torch.rand(n, 1, generator=g, device="cuda") * 14
    for at in range(0, n, 1024):                 # in parts, to keep the 32-bit copy small
        part = torch.randn(min(1024, n - at), V, generator=g, device="cuda") * 2 - 1
        t = targets[at:at + 1024, None]
        part.scatter_add_(1, t, lift[at:at + 1024])
        if case["allowed"] < 1:
            kept = part.gather(1, t)
            part.masked_fill_(torch.rand(part.shape, generator=g, device="cuda") >= case["allowed"], -math.inf)
            part.scatter_(1, t, kept)
        z[at:at + 1024] = part
    if case["allowed"] < 1 and n > 1:
        z[n - 1] = -math.inf                     # a row whose mask leaves nothing
    order = torch.randperm(n, generator=g, device="cuda")
    targets[order[:int(n * case["padding"])]] = -100
    return z, targets


def _update(case, g):
    """A gradient's shape of spectrum: a few strong directions over noise."""
    b, m, n = case["batch"], case["rows"], case["cols"]
    u = torch.randn(b, m, 16, generator=g, device="cuda")
    v = torch.randn(b, 16, n, generator=g, device="cuda")
    x = torch.randn(b, m, n, generator=g, device="cuda").add_(u @ v, alpha=0.5).mul_(1e-3).to(DTYPES[case["dtype"]])
    return x if b > 1 else x[0]


def prepare(case, seed):
    g = _generator(seed)
    state = {"case": case}
    if case["op"] == "orthogonalize":
        state["grad"] = _update(case, g)
        return state
    z, t = _logits(case, g)
    state.update(logits=z, targets=t)
    if case["op"] == "backward":
        # what the forward pass left, and the gradients that reach it
        parts = [_plain_logprobs(z[at:at + 1024], t[at:at + 1024], case["scale"], 0) for at in range(0, case["rows"], 1024)]
        for key in ("entropy", "row_max", "log_sum"):
            state[key] = torch.cat([p[key] for p in parts])
        state["grad_logprobs"] = torch.randn(case["rows"], generator=g, device="cuda")
        state["grad_entropy"] = torch.randn(case["rows"], generator=g, device="cuda") * 0.1 if case["entropy"] else None
    return state


def _plain_logprobs(logits, targets, scale, top):
    z = logits.float()
    real = targets >= 0                                  # a negative target marks a padding row
    row_max = z.amax(1)
    some = row_max > -math.inf                           # whether the mask leaves anything
    base = torch.where(some, row_max, 0.0)
    x = (z - base[:, None]) * scale
    e = x.exp()
    # the sum without one occurrence of the largest (whose term is 1): a row that is all but
    # sure of one token keeps the digits of the others' small share
    others = torch.where(some, e.scatter(1, z.argmax(1, keepdim=True), 0.0).sum(1), 0.0)
    log_sum = others.log1p()
    entropy = log_sum - (e * x.clamp_min(-1e30)).sum(1) / (others + 1)
    logprobs = x.gather(1, targets.clamp_min(0)[:, None])[:, 0] - log_sum
    out = {"logprobs": torch.where(real, logprobs, 0.0), "entropy": torch.where(real & some, entropy, 0.0),
           "row_max": torch.where(real, row_max, 0.0), "log_sum": torch.where(real, log_sum, 0.0)}
    if top:
        # one whole number that orders by logit, then by lower id
        i = (z + 0.0).view(torch.int32)
        key = (i ^ ((i >> 31) & 0x7fffffff)).to(torch.int64) * 2 ** 32 + torch.arange(z.shape[1] - 1, -1, -1, device=z.device)
        ids = key.topk(top, dim=1).indices
        best = x.gather(1, ids) - log_sum[:, None]
        out["top_logprobs"] = torch.where(real[:, None], best, -math.inf)
        out["top_ids"] = torch.where(out["top_logprobs"] > -math.inf, ids, -1)
    return out


def _plain_backward(s):
    z, t, scale = s["logits"].float(), s["targets"], s["case"]["scale"]
    empty = s["row_max"] == -math.inf
    g = torch.where((t >= 0) & ~empty, s["grad_logprobs"], 0.0)
    logp = (z - torch.where(empty, 0.0, s["row_max"])[:, None]) * scale - s["log_sum"][:, None]
    p = logp.exp()
    # p less the token's one-hot, at the token as expm1(log p): p - 1 with the digits it
    # has left where p is near 1
    at = t.clamp_min(0)[:, None]
    grad = -g[:, None] * p.scatter(1, at, logp.gather(1, at).expm1())
    if s["grad_entropy"] is not None:
        h = torch.where((t >= 0) & ~empty, s["grad_entropy"], 0.0)
        grad -= h[:, None] * p * (logp.clamp_min(-1e30) + s["entropy"][:, None])
    return (torch.where(((t >= 0) & ~empty)[:, None], grad, 0.0) * scale).to(s["logits"].dtype)


def _plain_orthogonalize(grad):
    a, b, c = COEFFICIENTS
    x = grad.float()
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT if tall else x
    norm = x.square().sum((-2, -1), keepdim=True).sqrt()
    x = x / torch.where(norm > 0, norm, 1.0)
    for _ in range(STEPS):
        gram = x @ x.mT
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return (x.mT if tall else x).to(torch.bfloat16)


def run(state):
    case = state["case"]
    if own:
        import embedding_weight_grad_gb300 as ewg

        if case["op"] == "logprobs":
            r = ewg.token_logprobs(state["logits"], state["targets"], scale=case["scale"], top=case["top"])
            out = {"logprobs": r.logprobs, "entropy": r.entropy, "row_max": r.row_max, "log_sum": r.log_sum}
            if case["top"]:
                out.update(top_logprobs=r.top_logprobs, top_ids=r.top_ids)
            return out
        if case["op"] == "backward":
            return {"grad_logits": ewg.token_logprobs_backward(
                state["logits"], state["targets"], state["row_max"], state["log_sum"], state["grad_logprobs"],
                entropy=state["entropy"], grad_entropy=state["grad_entropy"], scale=case["scale"])}
        return {"update": ewg.orthogonalize_update(state["grad"], steps=STEPS, coefficients=COEFFICIENTS)}
    if case["op"] == "logprobs":
        return _plain_logprobs(state["logits"], state["targets"], case["scale"], case["top"])
    if case["op"] == "backward":
        return {"grad_logits": _plain_backward(state)}
    return {"update": _plain_orthogonalize(state["grad"])}


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "orthogonalize":
        r, c = sorted((case["rows"], case["cols"]))
        elements = case["batch"] * r * c
        # per step X X^T and A A, both symmetric, at half their products, and B X
        return {"bytes": elements * (size + 2), "flops": case["batch"] * STEPS * (3 * r * r * c + r ** 3)}
    n, V = case["rows"], case["vocab"]
    read = (n - int(n * case["padding"])) * V          # rows of padding need not be read
    if case["op"] == "logprobs":
        return {"bytes": read * size + n * (8 + 16 + 12 * case["top"]), "flops": 6 * read}
    return {"bytes": (read + n * V) * size + n * (8 + (20 if case["entropy"] else 12)), "flops": (7 if case["entropy"] else 5) * read}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "orthogonalize":
        # by its definition in 64 bits, on the smaller side's Gram matrix
        w = s["grad"].double()
        size = torch.linalg.vector_norm(w, dim=(-2, -1), keepdim=True)
        w = w / size.masked_fill(size == 0, 1.0)
        k1, k3, k5 = COEFFICIENTS
        wide = w.shape[-2] <= w.shape[-1]
        eye = torch.eye(min(w.shape[-2:]), dtype=torch.float64, device=w.device)
        for _ in range(STEPS):
            q = torch.matmul(w, w.mT) if wide else torch.matmul(w.mT, w)
            poly = k1 * eye + torch.matmul(q, k3 * eye + k5 * q)
            w = torch.matmul(poly, w) if wide else torch.matmul(w, poly)
        return {"update": w}
    rows = [_exact_rows(case, s, slice(at, at + 512)) for at in range(0, case["rows"], 512)]
    out = {key: torch.cat([r[key] for r in rows]) for key in rows[0] if rows[0][key] is not None}
    if case.get("top"):
        out["top_ids"] = None
    return out


def _exact_rows(case, s, part):
    z, t = s["logits"][part].double(), s["targets"][part]
    dead = (t < 0)
    logp = torch.log_softmax(z * case["scale"], dim=1)
    nothing = torch.isneginf(z).all(1)
    logp = logp.masked_fill(nothing[:, None], -math.inf)
    p = logp.exp()
    plogp = torch.where(p > 0, p * logp, 0.0)
    entropy = -plogp.sum(1)
    at = t.clamp(min=0)[:, None]
    if case["op"] == "logprobs":
        top_z = z.amax(1)
        log_sum = torch.where(nothing, 0.0, torch.logsumexp(z * case["scale"], 1) - top_z * case["scale"])
        out = {"logprobs": logp.gather(1, at)[:, 0].masked_fill(dead, 0.0), "entropy": entropy.masked_fill(dead, 0.0),
               "row_max": top_z.masked_fill(dead, 0.0), "log_sum": log_sum.masked_fill(dead, 0.0)}
        if case["top"]:
            out["top_logprobs"] = logp.sort(dim=1, descending=True).values[:, :case["top"]].masked_fill(dead[:, None], -math.inf)
            out["top_ids"] = None
        return out
    gl = s["grad_logprobs"][part].double().masked_fill(dead | nothing, 0.0)
    grad = -gl[:, None] * p
    grad.scatter_add_(1, at, gl[:, None])
    if s["grad_entropy"] is not None:
        ge = s["grad_entropy"][part].double().masked_fill(dead | nothing, 0.0)
        grad -= ge[:, None] * (plogp + p * entropy[:, None])
    return {"grad_logits": grad * case["scale"]}
