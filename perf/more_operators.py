"""The training-step operators between the vocabulary's two ends and the optimiser: what they
compute in plain torch, what a user's call of each looks like, and the sizes they are measured at.

Three operators:

* ``layer_norm``: rows normalised to mean 0 and variance 1, times a weight, plus a bias; with
  each row's mean and 1 / standard deviation;
* ``layer_norm_backward``: the gradient with respect to the rows, and the weight's and the
  bias's added to their main_grads;
* ``adamw_step``: one AdamW step of many tensors at once, the two moments held in 32 bits, or
  in 8 (e4m3, the second as its root) with a scale for every 256 elements.

With ``own`` false, ``run`` computes them with elementary torch operations in 32 bits;
with ``own`` true it calls ``embedding_weight_grad_gb300``.
"""
import math

import torch

own = False

EPS_NORM = 1e-5
LR, BETAS, EPS_ADAM = 1e-3, (0.9, 0.999), 1e-8
FIRST_STEP = 1000                       # of the optimiser's steps: in the middle of a training
BLOCK = 256                             # elements of a tensor that share an 8-bit state's scale
LARGEST_ROWS = 131072 * 8192            # elements of the largest rows drawn
LARGEST_TABLE = 129280 * 7168           # elements of the largest update drawn
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # serving: a single token's row at a hidden size of 7168
        {"name": "norm 1x7168", "op": "norm", "rows": 1, "hidden": 7168, "dtype": "bf16", "weight": "bf16",
         "bias": True, "offset": 0.0, "row_pad": 0},
        # odd sizes in fp32, rows whose mean is far from 0, no bias
        {"name": "norm 4097x1001", "op": "norm", "rows": 4097, "hidden": 1001, "dtype": "fp32", "weight": "fp32",
         "bias": False, "offset": 8.0, "row_pad": 0},
        # training: 8192 tokens at a hidden size of 7168, weights in fp32
        {"name": "norm 8192x7168", "op": "norm", "rows": 8192, "hidden": 7168, "dtype": "bf16", "weight": "fp32",
         "bias": True, "offset": 0.0, "row_pad": 0},
        # the largest: a batch of 131072 tokens at a hidden size of 8192
        {"name": "norm 131072x8192", "op": "norm", "rows": 131072, "hidden": 8192, "dtype": "bf16", "weight": "bf16",
         "bias": True, "offset": 0.0, "row_pad": 0},
        # the gradient of a small model's norm
        {"name": "norm backward 512x256", "op": "norm backward", "rows": 512, "hidden": 256, "dtype": "bf16",
         "weight": "fp32", "bias": True, "offset": 0.0, "row_pad": 0},
        # odd sizes in fp32
        {"name": "norm backward 4097x1001", "op": "norm backward", "rows": 4097, "hidden": 1001, "dtype": "fp32",
         "weight": "fp32", "bias": False, "offset": 8.0, "row_pad": 0},
        # a GPT-2-like hidden size and a large batch
        {"name": "norm backward 65536x1024", "op": "norm backward", "rows": 65536, "hidden": 1024, "dtype": "bf16",
         "weight": "fp32", "bias": True, "offset": 0.0, "row_pad": 0},
        # training: 8192 tokens at a hidden size of 7168
        {"name": "norm backward 8192x7168", "op": "norm backward", "rows": 8192, "hidden": 7168, "dtype": "bf16",
         "weight": "fp32", "bias": True, "offset": 0.0, "row_pad": 0},
        # the norms of a small model of 13 layers: 26 vectors, where latency counts
        {"name": "adamw 26x256", "op": "adamw", "bits": 32, "tensors": "26*256", "dtype": "fp32", "grad": "fp32",
         "copy": False, "shift": 0},
        # GPT-2-like: the embedding, the positions and the norms of 24 layers, fp32 masters with
        # bf16 copies for the next forward pass
        {"name": "adamw 50257x1024", "op": "adamw", "bits": 32, "tensors": "1*50257x1024+1*1024x1024+98*1024",
         "dtype": "fp32", "grad": "fp32", "copy": True, "shift": 0},
        # odd sizes, in buckets that start anywhere: bf16 weights without masters, 8-bit states
        {"name": "adamw 8 bits odd", "op": "adamw", "bits": 8, "tensors": "40*1001+3*4097x1001+17*333x77+1*1",
         "dtype": "bf16", "grad": "bf16", "copy": False, "shift": 3},
        # the largest: a table of 129280 x 7168 with 8-bit states
        {"name": "adamw 8 bits 129280x7168", "op": "adamw", "bits": 8, "tensors": "1*129280x7168", "dtype": "fp32",
         "grad": "fp32", "copy": True, "shift": 0},
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm backward", "adamw"])
    dtype = rng.choice(["bf16", "fp32"])
    if op == "adamw":
        bits = rng.choice([8, 32])
        left, groups = _log_uniform(rng, 1000, LARGEST_TABLE if bits == 8 else LARGEST_TABLE // 2), []
        while left > 0 and len(groups) < 8:
            rows, cols = _log_uniform(rng, 1, 65536), _log_uniform(rng, 1, 8192)
            if rng.random() < 0.5 or rows * cols > left:
                rows, cols = 1, min(cols, left)
            times = min(rng.choice([1, 1, 2, 12, 25]), left // (rows * cols))
            groups.append("%d*%s" % (times, "%dx%d" % (rows, cols) if rows > 1 else "%d" % cols))
            left -= times * rows * cols
        return {"op": op, "bits": bits, "tensors": "+".join(groups), "dtype": dtype,
                "grad": rng.choice(["bf16", "fp32"]), "copy": dtype == "fp32" and rng.random() < 0.5,
                "shift": rng.choice([0, 0, 1, 8])}
    hidden = _log_uniform(rng, 8, 8192)
    if rng.random() < 0.5:
        hidden = (hidden + 7) // 8 * 8                  # as most models have it
    elements = LARGEST_ROWS if dtype == "bf16" else LARGEST_ROWS // 2
    if op == "norm backward":
        elements //= 2
    return {"op": op, "rows": _log_uniform(rng, 1, min(131072, elements // hidden)), "hidden": hidden, "dtype": dtype,
            "weight": rng.choice(["bf16", "fp32"]), "bias": rng.random() < 0.5, "offset": rng.choice([0.0, 0.0, 8.0]),
            "row_pad": rng.choice([0, 0, 0, 5, 64])}


def _shapes(case):
    """[(elements, decays)] of the case's tensors, in order: matrices decay, vectors do not."""
    out = []
    for group in case["tensors"].split("+"):
        times, shape = group.split("*")
        out += [(math.prod(int(d) for d in shape.split("x")), "x" in shape)] * int(times)
    return out


def _rows(case, g):
    """Activations: channels of different strength and a few strong ones; rows of a wider buffer
    where row_pad is not 0."""
    n, H = case["rows"], case["hidden"]
    x = torch.empty(n, H + case["row_pad"], dtype=DTYPES[case["dtype"]], device="cuda")[:, :H]
    strength = torch.randn(H, generator=g, device="cuda").mul_(0.3).exp_()
    strength[::97] *= 8
    for at in range(0, n, 16384):                    # in parts, to keep the 32-bit copy small
        part = torch.randn(min(16384, n - at), H, generator=g, device="cuda")
        x[at:at + 16384] = part * strength + case["offset"]
    return x


def _prepare_norm(case, g):
    H = case["hidden"]
    state = {"case": case, "x": _rows(case, g)}
    state["weight"] = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(DTYPES[case["weight"]])
    state["bias"] = (0.1 * torch.randn(H, generator=g, device="cuda")).to(DTYPES[case["weight"]]) if case["bias"] else None
    if case["op"] == "norm backward":
        # what the forward pass left, the gradient that reaches it, and what the steps before left
        # in the main_grads
        state["mean"], state["rstd"] = (torch.cat(part) for part in zip(*(
            _moments(state["x"][at:at + 16384].float())[1:] for at in range(0, case["rows"], 16384))))
        state["grad"] = torch.empty_like(state["x"])
        for at in range(0, case["rows"], 16384):
            state["grad"][at:at + 16384] = torch.randn(min(16384, case["rows"] - at), H, generator=g, device="cuda")
        state["weight_main_grad"] = torch.randn(H, generator=g, device="cuda")
        state["bias_main_grad"] = torch.randn(H, generator=g, device="cuda") if case["bias"] else None
    return state


def _prepare_adamw(case, g):
    """Buckets that hold all tensors one after the other, and the tensors as views of them. With
    8-bit states each tensor begins with a block of its own."""
    shapes, unit = _shapes(case), BLOCK if case["bits"] == 8 else 1
    lengths = [(n + unit - 1) // unit * unit for n, _ in shapes]
    starts = [sum(lengths[:i]) for i in range(len(lengths))] if len(lengths) < 64 else \
        (torch.tensor(lengths).cumsum(0) - torch.tensor(lengths)).tolist()
    N, shift = sum(lengths), case["shift"]

    def bucket(dtype, fill):
        b = torch.zeros(N + shift, dtype=dtype, device="cuda")[shift:]
        for (n, _), at in zip(shapes, starts):
            for k in range(at, at + n, 1 << 27):     # in parts, to keep the 32-bit copy small
                b[k:min(k + (1 << 27), at + n)] = fill(min(1 << 27, at + n - k))
        return b

    def randn(n):
        return torch.randn(n, generator=g, device="cuda")

    # gradients and their averages differ by a factor of ten and more within a block; some
    # elements (of rows that do not occur) have had none so far
    def spread(n):
        return (randn(n) * 1.2).exp_() * 1e-3 * (torch.rand(n, generator=g, device="cuda") > 0.05)

    size = bucket(torch.float32, spread)
    state = {"case": case, "step": FIRST_STEP,
             "param": bucket(DTYPES[case["dtype"]], lambda n: randn(n) * 0.02),
             "grad": torch.zeros(N + shift, dtype=DTYPES[case["grad"]], device="cuda")[shift:],
             "copy": torch.zeros(N + shift, dtype=torch.bfloat16, device="cuda")[shift:] if case["copy"] else None,
             "lengths": torch.tensor(lengths, device="cuda"), "starts": torch.tensor(starts, dtype=torch.int32, device="cuda"),
             "decays": torch.tensor([0.1 if d else 0.0 for _, d in shapes], device="cuda"),
             "grad_scale": torch.rand((), generator=g, device="cuda") * 0.5 + 0.5}
    mean, root = torch.zeros_like(size), size
    for k in range(0, N, 1 << 27):
        part = size[k:k + (1 << 27)]
        state["grad"][k:k + (1 << 27)] = randn(part.numel()) * part
        mean[k:k + (1 << 27)] = randn(part.numel()) * part * 0.25
    if case["bits"] == 32:
        state.update(exp_avg=mean, exp_avg_sq=root.square())
    else:
        codes, scales = [], []
        for x in (mean, root):
            codes.append(torch.empty(N, dtype=torch.float8_e4m3fn, device="cuda"))
            scales.append(torch.empty(N // BLOCK, device="cuda"))
            for k in range(0, N, 1 << 27):
                b = x[k:k + (1 << 27)].view(-1, BLOCK)
                s = b.abs().amax(1) / 448
                codes[-1][k:k + (1 << 27)] = (b / torch.where(s > 0, s, 1.0)[:, None]).clamp_(-448, 448).view(-1).to(torch.float8_e4m3fn)
                scales[-1][k // BLOCK:(k + (1 << 27)) // BLOCK] = s
        state.update(exp_avg=codes[0], exp_avg_sq=codes[1], scales=torch.stack(scales, 1))
    state["views"] = [(at, n, d) for (n, d), at in zip(shapes, starts)]
    return state


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return _prepare_adamw(case, g) if case["op"] == "adamw" else _prepare_norm(case, g)


def _moments(x):
    """Rows less their mean; mean; 1 / standard deviation."""
    mean = x.mean(1)
    d = x - mean[:, None]
    return d, mean, (d.square().mean(1) + EPS_NORM).rsqrt()


def _plain_norm(s):
    d, mean, rstd = _moments(s["x"].float())
    y = d * rstd[:, None] * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return {"out": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _plain_norm_backward(s):
    g = s["grad"].float()
    n = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    u = g * s["weight"].float()
    dx = (u - u.mean(1, keepdim=True) - n * (u * n).mean(1, keepdim=True)) * s["rstd"][:, None]
    s["weight_main_grad"] += (g * n).sum(0)
    out = {"grad_x": dx.to(s["x"].dtype), "weight_main_grad": s["weight_main_grad"]}
    if s["bias"] is not None:
        s["bias_main_grad"] += g.sum(0)
        out["bias_main_grad"] = s["bias_main_grad"]
    return out


def _signed(k):
    """k mod 2^32 as a 32-bit number."""
    return (k + 2 ** 31) % 2 ** 32 - 2 ** 31


def _plain_round8(x, i, t, a, b, positive):
    """x in blocks of 256: e4m3 codes and scales. A value between two levels goes to the upper one
    where its place between them and a threshold add up to 1 or more; thresholds are
    frac(i A + t B) to 20 bits, for element i in step t, A and B the first two powers of
    the plastic number's inverse (for the root the other way round)."""
    biggest = x.abs().amax(1, keepdim=True)
    scale = biggest * (1 / 448)
    held = ~(scale < 2.0 ** -120)
    inverse = torch.where(held, 1 / scale, 0.0)
    # times 2^-120, e4m3's exponents and its steps below the smallest one are fp32's own
    bits = (x * inverse * 2.0 ** -120).view(torch.int32)
    threshold = ((i * _signed(a) + _signed(t * b)) >> 12) & 0xfffff
    code = (((bits & 0x7fffffff) + threshold) >> 20).clamp_(max=126)
    if positive:
        code = torch.where((code == 0) & (x > 0) & held, 1, code)    # a root is not rounded to 0
    code = (code + (bits < 0) * 128).to(torch.uint8)
    return code.view(torch.float8_e4m3fn), torch.where(held, scale, 0.0)


def _plain_adamw(s):
    case = s["case"]
    s["step"] += 1
    N, t, (b1, b2) = s["param"].numel(), s["step"], BETAS
    g = s["grad"].float() * s["grad_scale"]
    p = s["param"].float()
    if case["bits"] == 32:
        m, v = s["exp_avg"], s["exp_avg_sq"]
    else:
        m = (s["exp_avg"].float().view(-1, BLOCK) * s["scales"][:, :1]).view(-1)
        v = (s["exp_avg_sq"].float().view(-1, BLOCK) * s["scales"][:, 1:]).view(-1).square()
    m = m * b1 + g * (1 - b1)
    v = v * b2 + g * g * (1 - b2)
    root = v.sqrt()
    step = m * (LR / (1 - b1 ** t)) / (root * (1 / math.sqrt(1 - b2 ** t)) + EPS_ADAM)
    decay = torch.repeat_interleave(s["decays"], s["lengths"], output_size=N)
    p = p * (1 - LR * decay) - step
    s["param"].copy_(p)
    out = {"param": s["param"], "exp_avg": s["exp_avg"], "exp_avg_sq": s["exp_avg_sq"]}
    if case["copy"]:
        s["copy"].copy_(p)
        out["copy"] = s["copy"]
    if case["bits"] == 32:
        s["exp_avg"].copy_(m)
        s["exp_avg_sq"].copy_(v)
        return out
    i = torch.arange(N, dtype=torch.int32, device=p.device) - torch.repeat_interleave(s["starts"], s["lengths"], output_size=N)
    i = i.view(-1, BLOCK)
    m, scale_m = _plain_round8(m.view(-1, BLOCK), i, t, 0xC13FA9A9, 0x91E10DA5, False)
    root, scale_r = _plain_round8(root.view(-1, BLOCK), i, t, 0x91E10DA5, 0xC13FA9A9, True)
    s["exp_avg"].copy_(m.view(-1))
    s["exp_avg_sq"].copy_(root.view(-1))
    s["scales"][:, :1] = scale_m
    s["scales"][:, 1:] = scale_r
    return {**out, "scales": s["scales"]}


def _adamw_plan(s):
    """What a training program makes once: the tensors, their main_grads and their states."""
    import embedding_weight_grad_gb300 as ewg

    def views(b):
        return None if b is None else [b[at:at + n] for at, n, _ in s["views"]]

    states = {"exp_avg": views(s["exp_avg"]), "exp_avg_sq": views(s["exp_avg_sq"])}
    if s["case"]["bits"] == 8:
        states["scales"] = [s["scales"][at // BLOCK:(at + n + BLOCK - 1) // BLOCK] for at, n, _ in s["views"]]
    return ewg.adamw_plan(views(s["param"]), views(s["grad"]), state_bits=s["case"]["bits"], copies=views(s["copy"]),
                          weight_decay=[0.1 if d else 0.0 for _, _, d in s["views"]], **states)


def run(state):
    case = state["case"]
    if own:
        import embedding_weight_grad_gb300 as ewg

        if case["op"] == "norm":
            r = ewg.layer_norm(state["x"], state["weight"], state["bias"], eps=EPS_NORM)
            return {"out": r.out, "mean": r.mean, "rstd": r.rstd}
        if case["op"] == "norm backward":
            out = {"grad_x": ewg.layer_norm_backward(
                state["grad"], state["x"], state["mean"], state["rstd"], state["weight"],
                weight_main_grad=state["weight_main_grad"], bias_main_grad=state["bias_main_grad"]),
                "weight_main_grad": state["weight_main_grad"]}
            if state["bias"] is not None:
                out["bias_main_grad"] = state["bias_main_grad"]
            return out
        if "plan" not in state:
            state["plan"] = _adamw_plan(state)
        state["step"] += 1
        ewg.adamw_step(state["plan"], state["step"], lr=LR, betas=BETAS, eps=EPS_ADAM, grad_scale=state["grad_scale"])
        return {k: state[k] for k in ("param", "copy", "exp_avg", "exp_avg_sq", "scales") if state.get(k) is not None}
    if case["op"] == "norm":
        return _plain_norm(state)
    if case["op"] == "norm backward":
        return _plain_norm_backward(state)
    return _plain_adamw(state)


def work(case):
    size = {"bf16": 2, "fp32": 4}
    if case["op"] == "adamw":
        shapes = _shapes(case)
        N, blocks = sum(n for n, _ in shapes), sum((n + BLOCK - 1) // BLOCK for n, _ in shapes)
        state = 16 * N if case["bits"] == 32 else 4 * N + 16 * blocks
        return {"bytes": N * (2 * size[case["dtype"]] + size[case["grad"]] + 2 * case["copy"]) + state, "flops": 16 * N}
    n, H, es = case["rows"], case["hidden"], size[case["dtype"]]
    vectors = 2 if case["bias"] else 1
    if case["op"] == "norm":
        return {"bytes": 2 * n * H * es + vectors * H * size[case["weight"]] + 8 * n, "flops": 8 * n * H}
    # the weight is read; the main_grads are read and written
    return {"bytes": 3 * n * H * es + H * size[case["weight"]] + vectors * 8 * H + 8 * n, "flops": 14 * n * H}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(case, s)
    w = s["weight"].double()
    parts = range(0, case["rows"], 16384)
    if case["op"] == "norm":
        outs = []
        for at in parts:
            x = s["x"][at:at + 16384].double()
            var, mean = torch.var_mean(x, dim=1, correction=0)
            rstd = 1 / torch.sqrt(var + EPS_NORM)
            y = (x - mean.unsqueeze(1)).mul_(rstd.unsqueeze(1)).mul_(w)
            if case["bias"]:
                y += s["bias"].double()
            outs.append((y if case["dtype"] == "fp32" else y.float(), mean, rstd))
        return {k: torch.cat([o[j] for o in outs]) for j, k in enumerate(("out", "mean", "rstd"))}
    H = case["hidden"]
    dw, db, dx = torch.zeros_like(w), torch.zeros_like(w), []
    for at in parts:
        x, g = s["x"][at:at + 16384].double(), s["grad"][at:at + 16384].double()
        rstd = s["rstd"][at:at + 16384].double().unsqueeze(1)
        hat = (x - s["mean"][at:at + 16384].double().unsqueeze(1)).mul_(rstd)
        dw += torch.einsum("nh,nh->h", g, hat)
        db += g.sum(dim=0)
        g *= w
        along = torch.einsum("nh,nh->n", g, hat) / H
        d = rstd * (g - hat.mul_(along.unsqueeze(1)) - (g.sum(dim=1) / H).unsqueeze(1))
        dx.append(d if case["dtype"] == "fp32" else d.float())
    out = {"grad_x": torch.cat(dx), "weight_main_grad": s["weight_main_grad"].double() + dw}
    if case["bias"]:
        out["bias_main_grad"] = s["bias_main_grad"].double() + db
    return out


def _exact_adamw(case, s):
    """One tensor, and 2^26 elements of it, after the other."""
    (b1, b2), t, bits = BETAS, s["step"] + 1, case["bits"]
    scale = float(s["grad_scale"])
    kept = torch.float64 if s["param"].numel() < 1 << 28 else torch.float32
    out = {"param": torch.zeros_like(s["param"], dtype=kept), "exp_avg": torch.zeros_like(s["exp_avg"], dtype=kept),
           "exp_avg_sq": torch.zeros_like(s["exp_avg_sq"], dtype=kept)}
    if bits == 8:
        out["scales"] = torch.zeros_like(s["scales"], dtype=torch.float64)
    part = 1 << 26
    for at, n, decays in s["views"]:
        for lo in range(at, at + n, part):
            here = slice(lo, min(lo + part, at + n))
            count = here.stop - here.start
            grad = s["grad"][here].double() * scale
            mean, sq = s["exp_avg"][here].double(), s["exp_avg_sq"][here].double()
            if bits == 8:
                blocks = slice(here.start // BLOCK, (here.stop + BLOCK - 1) // BLOCK)
                each = s["scales"][blocks].double().repeat_interleave(BLOCK, 0)[:count]
                mean, sq = mean * each[:, 0], (sq * each[:, 1]) ** 2
            mean = torch.lerp(grad, mean, b1)
            sq = torch.lerp(grad * grad, sq, b2)
            w = s["param"][here].double()
            hat = mean / (1 - b1 ** t) / (torch.sqrt(sq / (1 - b2 ** t)) + EPS_ADAM)
            out["param"][here] = w - LR * ((0.1 if decays else 0.0) * w + hat)
            if bits == 32:
                out["exp_avg"][here], out["exp_avg_sq"][here] = mean, sq
                continue
            index = torch.arange(here.start - at, here.stop - at, device=w.device)
            for j, (key, x) in enumerate((("exp_avg", mean), ("exp_avg_sq", sq.sqrt()))):
                whole = torch.nn.functional.pad(x, (0, -count % BLOCK)).view(-1, BLOCK)
                unit = whole.abs().max(dim=1).values / 448
                out["scales"][blocks, j] = unit
                y = (x / unit.repeat_interleave(BLOCK)[:count]).nan_to_num(0.0)
                k = (0xC13FA9A9, 0x91E10DA5)
                late = torch.remainder(index * k[j] + t * k[1 - j], 2 ** 32).div(4096, rounding_mode="floor") / 2 ** 20
                step = torch.ldexp(torch.ones_like(y), (torch.frexp(y).exponent - 1).clamp(min=-6) - 3)
                level = torch.floor(y.abs() / step + late) * step
                if j:
                    level = torch.where(y > 0, level.clamp(min=2.0 ** -9), level)
                out[key][here] = level.clamp(max=448) * y.sign()
    if case["copy"]:
        out["copy"] = out["param"]
    return out
