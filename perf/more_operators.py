"""Cases of the operators around a block and behind the last one: the dense
layer whose bias, activation and residual are part of its product, the norms
before and after a block joined with its gate and residual scale, and the log
probabilities of given tokens with entropy and top alternatives; each forward
and backward.

Every operator is given here in a plain form (fp32 torch operations, rounded
once), as the call of this package (``own``), and in 64 bits from its
definition (``exact``).
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-5

# what the largest listed cases multiply, and hold in a row-major matrix
MOST_MACS = 16384 * 2048 * 8192
MOST_ELEMENTS = {"norms": 16384 * 4096, "norms_grad": 16384 * 4096, "logprobs": 4096 * 128000,
                 "logprobs_grad": 4096 * 128000}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token through an output projection, back onto the residual stream
        {"name": "linear_one_token", "op": "linear", "rows": 1, "k": 4096, "n": 4096, "dtype": "bf16", "act": "none",
         "bias": True, "residual": True, "keep": False},
        # the up projection of training or of long prompts; the pre-activation is kept for the gradient
        {"name": "linear_training", "op": "linear", "rows": 16384, "k": 2048, "n": 8192, "dtype": "bf16",
         "act": "gelu_tanh", "bias": True, "residual": False, "keep": True},
        # a small ragged batch, sizes that are no multiple of a tile, fp16
        {"name": "linear_grad_odd", "op": "linear_grad", "rows": 333, "k": 1000, "n": 2056, "dtype": "fp16",
         "act": "silu", "bias": True},
        # the gradients of a layer in training: of its input, weights and bias through the activation
        {"name": "linear_grad_training", "op": "linear_grad", "rows": 8192, "k": 2048, "n": 8192, "dtype": "bf16",
         "act": "gelu_tanh", "bias": True},
        # one token between two blocks of a decode step
        {"name": "norms_one_token", "op": "norms", "rows": 1, "n": 4096, "dtype": "bf16", "post": "rms", "pre": "rms",
         "gates": 1, "shift": False},
        # the prompts of eight samples, each with a gate of its own
        {"name": "norms_prompts", "op": "norms", "rows": 16384, "n": 4096, "dtype": "bf16", "post": "rms",
         "pre": "rms", "gates": 8, "shift": False},
        # a ragged batch of odd width with a gate for every token, fp32
        {"name": "norms_grad_odd", "op": "norms_grad", "rows": 1003, "n": 1111, "dtype": "fp32", "post": "none",
         "pre": "layer", "gates": 1003, "shift": True},
        # a training step's gradients between two blocks, eight samples
        {"name": "norms_grad_training", "op": "norms_grad", "rows": 16384, "n": 4096, "dtype": "bf16", "post": "rms",
         "pre": "rms", "gates": 8, "shift": False},
        # a decode step of sixteen requests under a grammar that forbids part of an odd vocabulary; fp32 logits
        {"name": "logprobs_decode", "op": "logprobs", "rows": 16, "v": 50257, "pad": 0, "dtype": "fp32", "top": 20,
         "masked": True, "scale": 1.25},
        # scoring of prompts over a large vocabulary
        {"name": "logprobs_scoring", "op": "logprobs", "rows": 4096, "v": 128000, "pad": 0, "dtype": "bf16", "top": 8,
         "masked": False, "scale": 1.0},
        # a small step over an odd vocabulary in padded rows
        {"name": "logprobs_grad_odd", "op": "logprobs_grad", "rows": 96, "v": 32003, "pad": 61, "dtype": "fp16",
         "masked": True, "scale": 0.8},
        # the gradient of a large step's loss with an entropy bonus
        {"name": "logprobs_grad_training", "op": "logprobs_grad", "rows": 4096, "v": 128000, "pad": 0,
         "dtype": "bf16", "masked": False, "scale": 1.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["linear", "linear_grad", "norms", "norms_grad", "logprobs", "logprobs_grad"])
        if op.startswith("linear"):
            c = {"op": op, "rows": _log(rng, 1, 16384), "k": 8 * _log(rng, 8, 1024), "n": 8 * _log(rng, 8, 1024),
                 "dtype": rng.choice(["bf16", "bf16", "fp16"]), "act": rng.choice(["none", "gelu_tanh", "silu", "relu"]),
                 "bias": rng.random() < 0.7}
            macs = c["rows"] * c["k"] * c["n"] * (2 if op == "linear_grad" else 1)
            if op == "linear":
                c.update(residual=rng.random() < 0.5, keep=c["act"] != "none" and rng.random() < 0.5)
            if macs <= MOST_MACS:
                return c
        elif op.startswith("norms"):
            rows, n = _log(rng, 1, 16384), _log(rng, 64, 16384)
            n = n if rng.random() < 0.4 else max(8, n // 8 * 8)
            divisors = [d for d in range(1, rows + 1) if rows % d == 0]
            c = {"op": op, "rows": rows, "n": n, "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                 "post": rng.choice(["none", "rms", "layer"]), "pre": rng.choice(["rms", "layer"]),
                 "gates": rng.choice([0, 1, rows, rng.choice(divisors)]), "shift": rng.random() < 0.4}
            size = 2 if c["dtype"] == "fp32" else 1
            if size * rows * n <= MOST_ELEMENTS[op]:
                return c
        else:
            c = {"op": op, "rows": _log(rng, 1, 4096), "v": _log(rng, 1000, 200000),
                 "pad": rng.choice([0, 0, rng.randrange(1, 130)]), "dtype": rng.choice(["bf16", "fp16", "fp32"]),
                 "masked": rng.random() < 0.4, "scale": rng.choice([1.0, 0.7, 1.25])}
            if op == "logprobs":
                c["top"] = rng.choice([0, 1, 5, 20, rng.randint(1, 32)])
            size = 2 if c["dtype"] == "fp32" else 1
            if size * c["rows"] * (c["v"] + c["pad"]) <= MOST_ELEMENTS[op]:
                return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    rows = case["rows"]

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        t = torch.randn(*shape, generator=gen, device="cuda")
        return t.mul_(std).add_(mean).to(dtype)

    s = {"case": case}
    if case["op"].startswith("linear"):
        k, n = case["k"], case["n"]
        s["x"] = normal(rows, k)
        s["w"] = normal(k, n, std=k ** -0.5)
        s["bias"] = normal(n, std=0.1, dtype=torch.float32) if case["bias"] else None
        if case["op"] == "linear":
            s["residual"] = normal(rows, n) if case["residual"] else None
            s["z"] = torch.empty(rows, n, dtype=dt, device="cuda") if case["keep"] else None
        else:
            s["z"] = normal(rows, n) if case["act"] != "none" else None
            s["dy"] = normal(rows, n, std=rows ** -0.5)
        return s
    if case["op"].startswith("norms"):
        n = case["n"]
        s["h"] = normal(rows, n, std=0.7, mean=0.1)
        s["x"] = normal(rows, n, std=1.5)
        shift = case["shift"]
        s["post_weight"] = normal(n, std=0.1, mean=1.0, dtype=torch.float32) if case["post"] != "none" else None
        s["post_bias"] = normal(n, std=0.1, dtype=torch.float32) if case["post"] != "none" and shift else None
        s["pre_weight"] = normal(n, std=0.1, mean=1.0, dtype=torch.float32)
        s["pre_bias"] = normal(n, std=0.1, dtype=torch.float32) if shift else None
        s["gate"] = normal(case["gates"], n, std=0.5, mean=0.5) if case["gates"] else None
        s["scale"], s["alpha"] = 0.5, 1.0
        if case["op"] == "norms_grad":  # the forward pass's stream is at hand
            s["x_out"] = _norms(s)[0]
            del s["x"]
            s["dy"] = normal(rows, n)
            s["dx_out"] = normal(rows, n)
        return s
    v, pad = case["v"], case["pad"]
    logits = normal(rows, v + pad, std=2.5)
    if case["masked"]:  # tokens that the request may not choose
        forbidden = torch.rand(rows, v + pad, generator=gen, device="cuda") < 0.3
        logits.masked_fill_(forbidden, float("-inf"))
        del forbidden
    s["logits"] = logits[:, :v]
    s["targets"] = torch.randint(0, v, (rows,), generator=gen, device="cuda")
    if case["masked"]:  # a given token is an allowed one; some rows have none
        at = torch.arange(rows, device="cuda")
        s["logits"][at, s["targets"]] = normal(rows)
        s["targets"][torch.rand(rows, generator=gen, device="cuda") < 0.1] = -1
    if case["op"] == "logprobs_grad":
        _, s["lse"], s["entropy"] = _logprobs(s, 0)
        s["dlogprob"] = normal(rows, std=1.0 / rows, mean=-1.0 / rows, dtype=torch.float32)
        s["dentropy"] = normal(rows, std=0.1 / rows, dtype=torch.float32)
        s["out"] = torch.empty(rows, v + pad, dtype=dt, device="cuda")[:, :v]
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state)
    if op == "logprobs":
        return _logprobs(state, state["case"]["top"])
    return {"linear": _linear, "linear_grad": _linear_grad, "norms": _norms, "norms_grad": _norms_grad,
            "logprobs_grad": _logprobs_grad}[op](state)


def _workspace(state, size):
    from memory_fusion_gb300 import cf
    if "workspace" not in state:  # kept by the caller, as for the other calls of the package
        state["workspace"] = cf.new_workspace(size)
    return state["workspace"]


def _own(s):
    from memory_fusion_gb300 import cf
    c = s["case"]
    if c["op"].startswith("linear"):
        ws = _workspace(s, cf.cf_gemm_linear_workspace_size(c["rows"], c["n"], c["k"]))
        if c["op"] == "linear":
            y = cf.gemm_linear(s["x"], s["w"], s["bias"], act=c["act"], residual=s["residual"], preact=s["z"],
                               workspace=ws)
            return [y] if s["z"] is None else [y, s["z"]]
        dx, dw, db = cf.gemm_linear_grad(s["dy"], s["x"], s["w"], act=c["act"], preact=s["z"], bias=c["bias"],
                                         workspace=ws)
        return [dx, dw] if db is None else [dx, dw, db]
    if c["op"].startswith("norms"):
        kw = dict(post=c["post"], post_weight=s["post_weight"], post_bias=s["post_bias"], pre=c["pre"],
                  pre_weight=s["pre_weight"], pre_bias=s["pre_bias"], gate=s["gate"], scale=s["scale"],
                  alpha=s["alpha"], eps=EPS)
        if c["op"] == "norms":
            ws = _workspace(s, cf.cf_stitch_workspace_size(c["rows"], c["n"]))
            return list(cf.stitch_block_norms(s["h"], s["x"], workspace=ws, **kw))
        ws = _workspace(s, cf.cf_stitch_block_norms_grad_workspace_size(c["rows"], c["n"]))
        g = cf.stitch_block_norms_grad(s["dy"], s["dx_out"], s["h"], s["x_out"], workspace=ws, **kw)
        return [t for t in g if t is not None]
    ws = _workspace(s, cf.cf_stitch_workspace_size(c["rows"], c["v"]))
    if c["op"] == "logprobs":
        got = cf.stitch_logprobs(s["logits"], s["targets"], scale=c["scale"], top=c["top"], entropy=True, workspace=ws)
        return [t for t in got if t is not None]
    return [cf.stitch_logprobs_grad(s["logits"], s["targets"], s["lse"], s["dlogprob"], entropy=s["entropy"],
                                    dentropy=s["dentropy"], scale=c["scale"], out=s["out"], workspace=ws)]


def _act(name, z):
    if name == "gelu_tanh":
        return z / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    return z * (z > 0) if name == "relu" else z


def _act_slope(name, z):
    if name == "gelu_tanh":
        p = 1.0 / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
        return p + 2.0 * z * p * (1.0 - p) * math.sqrt(2.0 / math.pi) * (1.0 + 3.0 * 0.044715 * z * z)
    if name == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p + z * p * (1.0 - p)
    return (z > 0).to(z.dtype)


def _linear(s):
    c, dt = s["case"], s["x"].dtype
    z = s["x"].float() @ s["w"].float()
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _act(c["act"], z)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    if s["z"] is None:
        return [y.to(dt)]
    s["z"].copy_(z)
    return [y.to(dt), s["z"]]


def _linear_grad(s):
    c, dt = s["case"], s["x"].dtype
    dz = s["dy"].float()
    if s["z"] is not None:
        dz = dz * _act_slope(c["act"], s["z"].float())
    out = [(dz @ s["w"].float().t()).to(dt), (s["x"].float().t() @ dz).to(dt)]
    return out + [dz.sum(0)] if c["bias"] else out


def _spread(kind, t):
    """What a norm subtracts from the values of each row, and divides them by."""
    if kind == "none":
        return 0.0, 1.0
    if kind == "rms":
        return 0.0, torch.sqrt((t * t).mean(1, keepdim=True) + EPS)
    mean = t.mean(1, keepdim=True)
    return mean, torch.sqrt(((t - mean) ** 2).mean(1, keepdim=True) + EPS)


def _normalised(kind, t, weight, bias):
    mean, root = _spread(kind, t)
    t = (t - mean) / root
    t = t if weight is None else t * weight
    return t if bias is None else t + bias


def _of_rows(gate, rows):
    """The gate of each row: the rows of a sample share one."""
    return gate.float().repeat_interleave(rows // gate.shape[0], 0)


def _norms(s):
    c, dt = s["case"], s["h"].dtype
    p = _normalised(c["post"], s["h"].float(), s["post_weight"], s["post_bias"]) * s["scale"]
    if s["gate"] is not None:
        p = p * _of_rows(s["gate"], c["rows"])
    x = s["alpha"] * s["x"].float() + p
    return [x.to(dt), _normalised(c["pre"], x, s["pre_weight"], s["pre_bias"]).to(dt)]


def _norm_grad(kind, hat, root, g):
    """The gradient of a norm's input, of the gradient of its normalised values."""
    if kind == "none":
        return g
    d = g - hat * (g * hat).mean(1, keepdim=True)
    if kind == "layer":
        d = d - g.mean(1, keepdim=True)
    return d / root


def _norms_grad(s):
    c, dt = s["case"], s["h"].dtype
    h, x, dy = s["h"].float(), s["x_out"].float(), s["dy"].float()
    mean, root = _spread(c["pre"], x)
    hat = (x - mean) / root
    grads = [(dy * hat).sum(0)] + ([dy.sum(0)] if s["pre_bias"] is not None else [])
    dx = s["dx_out"].float() + _norm_grad(c["pre"], hat, root, dy * s["pre_weight"])
    mean, root = _spread(c["post"], h)
    hat = (h - mean) / root
    dp, dgate = dx * s["scale"], []
    if s["gate"] is not None:
        p = hat if s["post_weight"] is None else hat * s["post_weight"]
        p = p if s["post_bias"] is None else p + s["post_bias"]
        dgate = [(dp * p).view(c["gates"], -1, c["n"]).sum(1).to(dt)]
        dp = dp * _of_rows(s["gate"], c["rows"])
    posts = [] if s["post_weight"] is None else [(dp * hat).sum(0)]
    posts += [] if s["post_bias"] is None else [dp.sum(0)]
    dh = _norm_grad(c["post"], hat, root, dp if s["post_weight"] is None else dp * s["post_weight"])
    return [dh.to(dt), (s["alpha"] * dx).to(dt)] + dgate + posts + grads


def _logprobs(s, top):
    z = s["logits"].float()
    order = None
    if top > 0:  # by value, equal ones by index: a key of both
        bits = (z + 0.0).view(torch.int32)
        key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).to(torch.int64) << 32
        key -= torch.arange(z.shape[1], device=z.device)
        order = (-key.topk(top, 1).values) & 0xFFFFFFFF
        del bits, key
    z = z * s["case"]["scale"]
    z = z - (high := z.amax(1, keepdim=True))
    e = torch.exp(z)
    total = e.sum(1)
    log_total = torch.log(total)
    entropy = log_total - (e * torch.where(e > 0, z, torch.zeros_like(z))).sum(1) / total
    given = z.gather(1, s["targets"].clamp(min=0)[:, None])[:, 0]
    logprob = torch.where(s["targets"] < 0, torch.zeros_like(given), given - log_total)
    out = [logprob, log_total + high[:, 0], entropy]
    if top > 0:
        out += [z.gather(1, order) - log_total[:, None], order]
    return out


def _logprobs_grad(s):
    z = s["logits"].float() * s["case"]["scale"] - s["lse"][:, None]
    p = torch.exp(z)
    dlogprob = torch.where(s["targets"] < 0, torch.zeros_like(s["dlogprob"]), s["dlogprob"])
    finite = torch.where(p > 0, z, torch.zeros_like(z))
    d = -p * (dlogprob[:, None] + s["dentropy"][:, None] * (finite + s["entropy"][:, None]))
    at = torch.arange(z.shape[0], device=z.device)
    d[at, s["targets"].clamp(min=0)] += dlogprob
    s["out"].copy_(d * s["case"]["scale"])
    return [s["out"]]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    rows = case["rows"]
    if case["op"].startswith("linear"):
        k, n = case["k"], case["n"]
        acted = case["act"] != "none"
        if case["op"] == "linear":
            more = rows * n * (int(case["residual"]) + int(case["keep"]))
            return {"bytes": size * (rows * (k + n) + k * n + more) + (4 * n if case["bias"] else 0),
                    "flops": 2 * rows * k * n}
        return {"bytes": 2 * size * (rows * k + k * n) + size * rows * n * (2 if acted else 1) +
                (4 * n if case["bias"] else 0), "flops": 4 * rows * k * n}
    if case["op"].startswith("norms"):
        n = case["n"]
        vectors = 4 * n * ((case["post"] != "none") * (1 + case["shift"]) + 1 + case["shift"])
        if case["op"] == "norms":
            return {"bytes": size * n * (4 * rows + case["gates"]) + vectors, "flops": 12 * rows * n}
        return {"bytes": size * n * (6 * rows + 2 * case["gates"]) + 2 * vectors, "flops": 30 * rows * n}
    cells = rows * case["v"]
    if case["op"] == "logprobs":
        return {"bytes": size * cells + rows * (20 + 12 * case["top"]), "flops": 6 * cells}
    return {"bytes": 2 * size * cells + 24 * rows, "flops": 7 * cells}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)

    def f64(t):
        return None if t is None else t.to(torch.float64)

    op, rows = case["op"], case["rows"]
    root = math.sqrt(2.0 / math.pi)

    def activated(z):
        if case["act"] == "gelu_tanh":
            return 0.5 * z * (1.0 + torch.tanh(root * (z + 0.044715 * z ** 3)))
        if case["act"] == "silu":
            return z * torch.sigmoid(z)
        return torch.clamp(z, min=0.0) if case["act"] == "relu" else z

    if op == "linear":
        z = f64(s["x"]) @ f64(s["w"])
        if s["bias"] is not None:
            z += f64(s["bias"])
        y = activated(z)
        if s["residual"] is not None:
            y = y + f64(s["residual"])
        return [y, z] if case["keep"] else [y]
    if op == "linear_grad":
        dz = f64(s["dy"])
        if s["z"] is not None:
            z = f64(s["z"])
            if case["act"] == "gelu_tanh":
                t = torch.tanh(root * (z + 0.044715 * z ** 3))
                slope = 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * root * (1.0 + 0.134145 * z * z)
            elif case["act"] == "silu":
                t = torch.sigmoid(z)
                slope = t * (1.0 + z * (1.0 - t))
            else:
                slope = torch.where(z > 0, torch.ones_like(z), torch.zeros_like(z))
            dz = dz * slope
        out = [dz @ f64(s["w"]).T, f64(s["x"]).T @ dz]
        return out + [dz.sum(0)] if case["bias"] else out

    if op.startswith("norms"):
        def norm(kind, t, weight, bias):
            if kind == "layer":
                t = t - t.mean(1, keepdim=True)
            if kind != "none":
                t = t * torch.rsqrt(t.square().mean(1, keepdim=True) + EPS)
            if weight is not None:
                t = t * weight
            return t if bias is None else t + bias

        n, samples = case["n"], case["gates"]
        names = ["post_weight", "post_bias", "pre_weight", "pre_bias"]
        vec = {k: f64(s[k]) for k in names}
        gate, h = f64(s["gate"]), f64(s["h"])

        def branch(h, gate, vec):
            p = norm(case["post"], h, vec["post_weight"], vec["post_bias"]) * s["scale"]
            return p if gate is None else (p.view(samples, -1, n) * gate[:, None, :]).view(rows, n)

        if op == "norms":
            x = s["alpha"] * f64(s["x"]) + branch(h, gate, vec)
            return [x, norm(case["pre"], x, vec["pre_weight"], vec["pre_bias"])]
        # by automatic differentiation, with the given stream as the second norm's input
        x = f64(s["x_out"]).requires_grad_()
        y = norm(case["pre"], x, vec["pre_weight"].requires_grad_(),
                 None if vec["pre_bias"] is None else vec["pre_bias"].requires_grad_())
        pres = [vec[k] for k in names[2:] if vec[k] is not None]
        dx, *dpres = torch.autograd.grad(y, [x] + pres, f64(s["dy"]))
        dx = dx + f64(s["dx_out"])
        leaves = [h] + ([] if gate is None else [gate]) + [vec[k] for k in names[:2] if vec[k] is not None]
        for t in leaves:
            t.requires_grad_()
        dh, *rest = torch.autograd.grad(branch(h, gate, vec), leaves, dx)
        return [dh, s["alpha"] * dx] + rest + list(dpres)

    # row by row block: a large vocabulary in 64 bits
    parts = []
    step = max(1, (1 << 27) // case["v"])
    for lo in range(0, rows, step):
        raw = f64(s["logits"][lo:lo + step])
        z = raw * case["scale"]
        logp = torch.log_softmax(z, 1)
        targets = s["targets"][lo:lo + step]
        none = targets < 0
        at = torch.arange(z.shape[0], device=z.device)
        if op == "logprobs":
            logprob = logp[at, targets.clamp(min=0)]
            logprob[none] = 0.0
            part = [logprob, torch.logsumexp(z, 1), -torch.xlogy(p := logp.exp(), p).sum(1)]
            if case["top"] > 0:
                order = raw.sort(dim=1, descending=True, stable=True).indices[:, :case["top"]]
                part += [logp.gather(1, order), order]
        else:
            p = torch.exp(z - f64(s["lse"][lo:lo + step, None]))
            dl = f64(s["dlogprob"][lo:lo + step]).masked_fill(none, 0.0)
            d = -p * dl[:, None]
            d[at, targets.clamp(min=0)] += dl
            d -= f64(s["dentropy"][lo:lo + step, None]) * (torch.xlogy(p, p) + p * f64(s["entropy"][lo:lo + step, None]))
            part = [d * case["scale"]]
        parts.append(part)
    return [torch.cat(column) for column in zip(*parts)]
