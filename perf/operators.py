"""Cases of the products whose rows choose their weights: the expert-grouped
GEMM in its three directions (forward with a fused GELU, gradient of the
input, gradient of the weights) and the low-rank adapters of many requests
beside a shared projection.

Every operator is given here in a plain form (fp32 torch products over
padded groups, rounded once), as the call of this package (``own``), and in
64 bits from its definition (``exact``).
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}

# the largest listed product: rows * K * N, and the bytes a drawn case may hold
MOST_MACS = 16384 * 2048 * 8192
MOST_BYTES = 1 << 30


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token with two of eight experts, the up projection of a decode step
        {"name": "up_one_token", "op": "forward", "rows": 2, "behind": 0, "groups": 8, "k": 1024, "n": 2048,
         "dtype": "bf16", "act": "gelu_tanh", "keep": False, "split": 1},
        # a decode batch over 32 experts: every group is a handful of rows, the weights are the work
        {"name": "up_decode_batch", "op": "forward", "rows": 250, "behind": 6, "groups": 32, "k": 2048, "n": 4096,
         "dtype": "bf16", "act": "gelu_tanh", "keep": False, "split": 2},
        # many small experts, sizes that are no multiple of a tile, fp16
        {"name": "up_many_experts_odd", "op": "forward", "rows": 4099, "behind": 0, "groups": 64, "k": 1000,
         "n": 2056, "dtype": "fp16", "act": "none", "keep": False, "split": 3},
        # prefill or training forward over eight large experts; the pre-activation is kept for the gradient
        {"name": "up_training", "op": "forward", "rows": 16384, "behind": 0, "groups": 8, "k": 2048, "n": 8192,
         "dtype": "bf16", "act": "gelu_tanh", "keep": True, "split": 4},
        # the gradient of the down projection's input, through the activation
        {"name": "input_grad_training", "op": "input_grad", "rows": 16384, "behind": 0, "groups": 16, "k": 4096,
         "n": 2048, "dtype": "bf16", "act": "gelu_tanh", "keep": False, "split": 5},
        # a small ragged batch with empty groups
        {"name": "input_grad_odd", "op": "input_grad", "rows": 333, "behind": 19, "groups": 12, "k": 1032, "n": 520,
         "dtype": "fp16", "act": "none", "keep": False, "split": 6},
        # the gradient of the weights of the training case
        {"name": "weight_grad_training", "op": "weight_grad", "rows": 16384, "behind": 0, "groups": 8, "k": 2048,
         "n": 8192, "dtype": "bf16", "act": "none", "keep": False, "split": 4},
        # a small step over many experts: short ragged sums
        {"name": "weight_grad_odd", "op": "weight_grad", "rows": 1003, "behind": 21, "groups": 24, "k": 520, "n": 1032,
         "dtype": "fp16", "act": "none", "keep": False, "split": 7},
        # one request that decodes one token with its adapter
        {"name": "lora_one_token", "op": "lora", "rows": 1, "behind": 0, "groups": 1, "k": 4096, "n": 4096,
         "dtype": "bf16", "rank": 16, "adapters": 4, "bias": False, "split": 8},
        # a decode batch: 64 requests, one row each, 24 adapters among them
        {"name": "lora_decode_batch", "op": "lora", "rows": 64, "behind": 0, "groups": 64, "k": 4096, "n": 4096,
         "dtype": "bf16", "rank": 16, "adapters": 24, "bias": True, "split": 9},
        # decoding rows and a few prompts in one batch, some requests without an adapter
        {"name": "lora_mixed_batch", "op": "lora", "rows": 1537, "behind": 31, "groups": 40, "k": 2048, "n": 2056,
         "dtype": "fp16", "rank": 24, "adapters": 12, "bias": True, "split": 10},
        # prompts of eight requests
        {"name": "lora_prompts", "op": "lora", "rows": 8192, "behind": 0, "groups": 8, "k": 4096, "n": 4096,
         "dtype": "bf16", "rank": 64, "adapters": 8, "bias": False, "split": 11},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["forward", "forward", "input_grad", "weight_grad", "lora", "lora"])
        c = {"op": op, "rows": _log(rng, 1, 16384), "k": 8 * _log(rng, 8, 1024), "n": 8 * _log(rng, 8, 1024),
             "dtype": rng.choice(["bf16", "bf16", "fp16"]), "split": rng.randrange(1 << 20)}
        c["behind"] = rng.choice([0, 0, rng.randrange(1, 40)])
        if op == "lora":
            c["groups"] = min(c["rows"], _log(rng, 1, 128))
            c.update(rank=8 * rng.randint(1, 8), adapters=_log(rng, 1, 64), bias=rng.random() < 0.5)
            held = c["adapters"] * c["rank"] * (c["k"] + c["n"]) + c["k"] * c["n"]
        else:
            c["groups"] = _log(rng, 1, 64)
            c["act"] = "none" if op == "weight_grad" else rng.choice(["none", "gelu_tanh"])
            c["keep"] = op == "forward" and c["act"] != "none" and rng.random() < 0.5
            held = c["groups"] * c["k"] * c["n"]
        held += c["rows"] * (c["k"] + 2 * c["n"])
        if c["rows"] * c["k"] * c["n"] <= MOST_MACS and 2 * held <= MOST_BYTES:
            return c


def _sizes(case):
    """Rows of each group: uneven, some groups empty where there are several; the same for a case always."""
    rng = random.Random(case["split"])
    g, rows = case["groups"], case["rows"]
    if case["op"] == "lora":  # every request has a row at least
        # a serving batch: most requests decode one row, the rest of the rows are prompts
        share = [rng.choice([0.0, 0.0, 1.0]) * rng.uniform(0.5, 1.5) if g > 8 else rng.uniform(0.5, 1.5)
                 for _ in range(g)]
        free, least = rows - g, 1
    else:
        share = [0.0 if g > 4 and rng.random() < 0.1 else rng.uniform(0.5, 1.5) for _ in range(g)]
        free, least = rows, 0
    if sum(share) == 0.0:
        share[rng.randrange(g)] = 1.0
    total = sum(share)
    sizes = [least + int(free * s / total) for s in share]
    left = rows - sum(sizes)
    while left > 0:
        i = rng.randrange(g)
        if share[i] > 0.0:
            sizes[i] += 1
            left -= 1
    return sizes


def _adapters(case):
    """The adapter of each request, -1 for none."""
    rng = random.Random(case["split"] + 1)
    return [-1 if case["groups"] > 4 and rng.random() < 0.15 else rng.randrange(case["adapters"])
            for _ in range(case["groups"])]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    g, k, n = case["groups"], case["k"], case["n"]
    total = case["rows"] + case["behind"]

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    sizes = _sizes(case)
    offsets = torch.tensor([0] + sizes, dtype=torch.int64).cumsum(0)
    # the plain form's plan: row i of group e sits at [e, i] of a padded batch
    group_of = torch.repeat_interleave(torch.arange(g), torch.tensor(sizes))
    within = torch.arange(case["rows"]) - offsets[group_of]
    s = {"case": case, "offsets": offsets.to(torch.int32).cuda(), "group": group_of.cuda(), "within": within.cuda(),
         "longest": max(sizes), "sizes": sizes}
    if case["op"] == "forward":
        s["x"] = normal(total, k)
        s["w"] = normal(g, k, n, std=k ** -0.5)
        s["y"] = torch.zeros(total, n, dtype=dt, device="cuda")
        s["z"] = torch.zeros(total, n, dtype=dt, device="cuda") if case["keep"] else None
    elif case["op"] == "input_grad":
        s["dy"] = normal(total, n)
        s["w"] = normal(g, k, n, std=n ** -0.5)
        s["z"] = normal(total, k) if case["act"] != "none" else None
        s["dx"] = torch.zeros(total, k, dtype=dt, device="cuda")
    elif case["op"] == "weight_grad":
        s["x"] = normal(total, k)
        s["dy"] = normal(total, n, std=total ** -0.5)
        s["dw"] = torch.zeros(g, k, n, dtype=dt, device="cuda")
    else:
        a, r = case["adapters"], case["rank"]
        s["x"] = normal(total, k)
        s["w"] = normal(k, n, std=k ** -0.5)
        s["bias"] = normal(n, std=0.1, dtype=torch.float32) if case["bias"] else None
        s["a"] = normal(a, k, r, std=k ** -0.5)
        s["b"] = normal(a, r, n, std=r ** -0.5)
        s["scale"] = torch.rand(a, generator=gen, device="cuda") + 0.5
        s["request_adapter"] = torch.tensor(_adapters(case), dtype=torch.int32).cuda()
        s["y"] = torch.zeros(total, n, dtype=dt, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    case = state["case"]
    if own:
        return _own(state)
    return {"forward": _forward, "input_grad": _input_grad, "weight_grad": _weight_grad, "lora": _lora}[case["op"]](state)


def _workspace(state, size):
    from memory_fusion_gb300 import cf
    if "workspace" not in state:  # kept by the caller, as for the other calls of the package
        state["workspace"] = cf.new_workspace(size)
    return state["workspace"]


def _own(s):
    from memory_fusion_gb300 import cf
    c = s["case"]
    total = c["rows"] + c["behind"]
    if c["op"] == "lora":
        ws = _workspace(s, cf.cf_gemm_lora_workspace_size(total, c["n"], c["k"], c["groups"], c["rank"]))
        return [cf.gemm_lora(s["x"], s["w"], s["bias"], s["a"], s["b"], s["offsets"], s["request_adapter"],
                             scale=s["scale"], out=s["y"], workspace=ws)]
    ws = _workspace(s, cf.cf_grouped_gemm_workspace_size(total, c["n"], c["k"], c["groups"]))
    if c["op"] == "forward":
        y = cf.grouped_gemm(s["x"], s["w"], s["offsets"], act=c["act"], preact=s["z"], out=s["y"], workspace=ws)
        return [y] if s["z"] is None else [y, s["z"]]
    if c["op"] == "input_grad":
        return [cf.grouped_gemm_dgrad(s["dy"], s["w"], s["offsets"], preact=s["z"], out=s["dx"], workspace=ws)]
    return [cf.grouped_gemm_wgrad(s["x"], s["dy"], s["offsets"], out=s["dw"], workspace=ws)]


def _padded(s, t):
    """The groups' rows of t in fp32, one group a batch entry, zeros behind the shorter ones."""
    out = torch.zeros(len(s["sizes"]), s["longest"], t.shape[1], dtype=torch.float32, device=t.device)
    out[s["group"], s["within"]] = t[: s["group"].shape[0]].float()
    return out


def _rows(s, padded, buffer):
    """The padded batch's rows back in order, rounded once, into the caller's buffer (rows behind the groups stay)."""
    buffer[: s["group"].shape[0]] = padded[s["group"], s["within"]].to(buffer.dtype)
    return buffer


def _sigmoid2(z):
    """1 / (1 + exp(-2u)) of the tanh form's argument u, so that GELU(z) = z * that."""
    u = math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)
    return 1.0 / (1.0 + torch.exp(-2.0 * u))


def _forward(s):
    z = torch.bmm(_padded(s, s["x"]), s["w"].float())
    y = z * _sigmoid2(z) if s["case"]["act"] == "gelu_tanh" else z
    out = [_rows(s, y, s["y"])]
    return out if s["z"] is None else out + [_rows(s, z, s["z"])]


def _input_grad(s):
    dx = torch.bmm(_padded(s, s["dy"]), s["w"].float().transpose(1, 2))
    if s["z"] is not None:
        z = _padded(s, s["z"])
        p = _sigmoid2(z)
        du = math.sqrt(2.0 / math.pi) * (1.0 + 3.0 * 0.044715 * z * z)
        dx = dx * (p + 2.0 * z * p * (1.0 - p) * du)
    return [_rows(s, dx, s["dx"])]


def _weight_grad(s):
    s["dw"].copy_(torch.bmm(_padded(s, s["x"]).transpose(1, 2), _padded(s, s["dy"])))
    return [s["dw"]]


def _lora(s):
    rows = s["group"].shape[0]
    y = s["x"][:rows].float() @ s["w"].float()
    if s["bias"] is not None:
        y = y + s["bias"]
    adapter = s["request_adapter"].long()
    of = adapter.clamp(min=0)
    scale = torch.where(adapter < 0, torch.zeros_like(s["scale"][of]), s["scale"][of])
    low = torch.bmm(_padded(s, s["x"]), s["a"].float()[of]) * scale[:, None, None]
    add = torch.bmm(low, s["b"].float()[of])
    s["y"][:rows] = (y + add[s["group"], s["within"]]).to(s["y"].dtype)
    return [s["y"]]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    sizes = _sizes(case)
    rows, k, n, size = case["rows"], case["k"], case["n"], 2
    used = sum(1 for t in sizes if t > 0)
    if case["op"] == "lora":
        adapters = _adapters(case)
        with_one = sum(t for t, a in zip(sizes, adapters) if a >= 0)
        kept = len({a for a in adapters if a >= 0})
        r = case["rank"]
        return {"bytes": size * (rows * (k + n) + k * n + kept * r * (k + n)) + (4 * n if case["bias"] else 0),
                "flops": 2 * rows * k * n + 2 * with_one * r * (k + n)}
    flops = 2 * rows * k * n
    if case["op"] == "weight_grad":
        return {"bytes": size * (rows * (k + n) + len(sizes) * k * n), "flops": flops}
    extra = rows * n if case["op"] == "forward" and case["keep"] else 0
    extra += rows * k if case["op"] == "input_grad" and case["act"] != "none" else 0
    return {"bytes": size * (rows * (k + n) + used * k * n + extra), "flops": flops}


# ---------------------------------------------------------------------------
# the definition in 64 bits, group by group
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    lo = 0

    def gelu(z):
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))

    def gelu_slope(z):
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 0.134145 * z * z)

    def f64(t):
        return t.to(torch.float64)

    if case["op"] == "forward":
        y, z = torch.zeros_like(s["y"], dtype=torch.float64), torch.zeros_like(s["y"], dtype=torch.float64)
        for e, t in enumerate(s["sizes"]):
            z[lo:lo + t] = f64(s["x"][lo:lo + t]) @ f64(s["w"][e])
            y[lo:lo + t] = gelu(z[lo:lo + t]) if case["act"] == "gelu_tanh" else z[lo:lo + t]
            lo += t
        return [y, z] if case["keep"] else [y]
    if case["op"] == "input_grad":
        dx = torch.zeros_like(s["dx"], dtype=torch.float64)
        for e, t in enumerate(s["sizes"]):
            dx[lo:lo + t] = f64(s["dy"][lo:lo + t]) @ f64(s["w"][e]).T
            lo += t
        if s["z"] is not None:
            dx[:lo] *= gelu_slope(f64(s["z"][:lo]))
        return [dx]
    if case["op"] == "weight_grad":
        dw = torch.zeros_like(s["dw"], dtype=torch.float64)
        for e, t in enumerate(s["sizes"]):
            dw[e] = f64(s["x"][lo:lo + t]).T @ f64(s["dy"][lo:lo + t])
            lo += t
        return [dw]
    y = torch.zeros_like(s["y"], dtype=torch.float64)
    w = f64(s["w"])
    for e, (t, ad) in enumerate(zip(s["sizes"], _adapters(case))):
        x = f64(s["x"][lo:lo + t])
        y[lo:lo + t] = x @ w + (f64(s["bias"]) if s["bias"] is not None else 0.0)
        if ad >= 0:
            y[lo:lo + t] += f64(s["scale"][ad]) * ((x @ f64(s["a"][ad])) @ f64(s["b"][ad]))
        lo += t
    return [y]
