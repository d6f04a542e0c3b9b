"""The training operators around a bank of projection matrices, as measured workloads.

Three operators, each with its backward pass: layer norm, the linear layer with bias, activation and
residual, and the linear layers of a stack of experts over ragged groups of rows, whose weight gradient
is the [g, m, n] gradient stack of a bank.  Sizes are those of the framework's banks (256 x 768,
2816 x 768, 4096 x 512, 512 x 4096, stacks of 24 and 32) and generic ones.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-5


def listed():
    return [
        # one token on its way through a block: the smallest call there is
        {"name": "norm_token", "op": "norm", "rows": 1, "cols": 768, "type": "bf16"},
        # a training batch of 64 sequences of 1024 tokens at the banks' model width
        {"name": "norm_batch", "op": "norm", "rows": 65536, "cols": 768, "type": "bf16"},
        # odd width and row count: rows that start at any 2-byte boundary
        {"name": "norm_grad_odd", "op": "norm_grad", "rows": 4099, "cols": 1601, "type": "fp16"},
        # the backward pass of the training batch, with the weight's and bias's gradients
        {"name": "norm_grad_batch", "op": "norm_grad", "rows": 65536, "cols": 768, "type": "bf16"},
        # one token through the down projection with its residual (weights stored [k, n], as the mlp
        # bank stores them): bound by the latency and the read of the weights
        {"name": "linear_token", "op": "linear", "rows": 1, "n": 768, "k": 2816, "kn": True, "act": "none",
         "residual": True, "keep": False, "type": "bf16"},
        # the up projection of a training batch, its preactivation kept for the backward pass
        {"name": "linear_batch", "op": "linear", "rows": 32768, "n": 2816, "k": 768, "kn": False, "act": "relu2",
         "residual": False, "keep": True, "type": "bf16"},
        # a short ragged batch: fewer tiles than compute units
        {"name": "linear_grad_ragged", "op": "linear_grad", "rows": 517, "n": 512, "k": 4096, "kn": False,
         "act": "gelu", "type": "fp16"},
        # the down projection's backward pass of a training batch, with the derivative of the activation
        {"name": "linear_grad_batch", "op": "linear_grad", "rows": 32768, "n": 768, "k": 2816, "kn": True,
         "act": "relu2", "type": "bf16"},
        # a few tokens over eight experts: bound by the read of the experts' weights, some have no rows
        {"name": "expert_few", "op": "expert", "rows": 64, "experts": 8, "n": 2816, "k": 768, "kn": False,
         "act": "silu", "type": "bf16"},
        # a training batch over 32 experts of the wide bank's shape
        {"name": "expert_batch", "op": "expert", "rows": 32768, "experts": 32, "n": 512, "k": 4096, "kn": False,
         "act": "none", "type": "bf16"},
        # a short batch over eight small experts, ragged row counts
        {"name": "expert_grad_few", "op": "expert_grad", "rows": 1000, "experts": 8, "n": 256, "k": 768, "kn": False,
         "act": "silu", "type": "fp16"},
        # the backward pass of a training batch over 24 experts: the gradient stack of the mlp bank
        {"name": "expert_grad_batch", "op": "expert_grad", "rows": 32768, "experts": 24, "n": 768, "k": 2816,
         "kn": True, "act": "relu2", "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "linear", "linear_grad", "expert", "expert_grad"])
    if op.startswith("norm"):
        cols = _log(rng, 32, 8192)
        if rng.random() < 0.6:
            cols = max(8, cols // 8 * 8)
        rows = min(_log(rng, 1, 65536), 65536 * 768 // cols)
        return {"op": op, "rows": rows, "cols": cols, "type": rng.choice(["bf16", "bf16", "fp16", "fp32"])}
    n, k = rng.choice([(768, 2816), (2816, 768), (256, 768), (768, 256), (512, 4096), (4096, 512), (0, 0), (0, 0)])
    if not n:
        n, k = _log(rng, 64, 4096), _log(rng, 64, 4096)
        if rng.random() < 0.75:
            n, k = n // 8 * 8, k // 8 * 8
    rows = min(_log(rng, 1, 32768), 32768 * 2816 * 768 // (n * k))
    case = {"op": op, "rows": rows, "n": n, "k": k, "kn": rng.random() < 0.5, "type": rng.choice(["bf16", "bf16", "fp16"]),
            "act": rng.choice(["none", "relu", "relu2", "gelu", "silu"])}
    if op == "linear":
        case |= {"residual": rng.random() < 0.5, "keep": rng.random() < 0.5}
    if op.startswith("expert"):
        case["experts"] = rng.choice([2, 5, 8, 24, 32])
    return case


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = TYPES[case["type"]]

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device="cuda") * scale

    s = dict(case)
    rows = case["rows"]
    if case["op"].startswith("norm"):
        cols = case["cols"]
        # a residual stream: features of different scale, an offset of their own, rows of different size
        s["x"] = ((normal(rows, cols) + 0.2 * normal(cols)) * torch.exp(0.5 * normal(cols)) * torch.exp(0.3 * normal(rows, 1))).to(t)
        s["weight"], s["bias"] = 1 + 0.1 * normal(cols), 0.1 * normal(cols)
        if case["op"] == "norm_grad":
            s["dy"] = normal(rows, cols, scale=0.01).to(t)
            xf = s["x"].float()
            s["mean"] = xf.mean(1)
            s["rstd"] = torch.rsqrt((xf - s["mean"][:, None]).square().mean(1) + EPS)
        return s
    n, k, e = case["n"], case["k"], case.get("experts")
    stack = () if e is None else (e,)
    s["w"] = normal(*stack, *((k, n) if case["kn"] else (n, k)), scale=k ** -0.5).to(t)
    if e is not None:
        # rows per expert as a router leaves them: uneven, some experts without a row
        r = np.random.RandomState(seed % (1 << 32))
        counts = r.multinomial(rows, r.dirichlet(np.full(e, 2.0)))
        s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
        s["most"] = int(counts.max())   # the largest group, for the plain form's padding
    if case["op"].endswith("grad"):
        s["dz"] = normal(rows, n, scale=0.01).to(t)
        s["prev"] = normal(rows, k).to(t)              # the preactivation of the layer before
        s["x"] = _act(s["prev"].float(), case["act"]).to(t)
    else:
        s["x"] = normal(rows, k).to(t)
        s["bias"] = normal(*stack, n, scale=0.1).to(t)
        if case.get("residual"):
            s["skip"] = normal(rows, n).to(t)
    return s


def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "relu2":
        return torch.clamp(z, min=0).square()
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "relu2":
        return 2 * torch.clamp(z, min=0)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    return torch.ones_like(z)


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    from orthogonalizing_polynomial_cascade_amd import anvil
    op = s["op"]
    if op == "norm":
        return anvil.anvil_layer_norm(s["x"], s["weight"], s["bias"], EPS)
    if op == "norm_grad":
        return anvil.anvil_layer_norm_grad(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"])
    if op == "linear":
        y, z = anvil.anvil_linear(s["x"], s["w"], s["bias"], residual=s.get("skip"), act=s["act"], w_kn=s["kn"],
                                  keep_preact=s["keep"])
        return [y, z] if s["keep"] else [y]
    if op == "linear_grad":
        dx = anvil.anvil_linear_grad_input(s["dz"], s["w"], preact=s["prev"], act=s["act"], w_kn=s["kn"])
        dw, db = anvil.anvil_linear_grad_weight(s["dz"], s["x"], w_kn=s["kn"])
        return [dx, dw, db]
    if op == "expert":
        y, _ = anvil.anvil_expert_linear(s["x"], s["w"], s["offsets"], s["bias"], act=s["act"], w_kn=s["kn"])
        return [y]
    dx = anvil.anvil_expert_grad_input(s["dz"], s["w"], s["offsets"], preact=s["prev"], act=s["act"], w_kn=s["kn"])
    dw, db = anvil.anvil_expert_grad_weight(s["dz"], s["x"], s["offsets"], w_kn=s["kn"])
    return [dx, dw, db]


def _run_plain(s):
    op, t = s["op"], s["x"].dtype
    x = s["x"].float()
    if op == "norm":
        mean = x.mean(1)
        d = x - mean[:, None]
        rstd = torch.rsqrt(d.square().mean(1) + EPS)
        return (d * rstd[:, None] * s["weight"] + s["bias"]).to(t), mean, rstd
    if op == "norm_grad":
        dy = s["dy"].float()
        h = (x - s["mean"][:, None]) * s["rstd"][:, None]
        gw = dy * s["weight"]
        dx = s["rstd"][:, None] * (gw - gw.mean(1, keepdim=True) - h * (gw * h).mean(1, keepdim=True))
        return dx.to(t), (dy * h).sum(0), dy.sum(0)
    w = s["w"].float()
    if op == "linear":
        z = torch.matmul(x, w if s["kn"] else w.t()) + s["bias"].float()
        y = _act(z, s["act"])
        if "skip" in s:
            y = y + s["skip"].float()
        return [y.to(t), z.to(t)] if s["keep"] else [y.to(t)]
    if op == "linear_grad":
        dz = s["dz"].float()
        dx = torch.matmul(dz, w.t() if s["kn"] else w) * _act_grad(s["prev"].float(), s["act"])
        dw = torch.matmul(x.t(), dz) if s["kn"] else torch.matmul(dz.t(), x)
        return [dx.to(t), dw, dz.sum(0)]
    # experts: each group of rows padded to the largest one, one batched product over the stack
    off = s["offsets"].long()
    place = torch.arange(s["most"], device=x.device)
    at = off[:-1, None] + place                                # [experts, most]: the rows of each group
    valid = (at < off[1:, None])[:, :, None]
    at = torch.clamp(at, max=x.shape[0] - 1)
    row = torch.arange(x.shape[0], device=x.device)
    owner = torch.searchsorted(off[1:], row, right=True)       # the expert of each row
    within = row - off[owner]
    if op == "expert":
        z = torch.bmm(torch.where(valid, x[at], 0.0), w if s["kn"] else w.transpose(1, 2).contiguous()) + s["bias"].float()[:, None]
        return [_act(z, s["act"]).to(t)[owner, within]]
    dz = torch.where(valid, s["dz"].float()[at], 0.0)
    xp = torch.where(valid, x[at], 0.0)
    dx = torch.bmm(dz, w.transpose(1, 2).contiguous() if s["kn"] else w)[owner, within] * _act_grad(s["prev"].float(), s["act"])
    dw = torch.bmm(xp.transpose(1, 2).contiguous(), dz) if s["kn"] else torch.bmm(dz.transpose(1, 2).contiguous(), xp)
    return [dx.to(t), dw, dz.sum(1)]


def work(case):
    rows, b = case["rows"], BYTES[case["type"]]
    if case["op"] == "norm":
        c = case["cols"]
        return {"bytes": 2 * rows * c * b + 8 * c + 8 * rows, "flops": 8 * rows * c}
    if case["op"] == "norm_grad":
        c = case["cols"]
        return {"bytes": 3 * rows * c * b + 12 * c + 8 * rows, "flops": 14 * rows * c}
    n, k, e = case["n"], case["k"], case.get("experts", 1)
    used = min(e, rows)   # the experts whose weights are read: at most one for each row
    if not case["op"].endswith("grad"):
        out = 1 + case.get("residual", False) + case.get("keep", False)
        return {"bytes": (rows * (k + n * out) + used * n * (k + 1)) * b, "flops": 2 * rows * n * k}
    # dz, x, weights and (where there is an activation) its preactivation in, input gradient and fp32 weight and
    # bias gradients out
    wide = 2 if case["act"] == "none" else 3
    return {"bytes": (rows * (n + wide * k) + used * n * k) * b + 4 * e * n * (k + 1), "flops": 4 * rows * n * k}


def exact(case, seed):
    """The definitions in 64 bits, group by group, from the same inputs."""
    s = {key: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for key, v in prepare(case, seed).items()}
    x, op = s["x"], case["op"]
    if op == "norm":
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = (var + EPS) ** -0.5
        return torch.addcmul(s["bias"], (x - mean.unsqueeze(1)) * rstd.unsqueeze(1), s["weight"]), mean, rstd
    if op == "norm_grad":
        cols = x.shape[1]
        r = s["rstd"].unsqueeze(1)
        h = (x - s["mean"].unsqueeze(1)) * r
        gw = s["dy"] * s["weight"]
        a = gw.sum(1, keepdim=True) / cols
        c = torch.linalg.vecdot(gw, h, dim=1).unsqueeze(1) / cols
        return r * (gw - a - h * c), torch.einsum("rc,rc->c", s["dy"], h), torch.einsum("rc->c", s["dy"])
    normal_cdf = torch.special.ndtr
    value = {"none": lambda z: z, "relu": torch.relu, "relu2": lambda z: torch.relu(z) ** 2,
             "gelu": lambda z: z * normal_cdf(z), "silu": lambda z: z * torch.sigmoid(z)}[case["act"]]
    slope = {"none": torch.ones_like, "relu": lambda z: torch.heaviside(z, torch.zeros_like(z)), "relu2": lambda z: 2 * torch.relu(z),
             "gelu": lambda z: normal_cdf(z) + z * torch.exp(-z ** 2 / 2) / math.sqrt(2 * math.pi),
             "silu": lambda z: torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z)}[case["act"]]
    grouped = op.startswith("expert")
    ends = s["offsets"].tolist() if grouped else [0, case["rows"]]
    weights = s["w"] if grouped else s["w"].unsqueeze(0)
    weights = weights.transpose(1, 2) if case["kn"] else weights          # [groups, n, k]
    if not op.endswith("grad"):
        bias = s["bias"] if grouped else s["bias"].unsqueeze(0)
        z = torch.cat([torch.addmm(bias[e], x[ends[e]:ends[e + 1]], weights[e].T) for e in range(len(weights))])
        y = value(z) + (s["skip"] if "skip" in s else 0)
        return [y, z] if case.get("keep") else [y]
    parts = [(s["dz"][ends[e]:ends[e + 1]], x[ends[e]:ends[e + 1]], weights[e]) for e in range(len(weights))]
    dx = torch.cat([dz @ w for dz, _, w in parts]) * slope(s["prev"])
    dw = torch.stack([xe.T @ dz if case["kn"] else dz.T @ xe for dz, xe, _ in parts])
    db = torch.stack([torch.ones(len(dz), dtype=dz.dtype, device=dz.device) @ dz for dz, _, _ in parts])
    return [dx, dw, db] if grouped else [dx, dw[0], db[0]]
