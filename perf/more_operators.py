"""The rest of a training step around the banks, as measured workloads.

Three operators: the gated linear layer (two projections, activation and product) with its backward pass, the
cross entropy of a linear head over a large vocabulary with its gradients, and the AdamW step of everything that
is no bank.  Sizes are the framework's (width 768, hidden 2816, the 768 x 50304 head) and generic ones.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
BLOCK = 256          # elements that share a scale of an 8-bit state
BETAS, EPS = (0.9, 0.95), 1e-8


def listed():
    return [
        # one token on its way through a feed-forward block: bound by latency and the read of the weights
        {"name": "gated_token", "op": "gated", "rows": 1, "n": 2816, "k": 768, "kn": False, "act": "silu", "bias": False,
         "keep": False, "type": "bf16"},
        # a training batch of 32 sequences of 1024 tokens, the preactivations kept for the backward pass
        {"name": "gated_batch", "op": "gated", "rows": 32768, "n": 2816, "k": 768, "kn": False, "act": "silu", "bias": False,
         "keep": True, "type": "bf16"},
        # odd widths and a short ragged batch: rows that start at any 2-byte boundary
        {"name": "gated_grad_odd", "op": "gated_grad", "rows": 517, "n": 1001, "k": 513, "kn": True, "act": "gelu", "type": "fp16"},
        # the backward pass of the training batch, from the gradient of the block's output
        {"name": "gated_grad_batch", "op": "gated_grad", "rows": 32768, "n": 2816, "k": 768, "kn": False, "act": "silu",
         "type": "bf16"},
        # the loss of a few tokens under the head: bound by the read of its weights
        {"name": "head_few", "op": "head", "rows": 5, "vocab": 50304, "k": 768, "kn": True, "type": "bf16"},
        # the loss of an evaluation batch
        {"name": "head_batch", "op": "head", "rows": 16384, "vocab": 50304, "k": 768, "kn": False, "type": "bf16"},
        # loss and gradients of a short ragged batch over a vocabulary and a width that no tile divides
        {"name": "head_grad_odd", "op": "head_grad", "rows": 1021, "vocab": 32003, "k": 777, "kn": False, "type": "fp16"},
        # loss and gradients of a training batch, the head stored [768, 50304]
        {"name": "head_grad_batch", "op": "head_grad", "rows": 16384, "vocab": 50304, "k": 768, "kn": True, "type": "bf16"},
        # the norms' weights and biases of a model: many tiny tensors, bound by latency
        {"name": "adamw_vectors", "op": "adamw", "matrices": 0, "size": 0, "vectors": 96, "least": 256, "most": 2816, "bits": 32,
         "param": "fp32", "grad": "fp32", "clip": False},
        # embedding and head with the norms: bf16 weights with the low halves of their fp32 masters
        {"name": "adamw_head", "op": "adamw", "matrices": 2, "size": 50304 * 768, "vectors": 50, "least": 256, "most": 2816,
         "bits": 32, "param": "split", "grad": "bf16", "clip": True},
        # tensors of every size from one element on, states in 8 bits: blocks that end anywhere
        {"name": "adamw_ragged_8", "op": "adamw", "matrices": 0, "size": 0, "vectors": 120, "least": 1, "most": 1000003, "bits": 8,
         "param": "fp32", "grad": "bf16", "clip": False},
        # embedding and head with the states in 8 bits
        {"name": "adamw_head_8", "op": "adamw", "matrices": 2, "size": 50304 * 768, "vectors": 50, "least": 256, "most": 2816,
         "bits": 8, "param": "split", "grad": "bf16", "clip": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated", "gated_grad", "head", "head_grad", "adamw", "adamw"])
    if op.startswith("gated"):
        n, k = rng.choice([(2816, 768), (768, 256), (512, 4096), (0, 0), (0, 0)])
        if not n:
            n, k = _log(rng, 64, 4096), _log(rng, 64, 4096)
            if rng.random() < 0.75:
                n, k = n // 8 * 8, k // 8 * 8
        case = {"op": op, "rows": min(_log(rng, 1, 32768), 32768 * 2816 * 768 // (n * k)), "n": n, "k": k, "kn": rng.random() < 0.5,
                "act": rng.choice(["silu", "silu", "gelu", "relu2", "relu", "none"]), "type": rng.choice(["bf16", "bf16", "fp16"])}
        if op == "gated":
            case |= {"bias": rng.random() < 0.5, "keep": rng.random() < 0.5}
        return case
    if op.startswith("head"):
        vocab, k = rng.choice([(50304, 768), (0, 0), (0, 0)])
        if not vocab:
            vocab, k = _log(rng, 1000, 100000), _log(rng, 64, 2048)
            if rng.random() < 0.75:
                vocab, k = vocab // 8 * 8, k // 8 * 8
        return {"op": op, "rows": min(_log(rng, 1, 16384), 16384 * 50304 * 768 // (vocab * k)), "vocab": vocab, "k": k,
                "kn": rng.random() < 0.5, "type": rng.choice(["bf16", "bf16", "fp16"])}
    matrices = rng.choice([0, 1, 2, 5])
    return {"op": "adamw", "matrices": matrices, "size": _log(rng, 10000, 2 * 50304 * 768 // matrices) if matrices else 0,
            "vectors": rng.choice([1, 7, 50, 200]), "least": rng.choice([1, 17, 256]), "most": _log(rng, 500, 100000),
            "bits": rng.choice([8, 32]), "param": rng.choice(["split", "fp32", "bf16", "fp16"]),
            "grad": rng.choice(["bf16", "fp32", "fp16"]), "clip": rng.random() < 0.5}


def _sizes(case):
    """Elements of each tensor of an AdamW case: the matrices, then vectors from the least to the most."""
    count, ratio = case["vectors"], case["most"] / case["least"]
    return [case["size"]] * case["matrices"] + [round(case["least"] * ratio ** (i / max(1, count - 1))) for i in range(count)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device="cuda") * scale

    s = dict(case)
    if case["op"] == "adamw":
        return _prepare_adamw(s, normal, seed)
    t, rows, k = TYPES[case["type"]], case["rows"], case["k"]
    if case["op"].startswith("gated"):
        n = case["n"]
        s["w"] = normal(*((k, 2 * n) if case["kn"] else (2 * n, k)), scale=k ** -0.5).to(t)
        s["x"] = normal(rows, k).to(t)
        if case["op"] == "gated":
            s["bias"] = normal(2 * n, scale=0.1).to(t) if case["bias"] else None
        else:
            s["down"] = normal(k, n, scale=n ** -0.5).to(t)      # h [rows, n] -> y [rows, k]
            s["dy"] = normal(rows, k, scale=0.01).to(t)
            s["z"] = normal(rows, 2 * n).to(t)
        return s
    vocab = case["vocab"]
    # a head in training: logits of a few units, the target's raised, as a model that has learnt something has them
    w = normal(vocab, k, scale=2 * k ** -0.5).to(t)
    s["targets"] = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    s["x"] = (normal(rows, k) + w[s["targets"]].float()).to(t)
    s["w"] = w.t().contiguous() if case["kn"] else w
    if rows > 8:
        s["targets"][torch.rand(rows, generator=g, device="cuda") < 0.05] = -1     # padding: no loss
    s["dloss"] = torch.full((rows,), 1 / rows, device="cuda")                      # the mean over the rows
    return s


def _prepare_adamw(s, normal, seed):
    sizes = _sizes(s)
    blocks = [-(-n // BLOCK) for n in sizes]
    total = sum(blocks)
    # one buffer for each kind of value, every tensor at a block of its own, zeros between
    owner = torch.repeat_interleave(torch.arange(len(sizes)), torch.tensor(blocks)).cuda()
    starts = torch.tensor([0] + blocks).cumsum(0)
    first = starts[:-1].cuda()[owner]
    index = (torch.arange(total, device="cuda") - first)[:, None] * BLOCK + torch.arange(BLOCK, device="cuda")
    there = index < torch.tensor(sizes).cuda()[owner][:, None]
    del index

    def values(scale):
        return torch.where(there, normal(total, BLOCK, scale=scale), torch.zeros((), device="cuda"))

    size = torch.exp(normal(total, 1))                 # gradients of different size from block to block
    s["grad"] = (values(1e-3) * size).to(TYPES[s["grad"]])
    p = values(0.05)
    if s["param"] == "split":                          # the master's upper and lower halves
        bits = p.view(torch.int32)
        s["p"] = (bits >> 16).to(torch.int16).view(torch.bfloat16)
        s["low"] = (bits & 0xFFFF).to(torch.int16)
    else:
        s["p"], s["low"] = p.to(TYPES[s["param"]]), None
    m, root = values(3e-4) * size, (values(1e-3) * size).abs()
    if s["bits"] == 32:
        s["m"], s["v"], s["m_scale"], s["v_scale"] = m, root.square(), None, None
    else:
        for name, v in (("m", m), ("v", root)):
            s[name + "_scale"] = v.abs().amax(1) / 448
            s[name] = (v / torch.clamp(s[name + "_scale"], min=1e-30)[:, None]).to(torch.float8_e4m3fn)
    # matrices decay, vectors do not and learn faster
    s["lr_mul"] = [1.0] * s["matrices"] + [2.0] * s["vectors"]
    s["wd_mul"] = [1.0] * s["matrices"] + [0.0] * s["vectors"]
    s["clip_by"] = torch.full((), 0.37, device="cuda") if s["clip"] else None
    s |= {"lr": 1e-3, "wd": 0.1, "step": 7, "seed": seed % 1000 + 1, "owner": owner, "first": first}
    if own:   # the optimizer that a program makes once: its tensors are pieces of the buffers
        from orthogonalizing_polynomial_cascade_amd import anvil

        def pieces(flat, per=BLOCK):
            ends = starts.tolist()
            return None if flat is None else [flat.view(-1)[e * per:e * per + (n if per > 1 else b)]
                                              for e, n, b in zip(ends, sizes, blocks)]

        s["plan"] = anvil.AdamW(pieces(s["p"]), pieces(s["grad"]), mantissas=pieces(s["low"]), state_bits=s["bits"],
                                m=pieces(s["m"]), v=pieces(s["v"]), m_scale=pieces(s["m_scale"], 1),
                                v_scale=pieces(s["v_scale"], 1), lr_mul=s["lr_mul"], wd_mul=s["wd_mul"])
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
    if op == "gated":
        h, z = anvil.anvil_gated_linear(s["x"], s["w"], s["bias"], act=s["act"], w_kn=s["kn"], keep_preact=s["keep"])
        return [h, z] if s["keep"] else [h]
    if op == "gated_grad":
        dz = anvil.anvil_gated_grad_input(s["dy"], s["down"], s["z"], act=s["act"])
        dx = anvil.anvil_linear_grad_input(dz, s["w"], w_kn=s["kn"])
        dw, _ = anvil.anvil_linear_grad_weight(dz, s["x"], w_kn=s["kn"], out_dtype=s["x"].dtype, want_bias=False)
        return [dz, dx, dw]
    if op == "head":
        return list(anvil.anvil_cross_entropy(s["x"], s["w"], s["targets"], w_kn=s["kn"]))
    if op == "head_grad":
        loss, lse = anvil.anvil_cross_entropy(s["x"], s["w"], s["targets"], w_kn=s["kn"])
        dx, dw = anvil.anvil_cross_entropy_grad(s["x"], s["w"], s["targets"], lse, s["dloss"], w_kn=s["kn"])
        return [loss, lse, dx, dw]
    anvil.anvil_adamw(s["plan"], s["lr"], s["step"], betas=BETAS, eps=EPS, weight_decay=s["wd"], grad_scale=s["clip_by"],
                      seed=s["seed"])
    return _adamw_state(s)


def _adamw_state(s):
    """What a step leaves: weights and states, the 8-bit ones with their scales."""
    return [s[name] for name in ("p", "low", "m", "v", "m_scale", "v_scale") if s[name] is not None]


def _run_plain(s):
    op = s["op"]
    if op == "adamw":
        return _plain_adamw(s)
    t, x = s["x"].dtype, s["x"].float()
    w = s["w"].float() if s["kn"] else s["w"].float().t()                # [k, columns]
    if op == "gated":
        z = torch.matmul(x, w)
        if s["bias"] is not None:
            z = z + s["bias"].float()
        gate, up = z.chunk(2, 1)
        h = (_act(gate, s["act"]) * up).to(t)
        return [h, z.to(t)] if s["keep"] else [h]
    if op == "gated_grad":
        gate, up = s["z"].float().chunk(2, 1)
        dh = torch.matmul(s["dy"].float(), s["down"].float())
        dz = torch.cat([dh * up * _act_grad(gate, s["act"]), dh * _act(gate, s["act"])], 1)
        dw = torch.matmul(x.t(), dz) if s["kn"] else torch.matmul(dz.t(), x)
        return [dz.to(t), torch.matmul(dz, w.t()).to(t), dw.to(t)]
    z = torch.matmul(x, w)
    most = z.amax(1, keepdim=True)
    lse = (torch.log(torch.exp(z - most).sum(1, keepdim=True)) + most)[:, 0]
    target = s["targets"]
    counts = (target >= 0) & (target < s["vocab"])
    at = torch.where(counts, target, 0)
    loss = torch.where(counts, lse - z.gather(1, at[:, None])[:, 0], 0.0)
    if op == "head":
        return [loss, lse]
    p = torch.exp(z - lse[:, None])
    p.scatter_add_(1, at[:, None], torch.full_like(at, -1, dtype=p.dtype)[:, None])
    p = p * torch.where(counts, s["dloss"], 0.0)[:, None]
    dw = torch.matmul(x.t(), p) if s["kn"] else torch.matmul(p.t(), x)
    return [loss, lse, torch.matmul(p, w.t()).to(t), dw.to(t)]


def _mix(h):
    """A hash of 32 bits, in the low half of 64-bit integers."""
    h = ((h ^ (h >> 16)) * 0x7A3C5EB5) & 0xFFFFFFFF
    h = ((h ^ (h >> 15)) * 0x5D8E36CB) & 0xFFFFFFFF
    return h ^ (h >> 16)


def _encode(v, dither, floor):
    """e4m3 codes and scales of fp32 rows: the largest magnitude of a row is 448 times its scale, and 20 bits of dither
    are added below the last kept bit.  `floor`: the least code of a value that is not zero."""
    most = v.abs().amax(1, keepdim=True)
    inverse = torch.where(most >= 2.0 ** -100, torch.full_like(most, 448.0) / most, 0.0)
    q = v.abs() * inverse
    small = q < 2.0 ** -6
    bits = torch.where(small, q + 2.0 ** -6, q).view(torch.int32)
    code = ((bits + dither.to(torch.int32)) >> 20) - torch.where(small, 968, 960)
    code = torch.clamp(code, max=126)
    code = torch.where((q > 0) & (code < floor), floor, code)
    code = torch.where(v < 0, code + 128, code).to(torch.uint8)
    return code.view(torch.float8_e4m3fn), torch.where(most >= 2.0 ** -100, most / torch.full_like(most, 448.0), 0.0)[:, 0]


def _plain_adamw(s):
    """On the whole buffers; every product and sum rounds on its own."""
    f32 = {"dtype": torch.float32, "device": s["p"].device}
    b1, b2 = BETAS
    one_b1, one_b2 = torch.tensor(1 - b1, **f32), torch.tensor(1 - b2, **f32)
    fix1 = torch.tensor(1 / (1 - b1 ** s["step"]), **f32)
    fix2 = torch.tensor(1 / math.sqrt(1 - b2 ** s["step"]), **f32)
    lr = torch.tensor(s["lr"], **f32) * torch.tensor(s["lr_mul"], **f32)[s["owner"]][:, None]
    keep = 1 - lr * (torch.tensor(s["wd"], **f32) * torch.tensor(s["wd_mul"], **f32)[s["owner"]][:, None])
    g = s["grad"].float()
    if s["clip_by"] is not None:
        g = g * s["clip_by"]
    if s["low"] is None:
        p = s["p"].float()
    else:
        p = ((s["p"].view(torch.int16).to(torch.int32) << 16) | (s["low"].to(torch.int32) & 0xFFFF)).view(torch.float32)
    m, v = s["m"].float(), s["v"].float()
    if s["bits"] == 8:
        m, v = m * s["m_scale"][:, None], (v * s["v_scale"][:, None]).square()
    m = m * torch.tensor(b1, **f32) + g * one_b1
    v = v * torch.tensor(b2, **f32) + (g * g) * one_b2
    root = torch.sqrt(v)
    p = p * keep - lr * ((m * fix1) / (root * fix2 + torch.tensor(EPS, **f32)))
    if s["low"] is None:
        s["p"].copy_(p)
    else:
        bits = p.view(torch.int32)
        s["p"].copy_((bits >> 16).to(torch.int16).view(torch.bfloat16))
        s["low"].copy_((bits & 0xFFFF).to(torch.int16))
    if s["bits"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return _adamw_state(s)
    key = _mix((s["seed"] + (s["owner"] + 1) * 0x9E3779B9) & 0xFFFFFFFF)[:, None]
    index = (torch.arange(len(s["p"]), device=g.device) - s["first"])[:, None] * BLOCK + torch.arange(BLOCK, device=g.device)
    h = _mix((index + key) & 0xFFFFFFFF)
    for name, value, dither, floor in (("m", m, h & 0xFFFFF, 0), ("v", root, h >> 12, 1)):
        codes, scale = _encode(value, dither, floor)
        s[name].copy_(codes)
        s[name + "_scale"].copy_(scale)
    return _adamw_state(s)


def work(case):
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        weight = {"split": 8, "fp32": 8, "bf16": 4, "fp16": 4}[case["param"]]
        state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
        return {"bytes": n * (weight + BYTES[case["grad"]] + state), "flops": 20 * n}
    rows, k, b = case["rows"], case["k"], BYTES[case["type"]]
    if case["op"] == "gated":
        n = case["n"]
        return {"bytes": (rows * (k + n * (3 if case["keep"] else 1)) + 2 * n * k) * b, "flops": 4 * rows * n * k}
    if case["op"] == "gated_grad":
        # dy, x, z and both weights in, dz, dx and dw out
        n = case["n"]
        return {"bytes": (rows * (3 * k + 4 * n) + 5 * n * k) * b, "flops": 10 * rows * n * k}
    vocab = case["vocab"]
    if case["op"] == "head":
        return {"bytes": (rows + vocab) * k * b + 16 * rows, "flops": 2 * rows * vocab * k}
    # logits once, two products with their gradient
    return {"bytes": 2 * (rows + vocab) * k * b + 20 * rows, "flops": 6 * rows * vocab * k}


def exact(case, seed):
    """The definitions in 64 bits from the same inputs."""
    s = {key: v.double() if torch.is_tensor(v) and v.is_floating_point() and case["op"] != "adamw" else v
         for key, v in prepare(case, seed).items()}
    if case["op"] == "adamw":
        return _exact_adamw(s)
    name = case.get("act")
    cdf = torch.special.ndtr
    value = {"none": lambda z: z, "relu": torch.relu, "relu2": lambda z: torch.relu(z) ** 2, "gelu": lambda z: z * cdf(z),
             "silu": lambda z: z * torch.sigmoid(z)}
    slope = {"none": torch.ones_like, "relu": lambda z: torch.heaviside(z, torch.zeros_like(z)), "relu2": lambda z: 2 * torch.relu(z),
             "gelu": lambda z: cdf(z) + z * torch.exp(-z ** 2 / 2) / math.sqrt(2 * math.pi),
             "silu": lambda z: torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z)}
    x, w = s["x"], s["w"].T if case["kn"] else s["w"]                    # [columns, k]
    if case["op"] == "gated":
        n, bias = case["n"], s["bias"] if s["bias"] is not None else torch.zeros(2 * case["n"], dtype=x.dtype, device=x.device)
        gate, up = torch.addmm(bias[:n], x, w[:n].T), torch.addmm(bias[n:], x, w[n:].T)
        h = value[name](gate) * up
        return [h, torch.cat([gate, up], 1)] if case["keep"] else [h]
    if case["op"] == "gated_grad":
        n = case["n"]
        gate, up, dh = s["z"][:, :n], s["z"][:, n:], s["dy"] @ s["down"]
        dgate, dup = dh * slope[name](gate) * up, dh * value[name](gate)
        dw = torch.cat([dgate.T @ x, dup.T @ x])
        return [torch.cat([dgate, dup], 1), dgate @ w[:n] + dup @ w[n:], dw.T if case["kn"] else dw]
    # the head, some rows at a time
    losses, sums, dxs, dw = [], [], [], torch.zeros_like(w)
    for at in range(0, case["rows"], 2048):
        rows = slice(at, at + 2048)
        z = x[rows] @ w.T
        lse, t = torch.logsumexp(z, 1), s["targets"][rows]
        valid = (t >= 0).double()
        hot = torch.clamp(t, min=0).unsqueeze(1)
        losses.append((lse - torch.gather(z, 1, hot).squeeze(1)) * valid)
        sums.append(lse)
        if case["op"] == "head_grad":
            p = torch.softmax(z, 1)
            p -= torch.zeros_like(p).scatter_(1, hot, 1.0)
            p *= (valid * s["dloss"][rows]).unsqueeze(1)
            dxs.append(p @ w)
            dw += p.T @ x[rows]
    out = [torch.cat(losses), torch.cat(sums)]
    return out + [torch.cat(dxs), dw.T if case["kn"] else dw] if case["op"] == "head_grad" else out


def _exact_adamw(s):
    owner, (b1, b2) = s["owner"], BETAS
    # the hyperparameters are numbers of 32 bits
    def number(v):
        return torch.tensor(v, dtype=torch.float32, device=owner.device).double()

    lr = (number(s["lr"]) * number(s["lr_mul"]))[owner].unsqueeze(1)
    wd = (number(s["wd"]) * number(s["wd_mul"]))[owner].unsqueeze(1)
    g = s["grad"].double() * (1 if s["clip_by"] is None else s["clip_by"].double())
    p, m, v = s["p"].double(), s["m"].double(), s["v"].double()
    if s["low"] is not None:   # the master's lower half, as a fraction of its upper half's last place
        upper = s["p"].view(torch.int16).int() * 65536
        p = (upper + (s["low"].int() + 65536) % 65536).view(torch.float32).double()
    if s["bits"] == 8:
        m, v = m * s["m_scale"].double().unsqueeze(1), (v * s["v_scale"].double().unsqueeze(1)) ** 2
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g ** 2
    p = (1 - lr * wd) * p - lr * (m / (1 - b1 ** s["step"])) / ((v / (1 - b2 ** s["step"])).sqrt() + EPS)
    low = [] if s["low"] is None else [None]
    if s["bits"] == 32:
        return [p] + low + [m, v]
    # the codes depend on the dither, the scales do not
    return [p] + low + [None, None, m.abs().amax(1) / 448, v.sqrt().amax(1) / 448]
