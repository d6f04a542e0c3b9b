"""AdamW over lists of tensors, on the GPU: bit for bit against the same operations on the CPU, and against 64 bits."""
import math

import numpy as np
import pytest
import torch

from tests import adamw_helpers as A

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZES = [1, 7, 8, 255, 256, 257, 0, 2047, 2048, 2049, 5000, 40000]
BETAS, EPS = (0.9, 0.95), 1e-8


def _place(v, shift):
    """A copy on the GPU that starts `shift` elements into a buffer."""
    buf = torch.zeros(v.numel() + shift, dtype=v.dtype if v.dtype != torch.float8_e4m3fn else torch.uint8, device="cuda")
    view = buf[shift:]
    view.copy_(v.view(torch.uint8) if v.dtype == torch.float8_e4m3fn else v)
    return view.view(torch.float8_e4m3fn) if v.dtype == torch.float8_e4m3fn else view


def _state(n, param, grad, bits, seed, lr_mul=1.0, wd_mul=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda scale: torch.randn(n, generator=g) * scale  # noqa: E731
    p, m, root = r(0.05), r(3e-4), r(1e-3).abs()
    s = {"grad": (r(1e-3) * torch.exp(2 * r(1))).to(TYPES[grad]), "mantissa": None, "m_scale": None, "v_scale": None,
         "lr_mul": lr_mul, "wd_mul": wd_mul}
    if param == "split":
        s["param"], s["mantissa"] = A.split(p)
    else:
        s["param"] = p.to(TYPES[param])
    if bits == 32:
        s["m"], s["v"] = m, root * root
    else:
        noise = torch.full((n,), 1 << 19)
        s["m"], s["m_scale"] = A.encode(m, noise, 0)
        s["v"], s["v_scale"] = A.encode(root, noise, 1)
    return s


NAMES = ("param", "mantissa", "grad", "m", "v", "m_scale", "v_scale")


def _plan(lib, states, shift=0):
    gpu = [{k: None if s[k] is None else _place(s[k], shift) for k in NAMES} for s in states]
    col = lambda k: [t[k] for t in gpu]  # noqa: E731
    bits = [32 if s["m"].dtype == torch.float32 else 8 for s in states]
    return lib.AdamW(col("param"), col("grad"), mantissas=col("mantissa"), state_bits=bits, m=col("m"), v=col("v"),
                     m_scale=col("m_scale"), v_scale=col("v_scale"), lr_mul=[s["lr_mul"] for s in states],
                     wd_mul=[s["wd_mul"] for s in states])


def _same_bits(got, want, what):
    got = got.cpu()
    assert got.dtype == want.dtype and got.shape == want.shape, what
    kind = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[got.element_size()]
    nan = torch.isnan(want.float()) if want.dtype != torch.int16 else torch.zeros(want.shape, dtype=torch.bool)
    a, b = got.contiguous().view(kind), want.contiguous().view(kind)
    assert torch.equal(a[~nan], b[~nan]), f"{what}: {int((a != b)[~nan].sum())} of {a.numel()} differ"
    assert torch.isnan(got.float()[nan]).all(), f"{what}: NaN"


def _compare(plan, states, what=""):
    for i, s in enumerate(states):
        for name, have in (("param", plan.params), ("mantissa", plan.mantissas), ("m", plan.m), ("v", plan.v),
                           ("m_scale", plan.m_scale), ("v_scale", plan.v_scale)):
            if s[name] is not None:
                _same_bits(have[i], s[name], f"{what} {name}[{i}] of {s['grad'].numel()}")


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("param", ["fp32", "bf16", "fp16", "split"])
def test_steps_bit_for_bit(gpu_lib, param, grad, bits):
    """Three steps of tensors of all sizes, with multipliers of their own, a clipping coefficient and new gradients."""
    states = [_state(n, param, grad, bits, 10 * i, 1 + 0.5 * (i % 3), float(i % 2)) for i, n in enumerate(SIZES)]
    plan = _plan(gpu_lib, states)
    for step in (1, 2, 3):
        clip = None if step == 1 else 0.3
        scale = None if clip is None else torch.tensor([clip], device="cuda")
        gpu_lib.anvil_adamw(plan, 1e-2, step, betas=BETAS, eps=EPS, weight_decay=0.1, grad_scale=scale, seed=step + 4)
        states = [A.step32(s, i, 1e-2, 0.1, BETAS, EPS, step, clip, step + 4) for i, s in enumerate(states)]
        _compare(plan, states, f"step {step}")
        for i, s in enumerate(states):
            s["grad"] = _state(s["grad"].numel(), param, grad, 32, 500 + 10 * i + step)["grad"]
            plan.grads[i].copy_(s["grad"])


@pytest.mark.parametrize("shift", [1, 3, 8])
def test_any_alignment(gpu_lib, shift):
    """Tensors that start at any element of a buffer, the kinds mixed in one plan."""
    kinds = [("split", "bf16", 8), ("fp32", "fp32", 32), ("fp16", "fp16", 8), ("bf16", "fp32", 32), ("fp32", "bf16", 8)]
    states = [_state(n, *kinds[i % 5], 3 * i) for i, n in enumerate(SIZES)]
    plan = _plan(gpu_lib, states, shift)
    gpu_lib.anvil_adamw(plan, 3e-3, 5, betas=BETAS, eps=EPS, weight_decay=0.01, seed=0xFFFFFFFF)
    _compare(plan, [A.step32(s, i, 3e-3, 0.01, BETAS, EPS, 5, None, 0xFFFFFFFF) for i, s in enumerate(states)])


@pytest.mark.parametrize("betas,eps,step", [((0.9, 0.95), 1e-8, 1), ((0.9, 0.999), 1e-6, 1000), ((0.0, 0.0), 1e-3, 1)])
def test_against_64_bits(gpu_lib, betas, eps, step):
    """Each value against the formula.  m and v are sums of two products of one sign or two: six roundings of their
    terms.  The update is a quotient of those: m's error, half of v's, a dozen roundings more, and the corrections' own
    (fp32 numbers of which 1 - beta is exact to 2^-24)."""
    u = 2.0 ** -24
    s = _state(100000, "fp32", "bf16", 32, 1)
    plan = _plan(gpu_lib, [s])
    gpu_lib.anvil_adamw(plan, 1e-2, step, betas=betas, eps=eps, weight_decay=0.1)
    f = lambda x: float(torch.tensor(x, dtype=torch.float32))  # noqa: E731
    p, m, v = A.step64(s["param"], s["grad"], s["m"], s["v"], f(1e-2), f(0.1), betas, eps, step, None)
    terms = betas[0] * s["m"].double().abs() + (1 - betas[0]) * s["grad"].double().abs()
    em = 6 * u * terms
    assert ((plan.m[0].double().cpu() - m).abs() <= em).all()
    assert ((plan.v[0].double().cpu() - v).abs() <= 6 * u * v + 2.0 ** -149).all()
    den = (v / (1 - betas[1] ** step)).sqrt() + eps
    update = f(1e-2) * (m.abs() / (1 - betas[0] ** step)) / den
    ep = f(1e-2) * em / (1 - betas[0] ** step) / den + 16 * u * update + 4 * u * (s["param"].double().abs() + p.abs())
    assert ((plan.params[0].double().cpu() - p).abs() <= ep).all()


def test_rounding_keeps_the_mean(gpu_lib):
    """Over many seeds the mean of what an 8-bit state holds is the value itself: each rounding is off by less than a step
    (2^-3 of the value, or 2^-9 of a scale below 2^-6 of one), so the mean of 400 stays within 6 / sqrt(400) steps.
    The least code of the root may only raise it."""
    n, seeds = 4096, 400
    s = _state(n, "fp32", "fp32", 8, 2)
    want = A.moments(s["grad"], A.decode(s["m"], s["m_scale"]), A.decode(s["v"], s["v_scale"]) ** 2, BETAS, None)
    want = (want[0], want[1].sqrt())
    sums = [torch.zeros(n, dtype=torch.float64) for _ in range(2)]
    plan = _plan(gpu_lib, [s])
    start = [t.clone() for t in (plan.m[0].view(torch.uint8), plan.m_scale[0], plan.v[0].view(torch.uint8), plan.v_scale[0])]
    held = []
    for seed in range(seeds):
        for t, v in zip((plan.m[0].view(torch.uint8), plan.m_scale[0], plan.v[0].view(torch.uint8), plan.v_scale[0]), start):
            t.copy_(v)
        gpu_lib.anvil_adamw(plan, 0.0, 1, betas=BETAS, eps=EPS, seed=seed)
        held.append([t.clone() for t in (plan.m[0].view(torch.uint8), plan.m_scale[0], plan.v[0].view(torch.uint8), plan.v_scale[0])])
    for m, ms, v, vs in held:
        sums[0] += A.decode(m.cpu().view(torch.float8_e4m3fn), ms.cpu()).double()
        sums[1] += A.decode(v.cpu().view(torch.float8_e4m3fn), vs.cpu()).double()
    for total, value, scale, floor in zip(sums, want, (held[0][1], held[0][3]), (0.0, 1.0)):
        scale = scale.cpu().double().repeat_interleave(256)[:n]
        value = value.double()
        step = torch.maximum(value.abs() * 2.0 ** -3, scale * 2.0 ** -9)
        off = total / seeds - value
        over = floor * scale * 2.0 ** -9
        assert (off <= 6 / math.sqrt(seeds) * step + over).all() and (off >= -6 / math.sqrt(seeds) * step).all()


def test_a_slow_second_moment_moves(gpu_lib):
    """A state that starts at the gradient's size follows one four times as large, a thousandth of the way each step: after
    700 steps v has gone 1 - 0.999^700 = 50% of the way in the mean over the elements, which rounding to the nearest code
    would never have left.  (The rounding's noise of one element stays in its code's step; over 65536 of them the mean is
    off by less than a tenth.)"""
    n = 65536
    one = torch.ones(n)
    codes, scale = A.encode(one, torch.zeros(n, dtype=torch.int64), 1)
    s = {"grad": 4 * one, "param": torch.zeros(n), "mantissa": None, "lr_mul": 1.0, "wd_mul": 0.0}
    # one larger element in each block holds the scale
    big = one.clone()
    big[::256] = 8.0
    s["v"], s["v_scale"] = A.encode(big, torch.zeros(n, dtype=torch.int64), 1)
    s["m"], s["m_scale"] = codes, scale
    s["grad"][::256] = 8.0
    plan = _plan(gpu_lib, [s])
    for step in range(1, 701):
        gpu_lib.anvil_adamw(plan, 0.0, step, betas=(0.9, 0.999), eps=EPS)
    v = A.decode(plan.v[0].cpu(), plan.v_scale[0].cpu()).double() ** 2
    rest = torch.ones(n, dtype=torch.bool)
    rest[::256] = False
    want = 16 - 15 * 0.999 ** 700
    assert abs(float(v[rest].mean()) - want) <= 0.1 * want


def test_zeros_and_small_blocks(gpu_lib):
    """Blocks of zeros stay zero (without a 0 / 0), blocks under 2^-100 are taken as zero, and a root that is not zero keeps a
    code however far below its block's largest it is."""
    n = 1024
    s = _state(n, "fp32", "fp32", 8, 3)
    for k in ("m", "v"):
        s[k] = torch.zeros(n, dtype=torch.uint8).view(torch.float8_e4m3fn)
        s[k + "_scale"] = torch.zeros(4)
    s["grad"][:256] = 0
    s["grad"][256:512] = 1e-32
    s["grad"][512:768] = 1e-9
    s["grad"][512] = 1e3
    plan = _plan(gpu_lib, [s])
    gpu_lib.anvil_adamw(plan, 1e-2, 1, betas=BETAS, eps=EPS, weight_decay=0.1, seed=9)
    want = A.step32(s, 0, 1e-2, 0.1, BETAS, EPS, 1, None, 9)
    _compare(plan, [want])
    codes = plan.v[0].cpu().view(torch.uint8)
    assert not codes[:512].any() and (codes[513:768] == 1).all() and torch.isfinite(plan.params[0]).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_nonfinite_gradients(gpu_lib, bits):
    """With 32-bit states a NaN or an infinity stays with its element; with 8-bit ones a NaN does, and an infinity takes
    its block's codes along (its scale is infinite), but no other element's weight in this step."""
    s = _state(3000, "fp32", "fp32", bits, 4)
    s["grad"][5], s["grad"][1000], s["grad"][2999] = float("nan"), float("inf"), -float("inf")
    plan = _plan(gpu_lib, [s])
    gpu_lib.anvil_adamw(plan, 1e-2, 2, betas=BETAS, eps=EPS, weight_decay=0.1, seed=1)
    _compare(plan, [A.step32(s, 0, 1e-2, 0.1, BETAS, EPS, 2, None, 1)])
    bad = torch.nonzero(~torch.isfinite(plan.params[0])).flatten().tolist()
    assert bad == [5, 1000, 2999]


def test_offsets_past_32_bits(gpu_lib):
    """A tensor of more than 2^32 elements: its last ones, and those about element 2^32."""
    n = (1 << 32) + 3000
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    plan = gpu_lib.AdamW([p], [g], state_bits=8)
    parts = [slice((1 << 32) - 2048, (1 << 32) + 512), slice((1 << 32) + 2048, n)]
    fill = torch.Generator().manual_seed(1)
    for part in parts:
        p[part] = torch.randn(part.stop - part.start, generator=fill).to(torch.bfloat16).cuda()
        g[part] = torch.randn(part.stop - part.start, generator=fill).to(torch.bfloat16).cuda()
    before = [(p[part].cpu(), g[part].cpu()) for part in parts]
    gpu_lib.anvil_adamw(plan, 1e-2, 1, betas=BETAS, eps=EPS, weight_decay=0.1, seed=3)
    for part, (pb, gb) in zip(parts, before):
        size = part.stop - part.start
        m, v = A.moments(gb, torch.zeros(size), torch.zeros(size), BETAS, None)
        root = A.root_of(v)
        w = A.weights(pb.float(), m, root, np.float32(1e-2), np.float32(0.1), BETAS, EPS, 1)
        _same_bits(p[part], w.to(torch.bfloat16), "param")
        h = A.dither(3, 0, torch.arange(part.start, part.stop) & 0xFFFFFFFF)
        codes, scale = A.encode(m, h & 0xFFFFF, 0)
        _same_bits(plan.m[0].view(torch.uint8)[part].view(torch.float8_e4m3fn), codes, "m")
        codes, scale = A.encode(root, h >> 12, 1)
        _same_bits(plan.v[0].view(torch.uint8)[part].view(torch.float8_e4m3fn), codes, "v")
        _same_bits(plan.v_scale[0][part.start // 256:-(-part.stop // 256)], scale, "scale")


def test_many_tensors(gpu_lib):
    states = [_state(1 + 37 * i % 900, "split" if i % 2 else "fp32", "bf16", 8 if i % 3 else 32, i) for i in range(1500)]
    plan = _plan(gpu_lib, states)
    gpu_lib.anvil_adamw(plan, 1e-3, 4, betas=BETAS, eps=EPS, weight_decay=0.1, seed=2)
    _compare(plan, [A.step32(s, i, 1e-3, 0.1, BETAS, EPS, 4, None, 2) for i, s in enumerate(states)])


def test_empty(gpu_lib):
    gpu_lib.anvil_adamw(gpu_lib.AdamW([], []), 1e-3, 1)
    none = torch.empty(0, device="cuda")
    gpu_lib.anvil_adamw(gpu_lib.AdamW([none], [none.clone()], state_bits=8), 1e-3, 1)


@pytest.mark.parametrize("bits", [32, 8])
def test_states_of_its_own(gpu_lib, bits):
    """States that are not given begin at zero, for matrices and for a single number."""
    g = torch.Generator().manual_seed(3)
    shapes = [(), (3, 5, 70), (1,), (256,)]
    params, grads = ([torch.randn(s, generator=g) for s in shapes] for _ in range(2))
    plan = gpu_lib.AdamW([p.cuda() for p in params], [v.cuda() for v in grads], state_bits=bits)
    for i, p in enumerate(params):
        assert plan.m[i].shape == plan.v[i].shape == p.shape and not plan.m[i].float().any() and not plan.v[i].float().any()
    gpu_lib.anvil_adamw(plan, 1e-2, 1, betas=BETAS, eps=EPS, weight_decay=0.1)
    for i, (p, v) in enumerate(zip(params, grads)):
        n = p.numel()
        s = {"param": p.view(-1), "mantissa": None, "grad": v.view(-1), "lr_mul": 1.0, "wd_mul": 1.0}
        zero = torch.zeros(n, dtype=torch.uint8).view(torch.float8_e4m3fn) if bits == 8 else torch.zeros(n)
        s |= {"m": zero, "v": zero, "m_scale": torch.zeros(-(-n // 256)), "v_scale": torch.zeros(-(-n // 256))}
        want = A.step32(s, i, 1e-2, 0.1, BETAS, EPS, 1, None, 1)
        _same_bits(plan.params[i].view(-1), want["param"], f"param {i}")
        _same_bits(plan.m[i].view(-1), want["m"], f"m {i}")
        _same_bits(plan.v[i].view(-1), want["v"], f"v {i}")


def test_gradients_elsewhere(gpu_lib):
    """bind() takes the gradients from other tensors, of another type too."""
    s = _state(3000, "fp32", "bf16", 32, 1)
    plan = _plan(gpu_lib, [s])
    other = dict(s, grad=_state(3000, "fp32", "fp32", 32, 2)["grad"])
    plan.bind([other["grad"].cuda()])
    gpu_lib.anvil_adamw(plan, 1e-3, 1, betas=BETAS, eps=EPS, weight_decay=0.1)
    _compare(plan, [A.step32(other, 0, 1e-3, 0.1, BETAS, EPS, 1, None, 1)])
    with pytest.raises(ValueError):
        plan.bind([])
    with pytest.raises(ValueError):
        plan.bind([torch.zeros(7, device="cuda")])


def test_a_refused_bind_changes_nothing(gpu_lib):
    """The plan goes on with the gradients that it has, and keeps them alive."""
    s = _state(3000, "fp32", "fp32", 32, 1)
    plan = _plan(gpu_lib, [s])
    had = plan.grads[0].data_ptr()
    with pytest.raises(gpu_lib.AnvilError):
        plan.bind([plan.params[0]])               # shares memory with what a step writes
    for bad in ([torch.zeros(7, device="cuda")], [plan.grads[0].double()], []):
        with pytest.raises((ValueError, TypeError)):
            plan.bind(bad)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu_lib.anvil_adamw(plan, 1e-3, 1, betas=BETAS, eps=EPS, weight_decay=0.1)
        with pytest.raises(RuntimeError, match="capture"):
            plan.bind([torch.zeros(3000, device="cuda")])
    assert plan.grads[0].data_ptr() == had
    graph.replay()
    _compare(plan, [A.step32(s, 0, 1e-3, 0.1, BETAS, EPS, 1, None, 1)])


def test_refusals(gpu_lib):
    p, g = torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
    for kw in ({"state_bits": 16}, {"mantissas": [None, None]}, {"lr_mul": [1.0, 2.0]}, {"m": [torch.zeros(3, device="cuda")]},
               {"state_bits": [8, 8]}):
        with pytest.raises(ValueError):
            gpu_lib.AdamW([p], [g], **kw)
    with pytest.raises(TypeError):   # a low half without a high one
        gpu_lib.AdamW([p], [g], mantissas=[torch.zeros(64, dtype=torch.int16, device="cuda")])
    for bad in (p.double(), None):
        with pytest.raises(TypeError):
            gpu_lib.AdamW([p], [bad])
    with pytest.raises(gpu_lib.AnvilError):   # one tensor twice
        gpu_lib.AdamW([p, p], [g, g])
    plan = gpu_lib.AdamW([p], [g])
    for kw in ({"step": 0}, {"step": 1, "betas": (1.0, 0.9)}, {"step": 1, "eps": -1.0}):
        with pytest.raises(gpu_lib.AnvilError):
            gpu_lib.anvil_adamw(plan, 1e-3, **kw)
    with pytest.raises(ValueError):
        gpu_lib.anvil_adamw(plan, 1e-3, 1, grad_scale=torch.zeros(2, device="cuda"))
    with pytest.raises(ValueError):
        gpu_lib.anvil_adamw_dev(plan, torch.zeros(4, device="cuda"))


def test_replayed_graph(gpu_lib):
    """A captured step with its scalars on the device, replayed with eager work between: after each replay the state is that
    of the eager calls on a second copy, and near the call that takes the scalars from the host."""
    states = [_state(n, "split", "bf16", 8 if i % 2 else 32, i) for i, n in enumerate((5000, 5000, 300, 2049))]
    captured, eager, host = (_plan(gpu_lib, states) for _ in range(3))
    scalars, scale = torch.zeros(5, device="cuda"), torch.tensor([0.5], device="cuda")

    def set_scalars(step):
        scalars.copy_(torch.tensor([1e-3 * step, 0.1, 1 - BETAS[0] ** step, math.sqrt(1 - BETAS[1] ** step), step]))

    set_scalars(1)
    for plan in (captured, eager):
        gpu_lib.anvil_adamw_dev(plan, scalars, betas=BETAS, eps=EPS, grad_scale=scale)
    gpu_lib.anvil_adamw(host, 1e-3, 1, betas=BETAS, eps=EPS, weight_decay=0.1, grad_scale=scale)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu_lib.anvil_adamw_dev(captured, scalars, betas=BETAS, eps=EPS, grad_scale=scale)
    for step in range(2, 6):
        set_scalars(step)
        graph.replay()
        gpu_lib.anvil_adamw_dev(eager, scalars, betas=BETAS, eps=EPS, grad_scale=scale)
        gpu_lib.anvil_adamw(host, 1e-3 * step, step, betas=BETAS, eps=EPS, weight_decay=0.1, grad_scale=scale)
        torch.cuda.synchronize()
        for name in ("params", "mantissas", "m", "v"):
            for a, b in zip(getattr(captured, name), getattr(eager, name)):
                kind = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
                assert torch.equal(a.view(kind), b.view(kind)), (step, name)
    # the reciprocal corrections are rounded once more on the device: 2^-24 of an update of at most lr each
    for a, b in zip(eager.params, host.params):
        assert (a.float() - b.float()).abs().max() <= 2.0 ** -7 * b.float().abs().max()


def test_captured_step_follows_its_gradients(gpu_lib):
    """bind() after a capture: the replay reads the new gradients, wherever the old ones went."""
    s = _state(5000, "fp32", "bf16", 32, 1)
    plan, again = _plan(gpu_lib, [s]), _plan(gpu_lib, [s])
    gpu_lib.anvil_adamw(plan, 0.0, 1)      # outside capture first
    for a, b in ((plan.m, again.m), (plan.v, again.v), (plan.params, again.params)):
        a[0].copy_(b[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu_lib.anvil_adamw(plan, 1e-3, 1, betas=BETAS, eps=EPS, weight_decay=0.1)
    other = dict(s, grad=_state(5000, "fp32", "fp16", 32, 2)["grad"])
    plan.bind([other["grad"].cuda()])
    graph.replay()
    _compare(plan, [A.step32(other, 0, 1e-3, 0.1, BETAS, EPS, 1, None, 1)])


def test_other_stream(gpu_lib):
    s = _state(100000, "fp32", "fp32", 8, 1)
    plan, side = _plan(gpu_lib, [s]), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    gpu_lib.anvil_adamw(plan, 1e-3, 1, betas=BETAS, eps=EPS, weight_decay=0.1, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    _compare(plan, [A.step32(s, 0, 1e-3, 0.1, BETAS, EPS, 1, None, 1)])


@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("bits", [32, 8])
def test_dropped_with_a_step_queued_on_another_stream(gpu_lib, bits, given):
    """The memory of the object's own states and plan is not handed out before the step has run, whether the stream is
    given or the current one."""
    n = 3 << 20
    side = torch.cuda.Stream()
    p, g = torch.ones(n, device="cuda"), torch.ones(n, device="cuda")
    plan = gpu_lib.AdamW([p], [g], state_bits=bits)
    held = [t for t in (plan.m[0], plan.v[0], plan.m_scale[0], plan.v_scale[0], plan._plan) if t is not None]
    sizes, was = [t.numel() * t.element_size() for t in held], {t.data_ptr() for t in held}
    del held
    a = torch.ones(8192, 8192, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(a)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(100):          # about a millisecond each
            torch.mm(a, a, out=out)
        if not given:
            gpu_lib.anvil_adamw(plan, 1e-2, 1, betas=BETAS, eps=EPS)
    if given:
        gpu_lib.anvil_adamw(plan, 1e-2, 1, betas=BETAS, eps=EPS, stream=side)
    del plan
    fresh = [torch.empty(size, dtype=torch.uint8, device="cuda") for size in sizes for _ in range(4)]
    again = was & {t.data_ptr() for t in fresh}
    assert side.query() or not again
    torch.cuda.synchronize()
    # m = 0.1, v = 0.05: the update is lr * 1 / (1 + eps)
    assert ((p - (1 - 1e-2)).abs() < 1e-6).all()


def _dev_step32(s, i, scalars, clip):
    """A.step32 with the corrections as the device forms them: fp32 reciprocals of the scalars."""
    lr, wd, one1, root2, seed = (np.float32(v) for v in scalars)

    def weights(p, m, root, lr, wd, betas, eps, step):
        fix1, fix2 = np.float32(1) / one1, np.float32(1) / root2
        with np.errstate(all="ignore"):
            return A._t(A._f(p) * (A._f(1.0) - lr * wd) - lr * ((A._f(m) * fix1) / (A._f(root) * fix2 + A._f(eps))))

    with pytest.MonkeyPatch.context() as patch:
        patch.setattr(A, "weights", weights)
        return A.step32(s, i, lr, wd, BETAS, EPS, None, clip, int(seed))


SCALARS = (3e-3, 0.1, 1 - BETAS[0] ** 7, math.sqrt(1 - BETAS[1] ** 7), 12345)
# each of them changed alone (lr, weight decay, both corrections, seed), and the extremes of the seed
CHANGES = [{}, {0: 5e-4}, {1: 0.0}, {1: 0.5}, {2: 1 - BETAS[0]}, {3: 1.0}, {4: 0}, {4: (1 << 24) - 1}]


def _dev_states():
    kinds = [("split", "bf16", 8), ("fp32", "fp32", 32), ("fp16", "fp16", 8), ("split", "bf16", 32), ("fp32", "bf16", 8)]
    return [_state(n, *kinds[i % 5], 7 * i, 1 + 0.5 * (i % 3), 0.5 + i % 2) for i, n in enumerate((5000, 2049, 300, 257, 40000))]


def test_scalar_changes_show_in_the_oracle():
    """What the next test compares depends on every scalar: each change gives other weights, or other codes."""
    states = _dev_states()
    base = [_dev_step32(s, i, SCALARS, 0.3) for i, s in enumerate(states)]
    for change in CHANGES[1:]:
        other = [_dev_step32(s, i, [change.get(k, v) for k, v in enumerate(SCALARS)], 0.3) for i, s in enumerate(states)]
        for a, b, s in zip(base, other, states):
            if 4 in change:
                assert torch.equal(a["param"], b["param"])
                assert s["m_scale"] is None or not torch.equal(a["m"].view(torch.uint8), b["m"].view(torch.uint8))
            else:
                low = "param" if a["mantissa"] is None else "mantissa"
                assert not torch.equal(a[low], b[low]), change


@pytest.mark.parametrize("change", CHANGES, ids=str)
def test_device_scalars_bit_for_bit(gpu_lib, change):
    """Every scalar, read from the device, against the same operations on the CPU: weights, low halves, states, scales."""
    scalars = [change.get(k, v) for k, v in enumerate(SCALARS)]
    states = _dev_states()
    plan = _plan(gpu_lib, states)
    gpu_lib.anvil_adamw_dev(plan, torch.tensor(scalars, dtype=torch.float32, device="cuda"), betas=BETAS, eps=EPS,
                            grad_scale=torch.tensor([0.3], device="cuda"))
    _compare(plan, [_dev_step32(s, i, scalars, 0.3) for i, s in enumerate(states)])


def test_device_corrections_differ_from_the_hosts_by_their_roundings(gpu_lib):
    """The factor 1 / (1 - beta1^t) is off by at most 2^-24 of itself from the host and by 2 * 2^-24 + 2^-48 from the
    device (its divisor is a number of 32 bits, and so is the quotient), the root's likewise: the quotients of an
    update are apart by at most 6 * 2^-24 and, with four roundings more in either, 14 * 2^-24 of the update, and the
    weights by that and their own last rounding."""
    u = 2.0 ** -24
    s = _state(100000, "fp32", "bf16", 32, 3)
    for step in (1, 7, 1000):
        host, dev = _plan(gpu_lib, [s]), _plan(gpu_lib, [s])
        gpu_lib.anvil_adamw(host, 1e-2, step, betas=BETAS, eps=EPS)
        gpu_lib.anvil_adamw_dev(dev, torch.tensor([1e-2, 0, 1 - BETAS[0] ** step, math.sqrt(1 - BETAS[1] ** step), 0],
                                                  device="cuda"), betas=BETAS, eps=EPS)
        a, b, was = (t.double().cpu() for t in (host.params[0], dev.params[0], s["param"]))
        assert ((a - b).abs() <= 14 * u * (a - was).abs() * (1 + 1e-3) + 2 * u * (a.abs() + was.abs())).all()
        assert torch.equal(host.m[0], dev.m[0]) and torch.equal(host.v[0], dev.v[0])
