"""Plain 64-bit forms of the training operators and the error bounds their GPU results are held to.

A 16-bit output is off by at most half a step of its type, eps / 2 relative to the value (plus half
of the smallest subnormal).  Before that rounding an fp32 sum of K products is off by the roundings of
its additions: each at most 2^-24 of the running sum, of independent signs, so their total stays
within a small multiple of 2^-24 sqrt(K) times the size of the sum, sqrt(sum of squared products)
(SIGMA times it here: sums of a few hundred thousand entries per test, each a normal deviate)."""
import math

import torch

SIGMA = 16.0
U32 = 2.0 ** -24
ACTS = ("none", "relu", "relu2", "gelu", "silu")


def act(z, name):
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if name == "relu2":
        return torch.where(z < 0, torch.zeros_like(z), z) ** 2
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return z.clone()


def act_slope(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "relu2":
        return 2 * torch.where(z < 0, torch.zeros_like(z), z)
    if name == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def half_step(want, dtype):
    f = torch.finfo(dtype)
    return f.eps / 2 * want.abs() * 1.01 + f.smallest_normal * f.eps / 2


def sum_error(p, q):
    """Bound on the fp32 accumulation error of p @ q (64-bit operands)."""
    k = max(1, p.shape[-1])
    return SIGMA * U32 * math.sqrt(k) * torch.sqrt((p * p) @ (q * q)) + 2 * U32 * (p @ q).abs()


def assert_within(got, want, tol, what):
    got = got.detach().double().cpu()
    want, tol = want.double().cpu(), tol.double().cpu()
    assert got.shape == want.shape, f"{what}: {tuple(got.shape)} against {tuple(want.shape)}"
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    fin = ~(nan | inf)
    assert torch.isfinite(got[fin]).all(), f"{what}: not finite where it should be"
    over = (got[fin] - want[fin]).abs() - tol[fin]
    if over.numel():
        worst = float(over.max())
        assert worst <= 0, f"{what}: {int((over > 0).sum())} of {over.numel()} entries out, worst by {worst:.3e}"


def clamp_offsets(offsets, rows):
    """The groups the kernels form: the running maximum of the offsets clamped to [0, rows]."""
    out, top = [], 0
    for v in offsets:
        top = max(top, min(max(int(v), 0), rows))
        out.append(top)
    return out


def linear(x, w, bias, residual, name, w_kn):
    """(y, z, bound on z's error before rounding) in 64 bits."""
    x, w = x.double(), w.double()
    wt = w if w_kn else w.t()
    z = x @ wt
    err = sum_error(x, wt)
    if bias is not None:
        z = z + bias.double()
        err = err + 2 * U32 * z.abs()
    y = act(z, name)
    if residual is not None:
        y = y + residual.double()
    return y, z, err


def forward_error(z, err, y, residual, name):
    """Bound on y's error before its rounding: z's through the activation's slope (at most 1.2, and
    2 |z| for the squared rectifier), eight fp32 roundings of the activation itself and the sum's."""
    slope = 2 * (z.abs() + err) if name == "relu2" else 1.2
    return slope * err + 16 * U32 * (act(z, name).abs() + z.abs() * U32) + 2 * U32 * y.abs()


def grad_input(dz, w, preact, name, add, w_kn):
    """(dx, bound on its error before rounding)."""
    dz, w = dz.double(), w.double()
    wt = w.t() if w_kn else w
    s = dz @ wt
    err = sum_error(dz, wt)
    if preact is not None and name != "none":
        slope = act_slope(preact.double(), name)
        err = err * slope.abs() + 32 * U32 * (s * slope).abs() + 8 * U32 * s.abs()
        s = s * slope
    if add is not None:
        s = s + add.double()
    return s, err + 2 * U32 * s.abs()


def grad_weight(dz, x, w_kn):
    """((dw, bound), (db, bound))."""
    dz, x = dz.double(), x.double()
    p, q = (x.t(), dz) if w_kn else (dz.t(), x)
    ones = torch.ones(1, dz.shape[0], dtype=torch.float64)
    return (p @ q, sum_error(p, q)), ((ones @ dz)[0], sum_error(ones, dz)[0])
