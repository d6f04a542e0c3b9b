"""Layer norm and its backward pass on the GPU against a plain form in 64 bits."""
import math

import pytest
import torch

from tests.layer_helpers import SIGMA, U32, assert_within, half_step

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _data(rows, cols, dtype, seed, pitch=None, offset=0.0):
    """x [rows, cols] on the GPU in rows `pitch` apart (a NaN-filled buffer around them)."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * (1 + torch.rand(cols, generator=g)) + offset
    buf = torch.full((max(rows, 1), (pitch or cols)), float("nan"), dtype=dtype, device="cuda")
    view = buf[:rows, :cols]
    view.copy_(x.to(dtype))
    return view


def _reference(x, w, b, eps):
    x = x.double().cpu()
    mean = x.mean(1)
    d = x - mean[:, None]
    var = (d * d).mean(1)
    rstd = (var + eps) ** -0.5
    h = d * rstd[:, None]
    y = h * (w.double().cpu() if w is not None else 1.0) + (b.double().cpu() if b is not None else 0.0)
    return y, mean, rstd, h


def _mean_error(x):
    """fp32 mean of a row: its additions' roundings and the division's."""
    x = x.double().cpu()
    n = x.shape[1]
    return (SIGMA * U32 * math.sqrt(n) * torch.sqrt((x * x).sum(1)) + 2 * U32 * x.sum(1).abs()) / n \
        + 2 * U32 * x.mean(1).abs()


def _check_forward(gpu_lib, x, w, b, eps, **kw):
    y, mean, rstd = gpu_lib.anvil_layer_norm(x, w, b, eps, **kw)
    torch.cuda.synchronize()
    want, mean_w, rstd_w, h = _reference(x, w, b, eps)
    em = _mean_error(x)
    assert_within(mean, mean_w, em, "mean")
    # the variance: the mean's error moves every deviation; then its own additions and the root
    er = (em * rstd_w) ** 2 + SIGMA * U32 * 4
    assert_within(rstd, rstd_w, rstd_w * er, "rstd")
    wa = w.double().cpu().abs() if w is not None else 1.0
    err = (em * rstd_w)[:, None] * wa + (er[:, None] + 8 * U32) * h.abs() * wa + 4 * U32 * want.abs()
    assert_within(y, want, err + half_step(want, x.dtype), "y")
    return y, mean, rstd


def _check_backward(gpu_lib, dy, x, w, mean, rstd, **kw):
    dx, dw, db = gpu_lib.anvil_layer_norm_grad(dy, x, w, mean, rstd, **kw)
    torch.cuda.synchronize()
    d, xd = dy.double().cpu(), x.double().cpu()
    m, r = mean.double().cpu()[:, None], rstd.double().cpu()[:, None]
    wd = w.double().cpu() if w is not None else torch.ones(x.shape[1], dtype=torch.float64)
    n, rows = x.shape[1], x.shape[0]
    h = (xd - m) * r
    g = d * wd
    a, c = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    want = r * (g - a - h * c)
    # h in fp32 carries the subtraction's rounding of x - mean, relative to the larger of both
    eh = 4 * U32 * ((xd.abs() + m.abs()) * r + h.abs())
    ea = SIGMA * U32 * math.sqrt(n) * torch.sqrt((g * g).sum(1, keepdim=True)) / n + 4 * U32 * a.abs()
    ec = SIGMA * U32 * math.sqrt(n) * torch.sqrt((g * h).square().sum(1, keepdim=True)) / n \
        + (g * eh).square().sum(1, keepdim=True).sqrt() * 4 / n + (g.abs() * eh).mean(1, keepdim=True) + 4 * U32 * c.abs()
    err = r * (ea + ec * h.abs() + eh * c.abs() + 8 * U32 * (g.abs() + a.abs() + (h * c).abs()))
    assert_within(dx, want, err + half_step(want, x.dtype), "dx")
    k = max(rows, 1)
    ew = SIGMA * U32 * math.sqrt(k) * (d * h).square().sum(0).sqrt() + (d.abs() * eh).sum(0) + 2 * U32 * (d * h).sum(0).abs()
    assert_within(dw, (d * h).sum(0), ew + 1e-45, "dweight")
    eb = SIGMA * U32 * math.sqrt(k) * d.square().sum(0).sqrt() + 2 * U32 * d.sum(0).abs()
    assert_within(db, d.sum(0), eb + 1e-45, "dbias")
    return dx, dw, db


# every register layout (one wave a row up to 2048 columns, a workgroup up to 8192, longer), its
# edges, odd widths, and row counts from one to more than one workgroup's
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 768), (3, 7), (5, 64), (2, 511), (9, 512), (9, 513),
                                       (130, 768), (7, 1024), (6, 1601), (5, 2048), (5, 2049), (3, 4096),
                                       (4, 5001), (2, 8192), (3, 8193), (2, 20000), (5000, 72)])
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
def test_norm_shapes(gpu_lib, rows, cols, kind):
    t = TYPES[kind]
    x = _data(rows, cols, t, 1 + rows + cols, pitch=cols + cols % 5)
    g = torch.Generator().manual_seed(rows * 31 + cols)
    w = (1 + 0.3 * torch.randn(cols, generator=g)).cuda()
    b = (0.3 * torch.randn(cols, generator=g)).cuda()
    if kind != "fp32" and cols % 2:
        w, b = w.to(t), b.to(t)
    _, mean, rstd = _check_forward(gpu_lib, x, w, b, 1e-5)
    dy = _data(rows, cols, t, 2 + rows + cols, pitch=cols + 3)
    _check_backward(gpu_lib, dy, x, w, mean, rstd)


@pytest.mark.parametrize("with_w,with_b", [(False, False), (True, False), (False, True)])
def test_norm_optional_parameters(gpu_lib, with_w, with_b):
    x = _data(33, 200, torch.bfloat16, 5)
    w = torch.linspace(0.5, 1.5, 200, device="cuda") if with_w else None
    b = torch.linspace(-1, 1, 200, device="cuda") if with_b else None
    _, mean, rstd = _check_forward(gpu_lib, x, w, b, 1e-6)
    _check_backward(gpu_lib, _data(33, 200, torch.bfloat16, 6), x, w, mean, rstd)


@pytest.mark.parametrize("cols", [100, 768, 3000])
def test_norm_large_offset(gpu_lib, cols):
    """A mean a thousand times the deviation: the deviations are summed about the mean."""
    x = _data(17, cols, torch.float32, 8, offset=1000.0)
    _check_forward(gpu_lib, x, None, None, 1e-5)


def test_norm_constant_rows(gpu_lib):
    """A row without deviation: rstd = eps^-1/2, y = bias; zero rows likewise."""
    x = torch.zeros(4, 96, dtype=torch.bfloat16, device="cuda")
    x[1] = 3.0
    x[2] = -0.5
    b = torch.linspace(-1, 1, 96, device="cuda")
    y, mean, rstd = gpu_lib.anvil_layer_norm(x, None, b, 1e-5)
    assert torch.equal(y, b.to(torch.bfloat16).expand(4, 96))
    assert torch.equal(mean.cpu(), torch.tensor([0.0, 3.0, -0.5, 0.0]))
    assert torch.allclose(rstd.cpu(), torch.full((4,), 1e-5 ** -0.5), rtol=4 * U32)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("cols", [96, 768, 3000, 9000])
def test_norm_nonfinite_stays_in_its_row(gpu_lib, bad, cols):
    x = _data(9, cols, torch.bfloat16, 3)
    clean = gpu_lib.anvil_layer_norm(x, None, None, 1e-5)[0].clone()
    x[4, cols // 2] = bad
    y, mean, rstd = gpu_lib.anvil_layer_norm(x, None, None, 1e-5)
    keep = [0, 1, 2, 3, 5, 6, 7, 8]
    assert torch.equal(y[keep], clean[keep])
    assert torch.isnan(y[4]).all()
    dy = _data(9, cols, torch.bfloat16, 4)
    dx, dw, db = gpu_lib.anvil_layer_norm_grad(dy, x, None, mean, rstd)
    assert torch.isfinite(dx[keep]).all() and torch.isnan(dx[4]).any()
    assert torch.isfinite(db).all()


@pytest.mark.parametrize("cols", [40, 9000])
def test_norm_no_rows(gpu_lib, cols):
    x = torch.empty(0, cols, dtype=torch.bfloat16, device="cuda")
    y, mean, rstd = gpu_lib.anvil_layer_norm(x)
    assert y.shape == (0, cols) and mean.numel() == 0
    dx, dw, db = gpu_lib.anvil_layer_norm_grad(x, x, None, mean, rstd)
    assert dx.shape == (0, cols)
    assert torch.count_nonzero(dw) == 0 and torch.count_nonzero(db) == 0


def test_norm_grad_against_differences(gpu_lib):
    """dx, dweight and dbias along random directions against central differences of the 64-bit
    forward: f(x) = sum c y.  The quotient's own error is h^2 times the third derivative, below
    1e-7 here; the gradients carry fp32 errors."""
    g = torch.Generator().manual_seed(11)
    rows, cols, eps, step = 6, 130, 1e-5, 1e-4
    x = torch.randn(rows, cols, generator=g)
    w, b = 1 + 0.2 * torch.randn(cols, generator=g), 0.1 * torch.randn(cols, generator=g)
    c = torch.randn(rows, cols, generator=g)
    xg = x.cuda()
    _, mean, rstd = gpu_lib.anvil_layer_norm(xg, w.cuda(), b.cuda(), eps)
    dx, dw, db = gpu_lib.anvil_layer_norm_grad(c.cuda(), xg, w.cuda(), mean, rstd)

    def f(x, w, b):
        return float((_reference(x, w, b, eps)[0] * c.double()).sum())

    for i in range(4):
        vx = torch.randn(rows, cols, generator=g).double()
        vw, vb = torch.randn(cols, generator=g).double(), torch.randn(cols, generator=g).double()
        X, W, B = x.double(), w.double(), b.double()
        for got, plus, minus, v in (
                (dx, f(X + step * vx, W, B), f(X - step * vx, W, B), vx),
                (dw, f(X, W + step * vw, B), f(X, W - step * vw, B), vw),
                (db, f(X, W, B + step * vb), f(X, W, B - step * vb), vb)):
            want = (plus - minus) / (2 * step)
            scale = float((got.double().cpu().abs() * v.abs()).sum())
            assert abs(float((got.double().cpu() * v).sum()) - want) <= 1e-5 * scale


def test_norm_repeats_bit_for_bit(gpu_lib):
    x = _data(4099, 768, torch.bfloat16, 21)
    dy = _data(4099, 768, torch.bfloat16, 22)
    _, mean, rstd = gpu_lib.anvil_layer_norm(x)
    first = gpu_lib.anvil_layer_norm_grad(dy, x, None, mean, rstd)
    for _ in range(3):
        again = gpu_lib.anvil_layer_norm_grad(dy, x, None, mean, rstd)
        assert all(torch.equal(p, q) for p, q in zip(first, again))


def test_norm_column_ranges_of_one_buffer(gpu_lib):
    """Input and output side by side in one buffer."""
    buf = torch.randn(20, 256, device="cuda").to(torch.bfloat16)
    x, y = buf[:, :100], buf[:, 128:228]
    want = gpu_lib.anvil_layer_norm(x.contiguous())[0]
    left = buf[:, :128].clone()
    right = buf[:, 228:].clone()
    gpu_lib.anvil_layer_norm(x, out=y)
    assert torch.equal(y, want)
    assert torch.equal(buf[:, :128], left) and torch.equal(buf[:, 228:], right)
    with pytest.raises(gpu_lib.AnvilError) as err:
        gpu_lib.anvil_layer_norm(x, out=buf[:, 50:150])
    assert err.value.status == gpu_lib.ANVIL_ERR_ALIAS


def test_norm_past_32_bit_offsets(gpu_lib):
    """Rows whose elements lie past 2^31 elements (and 2^32 bytes) from the first."""
    pitch, rows, cols = 1 << 20, 2100, 96
    big = torch.empty(rows * pitch, dtype=torch.bfloat16, device="cuda")
    x = big.view(rows, pitch)[:, 8:8 + cols]
    x.copy_(_data(rows, cols, torch.bfloat16, 31))
    y, mean, rstd = gpu_lib.anvil_layer_norm(x)
    want, m2, r2 = gpu_lib.anvil_layer_norm(x.contiguous())
    assert torch.equal(y, want) and torch.equal(mean, m2) and torch.equal(rstd, r2)
    dy = _data(rows, cols, torch.bfloat16, 32)
    got = gpu_lib.anvil_layer_norm_grad(dy, x, None, mean, rstd)
    ref = gpu_lib.anvil_layer_norm_grad(dy, x.contiguous(), None, mean, rstd)
    assert all(torch.equal(p, q) for p, q in zip(got, ref))


def test_norm_on_another_stream_and_in_a_graph(gpu_lib):
    x = _data(300, 768, torch.bfloat16, 41)
    dy = _data(300, 768, torch.bfloat16, 42)
    w = torch.linspace(0.5, 1.5, 768, device="cuda")
    y0, mean, rstd = gpu_lib.anvil_layer_norm(x, w)
    g0 = gpu_lib.anvil_layer_norm_grad(dy, x, w, mean, rstd)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y1 = gpu_lib.anvil_layer_norm(x, w, stream=s)[0]
    g1 = gpu_lib.anvil_layer_norm_grad(dy, x, w, mean, rstd, stream=s)
    s.synchronize()
    assert torch.equal(y0, y1) and all(torch.equal(p, q) for p, q in zip(g0, g1))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, m2, r2 = gpu_lib.anvil_layer_norm(x, w)
        g2 = gpu_lib.anvil_layer_norm_grad(dy, x, w, m2, r2)
    for seed in (43, 44, 45):
        x.copy_(_data(300, 768, torch.bfloat16, seed))
        graph.replay()
        torch.cuda.synchronize()
        ye, me, re = gpu_lib.anvil_layer_norm(x, w)
        ge = gpu_lib.anvil_layer_norm_grad(dy, x, w, me, re)
        assert torch.equal(y2, ye) and all(torch.equal(p, q) for p, q in zip(g2, ge))
