"""Linear layers (bias, activation, residual in the epilogue), their two gradient products and the
same over a stack of experts, on the GPU against plain forms in 64 bits."""
import pytest
import torch

from tests import layer_helpers as H

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _mat(rows, cols, t, seed, scale=1.0, pitch=None, shift=0):
    """[rows, cols] on the GPU: rows `pitch` apart, the first at element `shift` of a buffer that
    holds NaN everywhere else."""
    g = torch.Generator().manual_seed(seed)
    pitch = pitch or cols
    buf = torch.full((max(rows, 1) * pitch + shift + cols,), float("nan"), dtype=t, device="cuda")
    view = buf[shift:].as_strided((rows, cols), (pitch, 1))
    view.copy_((torch.randn(rows, cols, generator=g) * scale).to(t))
    return view


def _stack(e, n, k, t, seed, w_kn):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(e, *((k, n) if w_kn else (n, k)), generator=g) * max(k, 1) ** -0.5
    return w.to(t).cuda()


def _nan(*shape, t):
    return torch.full(shape, float("nan"), dtype=t, device="cuda")


def _check_forward(gpu_lib, x, w, bias, residual, act, w_kn, keep, t):
    rows, n = x.shape[0], w.shape[-1 if w_kn else -2]
    out = _nan(rows, n, t=t)
    pre = _nan(rows, n, t=t) if keep else None
    y, z = gpu_lib.anvil_linear(x, w, bias, residual=residual, act=act, w_kn=w_kn, preact=pre, out=out)
    torch.cuda.synchronize()
    cpu = lambda v: None if v is None else v.cpu()  # noqa: E731
    want, zw, ez = H.linear(x.cpu(), w.cpu(), cpu(bias), cpu(residual), act, w_kn)
    if keep:
        H.assert_within(z, zw, ez + H.half_step(zw, t), "preactivation")
    ey = H.forward_error(zw, ez, want, residual, act)
    H.assert_within(y, want, ey + H.half_step(want, t), "y")


def _check_backward(gpu_lib, dz, x, w, preact, add, act, w_kn, t):
    rows, n = dz.shape
    k = x.shape[1]
    dx = gpu_lib.anvil_linear_grad_input(dz, w, preact=preact, act=act, add=add, w_kn=w_kn,
                                         out=_nan(rows, k, t=t))
    torch.cuda.synchronize()
    cpu = lambda v: None if v is None else v.cpu()  # noqa: E731
    want, err = H.grad_input(dz.cpu(), w.cpu(), cpu(preact), act, cpu(add), w_kn)
    H.assert_within(dx, want, err + H.half_step(want, t), "dx")
    for out_t in (torch.float32, t):
        dw, db = gpu_lib.anvil_linear_grad_weight(dz, x, w_kn=w_kn, out=_nan(*w.shape, t=out_t))
        torch.cuda.synchronize()
        (ww, ew), (bw, eb) = H.grad_weight(dz.cpu(), x.cpu(), w_kn)
        H.assert_within(dw, ww, ew + H.half_step(ww, out_t), f"dw {out_t}")
        H.assert_within(db, bw, eb + 1e-45, "db")


# one row to more rows than a tile; widths below, at and past the tiles, odd ones, and one feature
SHAPES = [(1, 768, 256), (1, 1, 1), (2, 8, 8), (5, 72, 40), (17, 264, 136), (32, 64, 512), (33, 130, 67),
          (64, 64, 64), (65, 1, 300), (96, 300, 1), (130, 257, 515), (200, 768, 96), (257, 264, 520),
          (520, 520, 264), (1000, 40, 24), (300, 1024, 768)]


@pytest.mark.parametrize("rows,n,k", SHAPES)
@pytest.mark.parametrize("w_kn", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_linear_shapes(gpu_lib, rows, n, k, w_kn, kind):
    t = TYPES[kind]
    seed = rows * 7 + n * 3 + k
    act = H.ACTS[seed % 5]
    x = _mat(rows, k, t, seed)
    w = _stack(1, n, k, t, seed + 1, w_kn)[0]
    bias = torch.randn(n, generator=torch.Generator().manual_seed(seed + 2)).cuda()
    if seed % 2:
        bias = bias.to(t)
    residual = _mat(rows, n, t, seed + 3) if seed % 3 else None
    _check_forward(gpu_lib, x, w, bias, residual, act, w_kn, seed % 4 < 2, t)
    dz = _mat(rows, n, t, seed + 4, 0.1)
    add = _mat(rows, k, t, seed + 6, 0.1) if seed % 2 else None
    _check_backward(gpu_lib, dz, x, w, _mat(rows, k, t, seed + 5), add, act, w_kn, t)


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("n,k", [(768, 2816), (2816, 768), (4104, 200), (37, 1001), (5, 7), (4099, 513), (8, 4096)])
@pytest.mark.parametrize("w_kn", [False, True])
def test_linear_few_rows(gpu_lib, rows, n, k, w_kn):
    """Single tokens and a few: depths of less and more than a pass, ragged columns."""
    t = torch.float16 if n == 2816 else torch.bfloat16
    x = _mat(rows, k, t, 1, pitch=k + 3 if rows % 2 else k)
    w = _stack(1, n, k, t, 2, w_kn)[0]
    bias = torch.randn(n, generator=torch.Generator().manual_seed(3)).cuda()
    _check_forward(gpu_lib, x, w, bias, _mat(rows, n, t, 4), "silu", w_kn, True, t)
    _check_backward(gpu_lib, _mat(rows, n, t, 5, 0.1), x, w, _mat(rows, k, t, 6), _mat(rows, k, t, 7), "gelu", w_kn, t)


# enough tiles for the larger tile shapes, with ragged last rows, columns and depths
@pytest.mark.parametrize("rows,n,k", [(2100, 2000, 72), (5000, 2600, 136), (4100, 3336, 64), (700, 1288, 1032)])
@pytest.mark.parametrize("w_kn", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_linear_large_tiles(gpu_lib, rows, n, k, w_kn, kind):
    t = TYPES[kind]
    x, dz = _mat(rows, k, t, 1), _mat(rows, n, t, 4, 0.1)
    w = _stack(1, n, k, t, 2, w_kn)[0]
    bias = torch.randn(n, generator=torch.Generator().manual_seed(3)).cuda()
    _check_forward(gpu_lib, x, w, bias, _mat(rows, n, t, 5), "relu2", w_kn, True, t)
    _check_backward(gpu_lib, dz, x, w, _mat(rows, k, t, 6), None, "silu", w_kn, t)
    # the wide input gradient: the same tiles with the roles of n and k exchanged
    w2 = _stack(1, k, n, t, 7, w_kn)[0]
    dx = gpu_lib.anvil_linear_grad_input(x, w2, preact=dz, act="gelu", w_kn=w_kn, out=_nan(rows, n, t=t))
    want, err = H.grad_input(x.cpu(), w2.cpu(), dz.cpu(), "gelu", None, w_kn)
    H.assert_within(dx, want, err + H.half_step(want, t), "dx")


# widths that are no multiples of eight, with tiles for every CU and without
@pytest.mark.parametrize("rows,n,k", [(2100, 2003, 77), (4400, 1027, 130), (1500, 1285, 1601), (9000, 131, 203)])
@pytest.mark.parametrize("w_kn", [False, True])
def test_linear_large_odd(gpu_lib, rows, n, k, w_kn):
    t = torch.bfloat16
    x, dz = _mat(rows, k, t, 1), _mat(rows, n, t, 4, 0.1)
    w = _stack(1, n, k, t, 2, w_kn)[0]
    bias = torch.randn(n, generator=torch.Generator().manual_seed(3)).cuda()
    _check_forward(gpu_lib, x, w, bias, _mat(rows, n, t, 5), "gelu", w_kn, True, t)
    _check_backward(gpu_lib, dz, x, w, _mat(rows, k, t, 6), None, "relu2", w_kn, t)


@pytest.mark.parametrize("w_kn", [False, True])
def test_expert_large_odd(gpu_lib, w_kn):
    _expert_case(gpu_lib, 4900, [0, 700, 700, 1399, 1800, 2900, 3333, 4000, 4890], 1031, 131, w_kn, torch.bfloat16,
                 "silu", True)


@pytest.mark.parametrize("act", H.ACTS)
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("rows", [3, 300])
def test_linear_activations(gpu_lib, act, kind, rows):
    """Every activation over a wide range of preactivations, in both directions."""
    t = TYPES[kind]
    n, k = 136, 64
    x = _mat(rows, k, t, 50, 4.0)
    w = _stack(1, n, k, t, 51, False)[0]
    _check_forward(gpu_lib, x, w, None, _mat(rows, n, t, 52), act, False, True, t)
    _check_backward(gpu_lib, _mat(rows, n, t, 53), x, w, _mat(rows, k, t, 54, 4.0), None, act, False, t)


@pytest.mark.parametrize("w_kn", [False, True])
@pytest.mark.parametrize("rows,n,k,pad,shift", [(70, 264, 128, 8, 8), (70, 264, 128, 3, 0), (300, 128, 264, 0, 1),
                                                (300, 512, 256, 16, 16), (9, 256, 768, 5, 3)])
def test_linear_pitches_and_alignments(gpu_lib, rows, n, k, pad, shift, w_kn):
    t = torch.bfloat16
    x = _mat(rows, k, t, 60, pitch=k + pad, shift=shift)
    w = _stack(1, n, k, t, 61, w_kn)[0]
    res = _mat(rows, n, t, 62, pitch=n + 2 * pad, shift=shift)
    big_y, big_z = _nan(rows, n + pad, t=t), _nan(rows, n + 3 * pad, t=t)
    y, z = gpu_lib.anvil_linear(x, w, None, residual=res, act="silu", w_kn=w_kn, out=big_y[:, :n],
                                preact=big_z[:, 3 * pad:])
    y2, z2 = gpu_lib.anvil_linear(x.contiguous(), w, None, residual=res.contiguous(), act="silu", w_kn=w_kn,
                                  keep_preact=True)
    torch.cuda.synchronize()
    want, zw, ez = H.linear(x.cpu(), w.cpu(), None, res.cpu(), "silu", w_kn)
    H.assert_within(z, zw, ez + H.half_step(zw, t), "z")
    H.assert_within(y, want, H.forward_error(zw, ez, want, res, "silu") + H.half_step(want, t), "y")
    H.assert_within(y2, want, H.forward_error(zw, ez, want, res, "silu") + H.half_step(want, t), "y2")
    assert torch.isnan(big_y[:, n:]).all() and torch.isnan(big_z[:, :3 * pad]).all()
    dz = _mat(rows, n, t, 63, pitch=n + pad, shift=shift)
    pre = _mat(rows, k, t, 64, pitch=k + pad, shift=shift)
    _check_backward(gpu_lib, dz, x, w, pre, x, "gelu", w_kn, t)


@pytest.mark.parametrize("rows,n,k", [(0, 64, 64), (40, 64, 0), (40, 0, 64), (0, 33, 7)])
@pytest.mark.parametrize("w_kn", [False, True])
def test_linear_empty_sides(gpu_lib, rows, n, k, w_kn):
    """No depth: z is the bias alone and dw is empty; no rows: dw and db are zeros."""
    t = torch.bfloat16
    x, w = _mat(rows, k, t, 1), _stack(1, n, k, t, 2, w_kn)[0]
    b = torch.linspace(-1, 1, n, device="cuda") if n else torch.empty(0, device="cuda")
    y, z = gpu_lib.anvil_linear(x, w, b, act="relu", w_kn=w_kn, keep_preact=True)
    assert y.shape == (rows, n)
    if rows and n and k == 0:
        assert torch.equal(z, b.to(t).expand(rows, n)) and torch.equal(y, torch.relu(b).to(t).expand(rows, n))
    dz = _mat(rows, n, t, 3)
    dx = gpu_lib.anvil_linear_grad_input(dz, w, w_kn=w_kn)
    assert dx.shape == (rows, k) and (n > 0 or torch.count_nonzero(dx) == 0)
    dw, db = gpu_lib.anvil_linear_grad_weight(dz, x, w_kn=w_kn)
    if rows == 0:
        assert torch.count_nonzero(dw) == 0 and torch.count_nonzero(db) == 0


@pytest.mark.parametrize("rows,n,k", [(3000, 264, 136), (8200, 64, 520), (5000, 33, 77), (20000, 72, 64)])
@pytest.mark.parametrize("w_kn", [False, True])
def test_weight_gradient_over_many_rows(gpu_lib, rows, n, k, w_kn):
    """Row counts that are split over workgroups and joined."""
    t = torch.bfloat16
    dz, x = _mat(rows, n, t, 71, 0.1), _mat(rows, k, t, 72)
    dw, db = gpu_lib.anvil_linear_grad_weight(dz, x, w_kn=w_kn)
    (ww, ew), (bw, eb) = H.grad_weight(dz.cpu(), x.cpu(), w_kn)
    H.assert_within(dw, ww, ew + H.half_step(ww, torch.float32), "dw")
    H.assert_within(db, bw, eb, "db")
    again = gpu_lib.anvil_linear_grad_weight(dz, x, w_kn=w_kn)
    assert torch.equal(dw, again[0]) and torch.equal(db, again[1])
    none = gpu_lib.anvil_linear_grad_weight(dz, x, w_kn=w_kn, want_bias=False)
    assert none[1] is None and torch.equal(none[0], dw)


@pytest.mark.parametrize("rows,n,k", [(5, 64, 64), (300, 264, 128), (40, 33, 7)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_linear_nonfinite_stays_in_its_row(gpu_lib, rows, n, k, bad):
    t = torch.bfloat16
    x, w = _mat(rows, k, t, 81), _stack(1, n, k, t, 82, False)[0]
    clean = gpu_lib.anvil_linear(x, w, act="relu2")[0].clone()
    x[2, k // 2] = bad
    y, z = gpu_lib.anvil_linear(x, w, act="relu2", keep_preact=True)
    keep = [i for i in range(rows) if i != 2]
    assert torch.equal(y[keep], clean[keep])
    want = x[2].double() @ w.double().t()
    assert torch.equal(torch.isnan(z[2]), torch.isnan(want)) and not torch.isfinite(z[2]).any()
    assert torch.equal(torch.isnan(y[2]), torch.isnan(want))


@pytest.mark.parametrize("act", H.ACTS)
@pytest.mark.parametrize("rows,n", [(1, 1), (3, 8), (70, 768), (9, 77)])
def test_activation_grad(gpu_lib, act, rows, n):
    for t in (torch.bfloat16, torch.float16):
        dy, z = _mat(rows, n, t, 91, pitch=n + 5), _mat(rows, n, t, 92, 3.0, pitch=n + 2, shift=1)
        dz = gpu_lib.anvil_activation_grad(dy, z, act)
        s = H.act_slope(z.cpu().double(), act)
        want = dy.cpu().double() * s
        H.assert_within(dz, want, 32 * H.U32 * want.abs() + 8 * H.U32 * dy.cpu().double().abs()
                        + H.half_step(want, t), "dz")


def test_linear_grads_against_differences(gpu_lib):
    """The gradients of f = sum c y, y = act(x w^T + b) with x = act0(p), along random directions
    against central differences of the 64-bit forward.  The kernels round each of the entries they
    return to 16 bits (or sum fp32), so their inner product with a direction is off by a random sum of
    half steps: 2^-8 of the root of the summed squares, times four."""
    g = torch.Generator().manual_seed(5)
    rows, n, k, step = 40, 48, 64, 1e-4
    t = torch.bfloat16
    for name in ("gelu", "silu"):
        p = torch.randn(rows, k, generator=g).to(t)
        w = (torch.randn(n, k, generator=g) * k ** -0.5).to(t)
        b = torch.randn(n, generator=g)
        c = torch.randn(rows, n, generator=g).to(t)
        x = H.act(p.double(), name).to(t)
        _, z = gpu_lib.anvil_linear(x.cuda(), w.cuda(), b.cuda(), act=name, keep_preact=True)
        dz = gpu_lib.anvil_activation_grad(c.cuda(), z, name)
        dp = gpu_lib.anvil_linear_grad_input(dz, w.cuda(), preact=p.cuda(), act=name)
        dw, db = gpu_lib.anvil_linear_grad_weight(dz, x.cuda())

        def f(p, w, b):
            return float((H.act(H.act(p, name) @ w.t() + b, name) * c.double()).sum())

        P, W, B = p.double(), w.double(), b.double()
        for got, at in ((dp, 0), (dw, 1), (db, 2)):
            v = torch.randn(got.shape, generator=g).double()
            plus = [a + step * v if i == at else a for i, a in enumerate((P, W, B))]
            minus = [a - step * v if i == at else a for i, a in enumerate((P, W, B))]
            want = (f(*plus) - f(*minus)) / (2 * step)
            mine = got.double().cpu()
            # rounded: x, z and dz before it (each moves an entry of the sum by up to 2^-8 of its
            # size, independently), and the result itself
            tol = 4 * 4 * 2.0 ** -8 * float((mine * v).square().sum().sqrt())
            assert abs(float((mine * v).sum()) - want) <= tol, (name, at)


# ------------------------------------------------------------------------------------------------
# experts
# ------------------------------------------------------------------------------------------------

GROUPS = {
    "even": [0, 40, 80, 120, 160],
    "ragged": [0, 1, 1, 70, 199, 200, 333],
    "empty_ends": [0, 0, 0, 129, 129, 129],
    "gaps": [5, 37, 37, 100],                      # rows before the first and after the last
    "one": [0, 257],
    "none": [0, 0, 0],
    "bad": [-7, 60, 20, 90, 1 << 30, 100],          # decreasing, negative, past the rows
    "many": list(range(0, 391, 3)),
}
ROWS = {"even": 160, "ragged": 333, "empty_ends": 140, "gaps": 131, "one": 257, "none": 20, "bad": 150,
        "many": 400}


def _expert_case(gpu_lib, rows, offsets, n, k, w_kn, t, act, wide, keep=True):
    e = len(offsets) - 1
    off = torch.tensor(offsets, dtype=torch.int64 if wide else torch.int32, device="cuda")
    seed = rows + n + k
    x, dz = _mat(rows, k, t, seed), _mat(rows, n, t, seed + 1, 0.1)
    w = _stack(e, n, k, t, seed + 2, w_kn)
    bias = torch.randn(e, n, generator=torch.Generator().manual_seed(seed)).cuda()
    res, pre = _mat(rows, n, t, seed + 3), _mat(rows, k, t, seed + 4)
    y, z = gpu_lib.anvil_expert_linear(x, w, off, bias, residual=res, act=act, w_kn=w_kn,
                                       preact=_nan(rows, n, t=t) if keep else None, out=_nan(rows, n, t=t))
    dx = gpu_lib.anvil_expert_grad_input(dz, w, off, preact=pre, act=act, add=x, w_kn=w_kn, out=_nan(rows, k, t=t))
    dw, db = gpu_lib.anvil_expert_grad_weight(dz, x, off, w_kn=w_kn, out=_nan(*w.shape, t=torch.float32))
    torch.cuda.synchronize()
    b = H.clamp_offsets(offsets, rows)
    owned = torch.zeros(rows, dtype=torch.bool)
    for i in range(e):
        s = slice(b[i], b[i + 1])
        owned[s] = True
        if b[i + 1] > b[i]:
            want, zw, ez = H.linear(x[s].cpu(), w[i].cpu(), bias[i].cpu(), res[s].cpu(), act, w_kn)
            if keep:
                H.assert_within(z[s], zw, ez + H.half_step(zw, t), f"z {i}")
            H.assert_within(y[s], want, H.forward_error(zw, ez, want, res, act) + H.half_step(want, t), f"y {i}")
            want, err = H.grad_input(dz[s].cpu(), w[i].cpu(), pre[s].cpu(), act, x[s].cpu(), w_kn)
            H.assert_within(dx[s], want, err + H.half_step(want, t), f"dx {i}")
        (ww, ew), (bw, eb) = H.grad_weight(dz[s].cpu(), x[s].cpu(), w_kn)
        H.assert_within(dw[i], ww, ew + H.half_step(ww, torch.float32), f"dw {i}")
        H.assert_within(db[i], bw, eb + 1e-45, f"db {i}")
    free = (~owned).nonzero()[:, 0].cuda()
    for v, what in ((y, "y"), (dx, "dx")) + (((z, "z"),) if keep else ()):
        assert torch.count_nonzero(v[free]) == 0 and not torch.isnan(v[free]).any(), what


@pytest.mark.parametrize("groups", list(GROUPS))
@pytest.mark.parametrize("w_kn", [False, True])
@pytest.mark.parametrize("n,k", [(136, 72), (264, 512), (67, 33)])
def test_expert_groups(gpu_lib, groups, w_kn, n, k):
    t = torch.float16 if n == 136 else torch.bfloat16
    _expert_case(gpu_lib, ROWS[groups], GROUPS[groups], n, k, w_kn, t, H.ACTS[(n + len(groups)) % 5],
                 wide=w_kn, keep=n != 264)


@pytest.mark.parametrize("w_kn", [False, True])
def test_expert_large_groups(gpu_lib, w_kn):
    """Groups longer than a tile and a split, one of them most of the rows, one empty."""
    _expert_case(gpu_lib, 6000, [0, 4096, 4100, 4100, 5999], 264, 520, w_kn, torch.bfloat16, "relu2", False)


@pytest.mark.parametrize("experts", [2, 31, 61, 62, 63, 64, 65, 126, 127, 130])
@pytest.mark.parametrize("rows", [40, 3000])
def test_expert_counts(gpu_lib, experts, rows):
    """Group counts around one wave's 64 lanes, uneven groups, rows before and after them, and row
    counts that give few-row tiles and full ones."""
    g = torch.Generator().manual_seed(experts)
    cuts = torch.sort(torch.randint(1, rows - 2, (experts + 1,), generator=g))[0].tolist()
    _expert_case(gpu_lib, rows, cuts, 72, 136, experts % 2 == 0, torch.bfloat16, "silu", experts % 3 == 0)


@pytest.mark.parametrize("w_kn", [False, True])
@pytest.mark.parametrize("n,k", [(2304, 136), (1032, 1288)])
def test_expert_large_tiles(gpu_lib, w_kn, n, k):
    """Enough tiles for the largest tile shapes, groups that end inside them."""
    _expert_case(gpu_lib, 4900, [0, 700, 700, 1399, 1800, 2900, 3333, 4000, 4900], n, k, w_kn, torch.bfloat16,
                 "silu", True)


def test_expert_without_experts(gpu_lib):
    x = _mat(12, 16, torch.bfloat16, 1)
    off = torch.zeros(1, dtype=torch.int32, device="cuda")
    w = torch.empty(0, 24, 16, dtype=torch.bfloat16, device="cuda")
    y, _ = gpu_lib.anvil_expert_linear(x, w, off, out=_nan(12, 24, t=torch.bfloat16))
    assert torch.count_nonzero(y) == 0 and not torch.isnan(y).any()
    dw, db = gpu_lib.anvil_expert_grad_weight(_mat(12, 24, torch.bfloat16, 2), x, off)
    assert dw.shape == (0, 24, 16) and db.shape == (0, 24)


def test_experts_equal_single_layers(gpu_lib):
    """Each group alone through the single-matrix entry points, element for element within the two
    results' rounding (their tiles, and so their sums' order, may differ)."""
    t = torch.bfloat16
    offs = [0, 300, 300, 812, 1000]
    off = torch.tensor(offs, dtype=torch.int32, device="cuda")
    x, w = _mat(1000, 256, t, 5), _stack(4, 768, 256, t, 6, False)
    y, _ = gpu_lib.anvil_expert_linear(x, w, off, act="relu2")
    for i in range(4):
        s = slice(offs[i], offs[i + 1])
        if offs[i + 1] > offs[i]:
            one = gpu_lib.anvil_linear(x[s], w[i], act="relu2")[0].double()
            assert ((y[s].double() - one).abs() <= 2.0 ** -7 * one.abs() + 1e-5).all()


# ------------------------------------------------------------------------------------------------
# streams, graphs, far offsets
# ------------------------------------------------------------------------------------------------

def _block(lib, x, w1, w2, off, b1, stream=None):
    kw = {"stream": stream}
    h, z = lib.anvil_expert_linear(x, w1, off, b1, act="relu2", keep_preact=True, **kw)
    y, _ = lib.anvil_expert_linear(h, w2, off, residual=x, w_kn=True, **kw)
    dz1 = lib.anvil_expert_grad_input(y, w2, off, preact=z, act="relu2", w_kn=True, **kw)
    dw2, db2 = lib.anvil_expert_grad_weight(y, h, off, w_kn=True, **kw)
    dw1, db1 = lib.anvil_expert_grad_weight(dz1, x, off, **kw)
    return y, dz1, dw1, db1, dw2, db2


def test_layers_on_another_stream_and_in_a_graph(gpu_lib):
    t = torch.bfloat16
    x = _mat(700, 256, t, 1)
    w1, w2 = _stack(3, 520, 256, t, 2, False), _stack(3, 256, 520, t, 3, True)
    off = torch.tensor([0, 100, 500, 700], dtype=torch.int32, device="cuda")
    b1 = torch.randn(3, 520, device="cuda")
    eager = _block(gpu_lib, x, w1, w2, off, b1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = _block(gpu_lib, x, w1, w2, off, b1, stream=s)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(eager, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = _block(gpu_lib, x, w1, w2, off, b1)
    for i, offs in enumerate(([0, 100, 500, 700], [0, 0, 699, 700], [30, 31, 400, 512])):
        x.copy_(_mat(700, 256, t, 20 + i))
        off.copy_(torch.tensor(offs, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        now = _block(gpu_lib, x, w1, w2, off, b1)
        assert all(torch.equal(p, q) for p, q in zip(held, now)), i


@pytest.mark.parametrize("k", [64, 67])
def test_linear_past_32_bit_offsets(gpu_lib, k):
    """Activations whose rows lie past 2^31 elements from the first, as input, output and gradient."""
    t = torch.bfloat16
    pitch, rows, n = 1 << 20, 2300, 72
    big = torch.empty(rows * pitch, dtype=t, device="cuda").view(rows, pitch)
    x, out = big[:, :k], big[:, 1024:1024 + n]
    x.copy_(_mat(rows, k, t, 1))
    w = _stack(1, n, k, t, 2, False)[0]
    gpu_lib.anvil_linear(x, w, act="silu", out=out)
    want = gpu_lib.anvil_linear(x.contiguous(), w, act="silu")[0]
    assert torch.equal(out, want)
    dz = big[:, 2048:2048 + n]
    dz.copy_(_mat(rows, n, t, 3, 0.1))
    dw, db = gpu_lib.anvil_linear_grad_weight(dz, x)
    (ww, ew), (bw, eb) = H.grad_weight(dz.cpu(), x.cpu(), False)
    H.assert_within(dw, ww, ew + H.half_step(ww, torch.float32), "dw")
    H.assert_within(db, bw, eb, "db")


def test_caller_workspace(gpu_lib):
    t = torch.bfloat16
    dz, x = _mat(4096, 64, t, 1, 0.1), _mat(4096, 128, t, 2)
    need = gpu_lib.load().anvil_linear_grad_weight_workspace(0, 4096, 64, 128, 1)
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    a = gpu_lib.anvil_linear_grad_weight(dz, x, workspace=ws)
    b = gpu_lib.anvil_linear_grad_weight(dz, x)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(gpu_lib.AnvilError):
        gpu_lib.anvil_linear_grad_weight(dz, x, workspace=ws[:need - 256])
