"""The gated linear layer (two projections, activation and product in one kernel), its gradient through the layer
that follows, elementwise and over experts, on the GPU against plain forms in 64 bits."""
import pytest
import torch

from tests import gated_helpers as G
from tests import layer_helpers as H

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _mat(rows, cols, t, seed, scale=1.0, pitch=None, shift=0):
    """[rows, cols] on the GPU, rows `pitch` apart from element `shift` of a buffer of NaN on."""
    g = torch.Generator().manual_seed(seed)
    pitch = pitch or cols
    buf = torch.full((max(rows, 1) * pitch + shift + cols,), float("nan"), dtype=t, device="cuda")
    view = buf[shift:].as_strided((rows, cols), (pitch, 1))
    view.copy_((torch.randn(rows, cols, generator=g) * scale).to(t))
    return view


def _weight(n, k, t, seed, w_kn, stack=()):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*stack, *((k, n) if w_kn else (n, k)), generator=g) * max(k, 1) ** -0.5).to(t).cuda()


def _nan(*shape, t):
    return torch.full(shape, float("nan"), dtype=t, device="cuda")


def _check_forward(lib, x, w, bias, act, w_kn, keep, t):
    rows, both = x.shape[0], w.shape[-1 if w_kn else -2]
    pre = _nan(rows, both, t=t) if keep else None
    y, z = lib.anvil_gated_linear(x, w, bias, act=act, w_kn=w_kn, preact=pre, out=_nan(rows, both // 2, t=t))
    torch.cuda.synchronize()
    h, eh, zw, ez = G.forward(x.cpu(), w.cpu(), None if bias is None else bias.cpu(), act, w_kn)
    H.assert_within(y, h, eh + H.half_step(h, t), "y")
    if keep:
        H.assert_within(z, zw, ez + H.half_step(zw, t), "z")
    else:
        assert z is None


def _check_grad(lib, dy, w, z, act, w_kn, t):
    rows, k = dy.shape[0], z.shape[1] // 2
    dz = lib.anvil_gated_grad_input(dy, w, z, act=act, w_kn=w_kn, out=_nan(rows, 2 * k, t=t))
    torch.cuda.synchronize()
    want, err = G.grad(dy.cpu(), w.cpu(), z.cpu(), act, w_kn)
    H.assert_within(dz, want, err + H.half_step(want, t), "dz")


# one row to more rows than a tile; widths below, at and past the tiles' halves, odd ones, and one feature
SHAPES = [(1, 768, 256), (1, 1, 1), (2, 8, 8), (5, 72, 40), (17, 264, 136), (32, 32, 512), (33, 130, 67), (64, 64, 64),
          (65, 1, 300), (96, 300, 1), (130, 257, 515), (200, 768, 96), (257, 264, 520), (520, 520, 264), (1000, 40, 24)]


@pytest.mark.parametrize("rows,n,k", SHAPES)
@pytest.mark.parametrize("w_kn", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_shapes(gpu_lib, rows, n, k, w_kn, kind):
    t = TYPES[kind]
    seed = rows * 7 + n * 3 + k
    act = H.ACTS[seed % 5]
    bias = torch.randn(2 * n, generator=torch.Generator().manual_seed(seed)).cuda()
    bias = (bias, bias.to(t), None)[seed % 3]
    _check_forward(gpu_lib, _mat(rows, k, t, seed + 1), _weight(2 * n, k, t, seed + 2, w_kn), bias, act, w_kn, seed % 2 == 0, t)
    _check_grad(gpu_lib, _mat(rows, k, t, seed + 3, 0.1), _weight(k, n, t, seed + 4, w_kn), _mat(rows, 2 * n, t, seed + 5), act,
                w_kn, t)


@pytest.mark.parametrize("act", H.ACTS)
@pytest.mark.parametrize("n,k", [(136, 72), (67, 45)])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_activations(gpu_lib, act, n, k, kind):
    t = TYPES[kind]
    _check_forward(gpu_lib, _mat(70, k, t, 1, 3.0), _weight(2 * n, k, t, 2, False), None, act, False, True, t)
    z = _mat(70, 2 * n, t, 5, 3.0)
    _check_grad(gpu_lib, _mat(70, k, t, 3, 0.1), _weight(k, n, t, 4, False), z, act, False, t)
    dh = _mat(70, n, t, 6)
    got = gpu_lib.anvil_gated_activation_grad(dh, z, act=act, out=_nan(70, 2 * n, t=t))
    want, err = G.grad_from(dh.double().cpu(), torch.zeros(()), z.cpu(), act)
    H.assert_within(got, want, err + H.half_step(want, t), "dz of dh")


# enough tiles for the larger shapes, with ragged last rows, columns and depths, and odd widths
@pytest.mark.parametrize("rows,n,k", [(2100, 1000, 72), (5000, 1304, 136), (4100, 1672, 64), (700, 648, 1032), (2100, 1003, 77),
                                      (4400, 515, 130)])
@pytest.mark.parametrize("w_kn", [False, True])
def test_large_tiles(gpu_lib, rows, n, k, w_kn):
    t = torch.bfloat16 if n % 3 else torch.float16
    bias = torch.randn(2 * n, generator=torch.Generator().manual_seed(3)).cuda()
    _check_forward(gpu_lib, _mat(rows, k, t, 1), _weight(2 * n, k, t, 2, w_kn), bias, "gelu", w_kn, True, t)
    _check_grad(gpu_lib, _mat(rows, k, t, 3, 0.1), _weight(k, n, t, 4, w_kn), _mat(rows, 2 * n, t, 5), "silu", w_kn, t)


@pytest.mark.parametrize("pitch,shift", [(0, 0), (8, 8), (3, 1), (1, 0), (0, 5)])
@pytest.mark.parametrize("n,k", [(128, 64), (65, 33)])
def test_pitches_and_alignment(gpu_lib, pitch, shift, n, k):
    """Rows any pitch apart from any element on; what lies between them is neither read nor written."""
    t, rows = torch.bfloat16, 50
    x, z = _mat(rows, k, t, 1, pitch=k + pitch, shift=shift), _mat(rows, 2 * n, t, 5, pitch=2 * n + pitch, shift=shift)
    w, down = _weight(2 * n, k, t, 2, False), _weight(k, n, t, 4, True)
    _check_forward(gpu_lib, x, w, None, "silu", False, True, t)
    _check_grad(gpu_lib, _mat(rows, k, t, 3, 0.1, pitch=k + pitch, shift=shift), down, z, "silu", True, t)
    buf = _nan(rows * (n + pitch) + shift, t=t)
    out = buf[shift:].as_strided((rows, n), (n + pitch, 1))
    gpu_lib.anvil_gated_linear(x, w, out=out)
    assert torch.equal(out, gpu_lib.anvil_gated_linear(x.contiguous(), w)[0])
    rest = torch.ones_like(buf, dtype=torch.bool)
    rest[shift:].as_strided((rows, n), (n + pitch, 1)).fill_(False)
    assert torch.isnan(buf[rest]).all()


@pytest.mark.parametrize("n,k", [(136, 72), (67, 45)])
@pytest.mark.parametrize("w_kn", [False, True])
@pytest.mark.parametrize("offsets", [[0, 10, 10, 200, 260], [5, 37, 37, 100, 200], [0, 0, 0, 0, 260], [-7, 60, 20, 90, 1 << 30]])
def test_experts(gpu_lib, n, k, w_kn, offsets):
    """Each group through its own weights; rows without an expert give zeros, whatever z holds there."""
    t, rows, e = torch.bfloat16, 260, len(offsets) - 1
    for bits in (torch.int32, torch.int64):
        off = torch.tensor(offsets, dtype=bits, device="cuda")
        ends = H.clamp_offsets(offsets, rows)
        x, dy, z = _mat(rows, k, t, 1), _mat(rows, k, t, 2, 0.1), _mat(rows, 2 * n, t, 3)
        z[:ends[0]] = float("inf")
        w, down = _weight(2 * n, k, t, 4, w_kn, (e,)), _weight(k, n, t, 5, w_kn, (e,))
        bias = torch.randn(e, 2 * n, generator=torch.Generator().manual_seed(6)).cuda()
        y, zz = gpu_lib.anvil_expert_gated_linear(x, w, off, bias, act="silu", w_kn=w_kn, preact=_nan(rows, 2 * n, t=t),
                                                  out=_nan(rows, n, t=t))
        dz = gpu_lib.anvil_expert_gated_grad_input(dy, down, off, z, act="silu", w_kn=w_kn, out=_nan(rows, 2 * n, t=t))
        for part in (y, zz, dz):
            assert not part[:ends[0]].any() and not part[ends[-1]:].any()
        for i in range(e):
            s = slice(ends[i], ends[i + 1])
            h, eh, zw, ez = G.forward(x[s].cpu(), w[i].cpu(), bias[i].cpu(), "silu", w_kn)
            H.assert_within(y[s], h, eh + H.half_step(h, t), f"y {i}")
            H.assert_within(zz[s], zw, ez + H.half_step(zw, t), f"z {i}")
            want, err = G.grad(dy[s].cpu(), down[i].cpu(), z[s].cpu(), "silu", w_kn)
            H.assert_within(dz[s], want, err + H.half_step(want, t), f"dz {i}")


@pytest.mark.parametrize("w_kn", [False, True])
@pytest.mark.parametrize("act", ["relu2", "gelu"])
def test_experts_of_large_odd_widths(gpu_lib, w_kn, act):
    """Enough odd rows and columns for the larger tiles of the kernels of any width, in both directions."""
    t, rows, n, k, offsets = torch.float16, 4500, 1003, 45, [3, 1700, 1700, 4400]
    off = torch.tensor(offsets, device="cuda")
    x, dy, z = _mat(rows, k, t, 1, pitch=k + 2, shift=1), _mat(rows, k, t, 2, 0.1), _mat(rows, 2 * n, t, 3, pitch=2 * n + 1)
    w, down = _weight(2 * n, k, t, 4, w_kn, (3,)), _weight(k, n, t, 5, w_kn, (3,))
    bias = torch.randn(3, 2 * n, generator=torch.Generator().manual_seed(6)).to(t).cuda()
    y, zz = gpu_lib.anvil_expert_gated_linear(x, w, off, bias, act=act, w_kn=w_kn, preact=_nan(rows, 2 * n, t=t),
                                              out=_nan(rows, n, t=t))
    dz = gpu_lib.anvil_expert_gated_grad_input(dy, down, off, z, act=act, w_kn=w_kn, out=_nan(rows, 2 * n, t=t))
    for part in (y, zz, dz):
        assert not part[:3].any() and not part[4400:].any()
    for i in (0, 2):
        s = slice(offsets[i], offsets[i + 1])
        h, eh, zw, ez = G.forward(x[s].cpu(), w[i].cpu(), bias[i].cpu(), act, w_kn)
        H.assert_within(y[s], h, eh + H.half_step(h, t), f"y {i}")
        H.assert_within(zz[s], zw, ez + H.half_step(zw, t), f"z {i}")
        want, err = G.grad(dy[s].cpu(), down[i].cpu(), z[s].cpu(), act, w_kn)
        H.assert_within(dz[s], want, err + H.half_step(want, t), f"dz {i}")


def test_offsets_past_32_bits(gpu_lib):
    """z and dz of more than 2^32 elements: their last rows, by the tiles and by the kernels of any width."""
    t, rows = torch.bfloat16, 800000
    for n, k in ((2816, 64), (2817, 33)):
        x, w, down = _mat(rows, k, t, 1), _weight(2 * n, k, t, 2, False), _weight(k, n, t, 3, False)
        assert rows * 2 * n > 1 << 32
        y, z = gpu_lib.anvil_gated_linear(x, w, keep_preact=True)
        dz = gpu_lib.anvil_gated_grad_input(x, down, z)
        part = slice(rows - 70, rows)
        h, eh, zw, ez = G.forward(x[part].cpu(), w.cpu(), None, "silu", False)
        H.assert_within(y[part], h, eh + H.half_step(h, t), "y")
        H.assert_within(z[part], zw, ez + H.half_step(zw, t), "z")
        want, err = G.grad(x[part].cpu(), down.cpu(), z[part].cpu(), "silu", False)
        H.assert_within(dz[part], want, err + H.half_step(want, t), "dz")
        del x, w, y, z, dz


def test_a_single_row_of_any_pitch(gpu_lib):
    """The last row of a tensor whose rows lie further apart than a pitch may be."""
    t, far = torch.bfloat16, (1 << 22) + 8
    x = _mat(2, 72, t, 1, pitch=far)[1:]
    w, down = _weight(2 * 40, 72, t, 2, False), _weight(72, 40, t, 3, False)
    _check_forward(gpu_lib, x, w, None, "silu", False, True, t)
    _check_grad(gpu_lib, x, down, _mat(2, 80, t, 4, pitch=far)[1:], "silu", False, t)


def test_empty(gpu_lib):
    t = torch.bfloat16
    for rows, n, k in ((0, 16, 8), (3, 0, 8)):
        y, z = gpu_lib.anvil_gated_linear(_mat(rows, k, t, 1), _weight(2 * n, k, t, 2, False), keep_preact=True)
        assert y.shape == (rows, n) and z.shape == (rows, 2 * n)
        dz = gpu_lib.anvil_gated_grad_input(_mat(rows, k, t, 1), _weight(k, n, t, 2, False), _mat(rows, 2 * n, t, 3))
        assert dz.shape == (rows, 2 * n)
    # no experts: no row has one
    off = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, z = gpu_lib.anvil_expert_gated_linear(_mat(5, 8, t, 1), torch.empty(0, 32, 8, dtype=t, device="cuda"), off,
                                             preact=_nan(5, 32, t=t), out=_nan(5, 16, t=t))
    dz = gpu_lib.anvil_expert_gated_grad_input(_mat(5, 8, t, 1), torch.empty(0, 8, 16, dtype=t, device="cuda"), off, z,
                                               out=_nan(5, 32, t=t))
    assert not y.any() and not z.any() and not dz.any()
    # no inputs: z is the bias alone; no outputs: nothing reaches z
    bias = torch.randn(32, generator=torch.Generator().manual_seed(1)).cuda()
    y, z = gpu_lib.anvil_gated_linear(_mat(4, 0, t, 1), torch.empty(32, 0, dtype=t, device="cuda"), bias, act="relu", keep_preact=True)
    assert torch.equal(z, bias.to(t).expand(4, 32))
    h = torch.relu(bias[:16]) * bias[16:]
    assert torch.equal(y, h.to(t).expand(4, 16))
    dz = gpu_lib.anvil_gated_grad_input(_mat(4, 0, t, 1), torch.empty(0, 16, dtype=t, device="cuda"), z, out=_nan(4, 32, t=t))
    assert not dz.any()


def test_nonfinite_values_stay_in_their_place(gpu_lib):
    """An infinity or NaN of one element of x reaches its row alone, one of the weight its column pair alone."""
    t = torch.bfloat16
    for n, k in ((136, 72), (67, 45)):
        x, w = _mat(40, k, t, 1), _weight(2 * n, k, t, 2, False)
        clean, _ = gpu_lib.anvil_gated_linear(x, w)
        x[7, 3], x[20, 0] = float("inf"), float("nan")
        y, _ = gpu_lib.anvil_gated_linear(x, w)
        rows = [r for r in range(40) if r not in (7, 20)]
        assert torch.equal(y[rows], clean[rows]) and torch.isnan(y[20]).all() and not torch.isfinite(y[7]).any()
        x = _mat(40, k, t, 1)
        w[n + 5, 1] = float("nan")
        y, _ = gpu_lib.anvil_gated_linear(x, w)
        cols = [c for c in range(n) if c != 5]
        assert torch.equal(y[:, cols], clean[:, cols]) and torch.isnan(y[:, 5]).all()


def test_gradients_against_differences(gpu_lib):
    """dz, and from it dx, dw and dbias by the linear layer's gradients, against central differences of the 64-bit loss
    sum(y dy).  The kernels' z and dz are rounded to bf16 (2^-9 of each on average a third of a step); the sums over them
    stay within 2^-7 of their own size, which is what is asked of a directional derivative."""
    t, rows, n, k = torch.bfloat16, 96, 72, 40
    x, w = _mat(rows, k, t, 1), _weight(2 * n, k, t, 2, False)
    down, dy = _weight(k, n, t, 3, False), _mat(rows, k, t, 4)
    bias = 0.3 * torch.randn(2 * n, generator=torch.Generator().manual_seed(5)).cuda()
    _, z = gpu_lib.anvil_gated_linear(x, w, bias, keep_preact=True)
    dz = gpu_lib.anvil_gated_grad_input(dy, down, z)
    dx = gpu_lib.anvil_linear_grad_input(dz, w)
    dw, db = gpu_lib.anvil_linear_grad_weight(dz, x)

    def loss(xv, wv, bv):
        h, _, _, _ = G.forward(xv, wv, bv, "silu", False)
        return float(((h @ down.double().cpu().t()) * dy.double().cpu()).sum())

    at = [v.double().cpu() for v in (x, w, bias)]
    for i, grad in enumerate((dx, dw, db)):
        g = grad.double().cpu()
        step = [torch.zeros_like(v) for v in at]
        step[i] = g / g.norm() * 1e-4      # along the gradient: the slope is its norm
        up, low = [a + s for a, s in zip(at, step)], [a - s for a, s in zip(at, step)]
        slope = (loss(*up) - loss(*low)) / 2e-4
        assert abs(slope - float(g.norm())) <= 2.0 ** -7 * float(g.norm())


def test_replayed_graph(gpu_lib):
    """Forward and gradient captured and replayed on new inputs in the same buffers, with eager work between."""
    t = torch.bfloat16
    x, dy = _mat(200, 136, t, 1), _mat(200, 136, t, 2, 0.1)
    w, down = _weight(2 * 264, 136, t, 3, False), _weight(136, 264, t, 4, False)

    def step():
        y, z = gpu_lib.anvil_gated_linear(x, w, keep_preact=True)
        return y, gpu_lib.anvil_gated_grad_input(dy, down, z)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        x.copy_(_mat(200, 136, t, 10 + i))
        dy.copy_(_mat(200, 136, t, 20 + i, 0.1))
        graph.replay()
        got = [v.clone() for v in out]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
        torch.cuda.synchronize()


def test_other_stream(gpu_lib):
    t = torch.float16
    x, w = _mat(100, 72, t, 1), _weight(2 * 40, 72, t, 2, True)
    want = gpu_lib.anvil_gated_linear(x, w, w_kn=True)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gpu_lib.anvil_gated_linear(x, w, w_kn=True, stream=side)[0]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
