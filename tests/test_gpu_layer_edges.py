"""The training operators at the edges of their arguments."""
import pytest
import torch

from tests import layer_helpers as H

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _normal(*shape, t, seed, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(t).cuda()


# 128x128 and 256x256 tiles from copies, 64x64 and 128x128 tiles of any width
SUM_SHAPES = [(200, 96, 72), (6000, 776, 1032), (2048, 4104, 2056), (200, 97, 71), (2100, 1031, 1033), (40, 33, 7)]


@pytest.mark.parametrize("rows,n,k", SUM_SHAPES)
@pytest.mark.parametrize("w_kn", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_nonfinite_gradient_stays_in_its_column(gpu_lib, rows, n, k, w_kn, kind):
    """Infinities and NaN in some columns of dz reach the sums of those columns and no others."""
    t = TYPES[kind]
    dz, x = _normal(rows, n, t=t, seed=1, scale=0.1), _normal(rows, k, t=t, seed=2)
    clean = gpu_lib.anvil_linear_grad_weight(dz, x, w_kn=w_kn)
    inf = float("inf")
    marks = {0: (inf,), 5: (-inf,), 18: (float("nan"),), n - 1: (inf,), n - 9: (inf, -inf)}
    for c, values in marks.items():
        for i, v in enumerate(values):
            dz[(7 * c + 11 * i) % rows, c] = v
    dw, db = gpu_lib.anvil_linear_grad_weight(dz, x, w_kn=w_kn)
    (ww, ew), (bw, eb) = H.grad_weight(dz.cpu(), x.cpu(), w_kn)
    H.assert_within(db, bw, eb, "db")
    H.assert_within(dw, ww, ew + H.half_step(ww, torch.float32), "dw")
    rest = [c for c in range(n) if c not in marks]
    assert torch.equal(db[rest], clean[1][rest])


@pytest.mark.parametrize("n,k", [(264, 136), (67, 33)])
@pytest.mark.parametrize("w_kn", [False, True])
def test_nonfinite_gradient_stays_with_its_expert(gpu_lib, n, k, w_kn):
    t = torch.bfloat16
    ends = [0, 300, 300, 800, 1000]
    off = torch.tensor(ends, dtype=torch.int32, device="cuda")
    dz, x = _normal(1000, n, t=t, seed=3, scale=0.1), _normal(1000, k, t=t, seed=4)
    dz[299, 3], dz[300, 20], dz[999, 40] = float("inf"), float("nan"), -float("inf")
    dw, db = gpu_lib.anvil_expert_grad_weight(dz, x, off, w_kn=w_kn)
    for e in range(4):
        s = slice(ends[e], ends[e + 1])
        (ww, ew), (bw, eb) = H.grad_weight(dz[s].cpu(), x[s].cpu(), w_kn)
        H.assert_within(db[e], bw, eb + 1e-45, f"db {e}")
        H.assert_within(dw[e], ww, ew + H.half_step(ww, torch.float32), f"dw {e}")


@pytest.mark.parametrize("w_kn", [False, True])
@pytest.mark.parametrize("rows,n", [(1, 1), (40, 64), (5000, 33)])
def test_bias_gradient_of_a_layer_without_inputs(gpu_lib, rows, n, w_kn):
    """k = 0: the output is the bias alone, whose gradient is the sum of dz all the same."""
    t = torch.bfloat16
    dz = _normal(rows, n, t=t, seed=5)
    x = torch.empty(rows, 0, dtype=t, device="cuda")
    _, (want, err) = H.grad_weight(dz.cpu(), x.cpu(), w_kn)
    torch.full((1 << 18,), float("nan"), device="cuda")   # memory that the result may come from
    dw, db = gpu_lib.anvil_linear_grad_weight(dz, x, w_kn=w_kn)
    assert dw.numel() == 0
    H.assert_within(db, want, err, "db")
    assert gpu_lib.anvil_linear_grad_weight(dz, x, w_kn=w_kn, want_bias=False)[1] is None
    ends = [0, rows // 2, rows // 2, rows]
    off = torch.tensor(ends, dtype=torch.int64, device="cuda")
    dw, db = gpu_lib.anvil_expert_grad_weight(dz, x, off, w_kn=w_kn)
    assert dw.shape == ((3, 0, n) if w_kn else (3, n, 0)) and db.shape == (3, n)
    for e in range(3):
        _, (want, err) = H.grad_weight(dz[ends[e]:ends[e + 1]].cpu(), x[ends[e]:ends[e + 1]].cpu(), w_kn)
        H.assert_within(db[e], want, err + 1e-45, f"db {e}")


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_norm_statistics_without_columns(gpu_lib, kind):
    """No columns: the mean of nothing, 0 / 0, and what follows from it."""
    torch.zeros(1 << 18, device="cuda")   # memory that the statistics may come from
    y, mean, rstd = gpu_lib.anvil_layer_norm(torch.empty(300, 0, dtype=TYPES[kind], device="cuda"))
    assert y.shape == (300, 0) and mean.shape == rstd.shape == (300,)
    assert torch.isnan(mean).all() and torch.isnan(rstd).all()


@pytest.mark.parametrize("pitch", [1 << 24, (1 << 23) + 1])
@pytest.mark.parametrize("width", [768, 77])
def test_single_row_at_any_pitch(gpu_lib, pitch, width):
    """The last token of a long sequence: one row, whose stride is never taken."""
    t = torch.bfloat16
    n = 64
    x = _normal(1, width, t=t, seed=6).as_strided((1, width), (pitch, 1))
    dz = _normal(1, n, t=t, seed=7).as_strided((1, n), (pitch, 1))
    assert x.stride(0) == pitch
    flat, dflat = x.clone(memory_format=torch.contiguous_format).reshape(1, width), dz.reshape(-1).clone().reshape(1, n)
    w = _normal(n, width, t=t, seed=8)
    y, mean, rstd = gpu_lib.anvil_layer_norm(x)
    ref = gpu_lib.anvil_layer_norm(flat)
    assert all(torch.equal(p, q) for p, q in zip((y, mean, rstd), ref))
    got = gpu_lib.anvil_layer_norm_grad(x, x, None, mean, rstd)
    ref = gpu_lib.anvil_layer_norm_grad(flat, flat, None, mean, rstd)
    assert all(torch.equal(p, q) for p, q in zip(got, ref))
    out = torch.empty(1, n, dtype=t, device="cuda").as_strided((1, n), (pitch, 1))
    got = gpu_lib.anvil_linear(x, w, residual=dz, act="silu", keep_preact=True, out=out)
    ref = gpu_lib.anvil_linear(flat, w, residual=dflat, act="silu", keep_preact=True)
    assert all(torch.equal(p, q) for p, q in zip(got, ref))
    got = gpu_lib.anvil_linear_grad_input(dz, w, preact=x, act="gelu", add=x)
    assert torch.equal(got, gpu_lib.anvil_linear_grad_input(dflat, w, preact=flat, act="gelu", add=flat))
    got, ref = gpu_lib.anvil_linear_grad_weight(dz, x), gpu_lib.anvil_linear_grad_weight(dflat, flat)
    assert all(torch.equal(p, q) for p, q in zip(got, ref))
    assert torch.equal(gpu_lib.anvil_activation_grad(x, x, "relu2"), gpu_lib.anvil_activation_grad(flat, flat, "relu2"))


@pytest.mark.parametrize("cols", [12, 40, 600, 1100, 1601, 2100, 5000, 9001])
def test_norm_gradient_of_rows_near_the_end_of_the_range(gpu_lib, cols):
    """Rows of one value 2^120 with rstd 512: (0 - mean) rstd, as a column past the end would have it,
    is no fp32 value, while every column that is there has h = 0 and so dx = rstd (dy - mean(dy))."""
    x = torch.full((3, cols), 2.0 ** 120, device="cuda")
    dy = _normal(3, cols, t=torch.float32, seed=9)
    mean, rstd = torch.full((3,), 2.0 ** 120, device="cuda"), torch.full((3,), 512.0, device="cuda")
    dx, dw, db = gpu_lib.anvil_layer_norm_grad(dy, x, None, mean, rstd)
    d = dy.double().cpu()
    a = d.mean(1, keepdim=True)
    # the mean is a sum of cols products and two roundings, the rest four more
    ea = (H.SIGMA * H.U32 * cols ** 0.5 * d.square().sum(1, keepdim=True).sqrt()) / cols + 4 * H.U32 * a.abs()
    want = 512 * (d - a)
    H.assert_within(dx, want, 512 * (ea + 8 * H.U32 * (d.abs() + a.abs())), "dx")
    assert torch.count_nonzero(dw) == 0
    H.assert_within(db, d.sum(0), 4 * H.U32 * d.abs().sum(0), "db")


class _Borrowed:
    """A stream of another library: its handle under the name that torch's streams have."""

    def __init__(self, stream):
        self.cuda_stream = stream.cuda_stream


def test_streams_of_other_kinds(gpu_lib):
    """A handle, and an object that holds one, work as a torch stream does."""
    t = torch.bfloat16
    x, w = _normal(70, 64, t=t, seed=10), _normal(96, 64, t=t, seed=11)
    want = gpu_lib.anvil_linear(x, w, act="relu")[0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [gpu_lib.anvil_linear(x, w, act="relu", stream=k)[0] for k in (s, s.cuda_stream, _Borrowed(s))]
    s.synchronize()
    assert all(torch.equal(g, want) for g in got)


@pytest.mark.parametrize("n,k", [(96, 72), (97, 71)])
def test_subnormal_values_count(gpu_lib, n, k):
    """fp16 gradients below the smallest normal value are not taken as zero."""
    t = torch.float16
    dz, x = _normal(300, n, t=t, seed=12, scale=2e-6), _normal(300, k, t=t, seed=13)
    assert float(dz.abs().max()) < 2.0 ** -14
    dw, db = gpu_lib.anvil_linear_grad_weight(dz, x)
    (ww, ew), (bw, eb) = H.grad_weight(dz.cpu(), x.cpu(), False)
    H.assert_within(dw, ww, ew + H.half_step(ww, torch.float32), "dw")
    H.assert_within(db, bw, eb, "db")
    dx = gpu_lib.anvil_linear_grad_input(dz, x[:n].contiguous()[:, :k])
    want, err = H.grad_input(dz.cpu(), x[:n].cpu(), None, "none", None, False)
    H.assert_within(dx, want, err + H.half_step(want, t), "dx")


def test_outputs_on_another_stream_come_from_its_memory(gpu_lib):
    """A block that the current stream has just freed is not handed to a call on another stream."""
    t = torch.bfloat16
    x, w = _normal(1024, 64, t=t, seed=14), _normal(2048, 64, t=t, seed=15)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    freed = torch.empty(1024, 2048, dtype=t, device="cuda")
    at = freed.data_ptr()
    del freed
    y = gpu_lib.anvil_linear(x, w, stream=s)[0]
    assert y.data_ptr() != at
    s.synchronize()
    assert torch.equal(y, gpu_lib.anvil_linear(x, w)[0])
    # a bank call likewise
    grad = torch.randn(2, 64, 128, device="cuda")
    rails = [torch.zeros(2, 2, 64, 128, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    freed = torch.empty(2, 64, 128, dtype=t, device="cuda")
    at = freed.data_ptr()
    del freed
    other = gpu_lib.anvil_bank_step(grad, rails[0], 0.95, 0.85, 1.0, stream=s)
    assert other.data_ptr() != at
    s.synchronize()
    assert torch.equal(other, gpu_lib.anvil_bank_step(grad, rails[1], 0.95, 0.85, 1.0))
