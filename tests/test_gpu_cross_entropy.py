"""Cross entropy of a linear head and its gradients, on the GPU against plain forms in 64 bits."""
import pytest
import torch

from tests import head_helpers as C
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


def _weight(vocab, k, t, seed, w_kn, shift=0):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(*((k, vocab) if w_kn else (vocab, k)), generator=g) * 2 * max(k, 1) ** -0.5).to(t)
    buf = torch.full((w.numel() + shift,), float("nan"), dtype=t, device="cuda")
    view = buf[shift:].view(w.shape)
    view.copy_(w)
    return view


def _targets(rows, vocab, seed, bits=torch.int64, ignored=True):
    g = torch.Generator().manual_seed(seed)
    t = torch.randint(0, vocab, (rows,), generator=g)
    t[:2] = torch.tensor([0, vocab - 1])[:rows]       # the first and the last entry
    if ignored and rows > 4:
        t[3], t[4] = -1, vocab                        # just outside on either side
        t[torch.rand(rows, generator=g) < 0.1] = -100
    return t.to(bits).cuda()


def _nan(*shape, t):
    return torch.full(shape, float("nan"), dtype=t, device="cuda")


def _check(lib, x, w, targets, w_kn, t, seed=9):
    rows, k = x.shape
    loss, lse = lib.anvil_cross_entropy(x, w, targets, w_kn=w_kn)
    torch.cuda.synchronize()
    (lw, el), (sw, es) = C.forward(x.cpu(), w.cpu(), targets, w_kn)
    H.assert_within(lse, sw, es, "lse")
    H.assert_within(loss, lw, el, "loss")
    g = torch.Generator().manual_seed(seed)
    dloss = (torch.randn(rows, generator=g) / rows).cuda()
    for out_t in (torch.float32, t):
        dx, dw = lib.anvil_cross_entropy_grad(x, w, targets, lse, dloss, w_kn=w_kn, out=_nan(rows, k, t=t),
                                              dw_out=_nan(*w.shape, t=out_t))
        torch.cuda.synchronize()
        (xw, ex), (ww, ew) = C.gradients(x.cpu(), w.cpu(), targets, lse, dloss, w_kn, t)
        H.assert_within(dx, xw, ex + H.half_step(xw, t), "dx")
        H.assert_within(dw, ww, ew + H.half_step(ww, out_t), f"dw {out_t}")


# one row to more rows than a tile; vocabularies and widths below, at and past the tiles, odd ones
SHAPES = [(1, 1000, 64), (1, 1, 8), (2, 7, 3), (5, 4099, 72), (31, 64, 768), (32, 520, 40), (33, 1001, 67), (64, 128, 64),
          (65, 300, 1), (130, 515, 257), (200, 2056, 96), (257, 1032, 264), (520, 263, 520), (700, 3001, 45)]


@pytest.mark.parametrize("rows,vocab,k", SHAPES)
@pytest.mark.parametrize("w_kn", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_shapes(gpu_lib, rows, vocab, k, w_kn, kind):
    t = TYPES[kind]
    seed = rows * 7 + vocab * 3 + k
    bits = torch.int64 if seed % 2 else torch.int32
    _check(gpu_lib, _mat(rows, k, t, seed), _weight(vocab, k, t, seed + 1, w_kn), _targets(rows, vocab, seed, bits), w_kn, t)


# enough tiles for the larger shapes and several splits of the rows
@pytest.mark.parametrize("rows,vocab,k", [(2100, 4000, 72), (4100, 5003, 136), (3000, 2600, 520), (700, 20008, 264)])
@pytest.mark.parametrize("w_kn", [False, True])
def test_large_tiles(gpu_lib, rows, vocab, k, w_kn):
    t = torch.bfloat16 if vocab % 3 else torch.float16
    _check(gpu_lib, _mat(rows, k, t, 1), _weight(vocab, k, t, 2, w_kn), _targets(rows, vocab, 3), w_kn, t)


@pytest.mark.parametrize("w_kn", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_several_pieces(gpu_lib, w_kn, kind):
    """So many rows that the vocabulary is taken in pieces (of 1792 entries here), the last of them ragged: the pieces'
    sums against the same in 64 bits, for some rows and entries, and for all in one against the other layout."""
    t, rows, vocab, k = TYPES[kind], 270000, 2500, 16
    x, w = _mat(rows, k, t, 1), _weight(vocab, k, t, 2, w_kn)
    targets = _targets(rows, vocab, 3, torch.int32)
    loss, lse = gpu_lib.anvil_cross_entropy(x, w, targets, w_kn=w_kn)
    g = torch.Generator().manual_seed(4)
    dloss = torch.zeros(rows)
    some = torch.randperm(rows, generator=g)[:3000].sort()[0]
    dloss[some] = torch.randn(3000, generator=g) / 3000     # rows without a gradient leave dw to the others
    dloss = dloss.cuda()
    need = gpu_lib.load().anvil_cross_entropy_grad_workspace(1, 1, int(w_kn), 3, gpu_lib._code(x, "x", (1, 2)), rows, vocab, k)
    assert need < rows * vocab * 2                          # P is never whole
    dx, dw = gpu_lib.anvil_cross_entropy_grad(x, w, targets, lse, dloss, w_kn=w_kn, out=_nan(rows, k, t=t),
                                              dw_out=_nan(*w.shape, t=torch.float32))
    torch.cuda.synchronize()
    some = some.cuda()
    (lw, el), (sw, es) = C.forward(x[some].cpu(), w.cpu(), targets[some], w_kn)
    H.assert_within(loss[some], lw, el, "loss")
    H.assert_within(lse[some], sw, es, "lse")
    (xw, ex), (ww, ew) = C.gradients(x[some].cpu(), w.cpu(), targets[some], lse[some], dloss[some], w_kn, t)
    H.assert_within(dx[some], xw, ex + H.half_step(xw, t), "dx")
    H.assert_within(dw, ww, ew + H.half_step(ww, torch.float32), "dw")
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    rest[some] = False
    assert not dx[rest].any()


@pytest.mark.parametrize("pitch,shift,w_shift", [(0, 0, 0), (8, 8, 8), (8, 0, 3), (3, 1, 0), (1, 0, 1), (0, 5, 0)])
@pytest.mark.parametrize("vocab,k", [(1024, 64), (999, 33)])
@pytest.mark.parametrize("w_kn", [False, True])
def test_pitches_and_alignment(gpu_lib, pitch, shift, w_shift, vocab, k, w_kn):
    t, rows = torch.bfloat16, 70
    for r in (rows, 1):
        x = _mat(r, k, t, 1, pitch=k + pitch, shift=shift)
        _check(gpu_lib, x, _weight(vocab, k, t, 2, w_kn, w_shift), _targets(r, vocab, 3), w_kn, t)
    x, w, targets = _mat(rows, k, t, 1), _weight(vocab, k, t, 2, w_kn), _targets(rows, vocab, 3)
    _, lse = gpu_lib.anvil_cross_entropy(x, w, targets, w_kn=w_kn)
    dloss = torch.full((rows,), 1 / rows, device="cuda")
    buf = _nan(rows * (k + pitch) + shift, t=t)
    out = buf[shift:].as_strided((rows, k), (k + pitch, 1))
    gpu_lib.anvil_cross_entropy_grad(x, w, targets, lse, dloss, w_kn=w_kn, out=out)
    assert torch.equal(out, gpu_lib.anvil_cross_entropy_grad(x, w, targets, lse, dloss, w_kn=w_kn)[0])
    rest = torch.ones_like(buf, dtype=torch.bool)
    rest[shift:].as_strided((rows, k), (k + pitch, 1)).fill_(False)
    assert torch.isnan(buf[rest]).all()


def test_one_gradient_only(gpu_lib):
    t = torch.bfloat16
    x, w, targets = _mat(300, 72, t, 1), _weight(2000, 72, t, 2, False), _targets(300, 2000, 3)
    _, lse = gpu_lib.anvil_cross_entropy(x, w, targets)
    dloss = torch.full((300,), 1 / 300, device="cuda")
    dx, dw = gpu_lib.anvil_cross_entropy_grad(x, w, targets, lse, dloss)
    a, none = gpu_lib.anvil_cross_entropy_grad(x, w, targets, lse, dloss, want_weight=False)
    assert none is None and torch.equal(a, dx)
    none, b = gpu_lib.anvil_cross_entropy_grad(x, w, targets, lse, dloss, want_input=False)
    assert none is None and torch.equal(b, dw)


def test_large_logits_and_small_gradients(gpu_lib):
    """Logits of hundreds of units (no exponential of them is finite), and gradients far below fp16's range of mean
    losses: rows weighted by 1e-6 beside one of 1e-2."""
    for t in TYPES.values():
        x, w = _mat(200, 64, t, 1, 40.0), _weight(3000, 64, t, 2, False)
        _check(gpu_lib, x, w, _targets(200, 3000, 3), False, t)
    t = torch.float16
    x, w, targets = _mat(200, 64, t, 1), _weight(3000, 64, t, 2, False), _targets(200, 3000, 3, ignored=False)
    _, lse = gpu_lib.anvil_cross_entropy(x, w, targets)
    dloss = torch.full((200,), 1e-6, device="cuda")
    dloss[7] = 1e-2
    _, dw = gpu_lib.anvil_cross_entropy_grad(x, w, targets, lse, dloss, out_dtype=torch.float32)
    _, (ww, ew) = C.gradients(x.cpu(), w.cpu(), targets, lse, dloss, False, t)
    H.assert_within(dw, ww, ew + H.half_step(ww, torch.float32), "dw")
    dloss.fill_(1e-30)
    _, dw = gpu_lib.anvil_cross_entropy_grad(x, w, targets, lse, dloss, out_dtype=torch.float32)
    _, (ww, ew) = C.gradients(x.cpu(), w.cpu(), targets, lse, dloss, False, t)
    H.assert_within(dw, ww, ew + H.half_step(ww, torch.float32), "small dw")
    assert dw.any()


def test_ignored_rows_hold_anything(gpu_lib):
    """Rows without a target may hold infinities and NaN and a dloss of NaN: they have no loss and no gradient, and
    reach no other row's."""
    t = torch.bfloat16
    for k in (64, 45):
        x, w = _mat(150, k, t, 1), _weight(900, k, t, 2, False)
        targets = _targets(150, 900, 3)
        ignored = ~C.counts_of(targets, 900).cuda()
        clean = x.clone()
        clean[ignored] = 0
        x[ignored] = float("nan")
        x[4] = float("inf")
        dloss = torch.full((150,), 1 / 150, device="cuda")
        _, lse = gpu_lib.anvil_cross_entropy(clean, w, targets)
        want = gpu_lib.anvil_cross_entropy_grad(clean, w, targets, lse, dloss)
        loss, lse = gpu_lib.anvil_cross_entropy(x, w, targets)
        assert not loss[ignored].any() and torch.isnan(lse[ignored]).all()
        dloss[ignored] = float("nan")
        dx, _ = gpu_lib.anvil_cross_entropy_grad(x, w, targets, lse, dloss)
        assert torch.equal(dx, want[0]) and not dx[ignored].any()
        # dw = P^T x: a row of zeros in P meets the row's values, so those have to be finite for it
        _, dw = gpu_lib.anvil_cross_entropy_grad(clean, w, targets, lse, dloss)
        assert torch.equal(dw, want[1])


@pytest.mark.parametrize("bits", [torch.int32, torch.int64])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_large_dloss_of_ignored_rows(gpu_lib, kind, bits):
    """A finite dloss of a row without a target, however large, does not take part in an fp16 P's scale."""
    t = TYPES[kind]
    x, w, targets = _mat(150, 64, t, 1), _weight(900, 64, t, 2, False), _targets(150, 900, 3, bits)
    ignored = ~C.counts_of(targets, 900).cuda()
    dloss = torch.full((150,), 1 / 150, device="cuda")
    _, lse = gpu_lib.anvil_cross_entropy(x, w, targets)
    want = gpu_lib.anvil_cross_entropy_grad(x, w, targets, lse, dloss)
    dloss[ignored] = 1e30
    got = gpu_lib.anvil_cross_entropy_grad(x, w, targets, lse, dloss)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_offsets_past_32_bits(gpu_lib):
    """More than 2^32 logits, several pieces of more than 2^28 probabilities: the last rows' loss and dx, and dw of rows at
    both ends of the batch (the others have no target)."""
    t, rows, vocab, k = torch.bfloat16, 150000, 33000, 64
    x, w = _mat(rows, k, t, 1), _weight(vocab, k, t, 2, True)
    targets = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    some = torch.cat([torch.arange(40), torch.arange(rows - 40, rows)]).cuda()
    targets[some] = _targets(80, vocab, 3, torch.int32)
    loss, lse = gpu_lib.anvil_cross_entropy(x, w, targets, w_kn=True)
    dloss = torch.full((rows,), 1 / 80, device="cuda")
    dx, dw = gpu_lib.anvil_cross_entropy_grad(x, w, targets, lse, dloss, w_kn=True, out_dtype=torch.float32)
    xs, ts = x[some].cpu(), targets[some]
    (lw, el), (sw, es) = C.forward(xs, w.cpu(), ts, True)
    H.assert_within(loss[some], lw, el, "loss")
    H.assert_within(lse[some], sw, es, "lse")
    (xw, ex), (ww, ew) = C.gradients(xs, w.cpu(), ts, lse[some], dloss[some], True, t)
    H.assert_within(dx[some], xw, ex + H.half_step(xw, t), "dx")
    H.assert_within(dw, ww, ew + H.half_step(ww, torch.float32), "dw")
    assert not loss[40:-40].any() and not dx[40:-40].any()


def test_no_targets(gpu_lib):
    """Every row ignored: no loss and no gradient, and none of them NaN."""
    for t in TYPES.values():
        x, w = _mat(70, 40, t, 1), _weight(300, 40, t, 2, False)
        targets = torch.full((70,), -100, device="cuda")
        loss, lse = gpu_lib.anvil_cross_entropy(x, w, targets)
        dx, dw = gpu_lib.anvil_cross_entropy_grad(x, w, targets, lse, torch.zeros(70, device="cuda"))
        assert torch.isfinite(lse).all() and not loss.any() and not dx.any() and not dw.any()
        assert torch.isfinite(dx).all() and torch.isfinite(dw).all()


def test_a_single_row_of_any_pitch(gpu_lib):
    t, far = torch.bfloat16, (1 << 22) + 8
    for k in (64, 45):
        _check(gpu_lib, _mat(2, k, t, 1, pitch=far)[1:], _weight(900, k, t, 2, False), _targets(1, 900, 3), False, t)


def test_infinite_logits(gpu_lib):
    """An infinity or NaN in a row makes that row's loss NaN or infinite, no other's."""
    t = torch.bfloat16
    x, w, targets = _mat(300, 64, t, 1), _weight(900, 64, t, 2, False), _targets(300, 900, 3, ignored=False)
    clean, _ = gpu_lib.anvil_cross_entropy(x, w, targets)
    x[5, 1], x[200, 0], x[299, 63] = float("inf"), float("nan"), -float("inf")
    loss, lse = gpu_lib.anvil_cross_entropy(x, w, targets)
    rest = torch.ones(300, dtype=torch.bool, device="cuda")
    rest[[5, 200, 299]] = False
    assert torch.equal(loss[rest], clean[rest]) and not torch.isfinite(loss[~rest]).any()
    assert not torch.isfinite(lse[~rest]).any()


def test_empty(gpu_lib):
    t = torch.bfloat16
    w = _weight(50, 16, t, 1, False)
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    loss, lse = gpu_lib.anvil_cross_entropy(_mat(0, 16, t, 2), w, none)
    assert loss.shape == lse.shape == (0,)
    for out_t in (t, torch.float32):
        dx, dw = gpu_lib.anvil_cross_entropy_grad(_mat(0, 16, t, 2), w, none, lse, lse, dw_out=_nan(50, 16, t=out_t))
        assert dx.shape == (0, 16) and not dw.any() and torch.isfinite(dw).all()
    # no inputs: every logit is zero
    targets = torch.tensor([3, -1, 49], device="cuda")
    loss, lse = gpu_lib.anvil_cross_entropy(_mat(3, 0, t, 2), torch.empty(50, 0, dtype=t, device="cuda"), targets)
    want = torch.log(torch.tensor(50.0))
    assert (lse.cpu() - want).abs().max() < 1e-6 and float(loss[1]) == 0 and (loss[::2].cpu() - want).abs().max() < 1e-6


def test_gradients_against_differences(gpu_lib):
    """dx and dw against central differences of the 64-bit mean loss, along the gradient itself (see the gated layer's
    test): the rounded P and outputs stay within 2^-7 of the slope."""
    t, rows, vocab, k = torch.bfloat16, 90, 700, 48
    x, w, targets = _mat(rows, k, t, 1), _weight(vocab, k, t, 2, False), _targets(rows, vocab, 3)
    _, lse = gpu_lib.anvil_cross_entropy(x, w, targets)
    dloss = torch.full((rows,), 1 / rows, device="cuda")
    grads = gpu_lib.anvil_cross_entropy_grad(x, w, targets, lse, dloss)

    def loss(a, b):
        return float(C.forward(a, b, targets, False)[0][0].sum() / rows)

    at = [x.double().cpu(), w.double().cpu()]
    for i, grad in enumerate(grads):
        g = grad.double().cpu()
        step = [torch.zeros_like(v) for v in at]
        step[i] = g / g.norm() * 1e-3
        slope = (loss(*[a + s for a, s in zip(at, step)]) - loss(*[a - s for a, s in zip(at, step)])) / 2e-3
        assert abs(slope - float(g.norm())) <= 2.0 ** -7 * float(g.norm())


def test_replayed_graph(gpu_lib):
    """Loss and gradients captured and replayed on new inputs, two graphs with a workspace each, with eager work
    between."""
    t, rows, vocab, k = torch.float16, 260, 1500, 77
    x, w, targets = _mat(rows, k, t, 1), _weight(vocab, k, t, 2, True), _targets(rows, vocab, 3)
    dloss = torch.full((rows,), 1 / rows, device="cuda")

    def step():
        loss, lse = gpu_lib.anvil_cross_entropy(x, w, targets, w_kn=True)
        return (loss, lse) + gpu_lib.anvil_cross_entropy_grad(x, w, targets, lse, dloss, w_kn=True)

    step()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(step())
    for i in range(4):
        x.copy_(_mat(rows, k, t, 10 + i))
        targets.copy_(_targets(rows, vocab, 20 + i))
        for graph, out in zip(graphs, outs):
            graph.replay()
            got = [v.clone() for v in out]
            for a, b in zip(got, step()):
                assert torch.equal(a, b)
        torch.cuda.synchronize()


def test_other_stream(gpu_lib):
    t = torch.bfloat16
    x, w, targets = _mat(100, 45, t, 1), _weight(900, 45, t, 2, False), _targets(100, 900, 3)
    dloss = torch.full((100,), 1 / 100, device="cuda")
    loss, lse = gpu_lib.anvil_cross_entropy(x, w, targets)
    dx, dw = gpu_lib.anvil_cross_entropy_grad(x, w, targets, lse, dloss)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    loss2, lse2 = gpu_lib.anvil_cross_entropy(x, w, targets, stream=side)
    dx2, dw2 = gpu_lib.anvil_cross_entropy_grad(x, w, targets, lse2, dloss, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in ((loss, loss2), (lse, lse2), (dx, dx2), (dw, dw2)):
        assert torch.equal(a, b)


# pieces of 1792 entries and a ragged rest; and so many rows that the least piece, 1024 entries, is taken
@pytest.mark.parametrize("rows,vocab,k,w_kn,kind", [(270000, 2500, 16, False, "bf16"), (270000, 2500, 16, True, "bf16"),
                                                    (270000, 2500, 16, False, "fp16"), (270000, 2500, 16, True, "fp16"),
                                                    ((1 << 20) + 5, 1100, 8, False, "bf16")])
def test_several_pieces_of_every_row(gpu_lib, monkeypatch, rows, vocab, k, w_kn, kind):
    """A gradient at every row's loss: loss, log-sum-exp, dx and dw of all rows and entries against 64 bits, which are
    formed on the GPU (the plain forms fetch nothing here)."""
    t = TYPES[kind]
    x, w = _mat(rows, k, t, 1), _weight(vocab, k, t, 2, w_kn)
    targets = _targets(rows, vocab, 3, torch.int32)
    dloss = (torch.randn(rows, generator=torch.Generator().manual_seed(4)) / rows).cuda()
    loss, lse = gpu_lib.anvil_cross_entropy(x, w, targets, w_kn=w_kn)
    dx, dw = gpu_lib.anvil_cross_entropy_grad(x, w, targets, lse, dloss, w_kn=w_kn, out=_nan(rows, k, t=t),
                                              dw_out=_nan(*w.shape, t=torch.float32))
    torch.cuda.synchronize()
    with monkeypatch.context() as patch:
        patch.setattr(torch.Tensor, "cpu", lambda self: self)
        (lw, el), (sw, es) = C.forward(x, w, targets, w_kn)
        (xw, ex), (ww, ew) = C.gradients(x, w, targets, lse, dloss, w_kn, t)
    assert int(C.counts_of(targets, vocab).sum()) > 0.8 * rows and (ww.abs() > ew).double().mean() > 0.9   # bounds that say something
    H.assert_within(loss, lw, el, "loss")
    H.assert_within(lse, sw, es, "lse")
    H.assert_within(dx, xw, ex + H.half_step(xw, t), "dx")
    H.assert_within(dw, ww, ew + H.half_step(ww, torch.float32), "dw")


@pytest.mark.parametrize("w_kn", [False, True])
def test_more_than_2_30_weights(gpu_lib, monkeypatch, w_kn):
    """A head whose gradient's last entries lie past 2^30 elements and 2^32 bytes: everything against 64 bits on the GPU."""
    t, rows, vocab, k = torch.bfloat16, 70, 152064, 8192
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, k, generator=g, device="cuda").to(t)
    w = torch.empty((k, vocab) if w_kn else (vocab, k), dtype=t, device="cuda").normal_(0, 2 * k ** -0.5, generator=g)
    targets = _targets(rows, vocab, 3)
    dloss = (torch.randn(rows, generator=torch.Generator().manual_seed(4)) / rows).cuda()
    loss, lse = gpu_lib.anvil_cross_entropy(x, w, targets, w_kn=w_kn)
    dx, dw = gpu_lib.anvil_cross_entropy_grad(x, w, targets, lse, dloss, w_kn=w_kn, out=_nan(rows, k, t=t),
                                              dw_out=_nan(*w.shape, t=torch.float32))
    torch.cuda.synchronize()
    with monkeypatch.context() as patch:
        patch.setattr(torch.Tensor, "cpu", lambda self: self)
        (lw, el), (sw, es) = C.forward(x, w, targets, w_kn)
        (xw, ex), (ww, ew) = C.gradients(x, w, targets, lse, dloss, w_kn, t)
        H.assert_within(loss, lw, el, "loss")
        H.assert_within(lse, sw, es, "lse")
        H.assert_within(dx, xw, ex + H.half_step(xw, t), "dx")
        ew += H.half_step(ww, torch.float32)
        H.assert_within(dw, ww, ew, "dw")
