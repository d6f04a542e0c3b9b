"""Python binding of libanvil.so (ctypes): argument marshalling only.

Every function takes torch tensors that already live on the GPU, checks dtype, shape, device and
contiguity, and passes raw device pointers and the current HIP stream to the C ABI declared in
include/anvil.h.  All arithmetic happens in the library's HIP kernels; if the library is missing
the functions raise instead of computing anything another way.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libanvil.so")

ANVIL_OK = 0
ANVIL_ERR_INVALID_ARG = 1
ANVIL_ERR_UNSUPPORTED = 2
ANVIL_ERR_MISALIGNED = 3
ANVIL_ERR_ALIAS = 4
ANVIL_ERR_OOM = 5
ANVIL_ERR_HIP = 6
ANVIL_ERR_CAPTURING = 7
ANVIL_ERR_TOO_LARGE = 8
NOALLOC_SCRATCH_BYTES = 192 << 20   # ANVIL_NOALLOC_SCRATCH_BYTES of include/anvil.h

ANVIL_GRAD_F32 = 0
ANVIL_GRAD_BF16 = 1

# Every symbol include/anvil.h declares, with its ctypes signature (restype, argtypes).
_vp, _i64, _f, _i, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_int, ctypes.c_size_t
_d = ctypes.c_double
SIGNATURES = {
    "anvil_status_string": (ctypes.c_char_p, [_i]),
    "anvil_last_hip_error": (_i, []),
    "anvil_version": (_i, []),
    "anvil_bank_step": (_i, [_vp, _vp, _f, _f, _f, _vp, _i64, _i64, _i64, _vp]),
    "anvil_bank_step_ws": (_i, [_vp, _vp, _f, _f, _f, _vp, _i64, _i64, _i64, _vp, _sz, _vp]),
    "anvil_bank_step_noalloc": (_i, [_vp, _vp, _f, _f, _f, _vp, _i64, _i64, _i64, _vp]),
    "anvil_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "anvil_release_workspaces": (_i, []),
    "anvil_momentum": (_i, [_vp, _vp, _f, _f, _f, _vp, _i64, _i64, _i64, _vp]),
    "anvil_trace_slots": (_i64, [_i64, _i64]),
    "anvil_gram": (_i, [_vp, _vp, _vp, _i64, _i64, _i64, _vp]),
    "anvil_normalize": (_i, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp]),
    "anvil_poly": (_i, [_vp, _vp, _f, _f, _i64, _i64, _vp]),
    "anvil_apply": (_i, [_vp, _vp, _vp, _f, _i, _i64, _i64, _i64, _vp]),
    "anvil_bank_update": (_i, [_vp, _vp, _f, _f, _f, _vp, _vp, _d, _vp, _vp, _f, _vp,
                               _i64, _i64, _i64, _vp]),
    "anvil_bank_update_ws": (_i, [_vp, _vp, _f, _f, _f, _vp, _vp, _d, _vp, _vp, _f, _vp,
                                  _i64, _i64, _i64, _vp, _sz, _vp]),
    "anvil_equalizer_lanes": (_i64, [_i64, _i64]),
    "anvil_bank_step_dev": (_i, [_vp, _i, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _sz, _vp]),
    "anvil_bank_update_dev": (_i, [_vp, _i, _vp, _vp, _vp, _vp, _d, _vp, _vp, _vp, _i64, _i64,
                                   _i64, _vp, _sz, _vp]),
    "anvil_bank_step_maps": (_i, [_vp, _vp, _f, _f, _f, _vp, _i, _vp, _i64, _i64, _i64, _vp, _sz,
                                  _vp]),
    "anvil_equalize": (_i, [_vp, _vp, _d, _vp, _i64, _i64, _i64, _vp]),
    "anvil_decay_update": (_i, [_vp, _vp, _vp, _f, _vp, _vp, _i64, _i64, _i64, _vp]),
    "anvil_layer_norm": (_i, [_vp, _i64, _vp, _vp, _i, _f, _vp, _i64, _vp, _vp, _i, _i64, _i64,
                              _vp]),
    "anvil_layer_norm_grad": (_i, [_vp, _i64, _vp, _i64, _vp, _i, _vp, _vp, _vp, _i64, _vp, _vp,
                                   _i, _i64, _i64, _vp, _sz, _vp]),
    "anvil_layer_norm_grad_workspace": (_sz, [_i64, _i64]),
    "anvil_linear": (_i, [_vp, _i64, _vp, _i, _vp, _i, _i, _vp, _i64, _vp, _i64, _vp, _i64, _i,
                          _i64, _i64, _i64, _vp]),
    "anvil_linear_grad_input": (_i, [_vp, _i64, _vp, _i, _vp, _i64, _i, _vp, _i64, _vp, _i64, _i,
                                     _i64, _i64, _i64, _vp]),
    "anvil_linear_grad_weight": (_i, [_vp, _i64, _vp, _i64, _i, _vp, _i, _vp, _i, _i64, _i64,
                                      _i64, _vp, _sz, _vp]),
    "anvil_linear_grad_weight_workspace": (_sz, [_i, _i64, _i64, _i64, _i64]),
    "anvil_activation_grad": (_i, [_vp, _i64, _vp, _i64, _i, _vp, _i64, _i, _i64, _i64, _vp]),
    "anvil_expert_linear": (_i, [_vp, _i64, _vp, _i, _vp, _i, _i64, _vp, _i, _i, _vp, _i64, _vp,
                                 _i64, _vp, _i64, _i, _i64, _i64, _i64, _vp]),
    "anvil_expert_grad_input": (_i, [_vp, _i64, _vp, _i, _vp, _i, _i64, _vp, _i64, _i, _vp, _i64,
                                     _vp, _i64, _i, _i64, _i64, _i64, _vp]),
    "anvil_expert_grad_weight": (_i, [_vp, _i64, _vp, _i64, _i, _vp, _i, _i64, _vp, _i, _vp, _i,
                                      _i64, _i64, _i64, _vp, _sz, _vp]),
}

_lib = None


class AnvilError(RuntimeError):
    def __init__(self, fn: str, status: int, lib):
        self.status = status
        msg = lib.anvil_status_string(status).decode()
        if status == ANVIL_ERR_HIP:
            msg += f" (hipError {lib.anvil_last_hip_error()})"
        super().__init__(f"{fn}: {msg}")


def load(path: str | None = None):
    """Load libanvil.so (built in-tree by build.py) and declare its signatures."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is not built; run `python -m orthogonalizing_polynomial_cascade_amd.build`")
    lib = ctypes.CDLL(p)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _lib = lib
    return lib


def _check(fn: str, status: int):
    if status != ANVIL_OK:
        raise AnvilError(fn, status, load())


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _need(t, name, dtype, shape=None):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on the GPU (got {t.device})")
    if t.device.index is not None and t.device.index != torch.cuda.current_device():
        # the library launches on the current HIP device and takes plain device pointers
        raise ValueError(f"{name} is on {t.device}, not on the current device "
                         f"cuda:{torch.cuda.current_device()} (use torch.cuda.set_device)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")


def _gmn(grad):
    if grad.dim() != 3:
        raise ValueError("expected a [g, m, n] stack")
    return tuple(int(v) for v in grad.shape)


def workspace_bytes(g: int, m: int, n: int) -> int:
    return int(load().anvil_workspace_bytes(g, m, n))


def trace_slots(m: int, n: int) -> int:
    return int(load().anvil_trace_slots(m, n))


def release_workspaces():
    _check("anvil_release_workspaces", load().anvil_release_workspaces())


def anvil_bank_step(grad, velocity, momentum, fast_beta, fast_weight, out=None, workspace=None,
                    stream=None):
    """One ANVIL bank step on a [g, m, n] fp32 gradient stack.

    velocity (fp32 [2, g, m, n]) is updated in place; the bf16 update is written to `out`
    (allocated when None) and returned.  With `workspace` (a uint8 device tensor of at least
    workspace_bytes(g, m, n) bytes) the call allocates nothing.
    """
    import torch
    lib = load()
    _need(grad, "grad", torch.float32)
    g, m, n = _gmn(grad)
    _need(velocity, "velocity", torch.float32, (2, g, m, n))
    if out is None:
        out = _empty((g, m, n), torch.bfloat16, grad.device, stream)
    _need(out, "out", torch.bfloat16, (g, m, n))
    if workspace is None:
        st = lib.anvil_bank_step(_ptr(grad), _ptr(velocity), momentum, fast_beta, fast_weight,
                                 _ptr(out), g, m, n, _stream(stream))
        _check("anvil_bank_step", st)
    else:
        _need(workspace, "workspace", torch.uint8)
        st = lib.anvil_bank_step_ws(_ptr(grad), _ptr(velocity), momentum, fast_beta, fast_weight,
                                    _ptr(out), g, m, n, _ptr(workspace), workspace.numel(),
                                    _stream(stream))
        _check("anvil_bank_step_ws", st)
    return out


def anvil_bank_step_noalloc(grad, velocity, momentum, fast_beta, fast_weight, out, stream=None):
    """anvil_bank_step with the library's built-in device scratch: the C call allocates nothing.
    `out` (bf16 [g, m, n]) must be given; the bank's workspace_bytes(g, m, n) may be at most
    NOALLOC_SCRATCH_BYTES.  Calls on one device share that scratch (order them)."""
    import torch
    lib = load()
    _need(grad, "grad", torch.float32)
    g, m, n = _gmn(grad)
    _need(velocity, "velocity", torch.float32, (2, g, m, n))
    _need(out, "out", torch.bfloat16, (g, m, n))
    _check("anvil_bank_step_noalloc", lib.anvil_bank_step_noalloc(
        _ptr(grad), _ptr(velocity), momentum, fast_beta, fast_weight, _ptr(out), g, m, n,
        _stream(stream)))
    return out


def anvil_bank_step_maps(grad, velocity, momentum, fast_beta, fast_weight, maps, out=None,
                         workspace=None, stream=None):
    """The bank step with a caller-chosen list of (a, b, c) quintic maps (1 to 16 of them)."""
    import torch
    lib = load()
    _need(grad, "grad", torch.float32)
    g, m, n = _gmn(grad)
    _need(velocity, "velocity", torch.float32, (2, g, m, n))
    table = [float(v) for abc in maps for v in abc]
    if len(table) != 3 * len(maps):
        raise ValueError("maps must be (a, b, c) triples")
    host = (ctypes.c_float * max(1, len(table)))(*table)
    if out is None:
        out = _empty((g, m, n), torch.bfloat16, grad.device, stream)
    _need(out, "out", torch.bfloat16, (g, m, n))
    ws, wsb = None, 0
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8)
        ws, wsb = _ptr(workspace), workspace.numel()
    _check("anvil_bank_step_maps", lib.anvil_bank_step_maps(
        _ptr(grad), _ptr(velocity), momentum, fast_beta, fast_weight,
        ctypes.cast(host, ctypes.c_void_p), len(maps), _ptr(out), g, m, n, ws, wsb,
        _stream(stream)))
    return out


def _grad_dtype(grad):
    import torch
    if grad.dtype == torch.float32:
        return ANVIL_GRAD_F32
    if grad.dtype == torch.bfloat16:
        return ANVIL_GRAD_BF16
    raise TypeError("grad must be float32 or bfloat16")


def anvil_bank_step_dev(grad, velocity, scalars, out, workspace, stream=None):
    """The bank step with an fp32 or bf16 gradient and device scalars (fp32 [>= 3]: momentum,
    fast_beta, fast_weight) into fixed buffers; allocates nothing (graph-capturable)."""
    import torch
    lib = load()
    kind = _grad_dtype(grad)
    _need(grad, "grad", grad.dtype)
    g, m, n = _gmn(grad)
    _need(velocity, "velocity", torch.float32, (2, g, m, n))
    _need(scalars, "scalars", torch.float32)
    if scalars.numel() < 3:
        raise ValueError("scalars must hold momentum, fast_beta, fast_weight")
    _need(out, "out", torch.bfloat16, (g, m, n))
    _need(workspace, "workspace", torch.uint8)
    _check("anvil_bank_step_dev", lib.anvil_bank_step_dev(
        _ptr(grad), kind, _ptr(velocity), _ptr(scalars), _ptr(out), g, m, n, _ptr(workspace),
        workspace.numel(), _stream(stream)))
    return out


def anvil_bank_update_dev(grad, velocity, scalars, update, lane_energy, beta2, param, mantissa,
                          eff_lr, workspace, stream=None):
    """The whole bank update in the page's bank contract: device scalars (fp32 [4]: momentum,
    fast_beta, fast_weight, eff_wd), fixed buffers, caller workspace; graph-capturable."""
    import torch
    lib = load()
    kind = _grad_dtype(grad)
    _need(grad, "grad", grad.dtype)
    g, m, n = _gmn(grad)
    _need(velocity, "velocity", torch.float32, (2, g, m, n))
    _need(scalars, "scalars", torch.float32)
    if scalars.numel() < 4:
        raise ValueError("scalars must hold momentum, fast_beta, fast_weight, eff_wd")
    _need(update, "update", torch.bfloat16, (g, m, n))
    _need(lane_energy, "lane_energy", torch.float32)
    if lane_energy.numel() != g * equalizer_lanes(m, n):
        raise ValueError("lane_energy must hold g * lanes values")
    _need(param, "param", torch.bfloat16, (g, m, n))
    if mantissa.dtype not in (torch.int16, torch.uint16):
        raise TypeError("mantissa must be a 16-bit integer tensor")
    _need(mantissa, "mantissa", mantissa.dtype, (g, m, n))
    _need(eff_lr, "eff_lr", torch.float32, (g,))
    _need(workspace, "workspace", torch.uint8)
    _check("anvil_bank_update_dev", lib.anvil_bank_update_dev(
        _ptr(grad), kind, _ptr(velocity), _ptr(scalars), _ptr(update), _ptr(lane_energy), beta2,
        _ptr(param), _ptr(mantissa), _ptr(eff_lr), g, m, n, _ptr(workspace), workspace.numel(),
        _stream(stream)))
    return update


def anvil_momentum(grad, velocity, momentum, fast_beta, fast_weight, x_out=None, stream=None):
    import torch
    lib = load()
    _need(grad, "grad", torch.float32)
    g, m, n = _gmn(grad)
    _need(velocity, "velocity", torch.float32, (2, g, m, n))
    if x_out is None:
        x_out = _empty((g, m, n), torch.bfloat16, grad.device, stream)
    _need(x_out, "x_out", torch.bfloat16, (g, m, n))
    _check("anvil_momentum", lib.anvil_momentum(_ptr(grad), _ptr(velocity), momentum, fast_beta,
                                                fast_weight, _ptr(x_out), g, m, n, _stream(stream)))
    return x_out


def anvil_gram(x, a_out=None, trace_partials=None, want_trace=False, stream=None):
    """Gram of each matrix of the bf16 stack x; returns (a_out, trace_partials or None)."""
    import torch
    lib = load()
    _need(x, "x", torch.bfloat16)
    g, m, n = _gmn(x)
    s = min(m, n)
    if a_out is None:
        a_out = _empty((g, s, s), torch.bfloat16, x.device, stream)
    _need(a_out, "a_out", torch.bfloat16, (g, s, s))
    if want_trace and trace_partials is None:
        trace_partials = _empty((g, trace_slots(m, n)), torch.float32, x.device, stream)
    if trace_partials is not None:
        _need(trace_partials, "trace_partials", torch.float32, (g, trace_slots(m, n)))
    _check("anvil_gram", lib.anvil_gram(_ptr(x), _ptr(a_out), _ptr(trace_partials), g, m, n,
                                        _stream(stream)))
    return a_out, trace_partials


def anvil_normalize(x, a, trace_partials, d_out=None, stream=None):
    """In-place x <- bf16(x / d), a <- bf16(a / d^2); returns d (fp32 [g])."""
    import torch
    lib = load()
    _need(x, "x", torch.bfloat16)
    g, m, n = _gmn(x)
    s = min(m, n)
    _need(a, "a", torch.bfloat16, (g, s, s))
    _need(trace_partials, "trace_partials", torch.float32, (g, trace_slots(m, n)))
    if d_out is None:
        d_out = _empty((g,), torch.float32, x.device, stream)
    _need(d_out, "d_out", torch.float32, (g,))
    _check("anvil_normalize", lib.anvil_normalize(_ptr(x), _ptr(a), _ptr(trace_partials),
                                                  _ptr(d_out), g, m, n, _stream(stream)))
    return d_out


def anvil_poly(a, coef_b, coef_c, b_out=None, stream=None):
    import torch
    lib = load()
    _need(a, "a", torch.bfloat16)
    g, s, s2 = _gmn(a)
    if s != s2:
        raise ValueError("a must be a stack of square matrices")
    if b_out is None:
        b_out = _empty(a.shape, a.dtype, a.device, stream)
    _need(b_out, "b_out", torch.bfloat16, (g, s, s))
    _check("anvil_poly", lib.anvil_poly(_ptr(a), _ptr(b_out), coef_b, coef_c, g, s, _stream(stream)))
    return b_out


def anvil_apply(x, b, coef_a, split, c_out=None, stream=None):
    import torch
    lib = load()
    _need(x, "x", torch.bfloat16)
    g, m, n = _gmn(x)
    s = min(m, n)
    _need(b, "b", torch.bfloat16, (g, s, s))
    if c_out is None:
        c_out = _empty(x.shape, x.dtype, x.device, stream)
    _need(c_out, "c_out", torch.bfloat16, (g, m, n))
    _check("anvil_apply", lib.anvil_apply(_ptr(x), _ptr(b), _ptr(c_out), coef_a, int(bool(split)),
                                          g, m, n, _stream(stream)))
    return c_out


def equalizer_lanes(m: int, n: int) -> int:
    return int(load().anvil_equalizer_lanes(m, n))


def anvil_bank_update(grad, velocity, momentum, fast_beta, fast_weight, lane_energy, beta2,
                      param, mantissa, eff_wd, eff_lr, update=None, workspace=None, stream=None):
    """One whole bank update (step, equalizer, sign-aligned decay).

    grad fp32 [g,m,n]; velocity fp32 [2,g,m,n], lane_energy fp32 [g, lanes], param bf16 [g,m,n]
    and mantissa int16/uint16 [g,m,n] are updated in place; eff_lr fp32 [g].  Returns the
    equalized bf16 update."""
    import torch
    lib = load()
    _need(grad, "grad", torch.float32)
    g, m, n = _gmn(grad)
    _need(velocity, "velocity", torch.float32, (2, g, m, n))
    _need(lane_energy, "lane_energy", torch.float32)
    if lane_energy.numel() != g * equalizer_lanes(m, n):
        raise ValueError("lane_energy must hold g * lanes values")
    _need(param, "param", torch.bfloat16, (g, m, n))
    if mantissa.dtype not in (torch.int16, torch.uint16):
        raise TypeError("mantissa must be a 16-bit integer tensor")
    _need(mantissa, "mantissa", mantissa.dtype, (g, m, n))
    _need(eff_lr, "eff_lr", torch.float32, (g,))
    if update is None:
        update = _empty((g, m, n), torch.bfloat16, grad.device, stream)
    _need(update, "update", torch.bfloat16, (g, m, n))
    args = [_ptr(grad), _ptr(velocity), momentum, fast_beta, fast_weight, _ptr(update),
            _ptr(lane_energy), beta2, _ptr(param), _ptr(mantissa), eff_wd, _ptr(eff_lr), g, m, n]
    if workspace is None:
        _check("anvil_bank_update", lib.anvil_bank_update(*args, _stream(stream)))
    else:
        _need(workspace, "workspace", torch.uint8)
        _check("anvil_bank_update_ws", lib.anvil_bank_update_ws(*args, _ptr(workspace),
                                                                workspace.numel(), _stream(stream)))
    return update


def anvil_equalize(update, lane_energy, beta2, lane_scratch=None, stream=None):
    """In-place equalizer on a bf16 [g,m,n] update; lane_energy fp32 [g, lanes] in place."""
    import torch
    lib = load()
    _need(update, "update", torch.bfloat16)
    g, m, n = _gmn(update)
    lanes = equalizer_lanes(m, n)
    _need(lane_energy, "lane_energy", torch.float32)
    if lane_energy.numel() != g * lanes:
        raise ValueError("lane_energy must hold g * lanes values")
    if lane_scratch is None:
        lane_scratch = _empty(2 * g * lanes, torch.float32, update.device, stream)
    _need(lane_scratch, "lane_scratch", torch.float32)
    if lane_scratch.numel() < 2 * g * lanes:
        raise ValueError("lane_scratch must hold 2 * g * lanes values")
    _check("anvil_equalize", lib.anvil_equalize(_ptr(update), _ptr(lane_energy), beta2,
                                                _ptr(lane_scratch), g, m, n, _stream(stream)))
    return update


def anvil_decay_update(param, mantissa, update, eff_wd, eff_lr, gate, stream=None):
    """In-place sign-aligned decay of (param bf16, mantissa uint16) by the bf16 update."""
    import torch
    lib = load()
    _need(param, "param", torch.bfloat16)
    g, m, n = _gmn(param)
    if mantissa.dtype not in (torch.int16, torch.uint16):
        raise TypeError("mantissa must be a 16-bit integer tensor")
    _need(mantissa, "mantissa", mantissa.dtype, (g, m, n))
    _need(update, "update", torch.bfloat16, (g, m, n))
    _need(eff_lr, "eff_lr", torch.float32, (g,))
    _need(gate, "gate", torch.float32, (g, m, n))
    _check("anvil_decay_update", lib.anvil_decay_update(_ptr(param), _ptr(mantissa), _ptr(update),
                                                        eff_wd, _ptr(eff_lr), _ptr(gate), g, m, n,
                                                        _stream(stream)))


def rail_scalars(step: int):
    """(momentum, fast_beta, fast_weight) of a training step under the source's rail schedule:
    fast rail only before step 514, blend weight 0.4385 on the fast rail from step 514 on; fast
    beta 0.85 and Nesterov momentum 0.95 throughout (the pre-engage beta scheduler is not given)."""
    return 0.95, 0.85, (1.0 if step < 514 else 0.4385)


# ---------------------------------------------------------------------------------------------
# Training operators around a bank.  Activations are [rows, width] tensors whose rows may lie any
# pitch apart (the last dimension contiguous); weights, biases and offsets are contiguous.
# ---------------------------------------------------------------------------------------------

ANVIL_F32, ANVIL_BF16, ANVIL_F16 = 0, 1, 2
ACTIVATIONS = {"none": 0, "relu": 1, "relu2": 2, "gelu": 3, "silu": 4}
_SIXTEEN = (ANVIL_BF16, ANVIL_F16)
_torch = None
_codes = {}

# A call of a small layer lasts as long as its preparation on the host, so these checks read each
# property of a tensor once.


def _module():
    global _torch
    if _torch is None:
        import torch
        _codes.update({torch.float32: ANVIL_F32, torch.bfloat16: ANVIL_BF16,
                       torch.float16: ANVIL_F16})
        _torch = torch
    return _torch


def _device(t, name):
    """The index of the current device, which t has to be on."""
    torch = _module()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU (got {t.device})")
    index = t.get_device()
    if index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, not on the current device "
                         f"cuda:{torch.cuda.current_device()} (use torch.cuda.set_device)")
    return index


def _raw_stream(stream, device):
    """The HIP stream handle of `stream`, by default the current one."""
    if stream is None:
        return _torch._C._cuda_getCurrentRawStream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _code(t, name, allowed):
    code = _codes.get(t.dtype)
    if code not in allowed:
        raise TypeError(f"{name} has an unsupported dtype ({t.dtype})")
    return code


def _same(t, name, dtype, device):
    if not isinstance(t, _torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device} (got {t.device})")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")


def _rows(t, name):
    """Checks the layout of a [rows, width] operand; returns (rows, width, row pitch)."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be [rows, width] (got {t.dim()} dimensions)")
    rows, width = t.shape
    pitch, step = t.stride()
    if step != 1 and width > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if pitch < width:
        if rows > 1:
            raise ValueError(f"{name}: its rows overlap (pitch {pitch}, width {width})")
        pitch = width
    return rows, width, pitch


def _operand(t, name, dtype, device, rows, width):
    """(pointer, pitch) of a further [rows, width] operand, or (None, 0)."""
    if t is None:
        return None, 0
    _same(t, name, dtype, device)
    r, w, pitch = _rows(t, name)
    if r != rows or w != width:
        raise ValueError(f"{name} must have shape {(rows, width)} (got {tuple(t.shape)})")
    return t.data_ptr(), pitch


def _dense(t, name, dtype, device, shape):
    """Pointer of a contiguous operand of the given shape."""
    _same(t, name, dtype, device)
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape} (got {tuple(t.shape)})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _parameter(t, name, code, like, device, shape):
    """(pointer, dtype code) of an optional parameter: fp32 or of the dtype of `like`."""
    if t is None:
        return None, code
    if not isinstance(t, _torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    own = _code(t, name, (ANVIL_F32, code))
    return _dense(t, name, t.dtype, device, shape), own


def _other_stream(stream):
    """`stream` as a torch stream where it is not the current one, else None."""
    torch = _module()
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if handle == torch.cuda.current_stream().cuda_stream:
        return None
    return stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(handle)


def _empty(shape, dtype, device, stream):
    """torch.empty for a call on `stream`.  For another stream than the current one the memory is that
    stream's own: whatever used it before was queued there too, ahead of this call (memory of the
    current stream may still be in use by what is queued on it).  The current stream, where the
    caller goes on with the tensor, is recorded as its second user."""
    torch = _torch or _module()
    other = None if stream is None else _other_stream(stream)
    if other is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(other):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream())
    return t


def _act(name):
    code = ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)} (got {name!r})")
    return code


def _scratch(workspace, need, device, stream):
    """The workspace: the caller's, or one of `need` bytes (None for 0)."""
    if workspace is None:
        return _empty((need,), _torch.uint8, device, stream) if need else None
    _same(workspace, "workspace", _torch.uint8, device)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace


def anvil_layer_norm(x, weight=None, bias=None, eps=1e-5, out=None, stream=None):
    """Layer norm of each row of x (bf16, fp16 or fp32 [rows, cols]); weight and bias [cols] are
    fp32 or of x's dtype.  Returns (y, mean, rstd), the last two fp32 [rows] for the backward
    pass (NaN where there are no columns)."""
    torch = _module()
    device = _device(x, "x")
    code = _code(x, "x", (ANVIL_F32, ANVIL_BF16, ANVIL_F16))
    rows, cols, ldx = _rows(x, "x")
    w, w_code = _parameter(weight, "weight", code, x, device, (cols,))
    b, b_code = _parameter(bias, "bias", code, x, device, (cols,))
    if w is not None and b is not None and w_code != b_code:
        raise TypeError("weight and bias must have one dtype")
    if out is None:
        out = _empty((rows, cols), x.dtype, x.device, stream)
    y, ldy = _operand(out, "out", x.dtype, device, rows, cols)
    stats = _empty((2, rows), _torch.float32, x.device, stream)
    mean, rstd = stats.unbind()
    at = stats.data_ptr()
    status = load().anvil_layer_norm(x.data_ptr(), ldx, w, b, w_code if w is not None else b_code,
                                     eps, y, ldy, at, at + 4 * rows, code, rows, cols,
                                     _raw_stream(stream, device))
    if status:
        _check("anvil_layer_norm", status)
    if cols == 0:   # the library returns at once; the mean of nothing is 0 / 0
        with torch.cuda.stream(None if stream is None else _other_stream(stream)):
            stats.fill_(float("nan"))
    return out, mean, rstd


def anvil_layer_norm_grad(dy, x, weight, mean, rstd, out=None, workspace=None, stream=None):
    """Backward pass of anvil_layer_norm: returns (dx, dweight, dbias), the last two fp32 [cols].
    Without a weight (None) it was 1; dweight and dbias are returned all the same."""
    device = _device(x, "x")
    code = _code(x, "x", (ANVIL_F32, ANVIL_BF16, ANVIL_F16))
    rows, cols, ldx = _rows(x, "x")
    g, lddy = _operand(dy, "dy", x.dtype, device, rows, cols)
    w, w_code = _parameter(weight, "weight", code, x, device, (cols,))
    m = _dense(mean, "mean", _torch.float32, device, (rows,))
    r = _dense(rstd, "rstd", _torch.float32, device, (rows,))
    if out is None:
        out = _empty((rows, cols), x.dtype, x.device, stream)
    dx, lddx = _operand(out, "out", x.dtype, device, rows, cols)
    sums = _empty((2, cols), _torch.float32, x.device, stream)
    dweight, dbias = sums.unbind()
    at = sums.data_ptr()
    lib = load()
    ws = _scratch(workspace, lib.anvil_layer_norm_grad_workspace(rows, cols), device, stream)
    status = lib.anvil_layer_norm_grad(
        g, lddy, x.data_ptr(), ldx, w, w_code, m, r, dx, lddx, at, at + 4 * cols, code, rows, cols,
        ws.data_ptr() if ws is not None else None, ws.numel() if ws is not None else 0,
        _raw_stream(stream, device))
    if status:
        _check("anvil_layer_norm_grad", status)
    return out, dweight, dbias


def _weight(w, dtype, device, w_kn, experts):
    """(pointer, n, k) of a weight matrix or stack."""
    _same(w, "w", dtype, device)
    if not w.is_contiguous():
        raise ValueError("w must be contiguous")
    shape = w.shape
    if len(shape) != (2 if experts is None else 3):
        raise ValueError("w must be [n, k], or [experts, n, k] for experts")
    if experts is not None and shape[0] != experts:
        raise ValueError(f"w holds {shape[0]} experts, offsets {experts}")
    n, k = shape[-2:]
    return (w.data_ptr(), k, n) if w_kn else (w.data_ptr(), n, k)


def _offsets(offsets, device):
    """(pointer, bits, experts) of the row offsets."""
    if not isinstance(offsets, _torch.Tensor):
        raise TypeError("offsets must be a torch.Tensor")
    if offsets.dtype not in (_torch.int32, _torch.int64):
        raise TypeError("offsets must be int32 or int64")
    if offsets.get_device() != device:
        raise ValueError(f"offsets must be on cuda:{device} (got {offsets.device})")
    if offsets.dim() != 1 or offsets.numel() < 1 or not offsets.is_contiguous():
        raise ValueError("offsets must be a contiguous [experts + 1] tensor")
    return offsets.data_ptr(), 32 if offsets.dtype == _torch.int32 else 64, offsets.numel() - 1


def _linear(fn, x, w, offsets, bias, residual, act, w_kn, keep_preact, preact, out, stream):
    device = _device(x, "x")
    code = _code(x, "x", _SIXTEEN)
    dtype = x.dtype
    rows, k, ldx = _rows(x, "x")
    group = () if offsets is None else _offsets(offsets, device)
    experts = group[2] if group else None
    wp, n, wk = _weight(w, dtype, device, w_kn, experts)
    if k != wk:
        raise ValueError(f"x has width {k}, w takes {wk}")
    b, b_code = _parameter(bias, "bias", code, x, device,
                           (n,) if experts is None else (experts, n))
    r, ldr = _operand(residual, "residual", dtype, device, rows, n)
    if out is None:
        out = _empty((rows, n), dtype, x.device, stream)
    y, ldy = _operand(out, "out", dtype, device, rows, n)
    if preact is None and keep_preact:
        preact = _empty((rows, n), dtype, x.device, stream)
    z, ldz = _operand(preact, "preact", dtype, device, rows, n)
    status = getattr(load(), fn)(
        x.data_ptr(), ldx, wp, 1 if w_kn else 0, *group, b, b_code, _act(act), r, ldr, y, ldy, z,
        ldz, code, rows, n, k, _raw_stream(stream, device))
    if status:
        _check(fn, status)
    return out, preact


def _grad_input(fn, dz, w, offsets, preact, act, add, w_kn, out, stream):
    device = _device(dz, "dz")
    code = _code(dz, "dz", _SIXTEEN)
    dtype = dz.dtype
    rows, n, lddz = _rows(dz, "dz")
    group = () if offsets is None else _offsets(offsets, device)
    wp, wn, k = _weight(w, dtype, device, w_kn, group[2] if group else None)
    if n != wn:
        raise ValueError(f"dz has width {n}, w gives {wn}")
    z, ldz = _operand(preact, "preact", dtype, device, rows, k)
    a, lda = _operand(add, "add", dtype, device, rows, k)
    if out is None:
        out = _empty((rows, k), dtype, dz.device, stream)
    dx, lddx = _operand(out, "out", dtype, device, rows, k)
    status = getattr(load(), fn)(
        dz.data_ptr(), lddz, wp, 1 if w_kn else 0, *group, z, ldz, _act(act), a, lda, dx, lddx,
        code, rows, n, k, _raw_stream(stream, device))
    if status:
        _check(fn, status)
    return out


def _grad_weight(fn, dz, x, offsets, w_kn, out, out_dtype, want_bias, workspace, stream):
    device = _device(dz, "dz")
    code = _code(dz, "dz", _SIXTEEN)
    rows, n, lddz = _rows(dz, "dz")
    _same(x, "x", dz.dtype, device)
    x_rows, k, ldx = _rows(x, "x")
    if x_rows != rows:
        raise ValueError(f"x has {x_rows} rows, dz {rows}")
    group = () if offsets is None else _offsets(offsets, device)
    stack = (group[2],) if group else ()
    shape = stack + ((k, n) if w_kn else (n, k))
    if out is None:
        out = _empty(shape, out_dtype or _torch.float32, dz.device, stream)
    dw, out_code = _parameter(out, "out", code, dz, device, shape)
    if want_bias and k == 0 and n:
        # nothing of a weight, and the library returns at once; its bias has a gradient all the same,
        # which does not depend on x: one column of dz stands in for it
        return out, _grad_weight(fn, dz, dz[:, :1], offsets, w_kn, None, None, True, None, stream)[1]
    dbias = _empty(stack + (n,), _torch.float32, dz.device, stream) if want_bias else None
    lib = load()
    need = lib.anvil_linear_grad_weight_workspace(1 if w_kn else 0, rows, n, k,
                                                  stack[0] if stack else 1)
    ws = _scratch(workspace, need, device, stream)
    status = getattr(lib, fn)(
        dz.data_ptr(), lddz, x.data_ptr(), ldx, 1 if w_kn else 0, *group, dw, out_code,
        dbias.data_ptr() if want_bias else None, code, rows, n, k,
        ws.data_ptr() if ws is not None else None, ws.numel() if ws is not None else 0,
        _raw_stream(stream, device))
    if status:
        _check(fn, status)
    return out, dbias


def anvil_linear(x, w, bias=None, residual=None, act="none", w_kn=False, keep_preact=False,
                 preact=None, out=None, stream=None):
    """Linear layer y = act(x w^T + bias) + residual with w [n, k] (w_kn: x w, w [k, n]); x bf16 or
    fp16 [rows, k], act one of ACTIVATIONS, bias fp32 or of x's dtype.  Returns (y, z), z the
    preactivation x w^T + bias where keep_preact asks for it or `preact` receives it, else None."""
    return _linear("anvil_linear", x, w, None, bias, residual, act, w_kn, keep_preact, preact, out,
                   stream)


def anvil_linear_grad_input(dz, w, preact=None, act="none", add=None, w_kn=False, out=None,
                            stream=None):
    """dx = (dz w) * act'(preact) + add: the gradient of a linear layer's input x = act(preact)
    with respect to preact; add is a gradient that reaches it another way (a residual)."""
    return _grad_input("anvil_linear_grad_input", dz, w, None, preact, act, add, w_kn, out, stream)


def anvil_linear_grad_weight(dz, x, w_kn=False, out=None, out_dtype=None, want_bias=True,
                             workspace=None, stream=None):
    """(dw, dbias): dw = dz^T x [n, k] (w_kn: x^T dz [k, n]), fp32 or dz's dtype, and the fp32 sum of
    dz over the rows (None without want_bias)."""
    return _grad_weight("anvil_linear_grad_weight", dz, x, None, w_kn, out, out_dtype, want_bias,
                        workspace, stream)


def anvil_activation_grad(dy, preact, act, out=None, stream=None):
    """dz = dy * act'(preact), elementwise on [rows, n]."""
    device = _device(dy, "dy")
    code = _code(dy, "dy", _SIXTEEN)
    rows, n, lddy = _rows(dy, "dy")
    z, ldz = _operand(preact, "preact", dy.dtype, device, rows, n)
    if z is None:
        raise ValueError("preact must be given")
    if out is None:
        out = _empty((rows, n), dy.dtype, dy.device, stream)
    dz, lddz = _operand(out, "out", dy.dtype, device, rows, n)
    status = load().anvil_activation_grad(dy.data_ptr(), lddy, z, ldz, _act(act), dz, lddz, code,
                                          rows, n, _raw_stream(stream, device))
    if status:
        _check("anvil_activation_grad", status)
    return out


def anvil_expert_linear(x, w, offsets, bias=None, residual=None, act="none", w_kn=False,
                        keep_preact=False, preact=None, out=None, stream=None):
    """anvil_linear for a stack of experts: rows offsets[e] .. offsets[e + 1] - 1 of x go through
    w[e] (w [experts, n, k], bias [experts, n], offsets int32 or int64 [experts + 1] on the GPU).
    Rows outside every expert's range give zeros."""
    return _linear("anvil_expert_linear", x, w, offsets, bias, residual, act, w_kn, keep_preact,
                   preact, out, stream)


def anvil_expert_grad_input(dz, w, offsets, preact=None, act="none", add=None, w_kn=False, out=None,
                            stream=None):
    """anvil_linear_grad_input over the experts' groups of rows."""
    return _grad_input("anvil_expert_grad_input", dz, w, offsets, preact, act, add, w_kn, out,
                       stream)


def anvil_expert_grad_weight(dz, x, offsets, w_kn=False, out=None, out_dtype=None, want_bias=True,
                             workspace=None, stream=None):
    """anvil_linear_grad_weight over the experts' groups of rows: dw [experts, n, k], the gradient
    stack of the experts' bank, and dbias [experts, n]."""
    return _grad_weight("anvil_expert_grad_weight", dz, x, offsets, w_kn, out, out_dtype, want_bias,
                        workspace, stream)
