"""The AdamW step on the CPU: in fp32 with every operation rounded on its own, as the kernel's (so that results are
equal bit for bit), and in 64 bits.  The fp32 operations are numpy's, one rounding each whatever the CPU."""
import math

import numpy as np
import torch

BLOCK = 256


def master(param, mantissa):
    """fp32 values of a parameter, or of the two halves of its master."""
    if mantissa is None:
        return param.float()
    return ((param.view(torch.int16).int() << 16) | (mantissa.int() & 0xFFFF)).view(torch.float32)


def split(value):
    bits = value.view(torch.int32)
    return (bits >> 16).to(torch.int16).view(torch.bfloat16), (bits & 0xFFFF).to(torch.int16)


def _mix(h):
    h = ((h ^ (h >> 16)) * 0x7A3C5EB5) & 0xFFFFFFFF
    h = ((h ^ (h >> 15)) * 0x5D8E36CB) & 0xFFFFFFFF
    return h ^ (h >> 16)


def dither(seed, tensor, index):
    """The hash of each element, of which m takes the lowest 20 bits and the root of v the highest."""
    key = _mix(torch.tensor((seed + (tensor + 1) * 0x9E3779B9) & 0xFFFFFFFF))
    return _mix((index + key) & 0xFFFFFFFF)


def rows(v):
    """[n] as whole blocks, zeros past the end."""
    return torch.cat([v, v.new_zeros(-v.numel() % BLOCK)]).view(-1, BLOCK)


def _f(x):
    """A Python number, or a tensor, as numpy's fp32."""
    return x.numpy() if isinstance(x, torch.Tensor) else np.float32(x)


def _t(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32))


def decode(codes, scale):
    values = rows(codes.view(torch.uint8)).view(torch.float8_e4m3fn).float()
    return _t(_f(values) * _f(scale)[:, None]).view(-1)[:codes.numel()]


def encode(v, noise, least):
    """Codes and scales of fp32 values: floor of the value in steps of the e4m3 grid plus noise / 2^20."""
    n = v.numel()
    v, noise = rows(v), rows(noise)
    top = torch.where(torch.isnan(v), torch.zeros(()), v.abs()).amax(1, keepdim=True)
    there = top >= 2.0 ** -100
    with np.errstate(all="ignore"):
        inverse = torch.where(there, _t(_f(448.0) / _f(top)), torch.zeros(()))
        q = _t(np.abs(_f(v)) * _f(inverse))
        small = q < 2.0 ** -6
        bits = torch.where(small, _t(_f(q) + _f(2.0 ** -6)), q).view(torch.int32).long()
    code = ((bits + noise) >> 20) - torch.where(small, 968, 960)
    code = code.clamp(max=126)
    code = torch.where((q > 0) & (code < least), least, code)
    code = torch.where(torch.isnan(q), 127, code) + torch.where(v < 0, 128, 0)
    scale = torch.where(there, _t(_f(top) / _f(448.0)), torch.zeros(()))[:, 0]
    return code.to(torch.uint8).view(-1)[:n].view(torch.float8_e4m3fn), scale


def moments(grad, m, v, betas, clip):
    """m and v after the step, fp32 [n]."""
    with np.errstate(all="ignore"):
        g = _f(grad.float()) if clip is None else _f(grad.float()) * _f(clip)
        m = _f(m) * _f(betas[0]) + g * _f(1 - betas[0])
        return _t(m), _t(_f(v) * _f(betas[1]) + (g * g) * _f(1 - betas[1]))


def root_of(v):
    return _t(np.sqrt(_f(v)))


def weights(p, m, root, lr, wd, betas, eps, step):
    """fp32 weights after the step; lr and wd fp32 numbers with the multipliers in them."""
    fix1, fix2 = _f(1 / (1 - betas[0] ** step)), _f(1 / math.sqrt(1 - betas[1] ** step))
    with np.errstate(all="ignore"):
        return _t(_f(p) * (_f(1.0) - lr * wd) - lr * ((_f(m) * fix1) / (_f(root) * fix2 + _f(eps))))


def step32(state, i, lr, wd, betas, eps, step, clip, seed):
    """The state (dict of CPU tensors, flat) of tensor i after one step."""
    s = dict(state)
    eight = s["m"].dtype != torch.float32
    m, v = s["m"], s["v"]
    if eight:
        m, v = decode(m, s["m_scale"]), decode(v, s["v_scale"])
        with np.errstate(all="ignore"):
            v = _t(_f(v) * _f(v))
    m, v = moments(s["grad"], m, v, betas, clip)
    root = root_of(v)
    p = weights(master(s["param"], s["mantissa"]), m, root, _f(lr) * _f(s["lr_mul"]), _f(wd) * _f(s["wd_mul"]), betas, eps, step)
    if s["mantissa"] is None:
        s["param"] = p.to(s["param"].dtype)
    else:
        s["param"], s["mantissa"] = split(p)
    if not eight:
        s["m"], s["v"] = m, v
        return s
    h = dither(seed, i, torch.arange(m.numel()))
    s["m"], s["m_scale"] = encode(m, h & 0xFFFFF, 0)
    s["v"], s["v_scale"] = encode(root, h >> 12, 1)
    return s


def step64(p, grad, m, v, lr, wd, betas, eps, step, clip):
    """(p, m, v) in 64 bits, the hyperparameters the fp32 numbers that the step takes (but for its betas)."""
    g = grad.double() * (1 if clip is None else float(torch.tensor(clip, dtype=torch.float32)))
    m = betas[0] * m.double() + (1 - betas[0]) * g
    v = betas[1] * v.double() + (1 - betas[1]) * g * g
    return (1 - lr * wd) * p.double() - lr * (m / (1 - betas[0] ** step)) / ((v / (1 - betas[1] ** step)).sqrt() + eps), m, v
