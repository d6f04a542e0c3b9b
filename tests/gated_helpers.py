"""Plain 64-bit forms of the gated linear layer and its gradient, with bounds on the fp32 errors before the
results are rounded (see layer_helpers)."""
import torch

from tests import layer_helpers as H


def forward(x, w, bias, name, w_kn):
    """(h, bound on its error, z, bound on its error)."""
    _, z, ez = H.linear(x, w, bias, None, "none", w_kn)
    gate, up = z.chunk(2, -1)
    eg, eu = ez.chunk(2, -1)
    a = H.act(gate, name)
    h = a * up
    ea = H.forward_error(gate, eg, a, None, name)
    return h, ea * (up.abs() + eu) + a.abs() * eu + 2 * H.U32 * h.abs(), z, ez


def grad_from(dh, err, z, name):
    """(dz, bound) from dh with an error of `err`: the slope within thirty-two steps of fp32 (its terms may cancel:
    eight steps of the factor it is made of), the activation within sixteen."""
    gate, up = z.double().chunk(2, -1)
    slope, a = H.act_slope(gate, name), H.act(gate, name)
    dg, du = dh * up * slope, dh * a
    eg = err * (up * slope).abs() + 32 * H.U32 * dg.abs() + 8 * H.U32 * (dh * up).abs()
    eu = err * a.abs() + 32 * H.U32 * du.abs() + 16 * H.U32 ** 2 * (dh * gate).abs()
    return torch.cat([dg, du], -1), torch.cat([eg, eu], -1)


def grad(dy, w, z, name, w_kn):
    """(dz, bound) through the layer of weight w."""
    dh, err = H.grad_input(dy, w, None, "none", None, w_kn)
    return grad_from(dh, err, z, name)
