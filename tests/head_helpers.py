"""Plain 64-bit form of the linear head's cross entropy and its gradients, with bounds on the GPU's errors (see
layer_helpers).  exp2 of the hardware is within one step of fp32 of its argument's exact value; its argument
(s - lse) log2(e) has been rounded three times, each time by at most 2^-24 of the larger of |s log2 e| and
|lse log2 e|, and that error of an exponent is a relative error of the value."""
import math

import torch

from tests import layer_helpers as H


def _logits(x, w, w_kn):
    wt = w.double() if w_kn else w.double().t()
    x = x.double()
    return x @ wt, H.sum_error(x, wt), wt


def counts_of(targets, vocab):
    t = targets.long().cpu()
    return (t >= 0) & (t < vocab)


def forward(x, w, targets, w_kn):
    """((loss, bound), (lse, bound))."""
    s, es, _ = _logits(x, w, w_kn)
    lse = torch.logsumexp(s, 1)
    n = s.shape[1]
    top = s.abs().amax(1)
    # the weighted mean of the logits' errors is at most their largest; an exponent's roundings, the additions of n
    # terms of one sign in blocks (each at most n + 64 roundings), the logarithm's and the maximum's sum
    el = es.amax(1) + H.U32 * (8 * 1.45 * (top + lse.abs()) + math.sqrt(n) * H.SIGMA + 32 + 4 * lse.abs())
    ok = counts_of(targets, n)
    at = torch.where(ok, targets.long().cpu(), 0)[:, None]
    loss = torch.where(ok, lse - s.gather(1, at)[:, 0], 0.0)
    e = torch.where(ok, el + es.gather(1, at)[:, 0] + 2 * H.U32 * (lse.abs() + loss.abs()), 0.0)
    return (loss, e), (lse, el)


def gradients(x, w, targets, lse, dloss, w_kn, t):
    """((dx, bound), (dw, bound)) from the GPU's fp32 lse.  P is off by half a step of its type, by its exponent's
    error and by the logit's; what an fp16 P loses below its smallest number is 2^-25 of the largest, 2^14."""
    s, es, wt = _logits(x, w, w_kn)
    l = lse.double().cpu()[:, None]
    ok = counts_of(targets, s.shape[1])
    p = torch.exp(s - l)
    ep = p * (es + H.U32 * 8 * 1.45 * (s.abs() + l.abs()) + 4 * H.U32)
    hot = torch.zeros_like(p)
    hot[ok, targets.long().cpu()[ok]] = 1.0
    weight = torch.where(ok, dloss.double().cpu(), 0.0)[:, None]
    p = torch.where(ok[:, None], p - hot, 0.0) * weight
    ep = torch.where(ok[:, None], (ep + 2 * H.U32 * hot) * weight.abs() + 2 * H.U32 * p.abs(), 0.0)
    # fp32 and bf16 have no values between 0 and 2^-126 for the hardware's exp2 and for the matrix cores: an exponential
    # below 2^-126 is taken as 0, and so may be its product with dloss.  Either changes P by less than 2^-126 times
    # the weight or 1
    ep = ep + 2.0 ** -126 * (1 + weight.abs())
    ep = ep + torch.finfo(t).eps / 2 * (p.abs() + ep)
    if t == torch.float16:
        finite = weight[torch.isfinite(weight)].abs()
        ep = ep + (finite.max() if finite.numel() else 0.0) * 2.0 ** -38
    xd = x.double()
    dx, dw = p @ wt.t(), (xd.t() @ p if w_kn else p.t() @ xd)
    # sums of errors: of independent signs, so SIGMA times the root of their squares
    ex = H.SIGMA * torch.sqrt((ep * ep) @ (wt.t() ** 2)) + H.sum_error(p, wt.t())
    if w_kn:
        ew = H.SIGMA * torch.sqrt((xd.t() ** 2) @ (ep * ep)) + H.sum_error(xd.t(), p)
    else:
        ew = H.SIGMA * torch.sqrt((ep * ep).t() @ (xd ** 2)) + H.sum_error(p.t(), xd)
    return (dx, ex), (dw, ew)
