"""The AdamW operators' formulas in 64 bits, on the CPU, for one tensor at a time,
and bounds of what each rounding in the kernels can add.

u = 2^-24 is half a step of fp32 (relative), 2^-8 of bf16.  Terms of second order
are covered by a factor of 1.01.
"""
import math

import torch

BLOCK = 256
U = 2.0 ** -24
TINY = 2.0 ** -148   # a step of the smallest fp32 numbers


def step_tolerance(p, x, m, v, m1, v1, upd, p1, lr, wd, beta1, beta2, eps, t, u_extra):
    """Bounds of |kernel - formula| for the new m, v (32 bits) and p (before a rounding to bf16).

    m: beta1, 1-beta1 and x are rounded, so is their product, and the sum once more;
    v: the same with x twice; then the update's own operations (u_extra half
    steps), what m and v are off by, and the last two sums."""
    em = 1.01 * U * ((beta1 * m).abs() + 3 * ((1 - beta1) * x).abs() + m1.abs()) + TINY
    ev = 1.01 * U * (beta2 * v + 5 * (1 - beta2) * x * x + v1) + 4 * TINY
    c1, c2 = 1 / (1 - beta1 ** t), 1 / (1 - beta2 ** t)
    den = (v1 * c2).sqrt() + eps
    # |sqrt(v + ev) - sqrt(v)| <= min(ev / (2 sqrt(v - ev)), sqrt(ev)) with the root's own size
    low = (v1 - ev).clamp(min=0)
    er = torch.where(low > 0, ev / (2 * low.clamp(min=1e-300).sqrt()), ev.sqrt()).minimum(ev.sqrt())
    eu = upd.abs() * (u_extra * U + 1.01 * er * math.sqrt(c2) / den) + 1.01 * em * c1 / den
    ep = 1.01 * (abs(lr) * (eu + 3 * U * (wd * p).abs() + 3 * U * upd.abs()) + U * p1.abs()) + TINY
    return em, ev, ep


def step(p, g, m, v, t, lr, wd, scale=1.0, beta1=0.9, beta2=0.999, eps=1e-8):
    """(p, m, v) after a step, all in 64 bits, with the update u."""
    x = g * scale
    m1 = beta1 * m + (1 - beta1) * x
    v1 = beta2 * v + (1 - beta2) * x * x
    upd = (m1 / (1 - beta1 ** t)) / ((v1 / (1 - beta2 ** t)).sqrt() + eps)
    return p - lr * (upd + wd * p), m1, v1, upd


def blocks(x):
    """A flat tensor as [blocks, BLOCK], filled up with zeros."""
    return torch.nn.functional.pad(x, (0, -x.numel() % BLOCK)).view(-1, BLOCK)


def tops(m, v):
    """The largest |m| and sqrt(v) of each block in 64 bits (NaN where one is not finite)."""
    finite = blocks(m).isfinite().all(-1) & blocks(v).isfinite().all(-1)
    return [torch.where(finite, blocks(x).abs().amax(-1), math.nan) for x in (m, v.sqrt())]


def is_rounded(scale, top):
    """Whether each scale is its block's largest value in 64 bits rounded to fp32.

    Where that value lies in the middle of two fp32 numbers, to 64 bits' own
    rounding (1e-15 of it), either of them will do.  That is no rare event: after a
    step without a gradient the largest m is 0.9 times an fp32 number s, and 9 s / 10 is
    such a middle for every tenth s."""
    rounded = top.float()
    middle = (scale.double() - top).abs() <= (rounded.double() - top).abs() + 1e-15 * top
    return (scale == rounded) | (scale.isnan() & top.isnan()) | middle


def encode(m, v, sm, sr):
    """cm, cv (flat, of m's length) of moments in 64 bits with these scales, by looking
    at all values that a code can stand for; and how near (relative) the nearest border came."""
    n = m.numel()
    out, near = [], math.inf
    for x, top, steps in ((m, sm, 127), (v.sqrt(), sr, 255)):
        b = blocks(x)
        y = torch.where(top[:, None] > 0, b.abs() / top.double()[:, None], 0.0) * steps ** 2
        squares = torch.arange(steps + 1, dtype=torch.float64).square()
        borders = (squares[1:] + squares[:-1]) / 2
        code = torch.searchsorted(borders, y, right=True)          # y == border: the larger
        d = torch.minimum((y - borders[(code - 1).clamp(min=0)]).abs(), (y - borders[code.clamp(max=steps - 1)]).abs())
        near = min(near, float((d / y.clamp(min=0.5)).min()))
        if steps == 255:
            code = torch.where((b > 0) & (top[:, None] > 0), code.clamp(min=1), code)
        else:
            code = code * b.sign().nan_to_num().long()
        code = torch.where(top[:, None].isnan(), 0, code)
        out.append(code.view(-1)[:n].to(torch.int8 if steps == 127 else torch.uint8))
    return *out, near


def decode(cm, cv, sm, sr):
    """m and v in 64 bits of a flat tensor's codes and scales."""
    at = torch.arange(cm.numel()) // BLOCK
    c, q = cm.double(), cv.double()
    return c * c.abs() * sm.double()[at] / 127 ** 2, (q * q * sr.double()[at] / 255 ** 2) ** 2
