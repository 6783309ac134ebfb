"""The root-mean-square norm and its gradient in 64 bits, and the tolerances
their outputs are held to.

Forward: r is fp32 of a 64-bit value, off by half a step (2^-24) and the 64-bit
sum's own error (K + 8 steps of 2^-53 at most); with that r everything else is
a fixed order of fp32 roundings, so outputs are compared bit for bit.

Gradient, with u(T) = finfo(T).eps / 2:
- s is a sum of K products of three fp32 factors (three roundings each), in
  chains of at most 64 that five shuffles and at most 16 warps join: it is off
  by at most (3 + 64 + 5 + 16) 2^-24 S, S = sum |w dy h|;
- f = s r^2 / K and dx = dh + r (w dy - h f) take eight more roundings of
  terms no larger than |dh| + r |w dy| + r |h| |f|, and one to T;
- dw sums rows products of two roundings in chains of at most `rows` that 32 +
  32 parts join: (rows + 2 + 64 + 64) 2^-24 sum |dy h r|.
"""
import torch


def forward64(h, w, eps):
    """(y, r) of float64 h [rows, K]."""
    r = 1.0 / torch.sqrt((h * h).sum(-1) / h.shape[-1] + eps)
    return h * r[:, None] * w, r


def vjp64(dy, h, w, r, dh=None):
    """(dx, dw), all float64."""
    r = r[:, None]
    dx = r * w * dy - h * r ** 3 * (w * dy * h).sum(-1, keepdim=True) / h.shape[-1]
    return dx if dh is None else dx + dh, (dy * h * r).sum(0)


def vjp_tolerance(dy, h, w, r, dh, dtype):
    """(of dx, of dw) for float64 inputs."""
    rows, K = h.shape
    u, e = torch.finfo(dtype).eps / 2, 2.0 ** -24
    r = r[:, None]
    p = (w * dy * h)
    S, s = p.abs().sum(-1, keepdim=True), p.sum(-1, keepdim=True)
    f = s.abs() * r ** 2 / K
    df = 88 * e * S * r ** 2 / K
    dx, _ = vjp64(dy, h, w, r[:, 0], dh)
    size = r * (w * dy).abs() + r * h.abs() * f + (0 if dh is None else dh.abs())
    tol = u * dx.abs() + (1 + u) * (r * h.abs() * df + 8 * e * size)
    tol = tol + torch.finfo(dtype).smallest_normal * 2 * u + 2.0 ** -148
    return tol, (rows + 130) * e * (dy * h * r).abs().sum(0) + 2.0 ** -140
