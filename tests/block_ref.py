"""The feed-forward block's formulas in 64 bits on the CPU, with the bounds of the
kernels' errors, for the tests of its operators.

Bounds.  The kernels' exp2 and reciprocal are within an ulp (2^-23), products and sums
within half of one (U = 2^-24).
  logistic s(x): the exponent x log2 e is off by 1.5 U of itself (its rounding and the
  constant's), e^-x by |x| 1.5 U + 2^-23, and 1 + e^-x and the reciprocal add 2^-24 +
  2^-23: relatively (1 - s) (|x| 2^-23 + 2^-22) + 2^-22.
  normal Phi(-x) = q(x): the fit's 1.3e-7 = 2^-22.9, eight Horner steps on
  coefficients whose magnitudes add up to 1.9 of the sum (16 U), t's 2 ulp through a
  slope of at most 1 (2^-22), three products, and the exponent's roundings
  x^2 / 2 (3 U): relatively 2^-20 + x^2 2^-23.
  gelu's value alone is max(z, 0) - x 2^P(x), x = min(|z|, 6): the fit is within
  4.7e-8 < 2^-24 of x Phi(-x) up to 6 (6e-9 there, taken past it: 2^-26), seven Horner
  steps on terms that add up to A(x) < 1 + 1.16 x + 0.46 x^2 + 0.054 x^3 + 0.008 x^4 +
  0.0007 x^5 move P by 14 U A, so Phi by a factor ln 2 of that (10 U A), the exponential
  is off by 2 U and the last step by U of the result.
  tanh form: its inner x is off by 4 U of itself, which moves s by (1 - s) |x| 2^-22.
  An exponential below 2^-126 may be flushed: 2^-120 in all."""
import math

import torch

U = 2.0 ** -24
ROOT, CUBE = math.sqrt(2 / math.pi), 0.044715
TINY = 2.0 ** -120
BLOCK = 32
STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}     # a result's last rounding


def _logistic(x, inner=0.0):
    s, r = torch.sigmoid(x), torch.sigmoid(-x)
    return s, r, s * (r * (x.abs() * (2.0 ** -23 + inner) + 2.0 ** -22) + 2.0 ** -22) + TINY


def act(z, name):
    """(value, its error, slope, its error) of an fp32 z given in 64 bits."""
    a, one = z.abs(), torch.ones_like(z)
    if name == "none":
        return z, 0 * a, one, 0 * a
    if name == "relu":
        return z.clamp(min=0), 0 * a, (z > 0).double(), 0 * a
    if name == "gelu":
        # (erfc keeps the tail, which 1 + erf loses.)
        q = torch.special.erfc(a * math.sqrt(0.5)) / 2
        eq = q * (2.0 ** -20 + z * z * 2.0 ** -23) + TINY
        p = torch.special.erfc(z * -math.sqrt(0.5)) / 2
        ep = eq + U * p
        phi = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        ephi = phi * (z * z * 2.0 ** -23 + 2.0 ** -21) + TINY
        v, d = z * p, p + z * phi
        x = a.clamp(max=6.0)
        terms = 1 + 1.16 * x + 0.46 * x ** 2 + 0.054 * x ** 3 + 0.008 * x ** 4 + 0.0007 * x ** 5
        ev = 2.0 ** -24 + 2.0 ** -26 + x * q * U * (10 * terms + 2) + 2 * U * v.abs()
        return v, ev, d, ep + a * ephi + 3 * U * (p + a * phi)
    x, rate, inner = z, one, 0.0
    if name == "gelu_tanh":
        x, rate, inner = 2 * ROOT * (z + CUBE * z ** 3), 2 * ROOT * (1 + 3 * CUBE * z * z), 2.0 ** -22
    s, r, es = _logistic(x, inner)
    v = z * s
    # 1 - s is exact to an ulp of one: es and U; then products of a, s, 1 - s and rate.
    d = s + z * s * r * rate
    ed = es + a * rate * (es * (r + s) + s * U) + 6 * U * (s + a * s * r * rate)
    return v, a * es + U * v.abs(), d, ed


def checkpoint(z, F):
    """(codes, scales) of fp32 z [M, N] on the CPU, to the bit."""
    M, N = z.shape
    b = torch.nn.functional.pad(z.view(M, N // F, F), (0, -F % BLOCK)).view(M, N // F, -1, BLOCK)
    s = (b.abs().amax(3).double() / 127).float()        # one rounding: 127 is exact
    c = torch.where(s[..., None] > 0, b / s[..., None], 0.0).round().clamp(-127, 127)
    return c.view(M, N // F, -1)[:, :, :F].reshape(M, N).to(torch.int8), s.view(M, -1)


def restored(ck, ck_s, F):
    """fl(scale code) as fp32, [M, N]."""
    M, N = ck.shape
    each = ck_s.view(M, N // F, -1).repeat_interleave(BLOCK, 2)[:, :, :F].reshape(M, N)
    return ck.float() * each


def forward(z, F, name, residual=None):
    """(y, error) in 64 bits from the fp32 z, before y's rounding."""
    z = z.double()
    v, e, _, _ = act(z[:, :F], name)
    if z.shape[1] != F:
        u = z[:, F:]
        v, e = v * u, e * u.abs() + U * (v * u).abs()
    if residual is not None:
        v = v + residual.double()
        e = e + U * v.abs()
    return v, e


def backward(dy, z, F, name):
    """(dz, error) in 64 bits from dy and the restored fp32 z."""
    dy, z = dy.double(), z.double()
    v, ev, d, ed = act(z[:, :F], name)
    if z.shape[1] == F:
        g = dy * d
        return g, dy.abs() * ed + U * g.abs()
    u = z[:, F:]
    g, h = dy * u * d, dy * v
    return (torch.cat([g, h], 1),
            torch.cat([(dy * u).abs() * ed + 3 * U * g.abs(), dy.abs() * ev + 2 * U * h.abs()], 1))
