"""Attention in 64 bits and a derived bar for the 16-bit attention kernel.

With p the softmax weights of a row, A = sum_j p_j |v_j| per channel and n keys, the kernel's output is
off by at most, to first order:
  eps/2 |o|                  its rounding to the output type
  eps/2 A                    the rounding of each weight before the second product
  2 (ds + 7.6e-5) A          the weights themselves, in numerator and sum: ds the absolute error of the
                             exponent (natural units), 7.6e-5 the exp2 polynomial
  (n 2^-24 + n 2^-31) A'     fp32 accumulation of n terms; fp16 subnormal steps (2^-25 in units where the
                             row's largest weight is at least 2^7), A' = the largest |v| of the row's keys
ds: the scores are fp32 sums of d products; d 2^-24 sum_c |q_c k_c| bounds the sum, and one more
factor of two covers the multiply-add that forms the exponent: 2^-16 sum_c |q_c k_c| sm_scale for d <= 128.
"""
import math

import torch


def attend(q, k, v, seen, sm_scale):
    """q [h, n, d], k, v [h, m, d] (any float type), seen [n, m] -> (o, bar without the eps terms, A) in 64 bits."""
    q, k, v = q.double(), k.double(), v.double()
    x = q @ k.transpose(-1, -2) * sm_scale
    x = x.masked_fill(~seen, -math.inf)
    ds = 2.0 ** -16 * sm_scale * (q.abs() @ k.abs().transpose(-1, -2)).masked_fill(~seen, 0.0).amax(-1, keepdim=True)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top.isfinite(), top, torch.zeros_like(top)))
    l = p.sum(-1, keepdim=True)
    p = torch.where(l > 0, p / l.clamp(min=1e-300), torch.zeros_like(p))
    A = p @ v.abs()
    most = v.abs().amax(1, keepdim=True)
    n = x.shape[-1]
    return p @ v, 2 * (ds + 7.6e-5) * A + (n * 2.0 ** -24 + n * 2.0 ** -31) * most, A


def assert_attention(got, ref, extra, A):
    half = torch.finfo(got.dtype).eps / 2
    bar = 1.02 * (half * (ref.abs() + A) + extra) + (2.0 ** -24 if got.dtype == torch.float16 else 0.0)
    d = (got.double() - ref).abs()
    assert torch.isfinite(got).all()
    assert (d <= bar).all(), (float((d / bar).max()), float(d.max()))
