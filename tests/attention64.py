"""Plain 64-bit attention and the error bounds of the fp16 tensor-core kernels, for the
tests of tq_prompt_attention and tq_chunk_attention.

Bound of a row's output (unit roundoffs: fp16 u = 2^-11, fp32 2^-24), from the kernel's
roundings, with A = sum_j p_j |v_j| of the exact softmax weights p:
  * P is rounded to fp16: u A; below 2^-14 it is a subnormal with an absolute error of
    2^-25, and the sum it is divided by is at least 1: n 2^-25 max|v| for n tokens.
  * a score is a sum of 128 fp32 products scaled by scale: 128 * 2^-23 (the tensor core may
    truncate) of scale * sum_c |q_c k_c|, plus the rounding of the exponent's argument
    (2^-24 of up to 100) and of ex2 (2^-22).  A score error e moves the output by at most
    2 e A (numerator and denominator).
  * extra: rounding of the keys and values before the products (given by the caller).
  * an fp16 output: u |o| + 2^-25.
"""
import math

import torch

U16 = 2.0 ** -11


def attend64(q, k, v, first, scale=None):
    """q [n, Hq, 128], k, v [L, Hkv, 128] (float64); query i attends tokens 0 .. first + i.
    Returns (out, A, e): the output, sum p |v| and the score error bound [n, Hq, 1]."""
    n, Hq, d = q.shape
    L, Hkv = k.shape[0], k.shape[1]
    scale = 1.0 / math.sqrt(d) if not scale else scale
    G = Hq // Hkv
    out, A = torch.zeros_like(q), torch.zeros_like(q)
    e = torch.zeros((n, Hq, 1), dtype=torch.float64, device=q.device)
    if n == 0 or L == 0:
        return out, A, e
    i = torch.arange(n, device=q.device)[:, None]
    j = torch.arange(L, device=q.device)[None, :]
    see = j <= first + i
    for h in range(Hq):
        s = q[:, h] @ k[:, h // G].T * scale
        s = torch.where(see, s, -math.inf)
        p = torch.softmax(s, 1)
        p = torch.where(see, p, 0.0)
        vh = v[:, h // G]
        vz = torch.where(torch.isfinite(vh), vh, 0.0)
        out[:, h] = p @ vz
        A[:, h] = p @ vz.abs()
        mag = torch.where(see, q[:, h].abs() @ torch.nan_to_num(k[:, h // G], 0.0, 0.0, 0.0).abs().T, 0.0)
        e[:, h, 0] = mag.amax(1) * scale * 128 * 2.0 ** -23 + 100 * 2.0 ** -24 + 2.0 ** -22
    return out, A, e


def bound(out, A, e, n_tokens, vmax, fp16_out, extra=0.0):
    b = (U16 + 2 * e + extra) * A + n_tokens * 2.0 ** -25 * vmax
    if fp16_out:
        b = b + U16 * out.abs() + 2.0 ** -25
    return b
