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
  * keys and values rounded before the products: coordinates off by up to kabs (vabs) per
    token and by u of themselves; a score moves by scale (kabs sum|q_c| + u sum|q_c k_c|).
  * an fp16 output: u |o| + 2^-25.

The bound takes every rounding at its worst and all of one sign.  rms_bound takes them as
independent, for the root mean square over many outputs: P, the values' three roundings (two
in the rotation's products, one of the result) and the output's leave at most
u sqrt(5 / 3) of A; a score moves by scale |q| |k| / sqrt(128) * u sqrt(3 / 3) (the keys'
three), which moves the output by at most twice that share of A.  Rounded up: u (3 + 2 S) A,
S = scale |q| max|k| / sqrt(128)."""
import math

import torch

U16 = 2.0 ** -11


def attend64(q, k, v, first, scale=None, kabs=None, vabs=None, skip=None):
    """q [n, Hq, 128], k, v [L, Hkv, 128] (float64); query i attends tokens 0 .. first + i, but
    for those in skip [L].  kabs, vabs [L, Hkv]: coordinate errors of keys and values.
    Returns (out, A, e, V): the output, sum p |v|, the score error bound [n, Hq, 1] and the
    values' own error sum p (vabs + u |v|)."""
    n, Hq, d = q.shape
    L, Hkv = k.shape[0], k.shape[1]
    scale = 1.0 / math.sqrt(d) if not scale else scale
    G = Hq // Hkv
    out, A = torch.zeros_like(q), torch.zeros_like(q)
    e = torch.zeros((n, Hq, 1), dtype=torch.float64, device=q.device)
    V = torch.zeros_like(q)
    if n == 0 or L == 0:
        return out, A, e, V
    i = torch.arange(n, device=q.device)[:, None]
    j = torch.arange(L, device=q.device)[None, :]
    see = j <= first + i
    if skip is not None:
        see = see & ~skip[None, :]
    for h in range(Hq):
        s = q[:, h] @ k[:, h // G].T * scale
        s = torch.where(see, s, -math.inf)
        p = torch.where(see, torch.softmax(s, 1), 0.0)
        vh = v[:, h // G]
        vz = torch.where(torch.isfinite(vh), vh, 0.0)
        out[:, h] = p @ vz
        A[:, h] = p @ vz.abs()
        mag = torch.where(see, q[:, h].abs() @ torch.nan_to_num(k[:, h // G], 0.0, 0.0, 0.0).abs().T, 0.0)
        e[:, h, 0] = mag.amax(1) * scale * 128 * 2.0 ** -23 + 100 * 2.0 ** -24 + 2.0 ** -22
        if kabs is not None:
            off = torch.where(see, q[:, h].abs().sum(1, keepdim=True) * kabs[None, :, h // G] + U16 * mag, 0.0)
            e[:, h, 0] += scale * off.amax(1)
            V[:, h] = p @ vabs[:, h // G, None] + U16 * A[:, h]
    return out, A, e, V


def bound(out, A, e, V, n_tokens, vmax, fp16_out):
    b = (U16 + 2 * e) * A + V + n_tokens * 2.0 ** -25 * vmax
    if fp16_out:
        b = b + U16 * out.abs() + 2.0 ** -25
    return b


def rms_bound(A, q, k, n_heads_per, scale=None):
    """Per output, for the root mean square: q [n, Hq, 128], k [L, Hkv, 128]."""
    scale = 1.0 / math.sqrt(q.shape[2]) if not scale else scale
    kn = torch.nan_to_num(k, 0.0, 0.0, 0.0).norm(dim=2).amax(0).repeat_interleave(n_heads_per)
    S = scale * q.norm(dim=2) * kn / math.sqrt(128)
    return U16 * (3 + 2 * S)[..., None] * A
