"""Plain 64-bit forms and derived error bounds of the cached-serving operators.

The format of the 8-bit cache (see include/fa.h) and attention over a prefix
followed by a sequence's own rows, from their definitions, in numpy.  e4m3
codes are handled as the values they stand for (torch's table of the type).
"""

import numpy as np
import torch

import oracle

# the value of each of the 256 e4m3 codes
CODES = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()


def quantise(x):
    """(values of the codes, exponent bytes) of rows x [..., D] (float64)."""
    finite = np.where(np.isfinite(x), np.abs(x), 0.0)
    m, e = np.frexp(finite.max(-1))
    e = np.where(m <= 0.875, e - 9, e - 8)                  # 448 = 0.875 * 2^9
    e = np.maximum(np.where(m == 0, -127, e), -127)
    y = np.where(np.isfinite(x), x, 0.0) * np.exp2(-e.astype(np.float64))[..., None]
    _, ye = np.frexp(np.maximum(np.abs(y), 2.0 ** -6))      # normal from 2^-6 on
    step = np.exp2(ye - 4.0)                                # three bits after the leading one
    codes = np.rint(y / step) * step                        # rint: half to even
    return np.where(np.isfinite(x), codes, np.nan), (e + 127).astype(np.uint8)


def values(codes, exps):
    """Rows as numbers from uint8 code bits and exponent bytes."""
    return CODES[codes] * np.exp2(exps.astype(np.float64) - 127)[..., None]


def attend(q, k, v, scale, causal):
    """(O, L, A, S) for one key head: q [r, nq, D] (its query heads), keys and
    values [n, D].  A = sum_j w_j |v_j|, S = the largest sum_d |q_d k_jd| scale
    over the keys a row sees: what the rounding errors are relative to."""
    r, nq, D = q.shape
    n = k.shape[0]
    O, A = np.zeros_like(q), np.zeros_like(q)
    L, S = np.full((r, nq), -np.inf), np.zeros((r, nq))
    for g in range(r):
        O[g], L[g] = oracle.forward_cached_head(q[g], k, v, scale, causal)
        for i in range(nq):
            seen = n if not causal else max(0, n - nq + i + 1)
            if seen:
                w = np.exp(q[g, i] @ k[:seen].T * scale - L[g, i])
                A[g, i] = w @ np.abs(v[:seen])
                S[g, i] = (np.abs(q[g, i]) @ np.abs(k[:seen]).T).max() * scale
    return O, L, A, S


def o_bound(O, A, S, n, D, vmax, out_dtype, p_dtype):
    """How far an output may be off.

    A score is a float32 sum of D products (each at most one step of 2^-23 of
    the running sum, which S bounds) and enters 2^x with a step of 2^-23 of its
    own size and 2^-22 of the exponential's: e = (D + 4) 2^-23 S + 2^-22 relative to each weight.
    The weights are rounded to p_dtype (half a step u_p, and for fp16 2^-24
    absolute, for weights relative to their largest: fp16's subnormals end at
    2^-25, the 8-bit cache's weights in three e4m3 terms, c0 + c1 / 32 + c2 / 1024 times
    2^-4, at half of 2^-9 / 1024 / 16 = 2^-24), summed with n float32 additions in
    the numerator and in the denominator, and the quotient is rounded to
    out_dtype (half a step u_o)."""
    u_o, u_p = torch.finfo(out_dtype).eps / 2, torch.finfo(p_dtype).eps / 2
    e = (D + 4) * 2.0 ** -23 * S + 2.0 ** -22
    tiny = 2.0 ** -24 * n * vmax if p_dtype == torch.float16 else 0.0
    rel = u_p + 2 * e + 2 * n * 2.0 ** -23
    return u_o * np.abs(O) + (rel[..., None] * A + tiny) * (1 + u_o) + torch.finfo(out_dtype).smallest_normal * u_o


def lse_bound(L, S, n, D):
    """Scores as above; the sum of n exponentials, its logarithm (2^-22) and the
    result's own rounding."""
    e = (D + 4) * 2.0 ** -23 * S + 2.0 ** -22
    return e + n * 2.0 ** -23 + 2.0 ** -21 + 2.0 ** -22 * np.abs(np.where(np.isfinite(L), L, 0.0))
