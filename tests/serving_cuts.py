"""Inputs of the decoding steps over a cache in which no part of the keys can be lost or
counted twice unseen, their outputs in 64 bits, and bounds that hold for just these inputs.

Every 64 keys of a part (the prefix, a sequence's own rows; half a tile of either
pass) put their values into one channel of the head width, so that a channel
holds a handful of halves: one missing or doubled changes it by a tenth and more.  Scores
are small and exact: queries are -1, 0, 1, keys -1/8, 0, 1/8, so that a product of two rows
is a multiple of 1/8 below 32 whatever the order of its sum, and with scale 2^-4 no
weight is below a twentieth of the largest.  Keys and values are exact in e4m3, fp16 and bf16.
"""

import numpy as np
import torch

HALF = 64
SCALE = 2.0 ** -4

CASES = [
    # (B, H, Hk, nq, np, cap, lens, D, dtype, own8)
    (1, 2, 1, 1, 0, 40000, [39990], 128, torch.bfloat16, True),        # one unit over all CTAs
    (1, 2, 2, 1, 0, 40000, [39990], 64, torch.float16, True),
    (1, 3, 1, 2, 0, 30000, [29990], 64, torch.bfloat16, False),        # 16-bit rows
    (2, 4, 1, 5, 0, 12000, [11990, 7000], 128, torch.float16, False),  # 20 rows: one CTA an SM
    (5, 2, 1, 1, 0, 3000, [2990, 100, 0, 2000, 61], 128, torch.float16, True),  # runs over several sequences
    (3, 28, 1, 1, 0, 5000, [5000, 1, 3300], 64, torch.bfloat16, True),  # 28 rows: two groups of 16
    (1, 1, 1, 1, 19584, 12, [10], 64, torch.bfloat16, False),          # the prefix's halves over all CTAs
    (2, 7, 1, 1, 20000, 700, [640, 30], 128, torch.float16, True),
    (40, 8, 2, 2, 9990, 40, None, 128, torch.bfloat16, True),          # 320 rows a key head: pairs of tiles
    (40, 4, 1, 1, 16000, 300, None, 64, torch.float16, False),         # 160 rows: the second tile part-filled
    (4, 8, 2, 3, 5000, 6000, [5990, 1200, 77, 3000], 128, torch.float16, True),
    (3, 4, 1, 5, 1500, 9000, [8990, 40, 4444], 128, torch.bfloat16, False),
]


def lengths(case):
    B, cap = case[0], case[5]
    return case[6] if case[6] is not None else [(17 * b + 16) % (cap + 1) for b in range(B)]


def channels(np_, n, D):
    """The channel of each of np_ + n keys, and the half it belongs to (numbered over both parts)."""
    own = 0 if np_ == 0 else D // 4 * 3                        # the own rows' first channel
    a, b = np.arange(np_) // HALF, np.arange(n) // HALF
    ch = np.concatenate([a % max(own, 1), own + b % (D - own)])
    return ch, np.concatenate([a, (a[-1] + 1 if np_ else 0) + b])


def magnitudes(n):
    return 1 + (np.arange(n) % 8) / 8


def inputs(case, seed=0):
    """q [B, H, nq, D], the prefix's k, v [Hk, np, D] and the own k, v [B, Hk, cap, D], as numpy."""
    B, H, Hk, nq, np_, cap, _, D = case[:8]
    rng = np.random.default_rng(seed)
    q = rng.integers(-1, 2, (B, H, nq, D)).astype(np.float32)
    kp, k = (rng.integers(-1, 2, s).astype(np.float32) / 8 for s in ((Hk, np_, D), (B, Hk, cap, D)))
    ch, _ = channels(np_, cap, D)
    vp, v = np.zeros((np_, D), np.float32), np.zeros((cap, D), np.float32)
    vp[np.arange(np_), ch[:np_]] = magnitudes(np_)
    v[np.arange(cap), ch[np_:]] = magnitudes(cap)
    return q, kp, np.broadcast_to(vp, kp.shape).copy(), k, np.broadcast_to(v, k.shape).copy()


def halves(case, q, kp, k, b, h, causal=True):
    """(den, num, ch) for sequence b and key head h: for every query row of the key head and every half,
    the sum of its weights e^s and of its weights times its values; and the half's channel."""
    B, H, Hk, nq, np_, cap, _, D = case[:8]
    n, r = lengths(case)[b], H // Hk
    keys = np.concatenate([kp[h], k[b, h, :n]]).astype(np.float64)
    rows = q[b, h * r:(h + 1) * r].reshape(r * nq, D).astype(np.float64)
    ch, half = channels(np_, n, D)
    if len(keys) == 0:
        return np.zeros((r * nq, 0)), np.zeros((r * nq, 0)), ch
    e = np.exp(rows @ keys.T * SCALE)
    if causal:
        last = np_ + n - nq + np.tile(np.arange(nq), r)
        e *= np.arange(np_ + n)[None] <= last[:, None]
    starts = np.flatnonzero(np.diff(half, prepend=-1))
    mag = np.concatenate([magnitudes(np_), magnitudes(n)])
    return np.add.reduceat(e, starts, 1), np.add.reduceat(e * mag, starts, 1), ch[starts]


def outputs(den, num, ch, D):
    """(O [rows, D], L [rows]) from the halves."""
    O = np.zeros((den.shape[0], D))
    np.add.at(O.T, ch, num.T)
    total = den.sum(1)
    with np.errstate(divide="ignore", invalid="ignore"):
        return np.where(total[:, None] > 0, O / total[:, None], 0.0), np.log(total)


def bounds(O, L, n, out_dtype, p_dtype):
    """(of O, of L) for these inputs, with n keys in all.

    Weights.  |s| < 2, so a score times log2 e, its float32 factor off by 3 2^-24, in one rounded fma, is
    off by at most 4 * 2^-24 * 4 = 2^-20, and the exponential by 2^-22 relative: e = 2^-20 of a weight.  It is rounded to
    p_dtype, half a step u_p (nothing is near the subnormals: no weight is below 2^-5 of its reference, which is
    at most 2^8 off).
    Normaliser.  A thread of the own rows adds a key a tile, n / 128 of them at most; one of the prefix 64 of a
    tile in a row, then the tiles; then a tree of 7, and at most 305 states (a CTA each, and one), a factor (2^-22), a product and a sum each: d
    = (n / 128 + 64 + 8 + 3 * 305) 2^-23.
    Values.  The terms of a channel that are not zero, at most its halves' keys, each addition off by at most
    2^-23 (sums in the tensor core may be cut, not rounded), and the joins as above.
    The quotient is rounded to out_dtype, half a step u_o."""
    u_o, u_p = torch.finfo(out_dtype).eps / 2, torch.finfo(p_dtype).eps / 2
    e, joins = 2.0 ** -20, 3 * 305 * 2.0 ** -23
    d = (n / 128 + 64 + 8) * 2.0 ** -23 + joins
    terms = HALF * -(-n // (HALF * 16))                         # 16: the fewest channels of a part
    rel = u_p + 2 * e + d + terms * 2.0 ** -23 + joins
    finite = np.where(np.isfinite(L), np.abs(L), 0.0)
    return (rel + u_o) * (1 + u_o) * np.abs(O), e + d + 2.0 ** -22 * (1 + finite)
