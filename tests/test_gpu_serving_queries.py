"""How exactly the 8-bit cache's products take a query: elements far below the largest of their row."""

import numpy as np
import pytest
import torch

import exact_io_aware_37_gb300 as fa
import serving_ref as ref
from exact_io_aware_37_gb300 import synth
from parity import f64
from test_gpu_serving import BF16, DEV, F16, F32, bits, check, ok, outputs, reference


def query_term(q, k, scale):
    """What holding queries as three e4m3 terms may add to a score: an element is off by at most 2^-26 of the
    largest magnitude M in its row (a row is scaled by a power of two to between 112 and 224, the last term's step is
    2^-9 / 1024, half of it 2^-20, and fp16's half step below its normals 2^-25: (2^-20 + 2^-25) / 112 < 2^-26).
    q [..., D], keys k [n, D]."""
    return 2.0 ** -26 * np.abs(q).max(-1) * np.abs(k).sum(-1).max() * scale


def as_score_size(x, D):
    """The score size S whose share e = (D + 4) 2^-23 S of serving_ref's bounds covers scores that are off by x more.
    Weights are then off by a factor within e^-x .. e^x, and so is their sum: a quotient by at most e^(2 x) - 1, where the
    bound has 2 e, so e = (e^(2 x) - 1) / 2; lse by x, which is less.  A hundredth more for the product with the other
    roundings' factors, which are below 1.01."""
    return 1.01 * np.expm1(2 * x) / 2 / ((D + 4) * 2.0 ** -23)


def cache_of(k, v):
    c = fa.cache_alloc(1, 1, k.shape[2], k.shape[3])
    fa.fa_cache_write(k.to(DEV), v.to(DEV), c)
    return c


@pytest.mark.gpu
@pytest.mark.parametrize("dtype, D, log2", [(BF16, 128, 8), (BF16, 64, 12), (BF16, 128, 16), (BF16, 64, 20), (F16, 128, 8),
                                            (F16, 64, 15), (BF16, 128, -100), (BF16, 128, 100)])
def test_one_channel_far_above_the_others(dtype, D, log2):
    """The large channel meets zeros in the keys, so that the scores are the other channels'."""
    cap = 200
    k, v = (synth.normal((1, 1, cap, D), 500 + i, F32) for i in range(2))
    k[..., 0] = 0
    q = synth.normal((1, 3, 1, D), 502, F32)
    scale, apart = D ** -0.5, log2
    if abs(log2) == 100:                                    # the same at either end of the type's range
        q, scale, log2, apart = q * 2.0 ** log2, scale * 2.0 ** -log2, log2 + 18, 18
    q[..., 0] = 2.0 ** log2
    q = q.to(dtype).to(DEV)
    c = cache_of(k, v)
    o, lse = outputs(q)
    fa.fa_decode_cache(q, c, None, o.t, lse.t, True, scale)
    assert ok()
    scale = float(np.float32(scale))
    O, L, A, S = reference(q, None, None, c, [cap], scale, True)
    keys = ref.values(bits(c.k), bits(c.k_exp))[0, 0]
    more = query_term(f64(q), keys, scale)
    if apart <= 8:
        assert (more <= 2.0 ** -22 + (D + 4) * 2.0 ** -23 * S).all()    # no more than a score's own sum may lose
    check(o.t, lse.t, (O, L, A, S + as_score_size(more, D)), cap, F16, 64.0)


def test_the_term_against_the_format():
    """Three terms of a scaled query, as the kernel takes them, element by element in 64 bits."""
    codes = np.unique(ref.CODES[np.isfinite(ref.CODES)])

    def nearest(x):
        i = np.clip(np.searchsorted(codes, x), 1, len(codes) - 1)
        lo, hi = codes[i - 1], codes[i]
        return np.where(x - lo <= hi - x, lo, hi)

    rng = np.random.default_rng(5)
    for dtype in (torch.bfloat16, torch.float16):
        x = torch.from_numpy((rng.standard_normal((300, 64)) * 2.0 ** rng.integers(-30, 8, (300, 64))).astype(np.float32))
        x = x.to(dtype).double().numpy()
        big = np.abs(x).max(-1, keepdims=True)
        e = np.ceil(np.log2(big / 448))
        y = (x * 0.5 / 2.0 ** e).astype(np.float16).astype(np.float64)
        assert np.all(np.abs(y).max(-1) <= 224) and np.all(np.abs(y).max(-1) >= 112)
        rest, total = y, 0.0
        for i in range(3):
            t = nearest(rest)
            total = total + t / 32.0 ** i
            rest = (rest - t) * 32
        off = np.abs(total * 2 * 2.0 ** e - x)
        assert np.all(off <= 2.0 ** -26 * big) and np.all(off[np.abs(x) >= 2.0 ** -15 * big] == 0)


@pytest.mark.gpu
@pytest.mark.parametrize("where", ["own8", "own16", "prefix"])
@pytest.mark.parametrize("dtype, D", [(BF16, 128), (F16, 64)])
@pytest.mark.parametrize("size", [1e5, 8e6, -8e6])
def test_scores_up_to_the_stated_size(where, dtype, D, size):
    """Exact scores of up to 2^23 in magnitude: the largest decides, and ties share.
    Queries and keys are small whole numbers and the scale a power of two, so that a score is a multiple of the scale,
    the same whatever its sum's order.  The scale is at least 64, and float32 is off by less than two log2 units at this
    size, so a smaller score's weight is below e^-62 and only the largest (one, or two tied ones of the same bits) count."""
    n = 300
    g = torch.Generator().manual_seed(7)
    q = torch.randint(-1, 2, (1, 2, 1, D), generator=g).float()
    k = torch.randint(-4, 5, (1, 1, n, D), generator=g).float()
    k[0, 0, 200] = k[0, 0, 13]                              # for D = 128 the largest of the first row, in another tile
    v = torch.randn(1, 1, n, D, generator=g).to(torch.float8_e4m3fn).float()
    if size < 0:                                            # all scores far below zero
        q[..., 0], k[..., 0] = 16.0, -64.0
    dots = q.view(2, D).double() @ k.view(n, D).double().T
    scale = 2.0 ** np.floor(np.log2(abs(size) / float(dots.abs().max())))
    assert float(dots.abs().max()) * scale < 2.0 ** 23 and scale >= 64 and (size > 0 or float(dots.max()) < -500)
    qd, kd, vd = (x.to(dtype).to(DEV) for x in (q, k, v))
    none = torch.empty(1, 0, D, dtype=dtype, device=DEV)
    if where == "own8":
        o, lse = fa.decode_cache(qd, cache_of(k, v), scale=scale)
    elif where == "own16":
        o, lse = fa.decode_shared(qd, none, none, (kd, vd), scale=scale)
    else:
        o, lse = fa.decode_shared(qd, kd[0], vd[0], (none[None], none[None]), scale=scale)
    assert ok()
    w = (dots == dots.amax(-1, keepdim=True)).double()
    w /= w.sum(-1, keepdim=True)
    O, A = (w @ v.view(n, D).double()).numpy(), (w @ v.view(n, D).double().abs()).numpy()
    u = torch.finfo(dtype).eps / 2                          # of a weight and of the output; 2^-20 for the rest
    assert (np.abs(f64(o).reshape(2, D) - O) <= (u + 2.0 ** -20) * A + u * np.abs(O)).all()
    # the scale's factor to log2 units, the maximum and its way back: half a step of 2^-23 each
    L = torch.logsumexp(dots * scale, -1).numpy()
    assert (np.abs(f64(lse).reshape(2) - L) <= 2.0 ** -21 * (1 + np.abs(L))).all()
