"""The 8-bit cache and the decoding steps over it, on the GPU, against the
plain 64-bit forms of serving_ref.py under their derived bounds."""

import numpy as np
import pytest
import torch

import exact_io_aware_37_gb300 as fa
import serving_ref as ref
from exact_io_aware_37_gb300 import synth
from parity import Guarded, f64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def ok():
    torch.cuda.synchronize()
    return fa.fa_get_last_device_error() == 0


def int32(v):
    return None if v is None else torch.tensor(v, dtype=torch.int32, device=DEV)


def name(c):
    return "-".join(str(x).replace("torch.", "").replace(" ", "") for x in c)


def bits(t):
    return t.view(torch.uint8).cpu().numpy()


def random_cache(B, Hk, cap, D, seed):
    """A full cache written by the framework from N(0, 1) rows of unlike size."""
    c = fa.cache_alloc(B, Hk, cap, D)
    k, v = (synth.normal((B, Hk, cap, D), seed + i, F32) for i in range(2))
    g = torch.Generator().manual_seed(seed + 2)
    k, v = (x * 2.0 ** torch.randint(-3, 4, (B, Hk, cap, 1), generator=g) for x in (k, v))
    fa.fa_cache_write((k / 4).to(DEV), v.to(DEV), c)
    return c


# ---------------------------------------------------------------- write, read

ROWS = [
    # (B, H, n, cap, D, dtype, start, count)
    (1, 1, 1, 1, 64, BF16, None, None),
    (2, 3, 1, 7, 128, BF16, [6, 0], None),
    (3, 2, 17, 40, 64, F16, [0, 23, 5], [17, 0, 9]),
    (2, 5, 33, 33, 128, F32, None, [33, 1]),
    (1, 7, 129, 300, 64, F32, [171], None),
    (5, 1, 3, 64, 128, F16, [61, 1, 0, 30, 2], [3, 2, 1, 0, 3]),
    (1, 2, 1000, 1024, 128, BF16, [24], None),
]


@pytest.mark.parametrize("case", ROWS, ids=name)
def test_rows_written_and_read_back(case):
    B, H, n, cap, D, dtype, start, count = case
    k, v = (synth.normal((B, H, n, D), 90 + i, F32) * 2.0 ** (7 * i) for i in range(2))
    k, v = k.to(dtype), v.to(dtype)
    c = fa.cache_alloc(B, H, cap, D)
    for t in c:
        t.view(torch.uint8).fill_(0x5A)
    before = [bits(t).copy() for t in c]
    fa.fa_cache_write(k.to(DEV), v.to(DEV), c, int32(start), int32(count))
    assert ok()
    rows = np.zeros((B, H, cap), bool)
    s, m = start or [0] * B, count or [n] * B
    for b in range(B):
        rows[b, :, s[b]:s[b] + m[b]] = True
    for x, codes, exps, c0, e0 in ((k, c.k, c.k_exp, before[0], before[2]), (v, c.v, c.v_exp, before[1], before[3])):
        want, want_e = ref.quantise(f64(x))
        for b in range(B):
            at = slice(s[b], s[b] + m[b])
            assert np.array_equal(ref.CODES[bits(codes)[b, :, at]], want[b, :, :m[b]])
            assert np.array_equal(bits(exps)[b, :, at], want_e[b, :, :m[b]])
        assert np.array_equal(bits(codes)[~rows], c0[~rows])            # the other rows as they were
        assert np.array_equal(bits(exps)[~rows], e0[~rows])
    for out in (BF16, F16, F32):
        kr, vr = Guarded((B, H, n, D), out, DEV), Guarded((B, H, n, D), out, DEV)
        fa.fa_cache_read(c, kr.t, vr.t, int32(start), int32(count))
        assert ok() and kr.guards_intact() and vr.guards_intact()
        for got, codes, exps in ((kr.t, c.k, c.k_exp), (vr.t, c.v, c.v_exp)):
            val = ref.values(bits(codes), bits(exps))
            want = np.zeros((B, H, n, D))
            for b in range(B):
                want[b, :, :m[b]] = val[b, :, s[b]:s[b] + m[b]]
            assert torch.equal(got.cpu(), torch.from_numpy(want).to(F32).to(out))


def test_rows_at_the_borders_of_the_format():
    D = 64
    rows = np.zeros((12, D), np.float32)
    rows[1, 0] = 448.0
    rows[2, 0] = np.nextafter(np.float32(448), np.float32(449))         # just past: the next exponent
    rows[3, :] = 2.0 ** -149                                            # the smallest float
    rows[4, ::2] = 3.4e38
    rows[4, 1::2] = -1e-30
    rows[5, :4] = np.nan, np.inf, -np.inf, 5.0
    rows[6, :] = np.nan
    rows[7, :] = -np.inf
    rows[8, :] = np.linspace(-1, 1, D)
    rows[9, :] = 2.0 ** -130
    rows[10, :17] = 2.0 ** -np.arange(17)                               # through the codes' subnormals
    rows[10, 17:34] = 1.5 * 2.0 ** -np.arange(17)                       # ties on the way
    rows[11, 0], rows[11, 1] = 2.0 ** -126, 2.0 ** -127
    x = torch.from_numpy(rows).view(1, 1, 12, D).to(DEV)
    c = fa.cache_alloc(1, 1, 12, D)
    fa.fa_cache_write(x, -x, c)
    assert ok()
    want, want_e = ref.quantise(rows.astype(np.float64))
    got = ref.CODES[bits(c.k)[0, 0]]
    assert np.array_equal(bits(c.k_exp)[0, 0], want_e) and np.array_equal(bits(c.v_exp)[0, 0], want_e)
    assert np.array_equal(got, want, equal_nan=True)
    assert np.array_equal(ref.CODES[bits(c.v)[0, 0]], -want, equal_nan=True)
    k, _ = fa.cache_read(c, None, 12, dtype=F32)
    # 3.4e38 has code 256 at exponent 120: 2^128, past float32's range, so it reads back as infinity
    back = torch.from_numpy(want * np.exp2(want_e.astype(float) - 127)[:, None]).to(F32)
    assert back[4, 0] == float("inf") and np.array_equal(f64(k)[0, 0], f64(back), equal_nan=True)


def test_row_error_is_half_a_step_of_the_format():
    x = synth.normal((2, 2, 50, 128), 95, F32)
    c = fa.cache_alloc(2, 2, 50, 128)
    fa.fa_cache_write(x.to(DEV), x.to(DEV), c)
    k, v = fa.cache_read(c, None, 50, dtype=F32)
    assert torch.equal(k, v)
    # half a step: 2^-4 of the value, or of the smallest normal (2^-6 of a scale of at most amax / 224)
    floor = x.abs().amax(-1, keepdim=True) / 224 * 2.0 ** -6
    assert bool(((k.cpu() - x).abs() <= 2.0 ** -4 * torch.maximum(x.abs(), floor)).all())


BAD = [  # (start, count) of sequence 1 of 3, n = 4, cap = 10
    (-1, 2), (7, 4), (0, 5), (3, -1), (2 ** 31 - 1, 4), (-2 ** 31, 0),
]


@pytest.mark.parametrize("bad", BAD, ids=name)
def test_ranges_that_do_not_fit_are_skipped_and_reported(bad):
    B, H, n, cap, D = 3, 2, 4, 10, 64
    x = synth.normal((B, H, n, D), 96, BF16).to(DEV)
    start, count = int32([1, bad[0], 6]), int32([4, bad[1], 4])
    c = fa.cache_alloc(B, H, cap, D)
    for t in c:
        t.view(torch.uint8).fill_(0x33)
    fa.fa_cache_write(x, x, c, start, count)
    torch.cuda.synchronize()
    assert fa.fa_get_last_device_error() == -1
    assert bool((c.k.view(torch.uint8)[1] == 0x33).all()) and bool((c.k_exp[1] == 0x33).all())
    good = fa.cache_alloc(B, H, cap, D)
    for t in good:
        t.view(torch.uint8).fill_(0x33)
    fa.fa_cache_write(x, x, good, int32([1, 0, 6]), int32([4, 0, 4]))
    for a, b in zip(c, good):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    k, v = (torch.full((B, H, n, D), 7.0, dtype=F32, device=DEV) for _ in range(2))
    fa.fa_cache_read(c, k, v, start, count)
    torch.cuda.synchronize()
    assert fa.fa_get_last_device_error() == -1
    assert bool((k[1] == 7.0).all()) and bool((v[1] == 7.0).all()) and not bool((k[0] == 7.0).any())
    assert ok()


# ---------------------------------------------------------------- decoding

def reference(q, kp, vp, cache, lens, scale, causal, heads=None):
    """(O, L, A, S) in float64 over the prefix (or None) and the cache."""
    B, H, nq, D = q.shape
    Hk = cache[0].shape[1]
    r = H // Hk
    if len(cache) == 4:
        k, v = ref.values(bits(cache[0]), bits(cache[2])), ref.values(bits(cache[1]), bits(cache[3]))
    else:
        k, v = f64(cache[0]), f64(cache[1])
    out = [np.zeros((B, H, nq, D)), np.zeros((B, H, nq)), np.zeros((B, H, nq, D)), np.zeros((B, H, nq))]
    qn = f64(q)
    for b in range(B):
        for h in range(Hk):
            if heads is not None and (b, h) not in heads:
                continue
            kk, vv = k[b, h, :lens[b]], v[b, h, :lens[b]]
            if kp is not None:
                kk, vv = np.concatenate([f64(kp[h]), kk]), np.concatenate([f64(vp[h]), vv])
            for t, got in zip(out, ref.attend(qn[b, h * r:(h + 1) * r], kk, vv, scale, causal)):
                t[b, h * r:(h + 1) * r] = got
    return out


def check(o, lse, want, n, p_dtype, vmax):
    """o, lse against reference()'s, with the weights of at most n keys rounded to p_dtype."""
    O, L, A, S = want
    bound = ref.o_bound(O, A, S, n, o.shape[-1], vmax, o.dtype, p_dtype)
    lbound = ref.lse_bound(L, S, n, o.shape[-1])
    o, lse = f64(o), f64(lse)
    empty = np.isneginf(L)
    assert np.array_equal(np.isneginf(lse), empty) and np.all(o[empty] == 0)
    assert np.isfinite(o).all()
    assert (np.abs(o - O) <= bound).all(), f"O off by {np.abs(o - O).max():.3e}, {(np.abs(o - O) / bound).max():.2f} of the bound"
    d = np.abs(np.where(empty, 0, lse) - np.where(empty, 0, L))
    assert (d <= lbound).all(), f"lse off by {d.max():.3e}, {(d / lbound).max():.2f} of the bound"


def outputs(q):
    return Guarded(q.shape, q.dtype, DEV), Guarded(q.shape[:-1], F32, DEV)


CACHE = [
    # (B, H, Hk, nq, cap, lens, D, dtype, causal)
    (1, 1, 1, 1, 1, [1], 64, BF16, True),
    (1, 1, 1, 1, 16, [0], 128, BF16, True),                             # no key at all
    (2, 4, 2, 1, 100, [100, 37], 128, BF16, True),
    (3, 2, 2, 1, 2100, [2100, 1, 777], 128, F16, True),
    (4, 8, 1, 1, 300, [0, 300, 64, 65], 64, F16, True),                 # eight query heads a key head
    (2, 6, 2, 5, 129, [128, 129], 128, BF16, True),                     # 15 rows
    (2, 7, 1, 3, 700, [513, 2], 64, BF16, True),                        # 21 rows; fewer keys than queries
    (1, 16, 1, 8, 400, [399], 128, F16, True),                          # 128 rows
    (2, 12, 4, 8, 90, [17, 90], 64, BF16, False),                       # not causal
    (1, 33, 1, 1, 1000, [997], 128, BF16, False),
    (5, 3, 3, 2, 63, [0, 1, 2, 63, 31], 128, BF16, True),
    (1, 40, 1, 5, 257, [256], 64, F16, True),                           # 200 rows
    (1, 2, 1, 1, 40000, [39999], 128, BF16, True),
    (2, 3, 1, 8, 300, [300, 129], 64, BF16, True),                      # 24 rows
    (1, 4, 1, 5, 1000, [1000], 128, BF16, True),                        # 20 rows
    (1, 4, 2, 70, 500, [333], 128, F16, True),                          # a piece of a prompt: 140 rows
    (300, 2, 1, 1, 40, None, 64, F16, True),                            # more sequences than a block plans at once
    (3, 2, 2, 1, 1500, [1500, 0, 1409], 64, BF16, True),
]


@pytest.mark.parametrize("case", CACHE, ids=name)
def test_decode_cache_matches_the_reference(case):
    B, H, Hk, nq, cap, lens, D, dtype, causal = case
    if lens is None:
        lens = [int(x) for x in synth.varlen_lengths(B, 0, cap, 8)]
    c = random_cache(B, Hk, cap, D, 100)
    q = (synth.normal((B, H, nq, D), 103, F32) * 2).to(dtype).to(DEV)
    o, lse = outputs(q)
    fa.fa_decode_cache(q, c, int32(lens), o.t, lse.t, causal)
    assert ok() and o.guards_intact() and lse.guards_intact()
    want = reference(q, None, None, c, lens, D ** -0.5, causal)
    vmax = np.abs(ref.values(bits(c.v), bits(c.v_exp))).max()
    check(o.t, lse.t, want, max(lens), F16, vmax)
    # the same again: no atomics, so the same bits
    o2, lse2 = fa.decode_cache(q, c, int32(lens), causal=causal)
    assert torch.equal(o.t, o2) and torch.equal(lse.t, lse2)


SHARED = [
    # (B, H, Hk, nq, np, cap, lens, D, dtype, causal, own8)
    (1, 1, 1, 1, 1, 1, [1], 64, BF16, True, False),
    (2, 2, 1, 1, 127, 8, [0, 8], 128, F16, True, False),                # a sequence with no key of its own
    (3, 8, 8, 1, 301, 64, [64, 1, 30], 64, F16, True, False),
    (3, 8, 2, 1, 300, 64, [64, 1, 30], 128, BF16, True, True),
    (2, 4, 2, 5, 129, 20, [3, 0], 128, BF16, True, True),               # the first queries end inside the prefix
    (2, 3, 1, 8, 3, 20, [2, 1], 64, BF16, True, False),                 # ... or before it: rows with no key
    (40, 8, 2, 2, 1000, 33, None, 128, BF16, True, False),              # 320 rows a key head
    (5, 16, 1, 7, 515, 100, [100, 99, 7, 6, 8], 64, F16, True, True),   # 560 rows
    (2, 4, 4, 1, 0, 50, [50, 0], 128, BF16, True, False),               # no prefix: unequal 16-bit caches
    (2, 4, 4, 2, 640, 0, [0, 0], 64, BF16, True, False),                # nothing but the prefix
    (4, 6, 2, 3, 256, 40, [9, 40, 0, 2], 128, F16, False, True),        # not causal
    (16, 5, 1, 1, 20000, 128, None, 128, BF16, True, True),
    (129, 1, 1, 1, 128, 5, None, 64, F16, True, False),
    (2, 5, 1, 2, 200, 300, [300, 129], 128, BF16, True, False),         # 16-bit rows: 10, 24, 20, 15 rows a key head
    (2, 6, 1, 4, 200, 300, [257, 31], 128, F16, True, False),
    (2, 4, 1, 5, 200, 400, [400, 64], 64, BF16, True, False),
    (3, 15, 1, 1, 1, 700, [700, 0, 128], 64, F16, False, False),
    (2, 9, 3, 40, 384, 260, [260, 40], 128, BF16, True, False),         # 120 rows a key head
    (300, 4, 2, 1, 130, 6, None, 128, F16, True, True),                 # 600 rows, little of their own
    (7, 2, 2, 1, 128 * 153, 20, None, 64, BF16, True, True),            # one unit over all CTAs, and then some
    (5, 6, 6, 8, 9000, 183, None, 128, BF16, True, True),               # nearly all SMs for the prefix
    (40, 8, 2, 5, 200, 1500, None, 64, F16, True, True),                # few for it
    (9, 12, 2, 3, 3000, 900, None, 128, F16, True, False),
]


@pytest.mark.parametrize("case", SHARED, ids=name)
def test_decode_shared_matches_the_reference(case):
    B, H, Hk, nq, np_, cap, lens, D, dtype, causal, own8 = case
    if lens is None:
        lens = [int(x) for x in synth.varlen_lengths(B, 0, cap, 7)]
    q = (synth.normal((B, H, nq, D), 110, F32) * 2).to(dtype).to(DEV)
    kp, vp = (synth.normal((Hk, np_, D), 111 + i, dtype).to(DEV) for i in range(2))
    c = random_cache(B, Hk, cap, D, 113) if own8 and cap else tuple(
        synth.normal((B, Hk, cap, D), 113 + i, dtype).to(DEV) for i in range(2))
    o, lse = outputs(q)
    fa.fa_decode_shared(q, kp, vp, c, int32(lens), o.t, lse.t, causal)
    assert ok() and o.guards_intact() and lse.guards_intact()
    want = reference(q, kp, vp, c, lens, D ** -0.5, causal)
    # the prefix's weights are rounded to dtype, those of 8-bit rows to fp16: the coarser of the two
    vmax = 8.0 * (8 if own8 else 1)
    check(o.t, lse.t, want, np_ + max(lens), dtype, vmax)
    o2, lse2 = fa.decode_shared(q, kp, vp, c, int32(lens), causal=causal)
    assert torch.equal(o.t, o2) and torch.equal(lse.t, lse2)


def test_without_lengths_every_row_up_to_max_len_counts():
    B, H, Hk, D, cap = 2, 4, 2, 64, 96
    c = random_cache(B, Hk, cap, D, 120)
    q = synth.normal((B, H, 1, D), 121, BF16).to(DEV)
    for n in (96, 50):
        a = fa.decode_cache(q, c, None, max_len=n)
        b = fa.decode_cache(q, c, int32([n, n]))
        check(a[0], a[1], reference(q, None, None, c, [n, n], D ** -0.5, True), n, F16, 64.0)
        check(b[0], b[1], reference(q, None, None, c, [n, n], D ** -0.5, True), n, F16, 64.0)


@pytest.mark.parametrize("own8", [True, False])
def test_rows_after_the_length_are_never_used(own8):
    B, H, Hk, nq, np_, cap, D = 3, 4, 2, 2, 70, 200, 128
    lens = [200, 0, 77]
    q = synth.normal((B, H, nq, D), 130, BF16).to(DEV)
    kp, vp = (synth.normal((Hk, np_, D), 131 + i, BF16).to(DEV) for i in range(2))
    c = random_cache(B, Hk, cap, D, 133) if own8 else tuple(
        synth.normal((B, Hk, cap, D), 133 + i, BF16).to(DEV) for i in range(2))
    before = fa.decode_shared(q, kp, vp, c, int32(lens))
    for b in range(B):
        for t in c:
            if t.dtype == torch.uint8:
                t[b, :, lens[b]:] = 255
            elif own8:
                t.view(torch.uint8)[b, :, lens[b]:] = 0x7F              # NaN
            else:
                t[b, :, lens[b]:] = float("nan") if b else float("inf")
    after = fa.decode_shared(q, kp, vp, c, int32(lens))
    assert ok()
    assert torch.equal(before[0], after[0]) and torch.equal(before[1], after[1])


@pytest.mark.parametrize("own8", [True, False])
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_keys_that_the_mask_hides_do_not_reach_a_row(own8, bad):
    """Not finite in the newest token's key and value: the earlier queries of the
    same step, which do not see it, are as without it."""
    B, H, Hk, nq, np_, cap, D = 1, 4, 2, 3, 40, 150, 64
    q = synth.normal((B, H, nq, D), 140, BF16).to(DEV)
    kp, vp = (synth.normal((Hk, np_, D), 141 + i, BF16).to(DEV) for i in range(2))
    c = random_cache(B, Hk, cap, D, 143) if own8 else tuple(
        synth.normal((B, Hk, cap, D), 143 + i, BF16).to(DEV) for i in range(2))
    for n in (1, 2, 130, 150):
        clean = tuple(t.clone() for t in c)
        before = fa.decode_shared(q, kp, vp, clean, int32([n]))
        for t in clean[:2]:
            if own8:
                t.view(torch.uint8)[0, :, n - 1, 5:9] = 0x7F
            else:
                t[0, :, n - 1, 5:9] = float(bad)
        after = fa.decode_shared(q, kp, vp, clean, int32([n]))
        assert ok()
        assert torch.equal(before[0][:, :, :2], after[0][:, :, :2])
        assert torch.equal(before[1][:, :, :2], after[1][:, :, :2])
        assert bool(after[0][:, :, 2].isnan().any())                    # the row that sees it says so


def test_values_of_unlike_scale_keep_their_precision():
    """A row that attends to one key whose values are 2^60 times smaller (or
    larger) than its neighbours' gets that key's values."""
    D, cap = 128, 300
    for at, big in ((7, -30), (250, 30), (299, 90), (0, -100)):
        k = torch.zeros(1, 1, cap, D)
        k[0, 0, at, 0] = 16.0
        v = synth.normal((1, 1, cap, D), 150, F32)
        v[0, 0, at] *= 2.0 ** big
        c = fa.cache_alloc(1, 1, cap, D)
        fa.fa_cache_write(k.to(DEV), v.to(DEV), c)
        q = torch.zeros(1, 1, 1, D, dtype=BF16)
        q[..., 0] = 16.0
        o, lse = fa.decode_cache(q.to(DEV), c, None, scale=1.0)         # weight 1 - 300 e^-256
        assert ok()
        want = ref.values(bits(c.v)[0, 0, at], bits(c.v_exp)[0, 0, at])
        got = f64(o)[0, 0, 0]
        # the other keys' values are at most 6 each and their weights e^-256 < 2^-369
        assert (np.abs(got - want) <= 2.0 ** -8 * 1.01 * np.abs(want) + cap * 6 * 2.0 ** -369 + 2.0 ** -134).all()


@pytest.mark.parametrize("magnitude", [1e-30, 3e4, 3e38])
def test_queries_of_any_size(magnitude):
    """Queries far outside fp16's range against the 8-bit cache."""
    D, cap = 64, 200
    c = random_cache(1, 1, cap, D, 155)
    q = (synth.normal((1, 2, 1, D), 156, F32).clamp(-1, 1) * magnitude).to(BF16).to(DEV)
    scale = 1.0 / magnitude
    if scale < 1.2e-38:
        scale = 1.2e-38
    o, lse = torch.empty_like(q), torch.empty(1, 2, 1, device=DEV)
    fa.fa_decode_cache(q, c, None, o, lse, True, scale)
    assert ok()
    check(o, lse, reference(q, None, None, c, [cap], float(np.float32(scale)), True), cap, F16, 64.0)


@pytest.mark.parametrize("own8", [True, False])
def test_scores_that_rise_along_the_cache(own8):
    """Every tile's scores above the last one's by less than, about, and far more than
    what a reference allows; then by more than float32's exponents reach."""
    D, cap = 128, 1300
    q = torch.zeros(1, 3, 1, D, dtype=BF16)
    q[..., 0] = 1.0
    for step in (0.5, 3.0, 2.5 * np.log(2) * 4, 60.0, 400.0):
        k = torch.zeros(1, 1, cap, D)
        k[..., 0] = (torch.arange(cap) // 100 * step)
        v = synth.normal((1, 1, cap, D), 157, F32)
        if own8:
            c = fa.cache_alloc(1, 1, cap, D)
            fa.fa_cache_write(k.to(DEV), v.to(DEV), c)
        else:
            c = tuple(x.to(BF16).to(DEV) for x in (k, v))
        kp, vp = (torch.zeros(1, 0, D, dtype=BF16, device=DEV) for _ in range(2))
        o, lse = fa.decode_shared(q.to(DEV), kp, vp, c, scale=1.0)
        assert ok()
        want = reference(q, None, None, c, [cap], 1.0, True)
        check(o, lse, want, cap, F16 if own8 else BF16, 8.0)


def test_infinite_scores_weigh_nothing_or_everything():
    """-inf in a 16-bit key: as if it were not there, here for a whole first tile and a part of the second."""
    D, cap = 64, 300
    q = torch.zeros(1, 1, 1, D, dtype=BF16)
    q[..., 0] = 1.0
    k, v = (synth.normal((1, 1, cap, D), 158 + i, BF16) for i in range(2))
    kp, vp = (torch.zeros(1, 0, D, dtype=BF16, device=DEV) for _ in range(2))
    k[0, 0, :200, 0] = float("-inf")                                    # whole first tile, part of the second
    o, lse = fa.decode_shared(q.to(DEV), kp, vp, (k.to(DEV), v.to(DEV)), scale=1.0)
    assert ok()
    tail = tuple(x[:, :, 200:].contiguous() for x in (k, v))
    check(o, lse, reference(q, None, None, tail, [100], 1.0, True), 100, BF16, 8.0)


def test_lengths_out_of_range_are_skipped_and_reported():
    B, H, Hk, nq, np_, cap, D = 4, 2, 1, 2, 33, 20, 64
    q = synth.normal((B, H, nq, D), 160, BF16).to(DEV)
    kp, vp = (synth.normal((Hk, np_, D), 161 + i, BF16).to(DEV) for i in range(2))
    c = random_cache(B, Hk, cap, D, 163)
    good = fa.decode_shared(q, kp, vp, c, int32([20, 3, 5, 1]))
    none = tuple(torch.empty(B, Hk, 0, D, dtype=BF16, device=DEV) for _ in range(2))  # no rows of their own at all
    o, lse = torch.full_like(q, 9.0), torch.full((B, H, nq), 9.0, device=DEV)
    fa.fa_decode_shared(q, kp, vp, none, int32([0, 1, 0, -1]), o, lse, True)
    torch.cuda.synchronize()
    assert fa.fa_get_last_device_error() == -1
    assert bool((o[1::2] == 9.0).all()) and bool((lse[1::2] == 9.0).all()) and not bool((lse[::2] == 9.0).any())
    for bad in (-1, 21, 2 ** 31 - 1, -2 ** 31):
        o, lse = torch.full_like(q, 9.0), torch.full((B, H, nq), 9.0, device=DEV)
        fa.fa_decode_shared(q, kp, vp, c, int32([20, bad, 5, 1]), o, lse, True)
        torch.cuda.synchronize()
        assert fa.fa_get_last_device_error() == -1
        assert bool((o[1] == 9.0).all()) and bool((lse[1] == 9.0).all())
        for b in (0, 2, 3):  # a skipped sequence moves where the work is cut, not what comes out
            assert bool(((o[b] - good[0][b]).abs() <= 2.0 ** -6 * good[0][b].abs() + 2e-3).all())
            assert bool(((lse[b] - good[1][b]).abs() <= 1e-5).all())
    assert ok()


def test_a_batch_is_its_sequences():
    """What a sequence gets does not hang on the others in its batch."""
    B, H, Hk, nq, np_, cap, D = 6, 8, 2, 2, 200, 90, 64
    lens = [90, 1, 45, 0, 64, 33]
    q = synth.normal((B, H, nq, D), 170, F16).to(DEV)
    kp, vp = (synth.normal((Hk, np_, D), 171 + i, F16).to(DEV) for i in range(2))
    c = random_cache(B, Hk, cap, D, 173)
    o, lse = fa.decode_shared(q, kp, vp, c, int32(lens))
    for b in range(B):
        one = fa.Cache8(*(t[b:b + 1].contiguous() for t in c))
        o1, lse1 = fa.decode_shared(q[b:b + 1].contiguous(), kp, vp, one, int32(lens[b:b + 1]))
        want = reference(q[b:b + 1], kp, vp, one, lens[b:b + 1], D ** -0.5, True)
        check(o1, lse1, want, np_ + lens[b], F16, 64.0)
        check(o[b:b + 1], lse[b:b + 1], want, np_ + lens[b], F16, 64.0)


# ---------------------------------------------------------------- how calls are made

def test_decoding_replays_from_a_graph_on_new_lengths():
    """Write, then attend, captured once: replays follow the buffers' contents."""
    B, H, Hk, np_, cap, D = 3, 8, 2, 300, 128, 128
    c = fa.cache_alloc(B, Hk, cap, D)
    for t in c:
        t.view(torch.uint8).fill_(0x11)
    q, k, v = (torch.empty(B, h, 1, D, dtype=BF16, device=DEV) for h in (H, Hk, Hk))
    kp, vp = (synth.normal((Hk, np_, D), 180 + i, BF16).to(DEV) for i in range(2))
    lens = torch.tensor([5, 60, 127], dtype=torch.int32, device=DEV)
    at = lens - 1
    o, lse = torch.empty_like(q), torch.empty(B, H, 1, device=DEV)
    ws = torch.empty(fa.fa_decode_shared_workspace_size(q, kp, c), dtype=torch.uint8, device=DEV)

    def step(stream, c=c, ws=ws, o=o, lse=lse):
        fa.fa_cache_write(k, v, c, at, stream=stream)
        fa.fa_decode_shared(q, kp, vp, c, lens, o, lse, True, workspace=ws, stream=stream)

    def new(seed):
        for i, t in enumerate((q, k, v)):
            t.copy_(synth.normal(tuple(t.shape), seed + i, BF16))

    new(182)
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(torch.cuda.current_stream())
    for n, seed in (([9, 128, 1], 185), ([128, 2, 77], 188)):
        new(seed)
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        at.copy_(lens - 1)
        eager = fa.Cache8(*(t.clone() for t in c))
        ws.fill_(0xFF)                                                  # what a workspace holds does not matter
        o.fill_(float("nan"))
        g.replay()
        o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
        step(torch.cuda.current_stream(), eager, torch.empty_like(ws), o2, lse2)
        assert ok()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        for a, b in zip(c, eager):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        want = reference(q, kp, vp, c, n, D ** -0.5, True)
        check(o, lse, want, np_ + max(n), BF16, 64.0)


def test_two_streams_at_once():
    """Calls that overlap, each with scratch of its own, and two captured graphs
    replayed at once, each with its own workspace."""
    D, Hk, H = 128, 4, 8
    jobs = []
    for i, (B, np_, cap) in enumerate(((4, 2000, 700), (6, 900, 1500))):
        q = synth.normal((B, H, 1, D), 190 + i, BF16).to(DEV)
        kp, vp = (synth.normal((Hk, np_, D), 192 + 2 * i + j, BF16).to(DEV) for j in range(2))
        jobs.append((q, kp, vp, random_cache(B, Hk, cap, D, 196 + 3 * i), int32([cap - 7 * b for b in range(B)])))
    alone = [fa.decode_shared(*j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(DEV) for _ in jobs]
    for _ in range(20):
        got = []
        for j, s in zip(jobs, streams):
            got.append(fa.decode_shared(*j, stream=s))
        torch.cuda.synchronize()
        for (o, lse), (o2, lse2) in zip(got, alone):
            assert torch.equal(o, o2) and torch.equal(lse, lse2)
    graphs = []
    for j in jobs:
        o, lse = torch.empty_like(j[0]), torch.empty(j[0].shape[:-1], device=DEV)
        ws = torch.empty(fa.fa_decode_shared_workspace_size(j[0], j[1], j[3]), dtype=torch.uint8, device=DEV)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fa.fa_decode_shared(*j, o, lse, True, workspace=ws)
        graphs.append((g, o, lse, ws))
    for _ in range(20):
        for (g, *_), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    assert ok()
    for (_, o, lse, _), (o2, lse2) in zip(graphs, alone):
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_raw_stream_handles_are_taken():
    c = random_cache(1, 2, 64, 64, 205)
    q = synth.normal((1, 2, 1, 64), 206, BF16).to(DEV)
    want = fa.decode_cache(q, c)
    torch.cuda.synchronize()
    s = torch.cuda.Stream(DEV)
    got = fa.decode_cache(q, c, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_workspace_too_small_is_refused():
    c = random_cache(2, 2, 600, 64, 207)
    q = synth.normal((2, 2, 1, 64), 208, BF16).to(DEV)
    o, lse = torch.empty_like(q), torch.empty(2, 2, 1, device=DEV)
    n = fa.fa_decode_cache_workspace_size(q, c)
    with pytest.raises(fa.FAError, match="WORKSPACE"):
        fa.fa_decode_cache(q, c, None, o, lse, True, workspace=torch.empty(n - 1, dtype=torch.uint8, device=DEV))
    guard = torch.full((n + 512,), 0x5A, dtype=torch.uint8, device=DEV)
    fa.fa_decode_cache(q, c, None, o, lse, True, workspace=guard[256:256 + n])
    assert ok()
    assert bool((guard[:256] == 0x5A).all()) and bool((guard[256 + n:] == 0x5A).all())


def test_more_than_32_bits_of_cache():
    """Element offsets past 2^32: the last sequence's rows of a 5 GB cache."""
    B, Hk, cap, D = 5, 8, 1 << 20, 128
    c = fa.cache_alloc(B, Hk, cap, D)
    n = 100
    k, v = (synth.normal((B, Hk, n, D), 210 + i, BF16).to(DEV) for i in range(2))
    start = int32([0, 5, 0, 0, cap - n])
    fa.fa_cache_write(k, v, c, start, int32([0, n, 0, 0, n]))
    kr, vr = fa.cache_read(c, start, n, int32([0, n, 0, 0, n]), dtype=F32)
    assert ok()
    for b in (1, 4):
        for x, y in ((k, kr), (v, vr)):
            codes, exps = ref.quantise(f64(x[b, 7]))
            assert np.array_equal(f64(y[b, 7]), codes * np.exp2(exps.astype(float) - 127)[:, None])
    # all of the last sequence: zeros everywhere but in its last rows
    q = synth.normal((B, Hk, 1, D), 212, BF16).to(DEV)
    o, lse = fa.decode_cache(q, c, int32([0, 0, 0, 0, cap]))
    assert ok()
    one = fa.Cache8(*(t[4:, 7:, cap - n:].contiguous() for t in c))
    O, L, A, S = reference(q[4:, 7:], None, None, one, [n], D ** -0.5, True)
    zeros = cap - n                                                     # keys with score 0 and value 0
    m = np.logaddexp(L, np.log(zeros))
    shrink = np.exp(L - m)
    assert np.abs(f64(lse)[4:, 7:] - m).max() <= ref.lse_bound(m, S, 4096, D).max()
    bound = ref.o_bound(O * shrink[..., None], A * shrink[..., None], S, 4096, D, 8.0 / zeros, BF16, F16)
    assert (np.abs(f64(o)[4:, 7:] - O * shrink[..., None]) <= bound).all()
    assert bool((o[:4] == 0).all()) and bool((lse[:4] == float("-inf")).all())


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("dtype, D, Hk, group", [(BF16, 128, 2, 4), (F16, 64, 4, 1)])
def test_a_prompt_and_a_few_steps(dtype, D, Hk, group):
    """As a server uses them: a shared prompt through fa_fwd, its keys and values
    kept as the prefix; each step writes its tokens into the 8-bit cache and
    attends; drafted tokens that were not taken are overwritten; at the end the
    cache is read back and fa_fwd over prefix and cache agrees with the last step."""
    B, H, np_, cap = 3, Hk * group, 260, 64
    kp, vp = (synth.normal((1, Hk, np_, D), 220 + i, dtype).to(DEV) for i in range(2))
    qp = synth.normal((1, Hk, np_, D), 222, dtype).to(DEV)
    op, _ = fa.forward(qp, kp, vp, causal=True)                         # the prompt's own pass
    c = fa.cache_alloc(B, Hk, cap, D)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    for step, (nq, taken) in enumerate(((4, [4, 1, 2]), (1, [1, 1, 1]), (3, [1, 3, 2]), (2, [2, 2, 2]))):
        k, v = (synth.normal((B, Hk, nq, D), 230 + 10 * step + i, dtype).to(DEV) for i in range(2))
        q = synth.normal((B, H, nq, D), 232 + 10 * step, dtype).to(DEV)
        fa.fa_cache_write(k, v, c, lens)
        o, lse = fa.decode_shared(q, kp[0], vp[0], c, lens + nq)
        assert ok()
        now = [int(x) + nq for x in lens]
        check(o, lse, reference(q, kp[0], vp[0], c, now, D ** -0.5, True), np_ + max(now), dtype, 8.0)
        lens = lens + (int32(taken) if step < 3 else nq)
    n = int(lens[0])
    kr, vr = fa.cache_read(c, None, cap, lens, dtype=dtype)
    kk, vv = (torch.cat((x[0], y[0, :, :n]), 1)[None].contiguous() for x, y in ((kp, kr), (vp, vr)))
    qq = torch.zeros(1, Hk, np_ + n, D, dtype=dtype, device=DEV)
    qq[0, :, -nq:] = q[0].view(Hk, group, nq, D)[:, 0]                  # one query head a key head
    full, full_lse = fa.forward(qq, kk, vv, causal=True)
    mine = o[0].view(Hk, group, nq, D)[:, 0]
    # both are within the dtype's bound of the same exact values (the cache's values are exact in dtype)
    want = reference(q, kp[0], vp[0], c, [int(x) for x in lens], D ** -0.5, True)
    O, L, A, S = (x[:1].reshape((Hk, group, nq) + x.shape[3:])[:, 0] for x in want)
    both = 2 * ref.o_bound(O, A, S, np_ + n, D, 8.0, dtype, dtype)
    assert (np.abs(f64(mine) - f64(full[0, :, -nq:])) <= both).all()
    assert op.isfinite().all()
