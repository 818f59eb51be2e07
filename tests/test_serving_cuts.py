"""No part of the keys of a decoding step is lost or counted twice where the work is cut and joined
(inputs and bounds: serving_cuts.py)."""

import numpy as np
import pytest
import torch

import exact_io_aware_37_gb300 as fa
import serving_cuts as cuts

F32 = torch.float32


def name(c):
    return "-".join(str(x).replace("torch.", "").replace(" ", "") for x in c if not isinstance(x, list))


def p_dtype(case):
    """What the weights are rounded to: fp16 over the 8-bit cache, the queries' type elsewhere; the coarser."""
    return torch.float16 if case[9] and case[4] == 0 else case[8]


def differs(O, L, O2, L2, n, case):
    """Whether outputs near (O2, L2) cannot be taken for (O, L): further apart than both bounds, for every row."""
    bo, bl = cuts.bounds(O, L, n, case[8], p_dtype(case))
    bo2, bl2 = cuts.bounds(O2, L2, n, case[8], p_dtype(case))
    return ((np.abs(O - O2) > bo + bo2).any(1) | (np.abs(L - L2) > bl + bl2)).all()


@pytest.mark.parametrize("case", cuts.CASES, ids=name)
def test_a_lost_or_doubled_half_would_be_seen(case):
    D, np_ = case[7], case[4]
    q, kp, vp, k, v = cuts.inputs(case)
    lens = cuts.lengths(case)
    for b in sorted({0, int(np.argmin(lens)), len(lens) - 1}):
        den, num, ch = cuts.halves(case, q, kp, k, b, 0)
        # the rows that see every key (the last new token's): no half is hidden from them
        nq = case[3]
        rows = slice(nq - 1, None, nq)
        den, num = den[rows], num[rows]
        O, L = cuts.outputs(den, num, ch, D)
        n = np_ + lens[b]
        groups = [[i] for i in range(den.shape[1])] + [[i, i + 1] for i in range(0, den.shape[1] - 1, 2)]
        for part in groups:
            if den.shape[1] == len(part):
                continue                                    # nothing else to tell it from
            for times in (0, 2):
                w = np.ones(den.shape[1])
                w[part] = times
                assert differs(O, L, *cuts.outputs(den * w, num * w, ch, D), n, case), (b, part, times)


def test_the_reference_is_the_definition():
    """The halves' sums against the oracle's attention, on small cases of each kind."""
    import oracle
    for case in ((2, 4, 2, 2, 130, 200, [150, 1], 64, torch.float16, True), (1, 3, 1, 3, 0, 300, [257], 128, torch.bfloat16, False)):
        B, H, Hk, nq, np_, cap, lens, D = case[:8]
        q, kp, vp, k, v = (x.astype(np.float64) for x in cuts.inputs(case))
        for b in range(B):
            for h in range(H):
                g = h // (H // Hk)
                kk, vv = np.concatenate([kp[g], k[b, g, :lens[b]]]), np.concatenate([vp[g], v[b, g, :lens[b]]])
                O, L = oracle.forward_cached_head(q[b, h], kk, vv, cuts.SCALE, True)
                den, num, ch = cuts.halves(case, q, kp, k, b, g)
                O2, L2 = cuts.outputs(den, num, ch, D)
                at = slice(h % (H // Hk) * nq, h % (H // Hk) * nq + nq)
                assert np.allclose(O, O2[at], rtol=1e-12, atol=1e-15) and np.allclose(L, L2[at], rtol=1e-12)


def test_the_inputs_are_exact_in_every_type():
    for case in cuts.CASES[:2] + cuts.CASES[6:8]:
        for x in cuts.inputs(case):
            t = torch.from_numpy(x)
            for dt in (torch.bfloat16, torch.float16, torch.float8_e4m3fn):
                assert torch.equal(t, t.to(dt).float())
        q, kp, _, k, _ = cuts.inputs(case)
        keys = np.concatenate([kp[0], k[0, 0]])
        assert np.abs(q[0].reshape(-1, q.shape[-1]) @ keys.T * cuts.SCALE).max() < 1.5  # weights within 2^-5 .. 2^5


@pytest.mark.gpu
@pytest.mark.parametrize("case", cuts.CASES, ids=name)
def test_no_part_of_the_keys_is_lost_or_doubled(case):
    B, H, Hk, nq, np_, cap, _, D, dtype, own8 = case
    dev = torch.device("cuda:0")
    lens = cuts.lengths(case)
    q, kp, vp, k, v = cuts.inputs(case)
    qd, kpd, vpd, kd, vd = (torch.from_numpy(x).to(dtype).to(dev) for x in (q, kp, vp, k, v))
    if own8:
        cache = fa.cache_alloc(B, Hk, cap, D)
        fa.fa_cache_write(kd, vd, cache)
        kr, vr = fa.cache_read(cache, None, cap, dtype=F32)
        assert torch.equal(kr, kd.float()) and torch.equal(vr, vd.float())
    else:
        cache = (kd, vd)
    o, lse = fa.decode_shared(qd, kpd, vpd, cache, torch.tensor(lens, dtype=torch.int32, device=dev), scale=cuts.SCALE)
    torch.cuda.synchronize()
    assert fa.fa_get_last_device_error() == 0
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(B):
        for h in range(Hk):
            den, num, ch = cuts.halves(case, q, kp, k, b, h)
            O, L = cuts.outputs(den, num, ch, D)
            at = slice(h * (H // Hk), (h + 1) * (H // Hk))
            got, got_l = o[b, at].reshape(O.shape), lse[b, at].reshape(L.shape)
            bo, bl = cuts.bounds(O, L, np_ + lens[b], dtype, p_dtype(case))
            empty = np.isneginf(L)
            assert np.array_equal(np.isneginf(got_l), empty) and np.all(got[empty] == 0)
            off = np.abs(got - O) - bo
            assert (off <= 0).all(), (b, h, np.argwhere(off > 0)[:4], np.abs(got - O).max())
            d = np.abs(np.where(empty, 0, got_l) - np.where(empty, 0, L))
            assert (d <= bl).all(), (b, h, d.max(), bl.max())
