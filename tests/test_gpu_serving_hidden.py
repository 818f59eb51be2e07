"""A shared prefix whose last keys the mask hides from some rows: where a sequence's own
part is shorter than its new tokens, the first of them end inside the prefix."""

import numpy as np
import pytest
import torch

import exact_io_aware_37_gb300 as fa
from exact_io_aware_37_gb300 import synth
from test_gpu_serving import BF16, DEV, F16, int32, name, ok, random_cache

pytestmark = pytest.mark.gpu

HIDDEN = [
    # (B, H, Hk, nq, np, cap, lens, D, dtype, own8)
    (2, 4, 2, 3, 40, 150, [0, 130], 64, BF16, False),       # one tile, halves
    (3, 2, 2, 5, 300, 20, [3, 0, 20], 128, F16, True),
    (2, 3, 1, 8, 5, 20, [2, 8], 64, F16, False),            # fewer keys than new tokens
    (1, 2, 1, 60, 4000, 0, [0], 128, BF16, False),          # nothing of their own; hidden keys in both halves' slots
    (40, 8, 2, 2, 1000, 33, None, 128, BF16, True),         # 320 rows a key head: pairs of tiles
    (40, 4, 2, 2, 257, 9, None, 64, F16, False),            # 160 rows: the second tile part-filled
    (3, 1, 1, 150, 400, 160, [160, 0, 40], 128, F16, True), # hidden keys in two tiles; 450 rows
    (3, 1, 1, 150, 400, 160, [0, 40, 160], 64, BF16, False),
    (64, 4, 1, 2, 128, 4, [4] * 63 + [0], 128, BF16, False),  # only the last tile's rows are short
    (64, 4, 1, 2, 128, 4, [0] + [4] * 63, 64, BF16, True),    # only the first one's
    (30, 4, 4, 3, 20000, 6, [6] * 29 + [1], 64, F16, False),  # units cut over several CTAs
]


@pytest.mark.parametrize("case", HIDDEN, ids=name)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_hidden_prefix_values_do_not_reach_a_row(case, bad):
    """Values that are not finite at the prefix's end: rows that do not see them are bit for bit as
    without them, rows that do have them where they are and nowhere else."""
    B, H, Hk, nq, np_, cap, lens, D, dtype, own8 = case
    if lens is None:
        lens = [b % (nq + 1) for b in range(B)]
    q = synth.normal((B, H, nq, D), 300, dtype).to(DEV)
    kp, vp = (synth.normal((Hk, np_, D), 301 + i, dtype).to(DEV) for i in range(2))
    c = random_cache(B, Hk, cap, D, 303) if own8 else tuple(
        synth.normal((B, Hk, cap, D), 303 + i, dtype).to(DEV) for i in range(2))
    clean, clean_lse = fa.decode_shared(q, kp, vp, c, int32(lens))
    assert ok() and bool(clean.isfinite().all())
    last = [np_ + n - nq + np.arange(nq) for n in lens]     # the last key that a row sees
    hidden = sorted({int(x) + 1 for r in last for x in r if x + 1 < np_ and x >= 0})
    assert hidden
    for at in {hidden[0], hidden[-1], np_ - 1}:
        v = vp.clone()
        v[:, at, 5:9] = bad
        o, lse = fa.decode_shared(q, kp, v, c, int32(lens))
        assert ok()
        sees = torch.from_numpy(np.stack([r >= at for r in last])).to(DEV)[:, None, :, None]
        want = clean.clone()
        want[..., 5:9] = torch.where(sees, torch.full_like(want[..., 5:9], bad), want[..., 5:9])
        assert torch.equal(lse, clean_lse)
        assert torch.equal(o.isnan(), want.isnan())
        assert torch.equal(o.nan_to_num(0.0, 1e4, -1e4), want.nan_to_num(0.0, 1e4, -1e4))


@pytest.mark.parametrize("case", HIDDEN[:6], ids=name)
def test_hidden_prefix_keys_do_not_reach_a_row(case):
    B, H, Hk, nq, np_, cap, lens, D, dtype, own8 = case
    if lens is None:
        lens = [b % (nq + 1) for b in range(B)]
    q = synth.normal((B, H, nq, D), 310, dtype).to(DEV)
    kp, vp = (synth.normal((Hk, np_, D), 311 + i, dtype).to(DEV) for i in range(2))
    c = random_cache(B, Hk, cap, D, 313) if own8 else tuple(
        synth.normal((B, Hk, cap, D), 313 + i, dtype).to(DEV) for i in range(2))
    clean, clean_lse = fa.decode_shared(q, kp, vp, c, int32(lens))
    k = kp.clone()
    k[:, np_ - 1, 2:5] = float("nan")
    v = vp.clone()
    v[:, np_ - 1] = float("nan")
    o, lse = fa.decode_shared(q, k, v, c, int32(lens))
    assert ok()
    for b, n in enumerate(lens):
        for i in range(nq):
            if n - nq + i + 1 < 0:                          # the prefix's last key is hidden
                assert torch.equal(o[b, :, i], clean[b, :, i]) and torch.equal(lse[b, :, i], clean_lse[b, :, i])
            else:
                assert bool(o[b, :, i].isnan().all())
