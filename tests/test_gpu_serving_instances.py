"""Every compiled kernel of the decoding steps over a cache, each on a small case against the 64-bit
reference; and, without a GPU, that the cases reach them all."""

import pytest
import torch

import exact_io_aware_37_gb300 as fa
from exact_io_aware_37_gb300 import synth
from test_gpu_serving import BF16, DEV, F16, F32, bits, check, int32, ok, outputs, random_cache, ref, reference
from test_serving_plan import ask  # noqa: F401 (a fixture)

# query rows a key head, as (group, new tokens): every number of rows of a CTA, full and not, and numbers that take
# two row groups of 16 (25 .. 32) or of 24
ROWS = [(3, 1), (4, 1), (7, 1), (2, 4), (13, 1), (8, 2), (11, 2), (4, 6), (5, 5), (7, 4), (8, 4), (5, 8), (16, 3)]
LENS, CAP = [301, 0, 133], 320
OWN = [(kind, dtype, D) for kind in ("e4m3", "16") for dtype in (BF16, F16) for D in (64, 128)]

# (B, group, nq): rows of the batch that share a tile's halves, or fill pairs of tiles
BATCHES = [(3, 4, 1), (3, 4, 3), (40, 4, 1), (20, 4, 5)]
PREFIX = [(dtype, D) for dtype in (BF16, F16) for D in (64, 128)]


def name(c):
    return "-".join(str(x).replace("torch.", "") for x in c)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", ROWS, ids=name)
@pytest.mark.parametrize("own", OWN, ids=name)
def test_own_rows(own, rows):
    (kind, dtype, D), (group, nq) = own, rows
    B, Hk = len(LENS), 2
    q = (synth.normal((B, Hk * group, nq, D), 400, F32) * 2).to(dtype).to(DEV)
    none = tuple(torch.empty(Hk, 0, D, dtype=dtype, device=DEV) for _ in range(2))
    if kind == "e4m3":
        c = random_cache(B, Hk, CAP, D, 401)
        vmax = ref.np.abs(ref.values(bits(c.v), bits(c.v_exp))).max()
    else:
        c = tuple(synth.normal((B, Hk, CAP, D), 401 + i, dtype).to(DEV) for i in range(2))
        vmax = 8.0
    o, lse = outputs(q)
    fa.fa_decode_shared(q, *none, c, int32(LENS), o.t, lse.t, True)
    assert ok() and o.guards_intact() and lse.guards_intact()
    check(o.t, lse.t, reference(q, None, None, c, LENS, D ** -0.5, True), max(LENS), F16 if kind == "e4m3" else dtype, vmax)


@pytest.mark.gpu
@pytest.mark.parametrize("batch", BATCHES, ids=name)
@pytest.mark.parametrize("prefix", PREFIX, ids=name)
@pytest.mark.parametrize("causal", [True, False])
def test_prefix(prefix, batch, causal):
    (dtype, D), (B, group, nq) = prefix, batch
    Hk, np_, cap = 2, 333, 9
    q = (synth.normal((B, Hk * group, nq, D), 410, F32) * 2).to(dtype).to(DEV)
    kp, vp = (synth.normal((Hk, np_, D), 411 + i, dtype).to(DEV) for i in range(2))
    c = tuple(synth.normal((B, Hk, cap, D), 413 + i, dtype).to(DEV) for i in range(2))
    lens = [(3 * b + 4) % (cap + 1) for b in range(B)]
    o, lse = outputs(q)
    fa.fa_decode_shared(q, kp, vp, c, int32(lens), o.t, lse.t, causal)
    assert ok() and o.guards_intact() and lse.guards_intact()
    check(o.t, lse.t, reference(q, kp, vp, c, lens, D ** -0.5, causal), np_ + cap, dtype, 8.0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype, D", PREFIX)
def test_no_keys_at_all(dtype, D):
    """Neither a prefix nor room for rows: only the join runs."""
    q = synth.normal((2, 4, 3, D), 420, dtype).to(DEV)
    none = tuple(torch.empty(2, 0, D, dtype=dtype, device=DEV) for _ in range(2))
    held = tuple(torch.empty(2, 2, 0, D, dtype=dtype, device=DEV) for _ in range(2))
    o, lse = outputs(q)
    fa.fa_decode_shared(q, *none, held, None, o.t, lse.t, True)
    assert ok() and o.guards_intact() and lse.guards_intact()
    assert bool((o.t == 0).all()) and bool((lse.t == float("-inf")).all())


def test_the_cases_reach_every_kernel(ask):  # noqa: F811
    cta_rows = [r[0] for r in ask("rows", 64)]
    kinds = {("e4m3", BF16): 0, ("e4m3", F16): 0, ("16", BF16): 1, ("16", F16): 2}
    reached = {(kinds[kind, dtype], D, cta_rows[g * n - 1]) for kind, dtype, D in OWN for g, n in ROWS}
    assert reached == {tuple(x[:3]) for x in ask("instances")}
    assert {16, 24} <= {cta_rows[g * n - 1] for g, n in ROWS if g * n > cta_rows[g * n - 1]}    # several row groups
    # the prefix: halves or pairs, with and without hidden keys
    kinds = {(ask("plan", B, 2 * g, 2, n, 333, 9, 64, 2)[0][0], n > 1) for B, g, n in BATCHES}
    assert kinds == {(0, False), (0, True), (1, False), (1, True)}
    for B, g, n in BATCHES:
        lens = [(3 * b + 4) % 10 for b in range(B)]
        assert n == 1 or min(lens) < n - 1                  # some do hide keys
