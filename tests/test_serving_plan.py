"""How a decoding step is laid over the SMs, asked of the host code itself (no GPU needed)."""

import os
import subprocess

import pytest

from exact_io_aware_37_gb300 import build as fa_build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan") / "serving_plan")
    r = subprocess.run([fa_build.nvcc_path(), *fa_build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I",
                        fa_build.INCLUDE, "-I", fa_build.CSRC, os.path.join(HERE, "serving_plan.cu"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]

    def run(*args):
        out = subprocess.run([exe, *map(str, args)], capture_output=True, text=True, check=True).stdout
        return [[int(x) for x in line.split()] for line in out.splitlines()]
    return run


def test_the_plan_counts_the_ctas_that_an_sm_holds(ask):
    got = ask("instances")
    assert len(got) == 24
    for kind, D, rows, has, planned in got:
        assert has == planned, (kind, D, rows)
    assert {has for *_, has, _ in got} == {1, 2}


def test_both_passes_end_at_about_the_same_time_where_an_sm_holds_one_cta(ask):
    """24 rows of 16-bit keys, D = 128: a tile of the own rows took 1.14 to 1.2 us of a whole SM, a run 3 to 5, a step of the
    prefix 1.6 to 2.2.  The longer pass takes at most half again as long as the shorter (counting two CTAs an
    SM: 1.7 and 1.8 times in the last two)."""
    for B, H, Hk, nq, np_, cap in ((16, 32, 8, 5, 8192, 1024), (16, 24, 8, 8, 8192, 1024), (24, 32, 8, 5, 32768, 512),
                                   (12, 32, 8, 5, 60000, 3000), (8, 32, 8, 5, 65536, 2048)):
        (split, pairs, steps, units, ctas, per_cta, own_sms), = ask("plan", B, H, Hk, nq, np_, cap, 128, 2)
        assert ctas + own_sms == 152 and ctas * per_cta >= units * steps
        tiles = B * Hk * (0.55 * cap / 128 + 0.5)
        own = 6 + (1.17 * tiles + 4 * B * Hk) / own_sms
        prefix = 9 + 1.6 * per_cta
        assert max(own, prefix) <= 1.5 * min(own, prefix), (B, H, Hk, nq, np_, cap, own, prefix)
