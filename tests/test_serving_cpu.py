"""Cached serving without a GPU: the reference's own pins, and the refusals of
fa_cache_write, fa_cache_read, fa_decode_cache and fa_decode_shared."""

import ctypes

import numpy as np
import pytest
import torch

import exact_io_aware_37_gb300 as fa
import serving_ref as ref
from exact_io_aware_37_gb300 import build as fa_build

OK, INVALID, UNSUPPORTED, ALIGN, CUDA, WORKSPACE = 0, -1, -2, -3, -4, -6


@pytest.fixture(scope="module")
def lib():
    fa_build.build()
    return fa.lib()


# ---------------------------------------------------------------- the format

def test_reference_quantiser_picks_the_nearest_code():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((200, 64)) * np.exp2(rng.integers(-140, 120, (200, 1)))
    x = x.astype(np.float32).astype(np.float64)
    codes, exps = ref.quantise(x)
    grid = np.unique(ref.CODES[np.isfinite(ref.CODES)])
    y = x * np.exp2(127.0 - exps)[:, None]
    assert np.abs(y).max() <= 448
    assert np.all(np.isin(codes, grid))
    best = np.abs(y[..., None] - grid).min(-1)
    assert np.array_equal(np.abs(y - codes), best)
    # the exponent is the smallest: half the scale would not do
    assert np.all((np.abs(y).max(-1) * 2 > 448) | (exps == 0))


@pytest.mark.parametrize("amax, exp", [(448.0, 127), (449.0, 128), (224.0, 126), (0.0, 0), (2.0 ** -149, 0),
                                       (3.0e38, 247)])
def test_reference_exponents_at_the_borders(amax, exp):
    x = np.zeros((1, 64))
    x[0, 3] = amax
    assert ref.quantise(x)[1][0] == exp


def test_reference_rows_that_are_not_finite():
    x = np.ones((1, 64))
    x[0, :3] = np.nan, np.inf, -np.inf
    codes, exps = ref.quantise(x)
    assert np.isnan(codes[0, :3]).all() and exps[0] == 127 - 8 and np.all(codes[0, 3:] == 256)


# ---------------------------------------------------------------- the C ABI

P = 0x1000


def _rows(lib, write=True, **kw):
    a = dict(k=P, v=P, kc=P, vc=P, ke=P, ve=P, B=2, H=3, n=4, cap=8, D=128, start=P, count=P, dt=0)
    a.update(kw)
    dense, held = (a["k"], a["v"]), (a["kc"], a["vc"], a["ke"], a["ve"])
    f = lib.fa_cache_write if write else lib.fa_cache_read
    return f(*(dense + held if write else held + dense), a["B"], a["H"], a["n"], a["cap"], a["D"], a["start"],
             a["count"], a["dt"], None)


@pytest.mark.parametrize("write", [True, False])
def test_cache_rows_validation(lib, write):
    def f(**kw):
        return _rows(lib, write, **kw)
    assert f(D=32) == UNSUPPORTED and f(D=96) == UNSUPPORTED and f(dt=7) == UNSUPPORTED
    assert f(B=-1) == INVALID and f(H=-1) == INVALID and f(n=-1) == INVALID and f(cap=-1) == INVALID
    assert f(D=0) == INVALID
    assert f(n=9) == INVALID                                # more rows than the cache holds
    assert f(B=65536) == UNSUPPORTED and f(H=65536) == UNSUPPORTED
    assert f(B=60000, H=60000) == UNSUPPORTED
    assert f(B=4096, H=64, n=8192, cap=8192) == UNSUPPORTED  # 2^31 rows
    for name in ("k", "v", "kc", "vc"):
        assert f(**{name: None}) == INVALID
        assert f(**{name: P + 8}) == ALIGN
    for name in ("ke", "ve"):
        assert f(**{name: None}) == INVALID
    assert f(start=P + 2) == ALIGN and f(count=P + 1) == ALIGN
    assert f(B=0) == OK and f(H=0) == OK and f(n=0) == OK and f(n=0, cap=0, k=None) == OK


def _decode(lib, ws=0x100000, ws_bytes=1 << 34, **kw):
    a = dict(q=P, k=P, v=P, ke=P, ve=P, o=P, lse=P, B=2, H=8, Hk=2, nq=1, cap=512, max_len=500, D=128, scale=0.1,
             causal=1, lens=P, dt=0)
    a.update(kw)
    return lib.fa_decode_cache(a["q"], a["k"], a["v"], a["ke"], a["ve"], a["o"], a["lse"], a["B"], a["H"], a["Hk"],
                               a["nq"], a["cap"], a["max_len"], a["D"], a["scale"], a["causal"], a["lens"], a["dt"],
                               ws, ws_bytes, None)


def _shared(lib, ws=0x100000, ws_bytes=1 << 34, **kw):
    a = dict(q=P, kp=P, vp=P, k=P, v=P, ke=None, ve=None, o=P, lse=P, B=2, H=8, Hk=2, nq=1, np=100, cap=512,
             max_len=500, D=128, scale=0.1, causal=1, lens=P, dt=0)
    a.update(kw)
    return lib.fa_decode_shared(a["q"], a["kp"], a["vp"], a["k"], a["v"], a["ke"], a["ve"], a["o"], a["lse"], a["B"],
                                a["H"], a["Hk"], a["nq"], a["np"], a["cap"], a["max_len"], a["D"], a["scale"],
                                a["causal"], a["lens"], a["dt"], ws, ws_bytes, None)


@pytest.mark.parametrize("call", [_decode, _shared])
def test_decode_validation(lib, call):
    def f(**kw):
        return call(lib, **kw)
    assert f(D=32) == UNSUPPORTED and f(D=256) == UNSUPPORTED
    assert f(dt=1) == UNSUPPORTED and f(dt=7) == UNSUPPORTED        # float32 queries have no kernel
    for name in ("B", "H", "Hk", "nq", "cap", "max_len"):
        assert f(**{name: -1}) == INVALID
    assert f(Hk=0) == INVALID and f(Hk=3) == INVALID                # heads that do not divide
    assert f(max_len=513) == INVALID
    assert f(B=65536) == UNSUPPORTED and f(H=65536, Hk=1) == UNSUPPORTED
    assert f(B=32768, H=32768, Hk=1, nq=2) == UNSUPPORTED
    assert f(scale=0.0) == INVALID and f(scale=-1.0) == INVALID and f(scale=float("nan")) == INVALID
    assert f(scale=float("inf")) == INVALID
    assert f(causal=2) == INVALID
    for name in ("q", "o", "k", "v"):
        assert f(**{name: None}) == INVALID
        assert f(**{name: P + 4}) == ALIGN
    assert f(lse=None) == INVALID and f(lse=P + 2) == ALIGN and f(lens=P + 1) == ALIGN
    assert f(ws=None) == WORKSPACE and f(ws=0x100010) == WORKSPACE and f(ws_bytes=64) == WORKSPACE
    assert f(B=0) == OK and f(nq=0) == OK and f(H=0, Hk=0) == OK


def test_decode_exponents_and_prefix_pointers(lib):
    assert _decode(lib, ke=None) == INVALID and _decode(lib, ve=None) == INVALID
    assert _shared(lib, ke=P) == INVALID and _shared(lib, ve=P) == INVALID      # one without the other
    assert _shared(lib, kp=None) == INVALID and _shared(lib, vp=P + 8) == ALIGN
    assert _shared(lib, np=-1) == INVALID
    assert _shared(lib, np=(1 << 30) - 400, cap=512) == UNSUPPORTED


def test_workspace_sizes(lib):
    size, shared = lib.fa_decode_cache_workspace_size, lib.fa_decode_shared_workspace_size
    # refused or empty problems need nothing
    assert size(0, 8, 2, 1, 100, 128, 0) == 0 and size(1, 8, 3, 1, 100, 128, 0) == 0
    assert size(1, 8, 2, 0, 100, 128, 0) == 0 and size(1, 8, 2, 1, 100, 96, 0) == 0 and size(1, 8, 2, 1, 100, 128, 1) == 0
    for f in (lambda *a: size(*a), lambda *a: shared(*a[:4], 1000, *a[4:])):
        n = f(16, 32, 8, 2, 8192, 128, 0)
        assert n > 0 and n % 256 == 0
    assert shared(16, 32, 8, 2, 0, 8192, 128, 0) >= size(16, 32, 8, 2, 8192, 128, 0)


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU error path")
def test_valid_calls_without_gpu_report_cuda_error(lib):
    assert _rows(lib) == CUDA and _rows(lib, False, start=None, count=None) == CUDA
    assert _decode(lib) == CUDA and _decode(lib, lens=None) == CUDA
    assert _shared(lib) == CUDA and _shared(lib, ke=P, ve=P) == CUDA
    assert _shared(lib, np=0, kp=None, vp=None) == CUDA
    assert _shared(lib, max_len=0, cap=0, k=None, v=None) == CUDA
    assert b"" != lib.fa_last_error_detail()


# ---------------------------------------------------------------- the binding

def _cache(B=2, Hk=2, cap=16, D=64):
    return fa.cache_alloc(B, Hk, cap, D, device="cpu")


def test_binding_refuses_cpu_tensors(lib):
    k = torch.zeros(2, 2, 4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_cache_write(k, k, _cache())
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_cache_read(_cache(), k, k)
    q = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16)
    o, lse = torch.empty_like(q), torch.empty(2, 4, 1)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_decode_cache(q, _cache(), None, o, lse, True)
    kp = torch.zeros(2, 5, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_decode_shared(q, kp, kp, _cache(), None, o, lse, True)


def test_binding_refuses_caches_that_do_not_fit_the_queries(lib):
    q = torch.zeros(2, 5, 1, 64, dtype=torch.bfloat16)
    for bad in (q, q[:1, :4], torch.zeros(2, 4, 1, 128, dtype=torch.bfloat16), q[0]):
        with pytest.raises(ValueError):
            fa.fa_decode_cache(bad, _cache(), None, bad, bad, True)
    with pytest.raises(ValueError, match="max_len"):
        fa.fa_decode_cache(q[:, :4], _cache(), None, q[:, :4], q, True, max_len=17)
    c = _cache()
    q = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16)
    for bad in (fa.Cache8(c.k.float(), c.v, c.k_exp, c.v_exp), fa.Cache8(c.k, c.v, c.k_exp.int(), c.v_exp),
                fa.Cache8(c.k, c.v[:, :1], c.k_exp, c.v_exp), fa.Cache8(c.k, c.v, c.k_exp[..., :3], c.v_exp)):
        with pytest.raises(ValueError):
            fa.fa_decode_cache(q, bad, None, q, q, True)
    kv = torch.zeros(2, 2, 16, 64, dtype=torch.float16)             # not q's dtype
    with pytest.raises(ValueError):
        fa.fa_decode_shared(q, kv[0], kv[0], (kv, kv), None, q, q, True)


def test_new_cache_is_empty():
    c = fa.cache_alloc(2, 3, 5, 64, device="cpu")
    assert c.k.shape == c.v.shape == (2, 3, 5, 64) and c.k_exp.shape == c.v_exp.shape == (2, 3, 5)
    assert c.k.dtype == torch.float8_e4m3fn and not c.k.view(torch.uint8).any() and not c.k_exp.any()


def test_every_serving_signature_matches_the_header():
    """Argument counts of the binding's table against the declarations."""
    import os
    import re
    src = open(os.path.join(fa_build.INCLUDE, "fa.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    from exact_io_aware_37_gb300._lib import SIGNATURES
    for name in ("fa_cache_write", "fa_cache_read", "fa_decode_cache", "fa_decode_shared",
                 "fa_decode_cache_workspace_size", "fa_decode_shared_workspace_size"):
        args = [x.strip() for x in re.search(name + r"\((.*?)\);", src, flags=re.S).group(1).split(",")]
        types = SIGNATURES[name][1]
        assert len(args) == len(types), name
        for a, t in zip(args, types):
            want = ctypes.c_void_p if "*" in a else (ctypes.c_float if a.startswith("float") else
                                                     ctypes.c_size_t if a.startswith("size_t") else ctypes.c_int)
            assert t is want, (name, a)
