"""Refusals of the block-scaled FP8 operators, checked before any GPU work (fake addresses that
are never dereferenced), and the weight encoder."""
import ctypes
import os
import sys

import pytest
import torch

import swiglu_mlp_dfk_b200 as dfk
from swiglu_mlp_dfk_b200 import inputs as I

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    from swiglu_mlp_dfk_b200 import build
    build.build()
    return dfk.lib()


P, P2, P3, P4, P5, P6 = (ctypes.c_void_p(0x10000 * (i + 1)) for i in range(6))
MIS = ctypes.c_void_p(0x10008)   # not 16-byte aligned
ODD = ctypes.c_void_p(0x10002)   # not 4-byte aligned
BAD, SHAPE, ALIGN = dfk.DFK_ERR_INVALID_ARG, dfk.DFK_ERR_UNSUPPORTED_SHAPE, dfk.DFK_ERR_MISALIGNED


def quant(L, x=P, q=P2, s=P3, M=1, K=128):
    return L.dfk_quant_fp8_block(x, q, s, M, K, None)


def norm(L, x=P, res=P2, gamma=P3, eps=1e-5, out=P4, q=P5, s=P6, M=1, D=128):
    return L.dfk_add_rmsnorm_fp8_block(x, res, gamma, eps, out, q, s, M, D, None)


def gemm(L, qx=P, sx=P2, qw=P3, sw=P4, y=P5, M=1, K=128, N=128):
    return L.dfk_gemm_fp8_block(qx, sx, qw, sw, y, M, K, N, None)


def gate_up(L, qx=P, sx=P2, qg=P3, sg=P4, qu=P3, su=P4, h=None, qh=P5, sh=P6, M=1, D=128, F=128):
    return L.dfk_swiglu_gate_up_fp8_block(qx, sx, qg, sg, qu, su, h, qh, sh, M, D, F, None)


@pytest.mark.parametrize("fn,kw,status", [
    (quant, dict(M=-1), BAD), (quant, dict(K=0), BAD), (quant, dict(K=24), SHAPE),
    (quant, dict(x=None), BAD), (quant, dict(q=None), BAD), (quant, dict(s=None), BAD),
    (quant, dict(x=MIS), ALIGN), (quant, dict(q=MIS), ALIGN), (quant, dict(s=ODD), ALIGN),
    (norm, dict(M=-1), BAD), (norm, dict(D=-16), BAD), (norm, dict(D=120), SHAPE),
    (norm, dict(D=32784), SHAPE), (norm, dict(eps=-1.0), BAD), (norm, dict(eps=float("nan")), BAD),
    (norm, dict(eps=float("inf")), BAD), (norm, dict(x=None), BAD), (norm, dict(gamma=None), BAD),
    (norm, dict(out=None), BAD), (norm, dict(res=None), BAD), (norm, dict(q=None), BAD),
    (norm, dict(s=None), BAD), (norm, dict(res=MIS), ALIGN), (norm, dict(out=MIS), ALIGN),
    (norm, dict(gamma=MIS), ALIGN), (norm, dict(s=ODD), ALIGN),
    (gemm, dict(M=-1), BAD), (gemm, dict(N=0), BAD), (gemm, dict(K=8), SHAPE),
    (gemm, dict(qx=None), BAD), (gemm, dict(sx=None), BAD), (gemm, dict(qw=None), BAD),
    (gemm, dict(sw=None), BAD), (gemm, dict(y=None), BAD), (gemm, dict(qx=MIS), ALIGN),
    (gemm, dict(qw=MIS), ALIGN), (gemm, dict(y=MIS), ALIGN), (gemm, dict(sx=ODD), ALIGN),
    (gemm, dict(sw=ODD), ALIGN),
    (gate_up, dict(M=-1), BAD), (gate_up, dict(F=0), BAD), (gate_up, dict(D=8), SHAPE),
    (gate_up, dict(F=24), SHAPE), (gate_up, dict(h=P5), BAD), (gate_up, dict(qh=None), BAD),
    (gate_up, dict(sh=None), BAD), (gate_up, dict(qh=None, sh=None), BAD),
    (gate_up, dict(qu=None), BAD), (gate_up, dict(su=None), BAD), (gate_up, dict(qg=MIS), ALIGN),
    (gate_up, dict(qu=MIS), ALIGN), (gate_up, dict(qh=MIS), ALIGN), (gate_up, dict(sh=ODD), ALIGN),
    (gate_up, dict(su=ODD), ALIGN), (gate_up, dict(h=MIS, qh=None, sh=None), ALIGN),
    (quant, dict(M=2 ** 31 - 1), SHAPE), (quant, dict(K=2 ** 31 - 16), SHAPE),
    (norm, dict(M=2 ** 31 - 1), SHAPE), (gemm, dict(M=2 ** 31 - 1), SHAPE),
    (gemm, dict(K=2 ** 31 - 16), SHAPE), (gemm, dict(N=2 ** 31 - 1), SHAPE),
    (gate_up, dict(F=2 ** 31 - 16), SHAPE),
])
def test_refusals(L, fn, kw, status):
    assert fn(L, **kw) == status
    assert L.dfk_last_error().decode()


def test_no_tokens_is_a_no_op(L):
    assert quant(L, x=None, M=0) == 0
    assert norm(L, x=None, M=0) == 0
    assert gemm(L, qx=None, M=0) == 0
    assert gate_up(L, qx=None, M=0) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the behaviour without a device")
def test_valid_calls_fail_loudly_without_a_device(L):
    for fn in (quant, norm, gemm, gate_up):
        assert fn(L) == dfk.DFK_ERR_ARCH


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    for call in (lambda: dfk.dfk_quant_fp8_block(x),
                 lambda: dfk.dfk_add_rmsnorm_fp8_block(x, None, x[0], 1e-5),
                 lambda: dfk.dfk_gemm_fp8_block(x, x, x, x),
                 lambda: dfk.dfk_swiglu_gate_up_fp8_block(x, x, x, x, x, x)):
        with pytest.raises(dfk.DfkError) as e:
            call()
        assert e.value.status == BAD


def test_fast_calls_refuse_quietly(L):
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    f = dfk._fast
    for call, n in ((f.quant, 3), (f.norm, 7), (f.gemm, 5), (f.gate_up, 10)):
        for v in (x, None, 1, 1.0, "x", [x]):
            assert call(*[v] * n) is None
        assert call() is None and call(*[x] * (n + 1)) is None


def test_what_the_previous_call_may_write_is_no_read_only_memory():
    """The read-only path may serve what the memory held before the previous kernel wrote it: only
    gamma, weights and their scales, which are read early by contract, may take it."""
    import glob
    import re
    csrc = os.path.join(os.path.dirname(dfk.__file__), "csrc")
    loads = []
    for path in sorted(glob.glob(os.path.join(csrc, "fp8_block*.cu*"))):
        with open(path) as f:
            code = re.sub(r"//[^\n]*", "", f.read())
        assert "ld.global.nc" not in code
        loads += re.findall(r"(?:__ldg|ld_nc_v4)\(\s*((?:[^();]|\([^();]*\))*)\)", code)
    assert loads and all(re.search(r"gamma|p\.sw\[", arg) for arg in loads), loads


@pytest.mark.parametrize("compiler", ["false", "/nonexistent/g++"])
def test_a_build_without_a_cxx_compiler(monkeypatch, tmp_path, compiler):
    """The library is built and loaded without the module of the calls."""
    from swiglu_mlp_dfk_b200 import build
    monkeypatch.setenv("CXX", compiler)
    monkeypatch.setattr(build, "PKG", str(tmp_path))
    monkeypatch.setattr(build, "_calls_failed", False)
    with pytest.warns(RuntimeWarning, match="cannot be built"):
        assert build.build() == build.LIB
    assert not list(tmp_path.iterdir())
    build.build()                                # not tried, and not said, again


def test_a_module_of_the_calls_for_another_torch_is_not_loaded(L, monkeypatch):
    from swiglu_mlp_dfk_b200 import build
    assert dfk._fast is not None and os.path.exists(build.calls_path())
    monkeypatch.setattr(dfk, "_fast", None)
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "0.0.0")
        with pytest.warns(RuntimeWarning, match="cannot be loaded"):
            dfk._load_calls(L)
        assert dfk._fast is None
    dfk._load_calls(L)
    assert dfk._fast is not None


def test_a_module_of_the_calls_older_than_its_source_is_not_kept(monkeypatch, tmp_path):
    from swiglu_mlp_dfk_b200 import build
    monkeypatch.setattr(build, "PKG", str(tmp_path))
    monkeypatch.setattr(build, "_calls_failed", False)
    monkeypatch.setenv("CXX", "false")
    out = build.calls_path()
    open(out, "wb").close()
    build._build_calls(False, False)
    assert os.path.exists(out)                   # newer than its source
    os.utime(out, (0, 0))
    with pytest.warns(RuntimeWarning, match="cannot be built"):
        build._build_calls(False, False)
    assert not os.path.exists(out)


@pytest.mark.parametrize("nmat", [1, 2])
def test_the_listed_products_take_every_form(L, nmat):
    """A change in the choice of form that leaves one without a test fails here."""
    import math
    import random

    import fp8_block_forms as forms
    listed = forms.PLAIN if nmat == 1 else forms.GATED
    for sizes, form in listed:
        assert forms.form(nmat, *sizes) == form, sizes
    rng = random.Random(nmat)

    def spread(lo, hi):
        return int(math.exp(rng.uniform(math.log(lo), math.log(hi))))
    met = {forms.form(nmat, spread(1, 5000), 16 * spread(1, 1024), spread(1, 40000))
           for _ in range(100000)}
    assert met == {form for _, form in listed}


@pytest.mark.parametrize("N,K", [(1, 16), (128, 128), (129, 144), (300, 272)])
def test_weight_encoder(N, K):
    g = torch.Generator().manual_seed(N)
    w = torch.randn(N, K, generator=g)
    w[: min(N, 128), :128] = 0          # an all-zero block
    q, s = I.to_fp8_blocks(w)
    assert q.shape == (N, K) and q.dtype == torch.float8_e4m3fn
    assert s.shape == (-(-N // 128), -(-K // 128)) and s.dtype == torch.float32
    assert s[0, 0] == 2.0 ** -126 and (q[:128, :128].float() == 0).all()
    sf = s.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    err = (q.double() * sf - w.double()).abs()
    # half a step of E4M3: 2^-4 of the value, or 2^-10 of the scale below the normal range
    assert (err <= torch.maximum(w.double().abs() * 2.0 ** -4, sf * 2.0 ** -10) * (1 + 1e-6)).all()
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            top = w[128 * i:128 * i + 128, 128 * j:128 * j + 128].abs().max()
            assert s[i, j] == max((top / 448).item(), 2.0 ** -126)
