"""The block-scaled FP8 operators on the GPU against their definitions in 64 bits.

Tolerances, from the arithmetic:
  * a rounding is off by at most half a step: bf16 2^-8 of the value, E4M3 2^-4 of the value or,
    below its normal range, 2^-10 of the scale;
  * a product over groups of 128 in fp32: each of a group's 128 exact products enters the sum with
    at most one step 2^-23 of error, then each of the G groups is scaled (two roundings) and added
    (one): together (128 * 2^-23 + (G + 3) * 2^-24) times the sum of the terms' magnitudes;
  * SiLU's slope is below 1.1; __expf is within 2 + 1.2 |a| steps 2^-23 and the quotient and the
    product a few: (8 + 2 |a|) 2^-23 of the value.
"""
import os
import subprocess
import sys

import pytest
import torch

import swiglu_mlp_dfk_b200 as dfk
from swiglu_mlp_dfk_b200 import inputs as I

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import fp8_block_forms as forms

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from swiglu_mlp_dfk_b200 import build
    build.build()
    dfk.dfk_device_error()
    yield
    torch.cuda.synchronize()
    assert dfk.dfk_device_error() == 0


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rand_bf16(g, *shape, std=1.0):
    return (std * torch.randn(*shape, generator=g, device="cuda")).bfloat16()


def spread(q, s, dim_rows):
    """Scales of codes as a full matrix: s [G, M] (activations) or [N/128, G] (weights)."""
    M, K = q.shape
    s = s.double()
    s = s.t() if dim_rows else s.repeat_interleave(128, 0)[:M]
    return s.repeat_interleave(128, 1)[:, :K]


def values(q, s, activations=True):
    return q.view(E4M3).double() * spread(q, s, activations)


def activations(g, M, K):
    """8-bit activations made by plain torch operations."""
    G = -(-K // 128)
    x = torch.randn(M, K, generator=g, device="cuda") * \
        torch.exp(torch.randn(M, 1, generator=g, device="cuda"))
    p = torch.nn.functional.pad(x, (0, G * 128 - K)).view(M, G, 128)
    s = (p.abs().amax(2) / 448).clamp(min=2.0 ** -126)
    q = (p / s[:, :, None]).clamp(-448, 448).to(E4M3).view(M, -1)[:, :K].contiguous()
    return q, s.t().contiguous()


def weights(g, N, K, std=0.05):
    w = I.to_fp8_blocks(std * torch.randn(N, K, generator=g, device="cuda"))
    torch.cuda.synchronize()      # weights are read before the previous kernel has finished
    return w


def sum_error(G):
    return 128 * 2.0 ** -23 + (G + 3) * 2.0 ** -24


def product(q_x, s_x, q_w, s_w):
    """(x W^T, its error bound) in 64 bits."""
    x, w = values(q_x, s_x), values(q_w, s_w, False)
    return x @ w.t(), sum_error(s_x.shape[0]) * (x.abs() @ w.abs().t())


def check_rounded(y, ref, err, step):
    bad = (y.double() - ref).abs() > step * ref.abs() + err * (1 + step)
    assert not bad.any(), (int(bad.sum()), float((y.double() - ref).abs().max()))


def check_quantised(q, s, ref, err):
    """Codes and scales against the unrounded values `ref`, known to within `err`."""
    M, K = ref.shape
    G = -(-K // 128)
    pad = (0, G * 128 - K)
    top = torch.nn.functional.pad(ref.abs(), pad).view(M, G, 128).amax(2).t()
    off = torch.nn.functional.pad(err, pad).view(M, G, 128).amax(2).t()
    want = (top / 448).clamp(min=2.0 ** -126)
    assert ((s.double() - want).abs() <= off / 448 + 2.0 ** -23 * want).all()
    got, sf = values(q, s), spread(q, s, True)
    half = torch.maximum(2.0 ** -4 * ref.abs(), 2.0 ** -10 * sf)
    bad = (got - ref).abs() > half * (1 + 2.0 ** -20) + err * (1 + 2.0 ** -3)
    assert not bad.any(), (int(bad.sum()), float((got - ref).abs().max()))


def silu_mul(a, ea, u, eu):
    """SiLU(a) * u in 64 bits and how far it may be off."""
    f = a * torch.sigmoid(a)
    return f * u, 1.1 * ea * (u.abs() + eu) + f.abs() * eu + \
        (8 + 2 * a.abs()) * 2.0 ** -23 * (f * u).abs()


# ---- quantisation

def quant_reference(x):
    """Bitwise: fp32 division is correctly rounded on both sides."""
    M, K = x.shape
    G = -(-K // 128)
    p = torch.nn.functional.pad(x.float().cpu(), (0, G * 128 - K)).view(M, G, 128)
    s = (p.abs().amax(2) / 448).clamp(min=2.0 ** -126)
    q = (p / s[:, :, None]).clamp(-448, 448).to(E4M3).view(M, -1)[:, :K]
    return q.contiguous(), s.t().contiguous()


@pytest.mark.parametrize("M,K", [(1, 16), (1, 4096), (2, 112), (3, 128), (4, 144), (5, 2064),
                                 (7, 14336), (33, 688), (130, 256), (257, 1040), (1000, 272)])
def test_quant(M, K):
    x = rand_bf16(gen(M * 10000 + K), M, K)
    q, s = dfk.dfk_quant_fp8_block(x)
    wq, ws = quant_reference(x)
    assert torch.equal(s.cpu(), ws)
    assert torch.equal(q.cpu().view(torch.uint8), wq.view(torch.uint8))


def test_quant_every_bf16_pair_of_magnitudes():
    """Every positive bf16 mantissa against every largest-element mantissa: all the ties."""
    a = (torch.arange(128, dtype=torch.float64) / 128 + 1)
    x = torch.empty(128 * 8, 128, dtype=torch.float64)
    for e in range(8):
        x[e * 128:(e + 1) * 128, 1:] = (a[:127] * 2.0 ** -e)[None]
        x[e * 128:(e + 1) * 128, 0] = a * 2
    x[:, 2::2] *= -1
    x = x.cuda().bfloat16()
    q, s = dfk.dfk_quant_fp8_block(x)
    wq, ws = quant_reference(x)
    assert torch.equal(s.cpu(), ws)
    assert torch.equal(q.cpu().view(torch.uint8), wq.view(torch.uint8))


def test_quant_special_values():
    x = torch.zeros(6, 384, device="cuda", dtype=torch.bfloat16)
    x[1, :128] = 2.0 ** -133                       # the smallest bf16: scale at its floor
    x[2, 130] = float("nan")
    x[3, 5] = float("inf")
    x[3, 6] = 3.0
    x[4, 300] = torch.finfo(torch.bfloat16).max
    x[5, :] = -1.0
    q, s = dfk.dfk_quant_fp8_block(x)
    f = q.float()
    assert (s[:, 0] == 2.0 ** -126).all() and (f[0] == 0).all()
    assert s[0, 1] == 2.0 ** -126 and (f[1, :128] == 2.0 ** -7).all()
    assert torch.isnan(s[1, 2]) and torch.isnan(f[2, 128:256]).all()
    assert not torch.isnan(f[2, :128]).any() and not torch.isnan(f[2, 256:]).any()
    assert torch.isinf(s[0, 3]) and torch.isnan(f[3, 5]) and f[3, 6] == 0
    assert f[4, 300] == 448 and torch.isfinite(s[:, 4]).all()
    assert (f[5] == -448).all()


# ---- norm

@pytest.mark.parametrize("M,D", [(1, 16), (1, 4096), (2, 144), (3, 688), (5, 2064), (9, 4112),
                                 (17, 8192), (300, 256), (2, 16400), (3, 32768)])
@pytest.mark.parametrize("with_residual", [True, False])
def test_add_rmsnorm(M, D, with_residual):
    g = gen(M + D)
    x, res = rand_bf16(g, M, D), rand_bf16(g, M, D, std=3.0)
    gamma = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).bfloat16()
    q, s, r = dfk.dfk_add_rmsnorm_fp8_block(x, res if with_residual else None, gamma, 1e-5)
    if with_residual:
        assert torch.equal(r, (x.float() + res.float()).bfloat16())
    else:
        assert r is None
        r = x
    d = r.double()
    v = d / (d.square().mean(1, keepdim=True) + 1e-5).sqrt() * gamma.double()
    # a thread chains 32 squares at most, two butterflies add 10 more, then the mean, the root,
    # the quotient and two products: under 64 roundings of 2^-24, halved by the root
    check_quantised(q, s, v, 2.0 ** -18 * v.abs())


def test_add_rmsnorm_in_place_and_zero_rows():
    g = gen(5)
    x, res = rand_bf16(g, 4, 512), rand_bf16(g, 4, 512)
    x[2] = 0
    res[2] = 0
    gamma = torch.ones(512, device="cuda").bfloat16()
    q0, s0, r0 = dfk.dfk_add_rmsnorm_fp8_block(x, res, gamma, 1e-5)
    assert (q0[2].float() == 0).all() and (s0[:, 2] == 2.0 ** -126).all()
    for into in ("residual", "x"):
        a, b = x.clone(), res.clone()
        out = b if into == "residual" else a
        q, s, r = dfk.dfk_add_rmsnorm_fp8_block(a, b, gamma, 1e-5, residual_out=out)
        assert r is out and torch.equal(r, r0)
        assert torch.equal(q.view(torch.uint8), q0.view(torch.uint8)) and torch.equal(s, s0)


@pytest.mark.parametrize("M", [5, 1100])
def test_add_rmsnorm_in_place_of_every_size(M):
    g = gen(M)
    x, res = rand_bf16(g, M, 1040), rand_bf16(g, M, 1040)
    x[0, :8] = 2.0 ** -133                       # subnormal bf16 sums are kept
    res[0, :8] = 2.0 ** -133
    gamma = rand_bf16(g, 1040)
    q0, s0, r0 = dfk.dfk_add_rmsnorm_fp8_block(x, res, gamma, 1e-5)
    assert torch.equal(r0, (x.float() + res.float()).bfloat16())
    assert (r0[0, :8] == 2.0 ** -132).all()
    q, s, r = dfk.dfk_add_rmsnorm_fp8_block(x, res, gamma, 1e-5, residual_out=res)
    assert r is res and torch.equal(r, r0) and torch.equal(s, s0)
    assert torch.equal(q.view(torch.uint8), q0.view(torch.uint8))


def test_add_rmsnorm_all_zero_row_with_zero_eps_is_nan_as_the_formula():
    x = torch.zeros(2, 256, device="cuda", dtype=torch.bfloat16)
    x[1] = 1
    q, s, _ = dfk.dfk_add_rmsnorm_fp8_block(x, None, torch.ones_like(x[0]), 0.0)
    assert torch.isnan(s[:, 0]).all() and torch.isnan(q[0].float()).all()   # 0 * inf
    assert torch.isfinite(s[:, 1]).all() and (q[1].float() == 448).all()


@pytest.mark.parametrize("M", [9, 1100])
def test_add_rmsnorm_groups_near_the_scales_floor(M):
    """Groups whose largest value lies from 1/8 to 8 times 448 * 2^-126, the scale's floor."""
    D, steps = 8192, 64
    g = gen(M)
    x = (torch.randn(M, D, generator=g, device="cuda")
         * torch.linspace(1, 2, M, device="cuda")[:, None]).bfloat16()  # every factor of the root
    e = torch.linspace(-3, 3, steps, device="cuda").exp2() * 2.0 ** -118
    gamma = e.repeat_interleave(128).bfloat16()
    q, s, _ = dfk.dfk_add_rmsnorm_fp8_block(x, None, gamma, 1e-5)
    d = x.double()
    v = d / (d.square().mean(1, keepdim=True) + 1e-5).sqrt() * gamma.double()
    # as in test_add_rmsnorm, and a few steps 2^-149 where a value is subnormal
    check_quantised(q, s, v, 2.0 ** -18 * v.abs() + 2.0 ** -147)


@pytest.mark.parametrize("M", [3, 1100])
def test_add_rmsnorm_overflow_is_the_headers_rule(M):
    """An element whose normalised value passes fp32: infinite scale, its own code NaN, the
    others 0; the next group is untouched."""
    x = torch.ones(M, 256, device="cuda", dtype=torch.bfloat16)
    x[:, 5] = 2                            # 2 / sqrt(259 / 256) * 3.39e38; the ones stay finite
    gamma = torch.ones(256, device="cuda", dtype=torch.bfloat16)
    gamma[:128] = torch.finfo(torch.bfloat16).max
    q, s, _ = dfk.dfk_add_rmsnorm_fp8_block(x, None, gamma, 1e-5)
    f = q.float()
    assert torch.isinf(s[0]).all() and torch.isnan(f[:, 5]).all()
    f[:, 5] = 0
    assert (f[:, :128] == 0).all()
    assert torch.isfinite(s[1]).all() and (f[:, 128:] == 448).all()


# ---- products

SHAPES = [(1, 16, 1), (1, 128, 128), (2, 144, 130), (1, 4096, 512), (3, 2064, 1001),
          (16, 1040, 129), (17, 256, 688), (31, 688, 256), (33, 272, 96), (64, 512, 4096),
          (65, 512, 1032), (127, 640, 384), (128, 128, 257), (129, 1152, 640), (200, 400, 1000),
          (255, 2064, 255), (256, 256, 256), (257, 384, 520), (300, 14336, 200), (513, 144, 768),
          (777, 2064, 1001), (1024, 1024, 1024), (1100, 400, 5000), (2500, 144, 2056)]


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_gemm(M, K, N):
    g = gen(M * 7 + K * 3 + N)
    q_x, s_x = activations(g, M, K)
    q_w, s_w = weights(g, N, K)
    y = dfk.dfk_gemm_fp8_block(q_x, s_x, q_w, s_w)
    ref, err = product(q_x, s_x, q_w, s_w)
    check_rounded(y, ref, err, 2.0 ** -8)


@pytest.mark.parametrize("M,D,F", [s for s in SHAPES if s[1] < 4000 or s[0] < 100])
@pytest.mark.parametrize("fp8_out", [True, False])
def test_gate_up(M, D, F, fp8_out):
    if fp8_out:
        F = -(-F // 16) * 16
    g = gen(M * 5 + D + F)
    q_x, s_x = activations(g, M, D)
    wg, wu = weights(g, F, D), weights(g, F, D)
    out = dfk.dfk_swiglu_gate_up_fp8_block(q_x, s_x, *wg, *wu, fp8_out=fp8_out)
    ref, err = silu_mul(*product(q_x, s_x, *wg), *product(q_x, s_x, *wu))
    if fp8_out:
        check_quantised(*out, ref, err)
    else:
        check_rounded(out, ref, err, 2.0 ** -8)


# Sizes of the tensor-bound kernel's forms: pairs of CTAs, single CTAs (fewer rounds of tiles),
# clusters that share a tile's groups; odd columns, part tiles, shorter last groups.
@pytest.mark.parametrize("M,K,N", [(1100, 400, 5001), (2300, 272, 4112), (400, 272, 9008),
                                   (330, 144, 12296), (192, 14336, 4001), (150, 4112, 2048),
                                   (700, 656, 3002)])
@pytest.mark.parametrize("op", ["gemm", "fp8", "bf16"])
def test_forms_for_many_tokens(M, K, N, op):
    g = gen(M + K)
    q_x, s_x = activations(g, M, K)
    if op == "gemm":
        w = weights(g, N, K)
        check_rounded(dfk.dfk_gemm_fp8_block(q_x, s_x, *w), *product(q_x, s_x, *w), 2.0 ** -8)
        return
    if op == "fp8":
        N = -(-N // 16) * 16
    N = min(N, 6000) if K > 4000 else N
    wg, wu = weights(g, N, K), weights(g, N, K)
    out = dfk.dfk_swiglu_gate_up_fp8_block(q_x, s_x, *wg, *wu, fp8_out=op == "fp8")
    ref, err = silu_mul(*product(q_x, s_x, *wg), *product(q_x, s_x, *wu))
    if op == "fp8":
        check_quantised(*out, ref, err)
    else:
        check_rounded(out, ref, err, 2.0 ** -8)


# Clusters that add their shares of a part block of columns: two and four CTAs of the tensor-bound
# kernel with no column in their second 128 (plain), of both kernels with 16 or 48 in the last
# group (gated).
@pytest.mark.parametrize("M,K,N,op", [(150, 4112, 6465, "gemm"), (150, 6160, 3905, "gemm"),
                                      (20, 4096, 688, "fp8"), (40, 4096, 688, "fp8"),
                                      (130, 8208, 1808, "fp8"), (130, 8208, 1808, "bf16")])
def test_shared_sums_of_a_part_block(M, K, N, op):
    g = gen(M + N)
    q_x, s_x = activations(g, M, K)
    w = [weights(g, N, K) for _ in range(1 if op == "gemm" else 2)]

    def call():
        if op == "gemm":
            return (dfk.dfk_gemm_fp8_block(q_x, s_x, *w[0]),)
        out = dfk.dfk_swiglu_gate_up_fp8_block(q_x, s_x, *w[0], *w[1], fp8_out=op == "fp8")
        return out if op == "fp8" else (out,)

    out = call()
    ref, err = product(q_x, s_x, *w[0])
    if op != "gemm":
        ref, err = silu_mul(ref, err, *product(q_x, s_x, *w[1]))
    if op == "fp8":
        check_quantised(*out, ref, err)
    else:
        check_rounded(out[0], ref, err, 2.0 ** -8)
    again = [call() for _ in range(50)]      # back to back: the next call's CTAs take over at once
    assert all(same(out, o) for o in again)


def check_form(op, sizes, form):
    M, K, N = sizes
    nmat = 1 if op == "gemm" else 2
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert forms.form(nmat, M, K, N, sms) == form
    g = gen(M + K + N)
    q_x, s_x = activations(g, M, K)
    w = [weights(g, N, K) for _ in range(nmat)]
    ref, err = product(q_x, s_x, *w[0])
    if op == "gemm":
        check_rounded(dfk.dfk_gemm_fp8_block(q_x, s_x, *w[0]), ref, err, 2.0 ** -8)
        return
    ref, err = silu_mul(ref, err, *product(q_x, s_x, *w[1]))
    out = dfk.dfk_swiglu_gate_up_fp8_block(q_x, s_x, *w[0], *w[1], fp8_out=op == "fp8")
    if op == "fp8":
        check_quantised(*out, ref, err)
    else:
        check_rounded(out, ref, err, 2.0 ** -8)


@pytest.mark.parametrize("sizes,form", forms.PLAIN)
def test_gemm_in_every_form(sizes, form):
    check_form("gemm", sizes, form)


@pytest.mark.parametrize("sizes,form", forms.GATED)
@pytest.mark.parametrize("op", ["fp8", "bf16"])
def test_gate_up_in_every_form(op, sizes, form):
    check_form(op, sizes, form)


def test_codes_as_bytes():
    g = gen(8)
    q_x, s_x = activations(g, 70, 256)
    q_w, s_w = weights(g, 128, 256)
    u8 = torch.uint8
    y = dfk.dfk_gemm_fp8_block(q_x, s_x, q_w, s_w)
    assert torch.equal(y, dfk.dfk_gemm_fp8_block(q_x.view(u8), s_x, q_w.view(u8), s_w))
    q = torch.empty(70, 128, dtype=u8, device="cuda")
    want, s = dfk.dfk_quant_fp8_block(y)
    got, s2 = dfk.dfk_quant_fp8_block(y, q=q)
    assert got is q and torch.equal(q, want.view(u8)) and torch.equal(s, s2)


def test_silu_far_from_zero():
    """Gate values from -600 to 600: SiLU's limits, no overflow."""
    M, D, F = 40, 128, 128
    q_x = torch.zeros(M, D, device="cuda", dtype=E4M3)
    q_x[:, 0] = 1
    s_x = torch.linspace(-600, 600, M, device="cuda")[None].contiguous()
    q_w = torch.ones(F, D, device="cuda").to(E4M3)
    s_w = torch.ones(1, 1, device="cuda")
    h = dfk.dfk_swiglu_gate_up_fp8_block(q_x, s_x, q_w, s_w, q_w, s_w / 256, fp8_out=False)
    a = s_x[0].double()
    ref = (a * torch.sigmoid(a) * a / 256)[:, None].expand(M, F)
    assert torch.isfinite(h.float()).all()
    # below -80 exp(a) leaves fp32's normal range: there SiLU * up is under 1e-30
    assert ((h.double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -12) * ref.abs() + 1e-30).all()


@pytest.mark.parametrize("M", [40, 300, 1100])
def test_silu_of_the_lowest_gates(M):
    """Gates from -75 to -100, where e^a leaves fp32's normal range, beside a large up."""
    D, F = 128, 128
    q_x = torch.zeros(M, D, device="cuda", dtype=E4M3)
    q_x[:, 0] = 1
    s_x = torch.linspace(-100, -75, M, device="cuda")[None].contiguous()
    q_w = torch.ones(F, D, device="cuda").to(E4M3)
    s_w = torch.ones(1, 1, device="cuda")
    h = dfk.dfk_swiglu_gate_up_fp8_block(q_x, s_x, q_w, s_w, q_w, s_w * 2.0 ** 100, fp8_out=False)
    a, u = s_x[0].double(), s_x[0].double() * 2.0 ** 100
    ref = (a * torch.sigmoid(a) * u)[:, None]
    # the bound of silu_mul with nothing off before it, one step 2^-149 of the exponential and
    # half a step of its product with the gate, and bf16's rounding
    err = ((8 + 2 * a.abs()) * 2.0 ** -23)[:, None] * ref.abs()
    err = err + (1.5 * a.abs() * 2.0 ** -149 * u.abs())[:, None]
    check_rounded(h, ref.expand(M, F), err.expand(M, F), 2.0 ** -8)


def test_scales_of_every_block_count():
    """One code per group and block: y shows which scale met which."""
    M, K, N = 150, 656, 400
    G, B = 6, 4
    q_x = torch.zeros(M, K, device="cuda", dtype=E4M3)
    q_x[:, ::128] = 1
    q_w = torch.ones(N, K, device="cuda").to(E4M3)
    g = gen(3)
    s_x = torch.randn(G, M, generator=g, device="cuda").bfloat16().float()
    s_w = torch.randn(B, G, generator=g, device="cuda").bfloat16().float()
    y = dfk.dfk_gemm_fp8_block(q_x, s_x, q_w, s_w)
    ref, err = product(q_x, s_x, q_w, s_w)
    check_rounded(y, ref, err, 2.0 ** -8)


@pytest.mark.parametrize("M,K,N", [(5, 256, 136), (70, 272, 200), (300, 528, 392)])
def test_outputs_stay_inside_their_tensors(M, K, N):
    g = gen(M)
    q_x, s_x = activations(g, M, K)
    N16 = -(-N // 16) * 16
    wg, wu = weights(g, N16, K), weights(g, N16, K)

    def framed(shape, dtype):
        n = 1
        for d in shape:
            n *= d
        n *= torch.empty((), dtype=dtype).element_size()
        buf = torch.full((n + 512,), 0x5a, dtype=torch.uint8, device="cuda")
        return buf, buf[256:256 + n].view(dtype).view(shape)

    y_buf, y = framed((M, N16), torch.bfloat16)
    dfk.dfk_gemm_fp8_block(q_x, s_x, *wg, y=y)
    h_buf, h = framed((M, N16), torch.bfloat16)
    dfk.dfk_swiglu_gate_up_fp8_block(q_x, s_x, *wg, *wu, fp8_out=False, h=h)
    q_buf, q = framed((M, N16), E4M3)
    s_buf, s = framed((-(-N16 // 128), M), torch.float32)
    dfk.dfk_swiglu_gate_up_fp8_block(q_x, s_x, *wg, *wu, q_h=q, s_h=s)
    c_buf, c = framed((M, N16), E4M3)
    t_buf, t = framed((-(-N16 // 128), M), torch.float32)
    r_buf, r = framed((M, N16), torch.bfloat16)
    dfk.dfk_quant_fp8_block(h, q=c, s=t)
    dfk.dfk_add_rmsnorm_fp8_block(h, y, torch.ones_like(h[0]), 1e-5, residual_out=r, q=c, s=t)
    torch.cuda.synchronize()
    for b in (y_buf, h_buf, q_buf, s_buf, c_buf, t_buf, r_buf):
        assert (b[:256] == 0x5a).all() and (b[-256:] == 0x5a).all()
    assert torch.equal(y, dfk.dfk_gemm_fp8_block(q_x, s_x, *wg))


@pytest.mark.parametrize("M", [3, 40, 130, 300])
def test_a_token_that_is_nan_leaves_the_others(M):
    g = gen(M)
    x = rand_bf16(g, M, 512)
    wg, wu, wd = weights(g, 384, 512), weights(g, 384, 512), weights(g, 512, 384)

    def mlp(x):
        q, s, _ = dfk.dfk_add_rmsnorm_fp8_block(x, None, torch.ones_like(x[0]), 1e-5)
        q, s = dfk.dfk_swiglu_gate_up_fp8_block(q, s, *wg, *wu)
        return dfk.dfk_gemm_fp8_block(q, s, *wd)

    clean = mlp(x)
    x[1, 77] = float("nan")
    y = mlp(x)
    assert torch.isnan(y[1].float()).all()
    keep = torch.arange(M, device="cuda") != 1
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("M", [1, 16, 64, 100, 256, 700])
def test_same_bits_every_time(M):
    g = gen(M)
    q_x, s_x = activations(g, M, 2048)
    wg, wu = weights(g, 1024, 2048), weights(g, 1024, 2048)
    first = dfk.dfk_swiglu_gate_up_fp8_block(q_x, s_x, *wg, *wu)
    y0 = dfk.dfk_gemm_fp8_block(q_x, s_x, *wg)
    for _ in range(5):
        q, s = dfk.dfk_swiglu_gate_up_fp8_block(q_x, s_x, *wg, *wu)
        assert torch.equal(q.view(torch.uint8), first[0].view(torch.uint8))
        assert torch.equal(s, first[1])
        assert torch.equal(dfk.dfk_gemm_fp8_block(q_x, s_x, *wg), y0)


# ---- together, as a model's layer runs them

class Layer:
    """x -> norm of x + residual -> gate/up -> down, every intermediate in 8 bits."""

    def __init__(self, g, D, F):
        self.gamma = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).bfloat16()
        self.wg, self.wu, self.wd = weights(g, F, D), weights(g, F, D), weights(g, D, F)

    def __call__(self, x, res, stream=None):
        q, s, r = dfk.dfk_add_rmsnorm_fp8_block(x, res, self.gamma, 1e-5, stream=stream)
        qh, sh = dfk.dfk_swiglu_gate_up_fp8_block(q, s, *self.wg, *self.wu, stream=stream)
        return q, s, r, qh, sh, dfk.dfk_gemm_fp8_block(qh, sh, *self.wd, stream=stream)


@pytest.mark.parametrize("M", [1, 7, 64, 150, 600])
@pytest.mark.parametrize("D,F", [(256, 688), (1024, 3584)])
def test_layer(M, D, F):
    g = gen(M + D)
    layer = Layer(g, D, F)
    x, res = rand_bf16(g, M, D), rand_bf16(g, M, D)
    q, s, r, qh, sh, y = layer(x, res)
    d = r.double()
    v = d / (d.square().mean(1, keepdim=True) + 1e-5).sqrt() * layer.gamma.double()
    check_quantised(q, s, v, 2.0 ** -18 * v.abs())
    h, eh = silu_mul(*product(q, s, *layer.wg), *product(q, s, *layer.wu))
    check_quantised(qh, sh, h, eh)
    ref, err = product(qh, sh, *layer.wd)
    check_rounded(y, ref, err, 2.0 ** -8)


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("M", [1, 40, 300])
def test_layer_in_a_graph_and_on_two_streams(M):
    g = gen(M)
    layers = [Layer(g, 512, 1024) for _ in range(2)]
    xs = [(rand_bf16(g, M, 512), rand_bf16(g, M, 512)) for _ in range(2)]
    want = [l(*x) for l, x in zip(layers, xs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):          # both streams at once
        got = [l(*x, stream=st) for l, x, st in zip(layers, xs, streams)]
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, want))
    graphs, outs = [], []
    for l, x, st in zip(layers, xs, streams):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            outs.append(l(*x))
        graphs.append(gr)
    for _ in range(5):           # two captured graphs in flight at the same time
        for o in outs:
            for t in o:
                t.view(torch.uint8).fill_(7)
        torch.cuda.synchronize()
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(outs, want))
    for x, _ in xs:              # new inputs in the same buffers
        x.copy_(rand_bf16(g, M, 512))
    for gr in graphs:
        gr.replay()
    torch.cuda.synchronize()
    assert all(same(o, l(*x)) for o, l, x in zip(outs, layers, xs))


@pytest.mark.parametrize("M", [1, 16, 50, 200])
def test_a_chain_of_calls_in_the_same_buffers(M):
    """Every call rewrites what the call before the last one read, a hundred times over."""
    g = gen(M)
    n = 512
    w = [weights(g, n, n) for _ in range(3)]
    gamma = (1 + 0.1 * torch.randn(n, generator=g, device="cuda")).bfloat16()
    x0 = rand_bf16(g, M, n)

    def chain(fixed):
        x, res = x0.clone(), x0.clone()
        torch.cuda.synchronize()
        q = s = qh = sh = y = None
        if fixed:
            q, qh = (torch.empty(M, n, dtype=E4M3, device="cuda") for _ in range(2))
            s, sh = (torch.empty(4, M, device="cuda") for _ in range(2))
            y = x
        for i in range(100):
            a = dfk.dfk_add_rmsnorm_fp8_block(x, res, gamma, 1e-5, residual_out=res, q=q, s=s)
            if not fixed:
                torch.cuda.synchronize()
            b = dfk.dfk_swiglu_gate_up_fp8_block(a[0], a[1], *w[0], *w[1], q_h=qh, s_h=sh)
            if not fixed:
                torch.cuda.synchronize()
            x = dfk.dfk_gemm_fp8_block(*b, *w[2], y=y)
            if not fixed:
                torch.cuda.synchronize()
            c = dfk.dfk_quant_fp8_block(x, q=q, s=s)
            if not fixed:
                torch.cuda.synchronize()
            x = dfk.dfk_gemm_fp8_block(*c, *w[2], y=y)
            if not fixed:
                torch.cuda.synchronize()
        return x, res

    want = chain(False)
    assert torch.isfinite(want[1].float()).all()
    assert same(chain(True), want)


@pytest.mark.parametrize("B", [4, 100])
def test_decode_stack_in_block_scaled_fp8(B):
    from swiglu_mlp_dfk_b200.stack import DecodeStack
    x0, params = I.make_stack(3, B, 512, 1040, seed=B, w_std=0.05)
    st, ref = (DecodeStack(params, x0, fp8="block") for _ in range(2))
    st.step()
    ref.step_eager()
    st.capture()
    for _ in range(3):
        st.step()
        ref.step_eager()
        torch.cuda.synchronize()
        assert torch.equal(st.x, ref.x)
    for l in range(3):                     # one layer at a time, on its own input
        x = ref.layer_input(l).clone()
        with torch.cuda.stream(ref.stream):
            ref._layer(l)
        torch.cuda.synchronize()
        gamma, qg, sg, qu, su, qd, sd = ref.layers[l]
        d = x.double()
        v = d / (d.square().mean(1, keepdim=True) + ref.eps).sqrt() * gamma.double()
        check_quantised(*ref.xn, v, 2.0 ** -18 * v.abs())
        h, eh = silu_mul(*product(*ref.xn, qg, sg), *product(*ref.xn, qu, su))
        check_quantised(*ref.h, h, eh)
        check_rounded(ref.acts[l % 2], *product(*ref.h, qd, sd), 2.0 ** -8)
    with pytest.raises(ValueError):
        st.tune_variants()
    with pytest.raises(ValueError):
        DecodeStack(params, x0, fp8="rows")
    assert st.kernels_per_step() == 10 and st.bytes_per_step() > 3 * 3 * 512 * 1040


@pytest.mark.parametrize("given,meant", [(None, False), (0, False), (1, True), ("", False)])
def test_decode_stack_takes_any_truth_value(given, meant):
    from swiglu_mlp_dfk_b200.stack import DecodeStack
    x0, params = I.make_stack(1, 2, 256, 272, seed=1, w_std=0.05)
    a, b = DecodeStack(params, x0, fp8=given), DecodeStack(params, x0, fp8=meant)
    a.step()
    b.step()
    torch.cuda.synchronize()
    assert torch.equal(a.x, b.x) and a.kernels_per_step() == b.kernels_per_step()


def test_large_offsets():
    """Outputs whose offsets pass 32 bits: 70,000 tokens x 32,000 columns of bf16 (4.5 GB)."""
    M, K, N = 70000, 128, 32000
    g = gen(1)
    q_x, s_x = activations(g, M, K)
    q_w, s_w = weights(g, N, K)
    y = dfk.dfk_gemm_fp8_block(q_x, s_x, q_w, s_w)
    for lo in (0, 33554, 67100, M - 64):
        a, b = q_x[lo:lo + 64].contiguous(), s_x[:, lo:lo + 64].contiguous()
        ref, err = product(a, b, q_w, s_w)
        check_rounded(y[lo:lo + 64], ref, err, 2.0 ** -8)


def test_a_given_stream_in_a_capture_and_as_a_handle():
    g = gen(4)
    layer, x, res = Layer(g, 256, 512), rand_bf16(g, 9, 256), rand_bf16(g, 9, 256)
    want = layer(x, res)
    torch.cuda.synchronize()
    assert same(layer(x, res, stream=0), want)                    # the legacy default stream
    st = torch.cuda.Stream()
    got = layer(x, res, stream=st.cuda_stream)
    st.synchronize()
    assert same(got, want)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=st):
        out = layer(x, res, stream=st)
    for t in out:
        t.view(torch.uint8).fill_(3)
    torch.cuda.synchronize()
    gr.replay()
    torch.cuda.synchronize()
    assert same(out, want)


FIRST = r'''
import os, sys
sys.path.insert(0, os.environ["DFK_ROOT"])
sys.path.insert(0, os.path.join(os.environ["DFK_ROOT"], "tests"))
import torch
import swiglu_mlp_dfk_b200 as dfk
import test_gpu_fp8_block as t
g = t.gen(1)
layer, x, res = t.Layer(g, 512, 1024), t.rand_bf16(g, 300, 512), t.rand_bf16(g, 300, 512)
torch.cuda.synchronize()
gr = torch.cuda.CUDAGraph()
with torch.cuda.graph(gr):
    out = layer(x, res)
gr.replay()
torch.cuda.synchronize()
assert t.same(out, layer(x, res))
print("first call in a capture ok")
'''


def test_the_first_call_may_be_captured():
    r = subprocess.run([sys.executable, "-c", FIRST], env=dict(os.environ, DFK_ROOT=ROOT),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "capture ok" in r.stdout, r.stdout + r.stderr


def test_no_tokens():
    e = torch.empty(0, 256, device="cuda", dtype=torch.bfloat16)
    q, s = dfk.dfk_quant_fp8_block(e)
    assert q.shape == (0, 256) and s.shape == (2, 0)
    w = weights(gen(0), 64, 256)
    assert dfk.dfk_gemm_fp8_block(q, s, *w).shape == (0, 64)
    assert dfk.dfk_swiglu_gate_up_fp8_block(q, s, *w, *w)[0].shape == (0, 64)


def test_binding_refusals():
    g = gen(0)
    q, s = activations(g, 4, 256)
    qw, sw = weights(g, 128, 256)
    ok = dfk.dfk_gemm_fp8_block(q, s, qw, sw)
    for args, kw in (((q, s.t(), qw, sw), {}), ((q, s, qw.t(), sw), {}),
                     ((q, s, qw, sw[:, :1]), {}), ((q.float(), s, qw, sw), {}),
                     ((q, s.double(), qw, sw), {}), ((q, s, qw, sw), {"y": ok[:3]}),
                     ((q, s, qw, sw), {"y": ok.float()}), ((q[0], s, qw, sw), {}),
                     ((q, s, qw, sw.cpu()), {}), ((q, s, None, sw), {})):
        with pytest.raises(dfk.DfkError) as e:
            dfk.dfk_gemm_fp8_block(*args, **kw)
        assert e.value.status == dfk.DFK_ERR_INVALID_ARG
    x = torch.zeros(4, 200, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(dfk.DfkError) as e:
        dfk.dfk_quant_fp8_block(x)            # 200 % 16
    assert e.value.status == dfk.DFK_ERR_UNSUPPORTED_SHAPE
    with pytest.raises(dfk.DfkError):
        dfk.dfk_quant_fp8_block(torch.zeros(8, 64, device="cuda", dtype=torch.bfloat16).t())
    with pytest.raises(dfk.DfkError):
        dfk.dfk_swiglu_gate_up_fp8_block(q, s, qw, sw, qw, sw, h=ok)
    with pytest.raises(dfk.DfkError):
        dfk.dfk_swiglu_gate_up_fp8_block(q, s, qw, sw, qw, sw, fp8_out=False, q_h=q)


def test_sizes_beyond_a_c_int_are_refused():
    # 2^32 + 16 would arrive as 16
    x = torch.empty(1, 2 ** 32 + 16, device="cuda", dtype=torch.uint8)
    s = torch.empty(2 ** 25 + 1, 1, device="cuda")
    sw = torch.empty(1, 2 ** 25 + 1, device="cuda")
    for call in (lambda: dfk.dfk_gemm_fp8_block(x, s, x, sw),
                 lambda: dfk.dfk_swiglu_gate_up_fp8_block(x, s, x, sw, x, sw),
                 lambda: dfk.dfk_quant_fp8_block(torch.empty(1, 2 ** 32 + 16, device="cuda",
                                                             dtype=torch.bfloat16))):
        with pytest.raises(dfk.DfkError) as e:
            call()
        assert e.value.status == dfk.DFK_ERR_UNSUPPORTED_SHAPE


def every_call(q, s, w, x, gamma):
    """One call of each kind: with new outputs, given ones, bf16 and codes, no tokens."""
    u8 = torch.uint8
    M, K = x.shape
    N = w[0][0].shape[0]
    yield dfk.dfk_quant_fp8_block(x)
    qo, so = torch.empty(M, K, device="cuda", dtype=u8), torch.empty(-(-K // 128), M, device="cuda")
    out = dfk.dfk_quant_fp8_block(x, q=qo, s=so)
    assert out[0] is qo and out[1] is so
    yield out
    yield dfk.dfk_quant_fp8_block(x[:0])
    yield dfk.dfk_add_rmsnorm_fp8_block(x, None, gamma, 1e-5)
    yield dfk.dfk_add_rmsnorm_fp8_block(x, x, gamma, 0)
    r = x.clone()
    out = dfk.dfk_add_rmsnorm_fp8_block(x, r, gamma, 1e-5, residual_out=r)
    assert out[2] is r
    yield out
    yield (dfk.dfk_gemm_fp8_block(q, s, *w[0]),)
    yield (dfk.dfk_gemm_fp8_block(q.view(u8), s, w[0][0].view(u8), w[0][1]),)
    y = torch.empty(M, N, device="cuda", dtype=torch.bfloat16)
    assert dfk.dfk_gemm_fp8_block(q, s, *w[0], y=y) is y
    yield (y,)
    yield dfk.dfk_swiglu_gate_up_fp8_block(q, s, *w[0], *w[1])
    yield (dfk.dfk_swiglu_gate_up_fp8_block(q, s, *w[0], *w[1], fp8_out=False),)
    qh, sh = torch.empty(M, N, device="cuda", dtype=u8), torch.empty(-(-N // 128), M, device="cuda")
    out = dfk.dfk_swiglu_gate_up_fp8_block(q, s, *w[0], *w[1], q_h=qh, s_h=sh)
    assert out[0] is qh and out[1] is sh
    yield out


@pytest.mark.parametrize("M", [1, 5, 70])
def test_both_host_paths_make_the_same_calls(M, monkeypatch):
    dfk.lib()
    assert dfk._fast is not None
    g = gen(M)
    q, s = activations(g, M, 272)
    w = weights(g, 400, 272), weights(g, 400, 272)
    x = torch.randn(M, 272, device="cuda", dtype=torch.bfloat16)
    gamma = torch.rand(272, device="cuda").bfloat16()

    def run():
        return [tuple(t if t is None else t.clone() for t in out)
                for out in every_call(q, s, w, x, gamma)]
    fast = run()
    with torch.inference_mode():
        inside = run()
    monkeypatch.setattr(dfk, "_fast", None)
    plain = run()
    for a, b, c in zip(fast, plain, inside):
        assert len(a) == len(b) == len(c)
        for t, u, v in zip(a, b, c):
            assert (t is None) == (u is None) == (v is None)
            if t is not None:
                assert t.dtype == u.dtype and t.shape == u.shape and t.stride() == u.stride()
                assert t.numel() == 0 or (torch.equal(t.view(torch.uint8), u.view(torch.uint8))
                                          and torch.equal(t.view(torch.uint8), v.view(torch.uint8)))


def test_fast_calls_leave_the_unusual_to_the_binding():
    g = gen(3)
    q, s = activations(g, 4, 256)
    qw, sw = weights(g, 128, 256)
    x = torch.randn(4, 256, device="cuda", dtype=torch.bfloat16)
    gamma = torch.ones(256, device="cuda", dtype=torch.bfloat16)
    dfk.lib()
    f = dfk._fast
    y = f.gemm(q, s, qw, sw, None)
    assert torch.equal(y, dfk.dfk_gemm_fp8_block(q, s, qw, sw))
    for args in ((q.cpu(), s, qw, sw, None), (q, s.t(), qw, sw, None), (q, s, qw.t(), sw, None),
                 (q, s, qw, sw[:, :1], None), (q, s, qw, sw, y[:3]), (q, s, qw, sw, y.float()),
                 (q.float(), s, qw, sw, None), (q[0], s, qw, sw, None), (q, s, qw, sw),
                 (q, s, None, sw, None), (q, s.double(), qw, sw, None), (q, s, qw, 1.0, None)):
        assert f.gemm(*args) is None
    for args in ((x.float(), None, None), (x.t(), None, None), (x[:, :200].contiguous(), None, None),
                 (x, q[:2], None), (x, None, s.t()), (x, x, None), (x.cpu(), None, None)):
        assert f.quant(*args) is None
    for args in ((x, x, gamma[:128], 1e-5, None, None, None), (x, x[:2], gamma, 1e-5, None, None, None),
                 (x, None, gamma, 1e-5, x, None, None), (x, x, gamma, 1, None, None, None),
                 (x, x, gamma, -1.0, None, None, None), (x, x, x, 1e-5, None, None, None)):
        assert f.norm(*args) is None
    for args in ((q, s, qw, sw, qw[:64], sw, True, None, None, None),
                 (q, s, qw, sw, qw, sw, True, y, None, None), (q, s, qw, sw, qw, sw, 1, None, None, None),
                 (q, s, qw, sw, qw, sw, False, None, q, None)):
        assert f.gate_up(*args) is None


def test_calls_from_several_threads():
    import threading
    g = gen(9)
    q, s = activations(g, 33, 512)
    w = weights(g, 384, 512)
    want = dfk.dfk_gemm_fp8_block(q, s, *w)
    torch.cuda.synchronize()
    wrong = []

    def work():
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(200):
                y = dfk.dfk_gemm_fp8_block(q, s, *w)
            torch.cuda.current_stream().synchronize()
            if not torch.equal(y, want):
                wrong.append(1)
    ts = [threading.Thread(target=work) for _ in range(4)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not wrong


CHILD = r'''
import os, sys
sys.path.insert(0, os.environ["DFK_ROOT"])
sys.path.insert(0, os.path.join(os.environ["DFK_ROOT"], "tests"))
import swiglu_mlp_dfk_b200 as dfk
assert dfk.LIB_PATH.endswith("libdfk_checked.so")
import test_gpu_fp8_block as t
for M, K in ((1, 16), (5, 2064), (130, 256)):
    t.test_quant(M, K)
for M, D in ((3, 688), (2, 16400)):
    t.test_add_rmsnorm(M, D, True)
for M, K, N in ((1, 16, 1), (3, 2064, 1001), (33, 272, 96), (129, 1152, 640), (257, 384, 520)):
    t.test_gemm(M, K, N)
    t.test_gate_up(M, K, N, True)
    t.test_gate_up(M, K, N, False)
t.test_forms_for_many_tokens(1100, 400, 5001, "gemm")
t.test_forms_for_many_tokens(150, 4112, 2048, "fp8")
t.test_forms_for_many_tokens(700, 656, 3002, "gemm")
t.test_forms_for_many_tokens(330, 144, 12296, "bf16")
st = dfk.dfk_device_status()
assert st[0] == 0, st
print("checked ok")
'''


def test_checked_build():
    env = dict(os.environ, DFK_CHECKED="1", DFK_ROOT=ROOT)
    r = subprocess.run([sys.executable, "-c", CHILD], env=env, capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0 and "checked ok" in r.stdout, r.stdout + r.stderr


CHILD_FORMS = r'''
import os, sys
sys.path.insert(0, os.environ["DFK_ROOT"])
sys.path.insert(0, os.path.join(os.environ["DFK_ROOT"], "tests"))
import swiglu_mlp_dfk_b200 as dfk
assert dfk.LIB_PATH.endswith("libdfk_checked.so")
import test_gpu_fp8_block as t
for op, listed in (("gemm", t.forms.PLAIN), ("fp8", t.forms.GATED), ("bf16", t.forms.GATED)):
    for sizes, form in listed:
        t.check_form(op, sizes, form)
t.test_add_rmsnorm(1100, 1040, True)
st = dfk.dfk_device_status()
assert st[0] == 0, st
print("checked ok")
'''


def test_checked_build_in_every_form():
    env = dict(os.environ, DFK_CHECKED="1", DFK_ROOT=ROOT)
    r = subprocess.run([sys.executable, "-c", CHILD_FORMS], env=env, capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0 and "checked ok" in r.stdout, r.stdout + r.stderr
