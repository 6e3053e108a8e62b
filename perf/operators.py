"""Cases for the block-scaled FP8 operators: quantisation of activations, RMSNorm with the
residual's addition, the gated gate/up product and the plain product.

Shared by all four: E4M3 codes with one fp32 scale per token and group of 128 along the
reduction for activations (scales [groups][tokens]), one per 128 x 128 block for weights.

    quant:    a = max |v| of the group, s = max(a / 448, 2^-126), q = E4M3(v / s)
    norm:     r = bf16(x + residual), v = r / sqrt(mean r^2 + eps) * gamma, then as quant
    gemm:     y = sum over groups of s_x s_w (q_x . q_w), rounded to bf16
    gate_up:  h = SiLU(gate) * up of two such products, quantised along d_ff or rounded to bf16

``own`` False: elementary torch operations in 32 bits.  True: the framework's calls.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
EPS = 1e-5
TINY = 2.0 ** -126


def listed():
    return [
        # one decoded token: attention's output on its way to the output projection
        {"name": "quant_token", "op": "quant", "M": 1, "K": 4096},
        # a long prompt's bf16 MLP activations
        {"name": "quant_prompt", "op": "quant", "M": 2047, "K": 14336},
        # the norm in front of the MLP at one decoded token, and over a prompt of the wide model
        {"name": "norm_token", "op": "norm", "M": 1, "K": 4096},
        {"name": "norm_prompt", "op": "norm", "M": 4096, "K": 8192},
        # the 4096 / 14336 layer's gate and up projections: one token, a full decode batch, a prompt
        {"name": "gate_up_token", "op": "gate_up", "M": 1, "K": 4096, "N": 14336, "fp8_out": True},
        {"name": "gate_up_batch", "op": "gate_up", "M": 64, "K": 4096, "N": 14336, "fp8_out": True},
        {"name": "gate_up_prompt", "op": "gate_up", "M": 4096, "K": 4096, "N": 14336, "fp8_out": True},
        # the tiny layer (a last group of 48) over a short prompt, h kept in bf16
        {"name": "gate_up_tiny", "op": "gate_up", "M": 333, "K": 256, "N": 688, "fp8_out": False},
        # the same layer's down projection at one token and over a prompt
        {"name": "down_token", "op": "gemm", "M": 1, "K": 14336, "N": 4096},
        {"name": "down_prompt", "op": "gemm", "M": 4096, "K": 14336, "N": 4096},
        # the packed QKV projection at a small decode batch
        {"name": "qkv_batch", "op": "gemm", "M": 16, "K": 4096, "N": 6144},
        # odd everything: tokens, output columns, a last group of 16
        {"name": "gemm_odd", "op": "gemm", "M": 777, "K": 2064, "N": 1001},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "norm", "gate_up", "gemm"])
    while True:
        case = {"op": op, "M": _spread(rng, 1, 8192), "K": 16 * _spread(rng, 8, 1024)}
        if op in ("gate_up", "gemm"):
            case["N"] = _spread(rng, 64, 16384)
            if op == "gate_up":
                case["fp8_out"] = rng.random() < 0.7
                if case["fp8_out"]:
                    case["N"] = -(-case["N"] // 16) * 16
            cost = case["M"] * case["K"] * case["N"] * (2 if op == "gate_up" else 1)
            if cost > 2 * 4096 * 4096 * 14336:
                continue
        elif case["M"] * case["K"] > 4096 * 8192:
            continue
        return case


# ---- inputs

def _groups(K):
    return -(-K // 128)


def _activations(g, M, K):
    """bf16 activations: normal noise, a few channels an order of magnitude larger (as hidden
    states have), a spread of token magnitudes."""
    x = torch.randn(M, K, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(M, 1, generator=g, device="cuda"))
    big = torch.rand(K, generator=g, device="cuda") < 0.01
    return (x * torch.where(big, 10.0, 1.0)).bfloat16()


def _codes(g, M, K):
    """8-bit activations with their scales, made from bf16 ones."""
    x = torch.nn.functional.pad(_activations(g, M, K).float(), (0, _groups(K) * 128 - K))
    x = x.view(M, _groups(K), 128)
    s = (x.abs().amax(2) / 448).clamp(min=TINY)
    q = (x / s[:, :, None]).clamp(-448, 448).to(E4M3).view(M, -1)[:, :K].contiguous()
    return q, s.t().contiguous()


def _weights(g, N, K):
    """Weights N(0, 0.02) as E4M3 codes with one scale per 128 x 128 block."""
    w = 0.02 * torch.randn(N, K, generator=g, device="cuda")
    w = torch.nn.functional.pad(w, (0, _groups(K) * 128 - K, 0, _groups(N) * 128 - N))
    w = w.view(_groups(N), 128, _groups(K), 128)
    s = w.abs().amax((1, 3)) / 448
    q = (w / s[:, None, :, None]).clamp(-448, 448).to(E4M3).view(_groups(N) * 128, -1)
    return q[:N, :K].contiguous(), s.contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    M, K = case["M"], case["K"]
    st = dict(case)
    if case["op"] in ("quant", "norm"):
        st["x"] = _activations(g, M, K)
        if case["op"] == "norm":
            st["residual"] = _activations(g, M, K)
            st["gamma"] = (1 + 0.1 * torch.randn(K, generator=g, device="cuda")).bfloat16()
    else:
        st["q_x"], st["s_x"] = _codes(g, M, K)
        st["w"] = [_weights(g, case["N"], K) for _ in range(2 if case["op"] == "gate_up" else 1)]
    return st


# ---- plain forms

def _plain_quant(v):
    M, K = v.shape
    G = _groups(K)
    v = torch.nn.functional.pad(v, (0, G * 128 - K)).view(M, G, 128)
    s = (v.abs().amax(2) / 448).clamp(min=TINY)
    q = (v / s[:, :, None]).clamp(-448, 448).to(E4M3).view(M, G * 128)[:, :K]
    return q.contiguous(), s.t().contiguous()


def _plain_product(q_x, s_x, q_w, s_w):
    K, N = q_x.shape[1], q_w.shape[0]
    x = q_x.float() * s_x.t().repeat_interleave(128, 1)[:, :K]
    w = q_w.float() * s_w.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return x @ w.t()


def _plain(st):
    if st["op"] == "quant":
        return _plain_quant(st["x"].float())
    if st["op"] == "norm":
        r = (st["x"].float() + st["residual"].float()).bfloat16()
        f = r.float()
        v = f / torch.sqrt((f * f).mean(1, keepdim=True) + EPS) * st["gamma"].float()
        return (*_plain_quant(v), r)
    a = _plain_product(st["q_x"], st["s_x"], *st["w"][0])
    if st["op"] == "gemm":
        return a.bfloat16()
    h = a / (1 + torch.exp(-a)) * _plain_product(st["q_x"], st["s_x"], *st["w"][1])
    return _plain_quant(h) if st["fp8_out"] else h.bfloat16()


def run(st):
    if not own:
        return _plain(st)
    import swiglu_mlp_dfk_b200 as dfk
    if st["op"] == "quant":
        return dfk.dfk_quant_fp8_block(st["x"])
    if st["op"] == "norm":
        return dfk.dfk_add_rmsnorm_fp8_block(st["x"], st["residual"], st["gamma"], EPS)
    if st["op"] == "gemm":
        return dfk.dfk_gemm_fp8_block(st["q_x"], st["s_x"], *st["w"][0])
    return dfk.dfk_swiglu_gate_up_fp8_block(st["q_x"], st["s_x"], *st["w"][0], *st["w"][1],
                                            fp8_out=st["fp8_out"])


def work(case):
    M, K = case["M"], case["K"]
    scales = 4 * M * _groups(K)
    if case["op"] == "quant":
        return {"bytes": 3 * M * K + scales, "flops": 3 * M * K}
    if case["op"] == "norm":
        return {"bytes": 7 * M * K + 2 * K + scales, "flops": 8 * M * K}
    N, mats = case["N"], 2 if case["op"] == "gate_up" else 1
    out = M * N + 4 * M * _groups(N) if case.get("fp8_out") else 2 * M * N
    weights = mats * (N * K + 4 * _groups(N) * _groups(K))
    return {"bytes": M * K + scales + weights + out, "flops": 2 * mats * M * N * K}


# ---- the definitions in 64 bits

def _e4m3_nearest(u):
    """u rounded to the nearest E4M3 value (4 significant bits, smallest step 2^-9), half to even."""
    e = torch.frexp(u)[1].clamp(min=-5) - 4
    return torch.ldexp(torch.round(torch.ldexp(u, -e)), e).clamp(-448, 448)


def _exact_quant(v):
    M, K = v.shape
    of = torch.arange(K, device=v.device) // 128
    top = torch.zeros(M, _groups(K), dtype=torch.float64, device=v.device)
    top = top.scatter_reduce(1, of.expand(M, K), v.abs(), "amax")
    s = torch.clamp(top / 448, min=TINY)
    return _e4m3_nearest(v / s[:, of]), s.t()


def _exact_product(q_x, s_x, q_w, s_w):
    n = torch.arange(q_w.shape[0], device=q_w.device) // 128
    y = torch.zeros(q_x.shape[0], q_w.shape[0], dtype=torch.float64, device=q_x.device)
    for k in range(s_x.shape[0]):
        part = slice(128 * k, 128 * (k + 1))
        p = q_x[:, part].double() @ q_w[:, part].double().t()
        y += p * s_x[k].double()[:, None] * s_w[n, k].double()[None, :]
    return y


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quant":
        return _exact_quant(st["x"].double())
    if case["op"] == "norm":
        r = (st["x"].double() + st["residual"].double()).bfloat16()  # the stored sum has 16 bits
        d = r.double()
        v = d * torch.rsqrt(d.square().mean(1, keepdim=True) + EPS) * st["gamma"].double()
        return (*_exact_quant(v), r.double())
    a = _exact_product(st["q_x"], st["s_x"], *st["w"][0])
    if case["op"] == "gemm":
        return a
    h = a * torch.sigmoid(a) * _exact_product(st["q_x"], st["s_x"], *st["w"][1])
    return _exact_quant(h) if case["fp8_out"] else h
