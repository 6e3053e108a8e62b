"""Outputs that a call allocates for a given stream.

Memory freed on the current stream may still be written by work queued there, and nothing orders
a given stream after that work: the output must not come from it.  And the caller goes on with the
output on the current stream, so its memory must not go to the given stream's next output before
that use has ended.
"""
import pytest
import torch

import swiglu_mlp_dfk_b200 as dfk
from swiglu_mlp_dfk_b200 import inputs as I

pytestmark = pytest.mark.gpu
B, D, F = 8, 4096, 4096     # outputs of 64 KB and scales of 1 KB
SLEEP = 20_000_000          # cycles, about 10 ms


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


@pytest.fixture(scope="module")
def data():
    g = torch.Generator(device="cuda")
    g.manual_seed(0)

    def rand(*shape, std=1.0):
        return (std * torch.randn(*shape, generator=g, device="cuda")).bfloat16()
    d = {"x": [rand(B, D), rand(B, D)], "gamma": 1 + rand(D, std=0.1), "w": rand(F, D, std=0.02),
         "u": rand(F, D, std=0.02), "h_all": rand(2, 4, 256), "w_all": rand(2, D, 256, std=0.02)}
    d["rows"], d["blocks"] = I.to_fp8_rows(d["w"]), I.to_fp8_blocks(d["w"])
    d["codes"] = [dfk.dfk_quant_fp8_block(x) for x in d["x"]]
    torch.cuda.synchronize()
    return d


CALLS = {
    "swiglu_gate_up": lambda d, i, s: dfk.dfk_swiglu_gate_up(d["x"][i], d["w"], d["u"], stream=s),
    "rmsnorm_swiglu_gate_up": lambda d, i, s: dfk.dfk_rmsnorm_swiglu_gate_up(
        d["x"][i], d["gamma"], 1e-5, d["w"], d["u"], stream=s),
    "down_proj": lambda d, i, s: dfk.dfk_down_proj(d["x"][i], d["w"], stream=s),
    "down_proj_static_scratch": lambda d, i, s: dfk.dfk_down_proj_static_scratch(
        d["x"][i], d["w"], stream=s),
    "swiglu_gate_up_fp8": lambda d, i, s: dfk.dfk_swiglu_gate_up_fp8(
        d["x"][i], *d["rows"], *d["rows"], stream=s),
    "rmsnorm_swiglu_gate_up_fp8": lambda d, i, s: dfk.dfk_rmsnorm_swiglu_gate_up_fp8(
        d["x"][i], d["gamma"], 1e-5, *d["rows"], *d["rows"], stream=s),
    "down_proj_fp8": lambda d, i, s: dfk.dfk_down_proj_fp8(d["x"][i], *d["rows"], stream=s),
    "rmsnorm_qkv_proj": lambda d, i, s: dfk.dfk_rmsnorm_qkv_proj(
        d["x"][i], d["gamma"], 1e-5, d["w"], 2048, 1024, 1024, stream=s),
    "gemv": lambda d, i, s: dfk.dfk_gemv(d["x"][i], d["w"], stream=s),
    "rmsnorm": lambda d, i, s: dfk.dfk_rmsnorm(d["x"][i], d["gamma"], 1e-5, stream=s),
    "rms_rescale": lambda d, i, s: dfk.dfk_rms_rescale(d["x"][i], stream=s),
    "silu": lambda d, i, s: dfk.dfk_silu(d["x"][i], stream=s),
    "mul": lambda d, i, s: dfk.dfk_mul(d["x"][i], d["x"][0], stream=s),
    "quant_fp8_block": lambda d, i, s: dfk.dfk_quant_fp8_block(d["x"][i], stream=s),
    "add_rmsnorm_fp8_block": lambda d, i, s: dfk.dfk_add_rmsnorm_fp8_block(
        d["x"][i], d["x"][0], d["gamma"], 1e-5, stream=s),
    "gemm_fp8_block": lambda d, i, s: dfk.dfk_gemm_fp8_block(
        *d["codes"][i], *d["blocks"], stream=s),
    "swiglu_gate_up_fp8_block": lambda d, i, s: dfk.dfk_swiglu_gate_up_fp8_block(
        *d["codes"][i], *d["blocks"], *d["blocks"], stream=s),
    "swiglu_gate_up_fp8_block bf16": lambda d, i, s: dfk.dfk_swiglu_gate_up_fp8_block(
        *d["codes"][i], *d["blocks"], *d["blocks"], fp8_out=False, stream=s),
}


def outputs(out):
    return [t for t in (out if isinstance(out, tuple) else (out,)) if t is not None]


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("name", CALLS)
def test_the_output_is_not_memory_that_the_current_stream_still_writes(data, name):
    call = CALLS[name]
    want = [t.clone() for t in outputs(call(data, 0, None))]
    side = torch.cuda.Stream()
    outputs(call(data, 0, side))               # decisions and workspaces of this stream
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    for stream in (side, side.cuda_stream):
        doomed = [torch.empty_like(t) for t in want for _ in range(4)]
        torch.cuda._sleep(SLEEP)
        for t in doomed:
            t.view(torch.uint8).fill_(0x5a)
        del doomed, t                          # free for the current stream, which has yet to write
        got = outputs(call(data, 0, stream))
        torch.cuda.synchronize()
        assert same(got, want)


@pytest.mark.parametrize("name", CALLS)
def test_the_output_lives_until_the_current_stream_has_read_it(data, name):
    call = CALLS[name]
    side = torch.cuda.Stream()
    want = [t.clone() for t in outputs(call(data, 0, None))]
    outputs(call(data, 1, side))
    torch.cuda.synchronize()
    got = outputs(call(data, 0, side))
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(SLEEP)
    kept = [t.clone() for t in got]            # queued behind the sleep
    del got
    for _ in range(4):                         # other values, into whatever memory is free there
        again = outputs(call(data, 1, side))
    torch.cuda.synchronize()
    assert same(kept, want) and len(again) == len(want)


def test_the_legacy_default_stream_as_a_handle(data):
    want = [t.clone() for t in outputs(dfk.dfk_quant_fp8_block(data["x"][0]))]
    with torch.cuda.stream(torch.cuda.Stream()):
        got = outputs(dfk.dfk_quant_fp8_block(data["x"][0], stream=0))
    torch.cuda.synchronize()
    assert same(got, want)
    assert dfk._torch_stream(0, got[0].device).cuda_stream == 0


def test_the_emulated_allreduce(data):
    side = torch.cuda.Stream()
    want = dfk.dfk_tp_down_proj_allreduce_emulated(data["h_all"], data["w_all"])
    torch.cuda.synchronize()
    doomed = [torch.empty_like(want) for _ in range(4)]
    torch.cuda._sleep(SLEEP)
    for t in doomed:
        t.fill_(1.0)
    del doomed, t
    got = dfk.dfk_tp_down_proj_allreduce_emulated(data["h_all"], data["w_all"], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
