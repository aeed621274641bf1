"""Refusals of the MXFP4 calls and of the few-token layer: argument errors are
found on the host before anything is enqueued (no GPU needed)."""
import ctypes
import os

import pytest
import torch

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def B():
    from sparse_mixture_experts_renormalised_amd import binding
    if not os.path.exists(binding.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    binding.lib()
    return binding


def quant(B, dtype=1, rows=4, d=64, x=4096, stride=64, codes=4096, scales=4096, wide=None):
    return B.lib().moe_quantize_mxfp4(dtype, rows, d, P(x), stride, P(codes), P(scales), P(wide), None)


def test_quantize_refusals(B):
    assert quant(B, rows=0, x=None) == 0                        # nothing to do
    for bad in ({"dtype": 2}, {"rows": -1}, {"d": 0}, {"d": -32}, {"x": None}, {"codes": None},
                {"scales": None}, {"x": 4104}, {"codes": 4104}, {"scales": 4100}, {"wide": 4104},
                {"stride": 63}, {"stride": 68}, {"dtype": 0, "stride": 66}, {"stride": -64}):
        assert quant(B, **bad) == -1, bad
    for bad in ({"d": 16}, {"d": 100, "stride": 104}, {"rows": 1 << 50}):
        assert quant(B, **bad) == -2, bad


def linear(B, g=3, n=64, k=128, xr=8, xc=4096, xs=4096, idx=None, off=4096, rows=8, wc=4096, ws_=4096,
           bias=None, silu=0, y=4096, ws=None, nbytes=0):
    return B.lib().moe_grouped_linear_mxfp4(g, n, k, xr, P(xc), P(xs), P(idx), P(off), rows, P(wc),
                                            P(ws_), P(bias), silu, P(y), P(ws), nbytes, None)


def test_linear_refusals(B):
    assert linear(B, rows=0, xc=None, y=None) == 0
    for bad in ({"g": 0}, {"n": 0}, {"k": 0}, {"rows": -1}, {"silu": 2}, {"xc": None}, {"xs": None},
                {"off": None}, {"wc": None}, {"ws_": None}, {"y": None}, {"xc": 4104}, {"xs": 4100},
                {"idx": 4100}, {"off": 4100}, {"wc": 4104}, {"ws_": 4100}, {"bias": 4104}, {"y": 4104},
                {"ws": 4100, "nbytes": 1 << 40}, {"xr": -1}, {"xr": 7}, {"xr": 0, "idx": 4096}):
        assert linear(B, **bad) == -1, bad
    for bad in ({"n": 60}, {"k": 64}, {"k": 192}, {"g": 1089}, {"rows": 1 << 31, "xr": 1 << 31},
                {"xr": 1 << 26}, {"k": 1 << 20, "n": 1 << 13}):
        assert linear(B, **bad) == -2, bad
    need = B.grouped_linear_mxfp4_workspace_size(3, 64, 128, 8)
    if need:
        assert linear(B, ws=4096, nbytes=need - 1) == -3
    assert B.grouped_linear_mxfp4_workspace_size(3, 64, 100, 8) == 0


def few(B, cfg, w, x=4096, y=4096, ws=4096, nbytes=1 << 40, idx=None, gate=None, counts=None, mx=False):
    fn = B.lib().moe_layer_forward_few_mxfp4 if mx else B.lib().moe_layer_forward_few
    return fn(ctypes.byref(cfg), ctypes.byref(w), P(x), P(y), P(idx), P(gate), P(counts), P(ws),
              nbytes, None)


def test_few_refusals(B):
    good = B.config(4, 128, 8, 2, 1, 256, "bf16")
    w = B.Weights(w_router=4096, w1=4096, w2=4096, ws1=4096, ws2=4096)
    need = B.few_workspace_size(good)
    assert need > 0
    assert few(B, B.config(0, 128, 8, 2, 1, 256, "bf16"), B.Weights(), x=None, y=None, ws=None) == 0
    assert few(B, good, w, nbytes=need - 1) == -3 and few(B, good, w, ws=None) == -3
    for bad in ({"x": None}, {"y": None}, {"x": 4104}, {"y": 4104}, {"ws": 4100}, {"idx": 4100},
                {"gate": 4100}, {"counts": 4100}):
        assert few(B, good, w, **bad) == -1, bad
    for field in ("w_router", "w1", "w2", "ws1", "ws2"):
        w2 = B.Weights(w_router=4096, w1=4096, w2=4096, ws1=4096, ws2=4096)
        setattr(w2, field, None)
        assert few(B, good, w2) == -1, field
    for field in ("w_router", "router_bias", "w1", "b1", "w2", "b2", "ws1", "bs1", "ws2", "bs2"):
        w2 = B.Weights(w_router=4096, w1=4096, w2=4096, ws1=4096, ws2=4096)
        setattr(w2, field, 4104)
        assert few(B, good, w2) == -1, field
    for cfg, want in [(B.config(17, 128, 8, 2, 1, 256, "bf16"), -2),
                      (B.config(4, 128, 8, 2, 1, 256, "bf16", dispatch_fp8=True), -2),
                      (B.config(4, 96, 8, 2, 1, 256, "bf16"), -2),
                      (B.config(4, 128, 8, 9, 1, 256, "bf16"), -1),
                      (B.config(4, 128, 2048, 2, 1, 256, "bf16"), -2),
                      (B.config(-1, 128, 8, 2, 1, 256, "bf16"), -1)]:
        assert few(B, cfg, w) == want
        assert B.few_workspace_size(cfg) == 0


def test_few_mxfp4_refusals(B):
    good = B.config(4, 128, 8, 2, 1, 256, "bf16")
    names = ("w_router", "w1", "w1_scales", "w2", "w2_scales", "ws1", "ws1_scales", "ws2", "ws2_scales")

    def table(**over):
        return B.WeightsMxfp4(**({n: 4096 for n in names} | over))

    assert few(B, good, table(), ws=None, mx=True) == -3
    for n in names:
        assert few(B, good, table(**{n: None}), mx=True) == -1, n
        assert few(B, good, table(**{n: 4100}), mx=True) == -1, n
    for n in ("router_bias", "b1", "b2", "bs1", "bs2"):
        assert few(B, good, table(**{n: 4104}), mx=True) == -1, n
    for cfg in (B.config(4, 128, 8, 2, 1, 256, "f32"), B.config(4, 192, 8, 2, 1, 256, "bf16"),
                B.config(4, 128, 8, 2, 1, 320, "bf16"), B.config(17, 128, 8, 2, 1, 256, "bf16")):
        assert few(B, cfg, table(), mx=True) == -2


def test_the_binding_refuses_what_is_not_on_the_gpu(B):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    c, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        B.quantize_mxfp4(x, c, s)
    with pytest.raises(ValueError, match="GPU"):
        B.grouped_linear_mxfp4(c, s, torch.zeros(2, dtype=torch.int32), c[None], s[None], x)
    with pytest.raises(ValueError, match="GPU"):
        B.layer_forward_few(B.config(4, 64, 8, 2, 0, 64, "bf16"), B.Weights(), x, x)
