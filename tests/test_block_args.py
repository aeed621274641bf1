"""Refusals of the calls that train the layer as a block: argument errors are found
on the host before anything is enqueued (no GPU needed)."""
import ctypes
import os

import pytest
import torch

P = ctypes.c_void_p
BIG = 1 << 50


@pytest.fixture(scope="module")
def B():
    from sparse_mixture_experts_renormalised_amd import binding
    if not os.path.exists(binding.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    binding.lib()
    return binding


def linear(B, dt=1, g=3, n=64, k=128, xr=8, x=4096, idx=None, off=4096, rows=8, w=4096, bias=None, silu=0,
           y=4096, pre=None, ws=4096, nbytes=BIG):
    return B.lib().moe_grouped_linear(dt, g, n, k, xr, P(x), P(idx), P(off), rows, P(w), P(bias), silu, P(y),
                                      P(pre), P(ws), nbytes, None)


def input_grad(B, dt=1, g=3, n=64, k=128, dy=4096, off=4096, rows=8, w=4096, pre=None, dx=4096, ws=4096,
               nbytes=BIG):
    return B.lib().moe_grouped_linear_input_grad(dt, g, n, k, P(dy), P(off), rows, P(w), P(pre), P(dx), P(ws),
                                                 nbytes, None)


def weight_grad(B, dt=1, gd=1, g=3, n=64, k=128, dy=4096, xr=8, x=4096, idx=None, off=4096, rows=8, dw=4096,
                db=None, acc=0, ws=4096, nbytes=BIG):
    return B.lib().moe_grouped_linear_weight_grad(dt, gd, g, n, k, P(dy), xr, P(x), P(idx), P(off), rows, P(dw),
                                                  P(db), acc, P(ws), nbytes, None)


SIZES = [({"dt": 2}, -1), ({"g": 0}, -1), ({"n": 0}, -1), ({"k": -64}, -1), ({"rows": -1}, -1),
         ({"g": 1089}, -2), ({"n": 72}, -2), ({"k": 32}, -2), ({"dt": 0, "n": 24, "gd": 0}, -2),
         ({"rows": 1 << 30, "xr": 1 << 30}, -2), ({"off": None}, -1), ({"off": 4100}, -1), ({"ws": 4104}, -1)]


def only(call, kw):
    names = call.__code__.co_varnames[:call.__code__.co_argcount]
    return {a: v for a, v in kw.items() if a in names}


@pytest.mark.parametrize("call", [linear, input_grad, weight_grad])
def test_linear_sizes(B, call):
    for kw, want in SIZES:
        assert call(B, **only(call, kw)) == want, kw
    need = B.grouped_linear_workspace_size("bf16", 3, 64, 128, 8)
    if need:
        assert call(B, nbytes=need - 1) == -3 and call(B, ws=None) == -3


def test_linear_refusals(B):
    assert linear(B, rows=0, x=None, y=None) == 0
    for bad in ({"x": None}, {"w": None}, {"y": None}, {"x": 4104}, {"idx": 4100}, {"w": 4104}, {"bias": 4104},
                {"y": 4104}, {"silu": 1, "pre": 4104}, {"silu": 2}, {"pre": 4096}, {"xr": 7}, {"xr": -1},
                {"xr": 0, "idx": 4096}):
        assert linear(B, **bad) == -1, bad
    assert input_grad(B, rows=0, dy=None, dx=None) == 0
    for bad in ({"dy": None}, {"w": None}, {"dx": None}, {"dy": 4104}, {"w": 4104}, {"pre": 4104}, {"dx": 4104}):
        assert input_grad(B, **bad) == -1, bad
    assert weight_grad(B, rows=0, acc=1, dw=None) == 0
    for bad in ({"dy": None}, {"x": None}, {"dw": None}, {"dy": 4104}, {"x": 4104}, {"dw": 4104}, {"db": 4104},
                {"idx": 4100}, {"acc": 2}, {"gd": 2}, {"xr": 7}, {"xr": 0, "idx": 4096}, {"rows": 0, "dw": None}):
        assert weight_grad(B, **bad) == -1, bad
    assert weight_grad(B, dt=0, gd=1) == -2
    assert B.grouped_linear_workspace_size("bf16", 3, 72, 128, 8) == 0


IN = ("residual", "branch", "y_rows", "slot_row", "topk_gate", "shared_out", "gate", "w_out", "b_out", "w_in",
      "b_in", "rng")
OUT = ("d_residual", "d_branch", "d_y_rows", "d_topk_gate", "d_gate", "d_w_out", "d_b_out", "d_w_in", "d_b_in")


def cfg_of(B, **kw):
    c = B.block(8, 64, "bf16", norm_out="rms", norm_in="layer", top_k=2, n_shared=1)
    for name, v in kw.items():
        setattr(c, name, v)
    return c


def join(B, cfg, out=4096, nxt=4096, bo=None, **t):
    s = B.BlockTensors(**{"residual": 4096, "branch": 4096, **t})
    return B.lib().moe_block_join(ctypes.byref(cfg), ctypes.byref(s), P(out), P(nxt), P(bo), None)


def grad(B, cfg, out=4096, d_out=4096, d_next=4096, ws=4096, nbytes=BIG, **t):
    s = B.BlockTensors(**{"branch": 4096, **{a: v for a, v in t.items() if a in IN}})
    g = B.BlockGrads(**{"d_branch": 4096, "d_w_in": 4096, **{a: v for a, v in t.items() if a in OUT}})
    return B.lib().moe_block_join_grad(ctypes.byref(cfg), ctypes.byref(s), P(out), P(d_out), P(d_next),
                                       ctypes.byref(g), P(ws), nbytes, None)


@pytest.mark.parametrize("call", [join, grad])
def test_block_sizes(B, call):
    nan = float("nan")
    for kw, want in [({"T": -1}, -1), ({"d_model": 0}, -1), ({"dtype": 2}, -1), ({"res_dtype": -1}, -1),
                     ({"norm_out": 3}, -1), ({"norm_in": -1}, -1), ({"eps": 0.0}, -1), ({"eps": nan}, -1),
                     ({"eps": float("inf")}, -1), ({"dropout_p": 1.0}, -1), ({"dropout_p": -0.1}, -1),
                     ({"dropout_p": nan}, -1), ({"dropout_p": 0.999995}, -1), ({"dropout_p": 0.1}, -1),
                     ({"dtype": 0, "res_dtype": 1}, -2), ({"d_model": 12}, -2), ({"d_model": 16392}, -2),
                     ({"T": 1 << 40}, -2)]:
        assert call(B, cfg_of(B, **kw)) == want, kw
    L = B.lib()
    assert L.moe_block_join(None, None, None, None, None, None) == -1
    assert L.moe_block_join_grad(None, None, None, None, None, None, None, 0, None) == -1


def test_join_refusals(B):
    c = cfg_of(B)
    assert join(B, cfg_of(B, T=0), residual=None, out=None, nxt=None) == 0
    rows = {"branch": None, "y_rows": 4096, "slot_row": 4096, "topk_gate": 4096, "shared_out": 4096}
    for bad in ({"residual": None}, {"out": None, "nxt": None}, {"y_rows": 4096, "slot_row": 4096, "topk_gate": 4096},
                {**rows, "slot_row": None}, {**rows, "topk_gate": None}, {**rows, "shared_out": None},
                {"residual": 4104}, {"branch": 4104}, {"gate": 4100}, {"w_out": 4100}, {"b_out": 4100},
                {"w_in": 4100}, {"b_in": 4100}, {"rng": 4104}, {"out": 4104}, {"nxt": 4104}, {**rows, "bo": 4104},
                {**rows, "y_rows": 4104}, {**rows, "slot_row": 4100}, {**rows, "topk_gate": 4100},
                {**rows, "shared_out": 4104}):
        assert join(B, c, **bad) == -1, bad
    assert join(B, cfg_of(B, top_k=0), **rows) == -1
    assert join(B, cfg_of(B, n_shared=-1), **rows) == -1
    assert join(B, cfg_of(B, top_k=65), **rows) == -2
    assert join(B, cfg_of(B, n_shared=65), **rows) == -2


def test_grad_refusals(B):
    c = cfg_of(B)
    assert grad(B, cfg_of(B, T=0), d_w_in=None) == 0
    slots = {"slot_row": 4096, "topk_gate": 4096, "y_rows": 4096, "d_topk_gate": 4096, "d_y_rows": 4096}
    for bad in ({"out": None}, {"branch": None}, {"branch": None, "d_branch": None, "d_gate": 4096},
                {**slots, "slot_row": None}, {**slots, "topk_gate": None}, {**slots, "y_rows": None},
                {**slots, "branch": None, "d_branch": None}, {"d_out": 4104}, {"d_next": 4104}, {"out": 4104},
                {"d_residual": 4104}, {"d_branch": 4104}, {**slots, "d_y_rows": 4104},
                {**slots, "d_topk_gate": 4100}, {"d_gate": 4100}, {"d_w_out": 4100}, {"d_b_out": 4100},
                {"d_w_in": 4100}, {"d_b_in": 4100}, {"ws": 4100}):
        assert grad(B, c, **bad) == -1, bad
    assert grad(B, cfg_of(B, top_k=65), **slots) == -2
    need = B.block_join_grad_workspace_size(c)
    assert need > 0 and grad(B, c, nbytes=need - 1) == -3 and grad(B, c, ws=None) == -3
    assert B.block_join_grad_workspace_size(cfg_of(B, d_model=12)) == 0


def drop(B, dt=1, rows=8, d=33, x=4096, y=4096, n=None, p=0.5, rng=4096):
    return B.lib().moe_dropout(dt, rows, d, P(x), P(y), P(n), p, P(rng), None)


def test_dropout_refusals(B):
    assert drop(B, rows=0, x=None, y=None) == 0
    for bad in ({"dt": 2}, {"rows": -1}, {"d": 0}, {"x": None}, {"y": None}, {"rng": None}, {"p": 1.0}, {"p": -0.01},
                {"p": float("nan")}, {"p": 0.999995}, {"x": 4104}, {"y": 4104}, {"n": 4098}, {"rng": 4104}):
        assert drop(B, **bad) == -1, bad
    assert drop(B, rows=1 << 40) == -2


def test_binding_refuses_shapes(B):
    """Tensors on the CPU, or of another shape or type, never reach the library."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int32)
    w = torch.zeros(2, 64, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        B.grouped_linear(x, off, w, x)
    with pytest.raises(ValueError):
        B.grouped_linear_input_grad(x, off, w, x)
    with pytest.raises(ValueError):
        B.grouped_linear_weight_grad(x, off, x, w)
    with pytest.raises(ValueError):
        B.dropout(x, x, 0.5, None)
    with pytest.raises(ValueError):
        B.block_join(B.block(4, 64, "bf16"), x, out=x)


def test_no_tokens_with_expert_rows(B):
    """A step without tokens: slot arrays are empty (and have no address), while expert rows
    and their gradients are usually buffers with room.  Sizes are checked all the same."""
    empty = cfg_of(B, T=0)
    rows = {"residual": None, "branch": None, "y_rows": 4096}
    assert join(B, empty, out=None, nxt=None, **rows) == 0
    assert join(B, empty, out=None, nxt=None, **rows, slot_row=4096) == 0
    asked = {"branch": None, "d_branch": None, "d_w_in": None, "y_rows": 4096, "d_y_rows": 4096, "d_topk_gate": 4096}
    assert grad(B, empty, out=None, d_out=None, d_next=None, ws=None, **asked) == 0
    for call in (lambda c: join(B, c, **rows), lambda c: grad(B, c, **asked)):
        assert call(cfg_of(B, T=0, top_k=0)) == -1
        assert call(cfg_of(B, T=0, n_shared=-1)) == -1
        assert call(cfg_of(B, T=0, top_k=65)) == -2
        assert call(cfg_of(B, T=0, n_shared=65)) == -2


@pytest.mark.parametrize("g,n,k,rows,most", [
    (8, 14336, 4096, 4096, 1 << 27),        # a training step on large experts
    (1, 1 << 20, 64, 4096, 1 << 27),        # sums too short for parts
    (1, 1 << 20, 8192, 4096, 1 << 27),      # so many outputs that they fill the chip
    (64, 1408, 2048, 4096, 1 << 27),
    (64, 1408, 2048, 500, 1 << 28),         # few rows: up to eight parts of 500 rows
])
def test_workspace_is_what_the_kernels_can_use(B, g, n, k, rows, most):
    assert 0 < B.grouped_linear_workspace_size("bf16", g, n, k, rows) <= most
