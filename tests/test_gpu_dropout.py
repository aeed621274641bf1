"""Dropout: the mask bit for bit against the generator's definition, values to one
rounding of their product (float32 factor: 2^-24, bf16 store: 2^-8)."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f32": torch.float32}
TOL = {"bf16": 2.0 ** -8 + 2.0 ** -23, "f32": 2.0 ** -23}


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sparse_mixture_experts_renormalised_amd import binding
    binding.lib()
    return binding


def rng_of(seed, stream):
    return torch.tensor([seed, stream], dtype=torch.int64, device="cuda")


def check(x, y, p, seed, stream, dtype):
    want = oracle.dropout(x.double().cpu().numpy(), p, seed, stream)
    got = y.double().cpu().numpy()
    assert np.array_equal(got == 0, want == 0)
    assert (np.abs(got - want) <= TOL[dtype] * np.abs(want)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d,p", [(1, 1, 0.5), (1, 7, 0.9), (3, 8, 0.1), (5, 33, 0.3), (17, 64, 0.5), (2, 4097, 0.01),
                                      (300, 5, 0.75), (9, 16, 0.9999)])
def test_mask_and_values(B, rows, d, p, dtype):
    print(f"[dropout] {rows}x{d} p={p} {dtype}", flush=True)
    x = (torch.rand(rows, d, generator=torch.Generator().manual_seed(rows)) + 0.5).to(T[dtype]).cuda()
    for seed, stream in ((0, 0), (-1, 5), (0x123456789ABCDEF, -(1 << 40) - 3)):
        y = torch.full_like(x, 7.0)
        B.dropout(x, y, p, rng_of(seed, stream))
        torch.cuda.synchronize()
        check(x, y, p, seed, stream, dtype)
        z = x.clone()
        B.dropout(z, z, p, rng_of(seed, stream))          # in place
        torch.cuda.synchronize()
        assert torch.equal(z, y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_are_not_there(B, dtype):
    x = torch.ones(11, 13, dtype=T[dtype], device="cuda")
    x[7:] = float("nan")
    for n, kept in ((7, 7), (0, 0), (-3, 0), (1, 1)):
        y = torch.full_like(x, 5.0)
        B.dropout(x, y, 0.4, rng_of(3, 4), n_rows=torch.tensor([n], dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        assert (y[kept:] == 5.0).all()
        if kept:
            check(x[:kept], y[:kept], 0.4, 3, 4, dtype)
    x[7:] = 1.0
    y = torch.full_like(x, 5.0)
    B.dropout(x, y, 0.4, rng_of(3, 4), n_rows=torch.tensor([1 << 30], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    check(x, y, 0.4, 3, 4, dtype)


def test_no_probability_copies(B):
    x = torch.randn(5, 33, device="cuda")
    y = torch.zeros_like(x)
    B.dropout(x, y, 0.0, None)
    assert torch.equal(x, y)
    y.zero_()
    B.dropout(x, y, 2.0 ** -18, None)                      # rounds to 0
    assert torch.equal(x, y)


def test_a_dropped_value_is_zero_whatever_it_was(B):
    x = torch.full((4, 256), float("nan"), device="cuda")
    x[1] = float("inf")
    y = torch.ones_like(x)
    B.dropout(x, y, 0.5, rng_of(1, 2))
    keep = torch.from_numpy(oracle.dropout_keep(1024, 0.5, 1, 2)).view(4, 256).cuda()
    assert (y[~keep] == 0).all() and not y[keep].isfinite().any()


def test_linear_in_x(B):
    """Its own gradient: <dropout(x), c> = <x, dropout(c)>, the same products in both."""
    g = torch.Generator().manual_seed(0)
    x, c = torch.randn(40, 100, generator=g).cuda(), torch.randn(40, 100, generator=g).cuda()
    y, d = torch.empty_like(x), torch.empty_like(x)
    B.dropout(x, y, 0.5, rng_of(9, 9))                     # factor 2: exact
    B.dropout(c, d, 0.5, rng_of(9, 9))
    assert torch.equal(y.double() * c.double(), x.double() * d.double())


def test_captured_with_new_numbers(B):
    x = torch.randn(33, 130, device="cuda")
    y, r = torch.empty_like(x), rng_of(1, 1)
    B.dropout(x, y, 0.3, r)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.dropout(x, y, 0.3, r)
    for step in range(3):
        r.copy_(torch.tensor([step, 7]))
        graph.replay()
        torch.cuda.synchronize()
        check(x, y, 0.3, step, 7, "f32")


def test_more_than_one_pass_of_the_grid(B):
    """More blocks of eight than the launch has threads, and a tail."""
    rows, d = 2049, 2051
    x = torch.ones(rows, d, device="cuda", dtype=torch.bfloat16)
    y = torch.empty_like(x)
    B.dropout(x, y, 0.5, rng_of(2, 3))
    got = y.view(-1).float().cpu().numpy()
    n = rows * d
    for first in (0, 8 * 256 * 2048 - 40, n - 77):
        m = min(77, n - first)
        assert np.array_equal(got[first:first + m] != 0, oracle.dropout_keep(m, 0.5, 2, 3, first=first))
    # standard deviation of the mean of n draws: 0.0005
    assert abs((got != 0).mean() - 0.5) < 0.0025
