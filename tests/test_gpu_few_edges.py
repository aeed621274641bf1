"""Edges of the few-token layer: kept gates that are very small, NaNs of unusual bits, zeros of
either sign, tokens that are not finite."""
import numpy as np
import pytest
import torch

import oracle
from test_gpu_few import B, Few  # noqa: F401  (B: the fixture)

pytestmark = pytest.mark.gpu


# T, d, N, f, factor of the capacity, bias of the Linears.  Small layers give every
# share one block of 32 hidden rows; the last one gives most shares three.
SMALL_GATES = [(1, 128, 6, 128, 0.0, True), (4, 128, 8, 128, 1.0, True), (6, 128, 8, 128, 2.0, True), (8, 256, 8, 384, 1.5, True),
               (16, 128, 12, 128, 1.5, False), (16, 256, 12, 384, 1.5, True), (16, 128, 12, 4096, 1.5, False)]


@pytest.mark.parametrize("lead", [11.0, 14.0, 18.0])
@pytest.mark.parametrize("case", SMALL_GATES, ids=lambda c: f"T{c[0]}-d{c[1]}-N{c[2]}-f{c[3]}")
def test_mxfp4_hidden_rows_of_small_gates(B, case, lead):  # noqa: F811
    """One expert's logit is far above the others', and its capacity drops it for the
    later tokens: what these tokens have left is an expert with a gate of about
    e^-lead.  Each token's output is checked against its own size: with E the error of
    a hidden value that the interface states (2^-12 of it or 2^-25 of the largest of
    its 32, tokens off by 2^-21 of the largest of theirs, float32 sums of n terms off by
    n 2^-24 of their magnitudes, SiLU's slope at most 1.1), the output is off by at most
    gate (|W2|_2 |E|_2 + the error of its own sums), the gate's own relative error
    (twice that of a logit), and 2^-8 of itself for the store."""
    T, d, N, f, cap, bias = case
    print(f"[few] small gates {case} lead={lead}", flush=True)
    L = Few(B, T, d, N, 2, 0, f, "mxfp4", cap=cap, bias=bias, router="gauss", seed=90 + T + d)
    L.rb[0] = lead
    L()
    torch.cuda.synchronize()
    ref, _ = L.reference()
    assert np.array_equal(L.idx.cpu().numpy(), ref["topk_idx"])
    h = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    x, y, wr = h(L.x), h(L.y), np.abs(h(L.wr))
    norm2 = {}
    alone = 0                                # tokens whose kept gates are all small
    for t in range(T):
        xm = np.repeat(np.abs(x[t]).reshape(-1, 32).max(1), 32)
        kept = [(int(e), ref["gates"][t, k]) for k, e in enumerate(ref["topk_idx"][t])
                if ref["slot_row"][t, k] >= 0]
        alone += bool(kept) and max(g for _, g in kept) < 1e-3
        dg = 2 * (d + 2) * 2.0 ** -24 * max((wr[e] @ np.abs(x[t]) + abs(float(L.rb[e]))
                                             for e in ref["topk_idx"][t]), default=0.0) + 2.0 ** -20
        tol = 2.0 ** -8 * np.linalg.norm(ref["y"][t])
        for e, g in kept:
            w1, w2 = h(L.w["w1"][e]), h(L.w["w2"][e])
            b1 = np.zeros(f) if not bias else h(L.w["b1"][e])
            b2 = np.zeros(d) if not bias else h(L.w["b2"][e])
            hid = oracle.silu(w1 @ x[t] + b1)
            dz = (2 * d + 1) * 2.0 ** -24 * (np.abs(w1) @ np.abs(x[t]) + np.abs(b1)) + \
                2.0 ** -21 * (np.abs(w1) @ xm)
            most = np.repeat(np.abs(hid).reshape(-1, 32).max(1), 32)
            dh = (2.0 ** -12 + 2.0 ** -20) * np.abs(hid) + 2.0 ** -25 * most + 1.1 * dz
            if e not in norm2:
                norm2[e] = np.linalg.norm(w2, 2)
            sums = (3 * f + 2) * 2.0 ** -24 * (np.abs(w2) @ np.abs(hid) + np.abs(b2))
            tol += (1 + dg) * g * (norm2[e] * np.linalg.norm(dh) + np.linalg.norm(sums)) + \
                dg * g * np.linalg.norm(w2 @ hid + b2)
        err = np.linalg.norm(y[t] - ref["y"][t])
        assert err <= tol, (t, err / max(np.linalg.norm(ref["y"][t]), 1e-300), err / max(tol, 1e-300))
    assert alone > 0 or T == 1


@pytest.mark.parametrize("bits", [0x7FFFFFFF, -1], ids=["plus", "minus"])
@pytest.mark.parametrize("kind", ["bf16", "mxfp4", "f32"])
@pytest.mark.parametrize("T", [1, 6, 16])
def test_nan_of_all_ones_in_the_router(B, T, kind, bits):  # noqa: F811
    """A NaN whose mantissa is all ones rounds to a NaN, not past it: a router bias that
    holds one makes NaN gates and with them outputs that are NaN throughout."""
    print(f"[few] NaN of all ones {kind} T={T}", flush=True)
    L = Few(B, T, 128, 2, 2, 1, 128, kind, router="gauss", seed=30 + T)
    L.rb.view(torch.int32)[1] = bits
    L()
    torch.cuda.synchronize()
    assert L.gate.isnan().all()
    assert L.y.isnan().all()


@pytest.mark.parametrize("bits", [0x7FFFFFFF, -1, 0x7FC00000], ids=["plus", "minus", "usual"])
def test_nan_gates_of_all_ones_in_the_combine(B, bits):  # noqa: F811
    T, d = 5, 128
    cfg = B.config(T, d, 4, 1, 0, 128, "bf16")
    rows = torch.randn(T, d, device="cuda").bfloat16()
    slot = torch.arange(T, dtype=torch.int32, device="cuda").view(T, 1)
    gate = torch.ones(T, 1, device="cuda")
    gate.view(torch.int32)[2] = bits
    y = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    B.combine(cfg, rows, slot, gate, None, y)
    torch.cuda.synchronize()
    assert y[2].isnan().all()
    keep = [0, 1, 3, 4]
    assert torch.equal(y[keep], rows[keep])


def test_every_rounding_to_bf16(B):  # noqa: F811
    """Gates of every sign, exponent and leading seven bits, with what follows below, at
    and above half a step, times rows of ones: the nearest bf16, ties to even."""
    high = torch.arange(65536, dtype=torch.int64, device="cuda") << 16
    bits = torch.cat([high | low for low in (0, 1, 0x7FFF, 0x8000, 0x8001, 0xFFFF)])
    T, d = bits.numel(), 64
    gate = (((bits + 2 ** 31) % 2 ** 32) - 2 ** 31).int().view(torch.float32).view(T, 1)
    rows = torch.ones(T, d, dtype=torch.bfloat16, device="cuda")
    slot = torch.arange(T, dtype=torch.int32, device="cuda").view(T, 1)
    y = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    B.combine(B.config(T, d, 4, 1, 0, 64, "bf16"), rows, slot, gate, None, y)
    torch.cuda.synchronize()
    nan = (bits & 0x7FFFFFFF) > 0x7F800000
    want = (bits + 0x7FFF + ((bits >> 16) & 1)) >> 16
    want[bits == 1 << 31] = 0                # the sum starts at +0
    got = y.view(torch.int16).long() & 0xFFFF
    assert y[nan].isnan().all()
    assert torch.equal(got[~nan], want[~nan].view(-1, 1).expand(-1, d))


@pytest.mark.parametrize("kind", ["bf16", "f32", "mxfp4"])
@pytest.mark.parametrize("T", [1, 9])
def test_zeros_of_either_sign_tie(B, T, kind):  # noqa: F811
    """Expert 0's logit is a product too small for float32 with a minus sign, -0; the
    others' are +0.  Equal values tie, and the lowest ids win."""
    print(f"[few] -0 ties {kind} T={T}", flush=True)
    L = Few(B, T, 4096, 6, 2, 0, 128, kind, seed=31 + T)
    L.x.fill_(2.0 ** -100)
    L.wr.zero_()
    L.wr[0] = -(2.0 ** -100)
    L()
    torch.cuda.synchronize()
    assert L.idx.cpu().tolist() == [[0, 1]] * T
    assert torch.all((L.gate - 0.5).abs() <= 1e-7)


def _micros(call, n=10):
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    least = float("inf")
    for _ in range(5):
        call()
        a.record()
        for _ in range(n):
            call()
        b.record()
        b.synchronize()
        least = min(least, a.elapsed_time(b) * 1e3 / n)
    return least


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("case", [(8, 2048, 64, 8, 2, 1408, "bf16"), (16, 2048, 32, 4, 1, 2048, "mxfp4"),
                                  (12, 512, 32, 4, 1, 768, "f32")], ids=lambda c: f"{c[6]}-T{c[0]}")
def test_tokens_that_are_not_finite_do_not_hold_a_step_up(B, case, bad):  # noqa: F811
    """A row of a padded batch may hold anything.  Its outputs are known not to be
    finite after the first terms of their sums: a step takes no longer for it, but for
    the little that finds it out (half again is allowed)."""
    L = Few(B, *case, seed=32)
    ref, A = L.reference()
    tol = L.bound(ref, A)
    usual = _micros(L)
    L.x[3] = bad
    held = _micros(L)
    print(f"[few] {case} {bad}: {usual:.1f} us, {held:.1f} us with such a token", flush=True)
    rest = [t for t in range(case[0]) if t != 3]
    assert not torch.isfinite(L.y[3].float()).any()
    # (not the same bits: the experts that token 3 meets now are others, and sums are cut
    # where all entries' chunks are)
    assert np.all((np.abs(L.y.double().cpu().numpy() - ref["y"]) <= tol)[rest])
    assert held <= 1.5 * usual + 5.0


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("case", [(8, 2048, 64, 8, 2, 1408, "bf16"), (16, 2048, 32, 4, 1, 2048, "mxfp4"),
                                  (12, 512, 32, 4, 1, 768, "f32")], ids=lambda c: f"{c[6]}-T{c[0]}")
def test_hidden_values_that_are_not_finite_do_not_hold_a_step_up(B, case, bad):  # noqa: F811
    """The same where one hidden value of an expert, its last, overflows or is NaN: no
    output of the tokens that the expert computes is finite, and those of the others
    are as before."""
    L = Few(B, *case, seed=33)
    ref, A = L.reference()
    tol = L.bound(ref, A)
    usual = _micros(L)
    T, d, N, f = case[0], case[1], case[2], case[5]
    e = int(ref["topk_idx"][1, 0])
    if case[6] == "mxfp4":
        L.w["k1"].view(N, f, d // 32)[e, f - 1, d // 32 - 1] = 255
    else:
        L.w["w1"][e, f - 1, d - 1] = bad
    held = _micros(L)
    print(f"[few] {case} {bad}: {usual:.1f} us, {held:.1f} us with such a value", flush=True)
    y = L.y.double().cpu().numpy()
    for t in range(T):
        if e in ref["topk_idx"][t]:
            assert not np.isfinite(y[t]).any(), t
        else:
            assert np.all(np.abs(y[t] - ref["y"][t]) <= tol[t]), t
    assert held <= 1.5 * usual + 5.0
