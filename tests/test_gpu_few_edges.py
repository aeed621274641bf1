"""Edges of the few-token layer: kept gates that are very small."""
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
