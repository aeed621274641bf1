"""The oracle of the training calls: the generator against published numbers, and
every gradient against differences of its forward (float64)."""
import numpy as np
import pytest

import oracle


def test_philox_known_answers():
    # known-answer vectors of the Random123 distribution
    full = 0xFFFFFFFF
    assert oracle.philox4x32([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert oracle.philox4x32([full] * 4, [full] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert oracle.philox4x32([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0]) == \
        [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_dropout_mask():
    a = oracle.dropout_keep(4000, 0.25, 7, 9)
    assert np.array_equal(oracle.dropout_keep(100, 0.25, 7, 9, first=1003), a[1003:1103])
    assert not np.array_equal(a, oracle.dropout_keep(4000, 0.25, 7, 10))
    assert not np.array_equal(a, oracle.dropout_keep(4000, 0.25, 8, 9))
    # 4000 draws of 0.75: standard deviation 0.007
    assert abs(a.mean() - 0.75) < 0.035
    assert oracle.dropout_cut(0.5 / 65536) == 0 and oracle.dropout_cut(1.5 / 65536) == 2
    y = oracle.dropout(np.ones(4000), 0.25, 7, 9)
    assert set(np.unique(y)) == {0.0, 4.0 / 3.0}


def diff(f, x, at, h=1e-6):
    """Derivative of the number f() along the element x[at]."""
    v = x[at]
    x[at] = v + h
    hi = f()
    x[at] = v - h
    lo = f()
    x[at] = v
    return (hi - lo) / (2 * h)


def test_linear_gradients_by_differences():
    rng = np.random.default_rng(0)
    offsets = np.array([0, 3, 3, 8])
    x, w, b = rng.normal(size=(5, 6)), rng.normal(size=(3, 4, 6)), rng.normal(size=(3, 4))
    index = rng.integers(0, 5, 8)
    c = rng.normal(size=(8, 4))

    def loss():
        return (c * oracle.grouped_linear(x, offsets, w, index, b)).sum()

    dw, db = oracle.grouped_linear_weight_grad(c, offsets, x, index)
    dx = np.zeros_like(x)
    np.add.at(dx, index, oracle.grouped_linear_input_grad(c, offsets, w))
    for at in [(0, 1, 2), (1, 0, 0), (2, 3, 5)]:
        assert diff(loss, w, at) == pytest.approx(dw[at], abs=1e-7)
    assert diff(loss, b, (2, 1)) == pytest.approx(db[2, 1], abs=1e-7)
    for at in [(0, 0), (3, 5), (4, 2)]:
        assert diff(loss, x, at) == pytest.approx(dx[at], abs=1e-7)


def test_silu_factor_by_differences():
    rng = np.random.default_rng(1)
    offsets = np.array([0, 2, 5])
    z, w, c = rng.normal(size=(5, 6)), rng.normal(size=(2, 4, 6)), rng.normal(size=(5, 4))

    def loss():
        return (c * oracle.grouped_linear(z / (1.0 + np.exp(-z)), offsets, w)).sum()

    dz = oracle.grouped_linear_input_grad(c, offsets, w, z)
    for at in [(0, 0), (1, 5), (4, 3)]:
        assert diff(loss, z, at) == pytest.approx(dz[at], abs=1e-7)


@pytest.mark.parametrize("norm_in", ["none", "rms", "layer"])
@pytest.mark.parametrize("norm_out", ["none", "rms", "layer"])
def test_block_gradients_by_differences(norm_out, norm_in):
    rng = np.random.default_rng(2)
    T, d, K, rows = 4, 16, 2, 7
    y, gates = rng.normal(size=(rows, d)), rng.random((T, K))
    slot = np.array([[0, 3], [-1, 6], [-1, -1], [2, -1]])
    shared = rng.normal(size=(2, T, d))
    t = {"residual": rng.normal(size=(T, d)), "gate": rng.random(T)}
    for n in ("w_out", "b_out", "w_in", "b_in"):
        t[n] = rng.normal(size=d)
    mask = (rng.random((T, d)) < 0.7) / 0.7
    c, e = rng.normal(size=(T, d)), rng.normal(size=(T, d))
    kw = dict(norm_out=norm_out, norm_in=norm_in, eps=1e-2, scale=0.7, mask=mask)

    def branch():
        return oracle.combine_rows(y, slot, gates, shared)

    def loss():
        out, nxt = oracle.block_join(branch=branch(), **t, **kw)
        return (c * out).sum() + (e * nxt).sum()

    out = oracle.block_join(branch=branch(), **t, **kw)[0]
    g = oracle.block_join_grad(c, e, out, branch(), gate=t["gate"], w_out=t["w_out"], b_out=t["b_out"],
                               w_in=t["w_in"], slot_row=slot, topk_gate=gates, y_rows=y, **kw)
    for at in [(0, 0), (1, 7), (2, 3), (3, 15)]:
        assert diff(loss, t["residual"], at) == pytest.approx(g["d_residual"][at], abs=1e-6)
        assert diff(loss, shared, (1, *at)) == pytest.approx(g["d_branch"][at], abs=1e-6)
    for name in ("gate", "w_out", "b_out", "w_in", "b_in"):
        for at in (0, 2, 3):
            assert diff(loss, t[name], at) == pytest.approx(g["d_" + name][at], abs=1e-6), name
    for at in [(0, 0), (0, 1), (1, 0), (1, 1), (2, 0), (3, 0)]:
        assert diff(loss, gates, at) == pytest.approx(g["d_topk_gate"][at], abs=1e-6)
    for row in range(rows):
        for j in (0, 9):
            want = g["d_y_rows"][row][j] if row in g["d_y_rows"] else 0.0
            assert diff(loss, y, (row, j)) == pytest.approx(want, abs=1e-6)
