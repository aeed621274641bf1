"""Plain CPU oracle, in float64, of the calls that train the layer as a block:
the single Linears of the experts and their gradients, the block around the
layer (norms, gate, residual) and its gradients, and the counter-based dropout.

TEST INFRASTRUCTURE ONLY, written from the definitions; it shares no code with
the HIP library and never calls it.
"""
from __future__ import annotations

import numpy as np

__all__ = ["philox4x32", "dropout_cut", "dropout_keep", "dropout", "grouped_linear",
           "grouped_linear_input_grad", "grouped_linear_weight_grad", "norm_rows", "combine_rows",
           "block_join", "block_join_grad"]

M32 = 0xFFFFFFFF


def philox4x32(counter, key, rounds=10):
    """Philox4x32 of Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
    easy as 1, 2, 3" (SC 2011): four words from a counter of four and a key of
    two, on Python integers."""
    c, k = [int(v) for v in counter], [int(v) for v in key]
    for _ in range(rounds):
        p, q = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(q >> 32) ^ c[1] ^ k[0], q & M32, (p >> 32) ^ c[3] ^ k[1], p & M32]
        k = [(k[0] + 0x9E3779B9) & M32, (k[1] + 0xBB67AE85) & M32]
    return c


def dropout_cut(p: float) -> int:
    """The probability in steps of 2^-16, ties to even."""
    return round(p * 65536)


def dropout_keep(n: int, p: float, seed: int, stream: int, first: int = 0):
    """Which of the elements first .. first + n - 1 stay."""
    cut, out = dropout_cut(p), []
    seed, stream = seed % 2 ** 64, stream % 2 ** 64
    for b in range(first // 8, (first + n + 7) // 8):
        w = philox4x32([b & M32, b >> 32, stream & M32, stream >> 32], [seed & M32, seed >> 32])
        for v in w:
            out += [(v & 0xFFFF) >= cut, (v >> 16) >= cut]
    return np.array(out[first % 8: first % 8 + n], dtype=bool)


def dropout(x, p, seed, stream):
    keep = dropout_keep(x.size, p, seed, stream).reshape(x.shape)
    return np.where(keep, x * (65536.0 / (65536 - dropout_cut(p))), 0.0)


def _silu(z):
    return z / (1.0 + np.exp(-z))


def grouped_linear(x, offsets, w, index=None, bias=None):
    """Rows before an activation: z[r] = x[index[r]] W_g^T + bias_g."""
    n = int(offsets[-1])
    z = np.zeros((n, w.shape[1]))
    for g in range(len(offsets) - 1):
        a, b = int(offsets[g]), int(offsets[g + 1])
        rows = x[a:b] if index is None else x[index[a:b]]
        z[a:b] = rows @ w[g].T + (0.0 if bias is None else bias[g])
    return z


def grouped_linear_input_grad(dy, offsets, w, pre=None):
    n = int(offsets[-1])
    dx = np.zeros((n, w.shape[2]))
    for g in range(len(offsets) - 1):
        a, b = int(offsets[g]), int(offsets[g + 1])
        dx[a:b] = dy[a:b] @ w[g]
    if pre is not None:
        s = 1.0 / (1.0 + np.exp(-pre[:n]))
        dx = dx * (s + pre[:n] * s * (1.0 - s))
    return dx


def grouped_linear_weight_grad(dy, offsets, x, index=None):
    """dw [G, n_out, k] and dbias [G, n_out]."""
    G = len(offsets) - 1
    dw, db = np.zeros((G, dy.shape[1], x.shape[1])), np.zeros((G, dy.shape[1]))
    for g in range(G):
        a, b = int(offsets[g]), int(offsets[g + 1])
        rows = x[a:b] if index is None else x[index[a:b]]
        dw[g], db[g] = dy[a:b].T @ rows, dy[a:b].sum(axis=0)
    return dw, db


def norm_rows(v, kind, eps):
    """Normalised rows and the factor r that made them."""
    if kind == "none":
        return v, np.ones((v.shape[0], 1))
    if kind == "layer":
        v = v - v.mean(axis=1, keepdims=True)
    r = 1.0 / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)
    return v * r, r


def combine_rows(y_rows, slot_row, topk_gate, shared_out=None):
    T, K = slot_row.shape
    b = np.zeros((T, y_rows.shape[1]))
    if shared_out is not None:
        b += shared_out.sum(axis=0)
    for t in range(T):
        for k in range(K):
            if slot_row[t, k] >= 0:
                b[t] += topk_gate[t, k] * y_rows[slot_row[t, k]]
    return b


def _or(v, other):
    return other if v is None else v


def block_join(residual, branch, norm_out, norm_in, eps, scale=1.0, gate=None, mask=None, w_out=None,
               b_out=None, w_in=None, b_in=None):
    """out and next; mask holds 0 or 1 / (1 - q) for every branch element."""
    h = residual
    if branch is not None:
        n = norm_rows(branch, norm_out, eps)[0] * _or(w_out, 1.0) + _or(b_out, 0.0)
        f = scale * (np.ones((len(branch), 1)) if gate is None else gate[:, None])
        h = h + f * _or(mask, 1.0) * n
    return h, norm_rows(h, norm_in, eps)[0] * _or(w_in, 1.0) + _or(b_in, 0.0)


def _norm_grad(g, hat, r, kind):
    if kind == "none":
        return g
    d = g - hat * (g * hat).mean(axis=1, keepdims=True)
    if kind == "layer":
        d = d - g.mean(axis=1, keepdims=True)
    return d * r


def block_join_grad(d_out, d_next, out, branch, norm_out, norm_in, eps, scale=1.0, gate=None, mask=None,
                    w_out=None, b_out=None, w_in=None, slot_row=None, topk_gate=None, y_rows=None):
    """Gradients of block_join's inputs, and of the expert rows and gates."""
    res = {}
    hat, r = norm_rows(out, norm_in, eps)
    dh = d_out + _norm_grad(d_next * _or(w_in, 1.0), hat, r, norm_in)
    res["d_residual"] = dh
    res["d_w_in"], res["d_b_in"] = (d_next * hat).sum(axis=0), d_next.sum(axis=0)
    if branch is None:
        return res
    hat, r = norm_rows(branch, norm_out, eps)
    u = scale * dh * _or(mask, 1.0)
    res["d_gate"] = (u * (hat * _or(w_out, 1.0) + _or(b_out, 0.0))).sum(axis=1)
    g = u if gate is None else u * gate[:, None]
    res["d_w_out"], res["d_b_out"] = (g * hat).sum(axis=0), g.sum(axis=0)
    db = res["d_branch"] = _norm_grad(g * _or(w_out, 1.0), hat, r, norm_out)
    if slot_row is not None:
        T, K = slot_row.shape
        res["d_topk_gate"], res["d_y_rows"] = np.zeros((T, K)), {}
        for t in range(T):
            for k in range(K):
                row = int(slot_row[t, k])
                if row >= 0:
                    res["d_y_rows"][row] = topk_gate[t, k] * db[t]
                    res["d_topk_gate"][t, k] = db[t] @ y_rows[row]
    return res
