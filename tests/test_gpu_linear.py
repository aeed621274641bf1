"""Single Linears of every expert and their gradients against float64.

Bounds, per output: float32 sums of n products are off by at most (n + 4) 2^-24
times the sum of magnitudes (every partial sum, and float32 products where the
inputs are float32, rounds once); SiLU and its derivative have slopes of at most
1.1 and the library's own are within 2^-19 (1 + |z|) relative (an exponent of
|z| 2^-23 and a few units of the reciprocal); a store to bf16 rounds by 2^-8
relative, one to float32 by 2^-24.  Weight gradients of n rows that are split into
parts add at most two roundings, which the 4 covers."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U = 2.0 ** -24


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sparse_mixture_experts_renormalised_amd import binding
    binding.lib()
    return binding


def f64(t):
    return t.double().cpu().numpy()


def close(got, ref, bound, what):
    """|got - ref| within bound plus the rounding of got's type."""
    g = f64(got)
    assert np.isfinite(g).all(), what
    over = np.abs(g - ref) - (bound + HALF[got.dtype] * (np.abs(ref) + bound))
    i = np.unravel_index(np.argmax(over), over.shape) if over.size else None
    assert not over.size or over[i] <= 0, f"{what}: {g[i]} for {ref[i]} at {i}, off by {abs(g[i] - ref[i]):.3e}"


def offsets_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def data(B, dtype, counts, n_out, k, seed, gather, room=5):
    gen = torch.Generator().manual_seed(seed)
    off = offsets_of(counts)
    rows, G = int(off[-1]), len(counts)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen) * std).to(T[dtype]).cuda()

    tokens = max(1, rows // 3) if gather else rows + room
    d = {"off": off, "offsets": torch.from_numpy(off).cuda(), "x": normal(tokens, k),
         "index": torch.randint(0, tokens, (rows + room,), generator=gen, dtype=torch.int32).cuda() if gather else None,
         "w": normal(G, n_out, k, std=k ** -0.5), "bias": normal(G, n_out), "dy": normal(rows + room, n_out),
         "z": normal(rows + room, k, std=2.0)}
    n = B.grouped_linear_workspace_size(dtype, G, n_out, k, rows + room)
    d["ws"] = torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda") if n else None
    d["src"] = None if d["index"] is None else d["index"].cpu().numpy()[:rows]
    d["rows"], d["room"] = rows, rows + room
    # rows behind the last group are not there: whatever they hold reaches nothing
    d["dy"][rows:] = float("nan")
    d["z"][rows:] = float("nan")
    if not gather:
        d["x"][rows:] = float("nan")
    return d


def acts(z):
    s = 1.0 / (1.0 + np.exp(-z))
    return z * s


CASES = [
    # counts, n_out, k
    ([1], 64, 64),
    ([0, 0, 3], 64, 128),
    ([5, 0, 64, 65, 63, 1, 0], 128, 320),
    ([0, 0, 0, 0], 64, 64),
    ([128, 127, 129, 33, 31, 2], 192, 64),
    ([257, 256, 255, 300, 0, 513], 320, 192),
    ([700], 576, 704),
    ([17] * 40 + [0] * 23 + [90], 64, 256),
    ([1, 2, 0, 1, 1, 0, 3], 1024, 1088),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_forward(B, case, dtype):
    counts, n_out, k = CASES[case]
    gather, silu, bias = case % 2 == 0, case % 3 != 1, case % 4 < 2
    print(f"[linear] forward {dtype} {counts[:8]} {k}->{n_out}", flush=True)
    d = data(B, dtype, counts, n_out, k, 100 + case, gather)
    y = torch.full((d["room"], n_out), 0.5, dtype=T[dtype], device="cuda")
    pre = torch.full_like(y, 0.25) if silu and case % 2 == 0 else None
    b = d["bias"] if bias else None
    B.grouped_linear(d["x"], d["offsets"], d["w"], y, row_index=d["index"], bias=b, silu=silu, pre=pre, ws=d["ws"])
    torch.cuda.synchronize()
    w, x, r = f64(d["w"]), f64(d["x"]), d["rows"]
    bb = f64(d["bias"]) if bias else None
    z = oracle.grouped_linear(x, d["off"], w, d["src"], bb)
    mag = oracle.grouped_linear(np.abs(x), d["off"], np.abs(w), d["src"], None if bb is None else np.abs(bb))
    bound = (k + 4) * U * mag
    assert (y[r:] == 0.5).all()
    if pre is not None:
        assert (pre[r:] == 0.25).all()
        close(pre[:r], z, bound, "pre")
    if silu:
        close(y[:r], acts(z), 1.1 * bound + 2.0 ** -19 * (1 + np.abs(z)) * np.abs(acts(z)), "y")
    else:
        close(y[:r], z, bound, "y")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_input_grad(B, case, dtype):
    counts, n_out, k = CASES[case]
    print(f"[linear] input gradient {dtype} {counts[:8]} {k}->{n_out}", flush=True)
    d = data(B, dtype, counts, n_out, k, 200 + case, False)
    for z in (None, d["z"]):
        dx = torch.full((d["room"], k), 0.5, dtype=T[dtype], device="cuda")
        B.grouped_linear_input_grad(d["dy"], d["offsets"], d["w"], dx, pre=z, ws=d["ws"])
        torch.cuda.synchronize()
        w, dy, r = f64(d["w"]), f64(d["dy"][:d["rows"]]), d["rows"]
        zz = None if z is None else f64(z[:r])
        ref = oracle.grouped_linear_input_grad(dy, d["off"], w, zz)
        plain = np.abs(oracle.grouped_linear_input_grad(dy, d["off"], w))
        mag = oracle.grouped_linear_input_grad(np.abs(dy), d["off"], np.abs(w))
        bound = 1.1 * (n_out + 4) * U * mag
        if zz is not None:
            bound = bound + 2.0 ** -19 * (1 + np.abs(zz)) * plain
        assert (dx[r:] == 0.5).all()
        close(dx[:r], ref, bound, "dx")


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_weight_grad(B, case, dtype, out):
    counts, n_out, k = CASES[case]
    gather = case % 2 == 1
    print(f"[linear] weight gradient {dtype}->{out} {counts[:8]} {k}->{n_out}", flush=True)
    d = data(B, dtype, counts, n_out, k, 300 + case, gather)
    G, r = len(counts), d["rows"]
    dw = torch.full((G, n_out, k), float("nan"), dtype=T[out], device="cuda")
    db = torch.full((G, n_out), float("nan"), dtype=T[out], device="cuda") if case % 3 != 2 else None
    call = dict(row_index=d["index"], ws=d["ws"])
    B.grouped_linear_weight_grad(d["dy"], d["offsets"], d["x"], dw, dbias=db, **call)
    torch.cuda.synchronize()
    dy, x = f64(d["dy"][:r]), f64(d["x"])
    ref, rb = oracle.grouped_linear_weight_grad(dy, d["off"], x, d["src"])
    mag, mb = oracle.grouped_linear_weight_grad(np.abs(dy), d["off"], np.abs(x), d["src"])
    n = np.array(counts, dtype=np.float64)
    bound, bb = (n + 4)[:, None, None] * U * mag, (n + 4)[:, None] * U * mb
    close(dw, ref, bound, "dw")
    if db is not None:
        close(db, rb, bb, "dbias")
    # added to what is there
    old = torch.full_like(dw, 3.0)
    B.grouped_linear_weight_grad(d["dy"], d["offsets"], d["x"], old, accumulate=True, **call)
    torch.cuda.synchronize()
    close(old, ref + 3.0, bound + U * (np.abs(ref) + 3.0), "accumulated dw")
    if db is not None:
        old = torch.full_like(db, 3.0)
        B.grouped_linear_weight_grad(d["dy"], d["offsets"], d["x"], dw, dbias=old, accumulate=True, **call)
        torch.cuda.synchronize()
        close(old, rb + 3.0, bb + U * (np.abs(rb) + 3.0), "accumulated dbias")


def test_nothing_to_do(B):
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((2, 64, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    db = torch.full((2, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    w = torch.ones_like(dw)
    n = B.grouped_linear_workspace_size("bf16", 2, 64, 64, 0)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    B.grouped_linear(x, off, w, x, ws=ws)
    B.grouped_linear_input_grad(x, off, w, x, ws=ws)
    B.grouped_linear_weight_grad(x, off, x, dw, dbias=db, ws=ws)
    torch.cuda.synchronize()
    assert (dw == 0).all() and (db == 0).all()
    dw.fill_(2.0)
    B.grouped_linear_weight_grad(x, off, x, dw, accumulate=True, ws=ws)
    torch.cuda.synchronize()
    assert (dw == 2).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_what_is_not_finite_stays_in_its_group(B, dtype):
    counts, n_out, k = [70, 3, 200, 64], 192, 128
    d = data(B, dtype, counts, n_out, k, 7, False)
    a, b = int(d["off"][1]), int(d["off"][2])
    clean = [torch.empty(d["room"], n_out, dtype=T[dtype], device="cuda"),
             torch.empty(d["room"], k, dtype=T[dtype], device="cuda"),
             torch.empty(4, n_out, k, dtype=T[dtype], device="cuda")]
    dirty = [torch.empty_like(t) for t in clean]

    def run(o):
        B.grouped_linear(d["x"], d["offsets"], d["w"], o[0], ws=d["ws"])
        B.grouped_linear_input_grad(d["dy"], d["offsets"], d["w"], o[1], ws=d["ws"])
        B.grouped_linear_weight_grad(d["dy"], d["offsets"], d["x"], o[2], ws=d["ws"])
        torch.cuda.synchronize()

    run(clean)
    d["x"][a:b] = float("inf")
    d["dy"][a:b] = float("nan")
    d["w"][1] = float("nan")
    run(dirty)
    for c, e in zip(clean[:2], dirty[:2]):
        assert torch.equal(c[:a], e[:a]) and torch.equal(c[b:d["rows"]], e[b:d["rows"]])
        assert not e[a:b].isfinite().any()
    assert torch.equal(clean[2][[0, 2, 3]], dirty[2][[0, 2, 3]]) and dirty[2][1].isnan().all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_other_streams_and_graphs(B, dtype):
    """Captured calls give the eager call's bits on every replay, with eager work
    between, and so do calls on another stream; each has its own workspace."""
    counts, n_out, k = [130, 0, 260, 7, 64], 320, 192
    d = data(B, dtype, counts, n_out, k, 11, True)
    dd = data(B, dtype, counts, n_out, k, 11, False)

    def outs():
        return [torch.full((d["room"], n_out), 0.5, dtype=T[dtype], device="cuda"),
                torch.full((d["room"], n_out), 0.5, dtype=T[dtype], device="cuda"),
                torch.full((d["room"], k), 0.5, dtype=T[dtype], device="cuda"),
                torch.full((5, n_out, k), 0.5, dtype=T[dtype], device="cuda"),
                torch.full((5, n_out), 0.5, dtype=T[dtype], device="cuda")]

    def run(o, ws, stream=None):
        B.grouped_linear(d["x"], d["offsets"], d["w"], o[0], row_index=d["index"], bias=d["bias"], silu=True,
                         pre=o[1], ws=ws, stream=stream)
        B.grouped_linear_input_grad(dd["dy"], d["offsets"], d["w"], o[2], pre=dd["z"], ws=ws, stream=stream)
        B.grouped_linear_weight_grad(dd["dy"], d["offsets"], d["x"], o[3], row_index=d["index"], dbias=o[4],
                                     ws=ws, stream=stream)

    def other_ws():
        return None if d["ws"] is None else torch.empty_like(d["ws"])

    ref, got, side = outs(), outs(), outs()
    run(ref, d["ws"])
    torch.cuda.synchronize()
    s, ws2, ws3 = torch.cuda.Stream(), other_ws(), other_ws()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(got, ws2)
    for _ in range(3):
        for t in got + side:
            t.fill_(0.5)
        torch.cuda.synchronize()
        g.replay()
        run(side, ws3, s)
        torch.cuda.synchronize()
        for a, b, c in zip(ref, got, side):
            assert torch.equal(a, b) and torch.equal(a, c)
        run(ref, d["ws"])


def steps_of_z():
    """Values before a SiLU, to where it leaves float32's normal numbers."""
    z = torch.cat([torch.linspace(-103.0, 100.0, 4000), torch.linspace(-3.0, 3.0, 1500), torch.tensor([0.0, -0.0]),
                   torch.logspace(-30, 30, 50), -torch.logspace(-30, 2, 42)])
    return torch.nn.functional.pad(z, (0, -len(z) % 16)).view(-1, 16).cuda()


def test_float32_silu_far_from_zero(B):
    """Rows through the identity, whose sums are exact.  With u = 2^-24: e = exp(-|z|) is within
    2.2 u, its product with z and 1 + e round by u each, the reciprocal is within 1.1 u and
    the last product rounds by u: 6.3 u of the value, which 6 and the store's own u cover;
    below the normal numbers e is off by 2^-149, times |z|."""
    z = steps_of_z()
    w = torch.eye(16, device="cuda").view(1, 16, 16).contiguous()
    off = torch.tensor([0, len(z)], dtype=torch.int32, device="cuda")
    n = B.grouped_linear_workspace_size("f32", 1, 16, 16, len(z))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    y, pre = torch.empty_like(z), torch.empty_like(z)
    B.grouped_linear(z, off, w, y, silu=True, pre=pre, ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(pre, z)
    v = f64(z)
    e = np.exp(-np.abs(v))
    ref = v * np.where(v >= 0, 1.0, e) / (1.0 + e)
    close(y, ref, 6 * U * np.abs(ref) + np.abs(v) * 2.0 ** -149, "y")


def test_float32_slope_far_from_zero(B):
    """Gradients of one through the identity.  With u = 2^-24: d = 1 / (1 + e) is within 3.2 u,
    e d within 6 u, the bracket within 5 u of its magnitudes and the product rounds by u: 12 u
    of s + |z| s (1 - s)."""
    z = steps_of_z()
    w = torch.eye(16, device="cuda").view(1, 16, 16).contiguous()
    off = torch.tensor([0, len(z)], dtype=torch.int32, device="cuda")
    n = B.grouped_linear_workspace_size("f32", 1, 16, 16, len(z))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    dx = torch.empty_like(z)
    B.grouped_linear_input_grad(torch.ones_like(z), off, w, dx, pre=z, ws=ws)
    torch.cuda.synchronize()
    v = f64(z)
    e = np.exp(-np.abs(v))
    d = 1.0 / (1.0 + e)
    s, rest = np.where(v >= 0, d, e * d), np.where(v >= 0, e * d, d)
    close(dx, s + v * s * rest, 12 * U * (s + np.abs(v) * s * rest) + (1 + np.abs(v)) * 2.0 ** -149, "dx")
