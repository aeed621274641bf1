"""MXFP4 quantisation and the grouped product on MXFP4 rows against the oracle:
codes, scale bytes and widened values bit for bit; products against float64 on
the values that the codes stand for.

The product's bound, per output: float32 sums of k exact products are off by at
most k * 2^-24 times the sum of magnitudes (each partial sum rounds once), SiLU
has a slope of at most 1.1 and the library's own about 2^-21 relative error, and
the store to bf16 rounds by 2^-8 relative."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sparse_mixture_experts_renormalised_amd import binding
    binding.lib()
    return binding


def quantize(B, x, wide=True):
    rows, d = x.shape
    codes = torch.full((rows, d // 2), 0x5A, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, d // 32), 0x5A, dtype=torch.uint8, device="cuda")
    w = torch.full((rows, d), 7.0, dtype=x.dtype, device="cuda") if wide else None
    B.quantize_mxfp4(x, codes, scales, w)
    torch.cuda.synchronize()
    return codes, scales, w


def check_quantized(x, codes, scales, w):
    c, s = oracle.quantize_mxfp4(x.double().cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), oracle.pack_mxfp4(c))
    if w is not None:
        ref = torch.from_numpy(oracle.dequantize_mxfp4(c, s)).to(x.dtype)
        got = w.cpu()
        assert torch.equal(got.isnan(), ref.isnan())
        assert torch.equal(got.nan_to_num(), ref.nan_to_num())


SHAPES = [(1, 32, 0), (1, 4096, 8), (3, 96, 8), (5, 32, 64), (7, 1408, 96), (300, 64, 0), (33, 7168, 8)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,d,pad", SHAPES)
def test_quantize(B, rows, d, pad, dtype):
    print(f"[mxfp4] quantize {rows}x{d}+{pad} {dtype}", flush=True)
    g = torch.Generator().manual_seed(rows * 131 + d)
    x = torch.randn(rows, d + pad, generator=g)
    # blocks of very different size, whole blocks of zeros, values on the format's borders
    x *= torch.exp2(torch.randint(-20, 20, (rows, (d + pad + 31) // 32), generator=g).float()
                    ).repeat_interleave(32, dim=1)[:, :d + pad]
    x[:, :32] = torch.randint(-24, 25, (rows, 32), generator=g) * 0.25
    if d > 32:
        x[-1, 32:64] = 0.0
    x = x.to(dtype).cuda()[:, :d]
    codes, scales, w = quantize(B, x)
    check_quantized(x, codes, scales, w)
    codes2, scales2, _ = quantize(B, x, wide=False)
    assert torch.equal(codes, codes2) and torch.equal(scales, scales2)


def test_quantize_every_bf16_value(B):
    # every finite bf16 as the largest of a block and as one of the others
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    v = bits[torch.isfinite(bits.float())]
    n = v.numel() // 32 * 32
    own = v[:n].view(-1, 32)                                    # neighbours in one block
    spread = v[:n].view(32, -1).t().contiguous()                # all binades in one block
    alone = torch.zeros(v.numel(), 32, dtype=torch.bfloat16)
    alone[:, 5] = v
    for name, x in (("own", own), ("spread", spread), ("alone", alone)):
        print(f"[mxfp4] every bf16 value: {name}", flush=True)
        x = x.cuda()
        check_quantized(x, *quantize(B, x))


def test_quantize_extreme_and_non_finite_blocks(B):
    big, tiny = float(np.finfo(np.float32).max), 2.0 ** -149
    x = torch.zeros(8, 64)
    x[0, 0], x[0, 1], x[0, 2] = big, -1.0, 1.74 * 2.0 ** 127
    x[1, 3], x[1, 4] = tiny, -tiny
    x[2, 1], x[2, 33] = float("inf"), 1.0
    x[3, 2] = float("nan")
    x[4, 40] = -float("inf")
    x[5, :] = 2.0 ** -126
    x[6, :] = -(2.0 ** -128)
    x[7, 0], x[7, 1] = 1.5 * 2.0 ** -125, 2.0 ** -130
    x = x.cuda()
    check_quantized(x, *quantize(B, x))


def test_quantize_more_elements_than_a_launch_takes(B):
    g = torch.Generator(device="cuda").manual_seed(8)
    block = torch.randn(4096, 2048, device="cuda", generator=g).bfloat16()
    n = 1025                                                    # 2^33 elements and a block more
    print("[mxfp4] quantize 8.6e9 elements", flush=True)
    x = block.repeat(n, 1)
    codes = torch.zeros(n * 4096, 1024, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(n * 4096, 64, dtype=torch.uint8, device="cuda")
    B.quantize_mxfp4(x, codes, scales)
    torch.cuda.synchronize()
    c, s, _ = quantize(B, block, wide=False)
    for i in range(n):
        assert torch.equal(codes[i * 4096:(i + 1) * 4096], c) and torch.equal(scales[i * 4096:(i + 1) * 4096], s), i


def mx_random(rng, rows, k, lo=-3, hi=3):
    codes = rng.integers(0, 16, (rows, k)).astype(np.uint8)
    scales = (127 + rng.integers(lo, hi, (rows, k // 32))).astype(np.uint8)
    return codes, scales


def run_linear(B, counts, n_out, k, index, silu, bias, seed=0, slack=3, tokens=None):
    rng = np.random.default_rng(seed)
    G, rows = len(counts), int(sum(counts))
    cap = rows + slack
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    src = tokens if index else cap
    xc, xs = mx_random(rng, src, k, -5, 1)
    wc, ws = mx_random(rng, G * n_out, k, -8, -2)
    idx = rng.integers(0, src, cap).astype(np.int32) if index else np.arange(cap, dtype=np.int32)
    b = torch.from_numpy(rng.normal(size=(G, n_out)).astype(np.float32)).bfloat16() if bias else None
    y = torch.full((cap, n_out), 123.0, dtype=torch.bfloat16, device="cuda")
    cu = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    need = B.grouped_linear_mxfp4_workspace_size(G, n_out, k, cap)
    args = dict(row_index=cu(idx) if index else None, bias=None if b is None else b.cuda(), silu=silu)
    dev = (cu(oracle.pack_mxfp4(xc)), cu(xs), cu(off), cu(oracle.pack_mxfp4(wc)).view(G, n_out, k // 2),
           cu(ws).view(G, n_out, k // 32))
    got = []
    for scratch in ([None, torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda")] if need else [None]):
        y.fill_(123.0)
        B.grouped_linear_mxfp4(*dev, y, ws=scratch, **args)
        torch.cuda.synchronize()
        got.append(y.double().cpu().numpy())
    X, Wt = oracle.dequantize_mxfp4(xc, xs)[idx], oracle.dequantize_mxfp4(wc, ws).reshape(G, n_out, k)
    for out in got:
        assert np.all(out[rows:] == 123.0)                      # rows behind the last group
        for g in range(G):
            a, z = off[g], off[g + 1]
            if a == z:
                continue
            ref, mag = X[a:z] @ Wt[g].T, np.abs(X[a:z]) @ np.abs(Wt[g]).T
            if b is not None:
                ref, mag = ref + b[g].double().numpy(), mag + np.abs(b[g].double().numpy())
            err = (k + 1) * 2.0 ** -24 * mag
            if silu:
                ref, err = oracle.silu(ref), 1.1 * err
                err = err + 2.0 ** -21 * np.abs(ref)
            err = err * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
            d = np.abs(out[a:z] - ref)
            assert np.all(d <= err), (g, float((d / err).max()))
    return got, dev, args


LINEAR = [
    # counts, n_out, k, index, silu, bias
    ([1], 8, 128, False, False, False),
    ([1], 64, 256, True, True, True),
    ([3, 0, 1, 5], 72, 384, True, False, True),
    ([0, 0, 17, 0], 40, 128, False, True, False),
    ([16, 33, 31], 136, 640, True, True, False),
    ([64, 65, 63, 0, 2], 264, 512, False, False, True),
    ([127, 128, 129], 256, 1408, True, True, True),
    ([255, 257, 256, 0, 1], 520, 256, True, False, False),
    ([513, 40], 248, 1024, False, True, True),
    ([300, 4, 0, 700], 1416, 2048, True, False, False),
    ([2] * 40 + [0] * 20 + [1] * 4, 512, 7168, True, True, False),
    ([0] * 5, 64, 128, False, False, False),
    ([0] * 1000 + [3] + [0] * 87, 16, 128, False, True, True),
    # small groups with tiles enough for all CUs, and the same with a third of them
    ([1, 2, 0, 7, 16, 17, 33, 64, 65, 8] * 12, 520, 384, True, True, True),
    ([1, 2, 0, 7, 16, 17, 33, 64, 65, 8] * 12, 248, 384, True, True, True),
    ([1] * 1088, 264, 128, False, False, False),
    ([0, 48] * 96, 256, 640, False, False, True),
    ([0, 16] * 96, 256, 640, True, False, False),
]


@pytest.mark.parametrize("case", LINEAR, ids=lambda c: f"{len(c[0])}g-{sum(c[0])}r-{c[1]}x{c[2]}")
def test_linear(B, case):
    counts, n_out, k, index, silu, bias = case
    print(f"[mxfp4] linear {counts[:6]}.. {n_out}x{k} index={index} silu={silu} bias={bias}", flush=True)
    run_linear(B, counts, n_out, k, index, silu, bias, seed=len(counts) + k, tokens=max(1, sum(counts) // 2))


@pytest.mark.parametrize("seed", range(8))
def test_linear_random(B, seed):
    rng = np.random.default_rng(100 + seed)
    G = int(rng.integers(1, 40))
    counts = (rng.integers(0, 2, G) * np.exp(rng.uniform(0, np.log(500), G))).astype(int).tolist()
    n_out, k = int(rng.integers(1, 150)) * 8, int(rng.integers(1, 20)) * 128
    print(f"[mxfp4] linear random {seed}: {counts} {n_out}x{k}", flush=True)
    run_linear(B, counts, n_out, k, bool(seed % 2), seed % 3 == 0, seed % 4 == 1, seed=seed, tokens=50,
               slack=int(rng.integers(0, 400)))


def test_linear_repeats_bit_exact_and_under_a_graph(B):
    counts = [300, 0, 5, 70]
    got, dev, args = run_linear(B, counts, 264, 768, True, True, True, seed=9, tokens=60)
    y = torch.zeros(sum(counts) + 3, 264, dtype=torch.bfloat16, device="cuda")
    need = B.grouped_linear_mxfp4_workspace_size(4, 264, 768, y.shape[0])
    ws = torch.empty(max(1, need), dtype=torch.uint8, device="cuda")
    B.grouped_linear_mxfp4(*dev, y, ws=ws, **args)
    torch.cuda.synchronize()
    ref = y.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.grouped_linear_mxfp4(*dev, y, ws=ws, **args)
    for _ in range(3):
        y.zero_()
        ws.fill_(0xFF)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y[:375], ref[:375]) and not y[375:].any()
        B.grouped_linear_mxfp4(*dev, y, ws=ws, **args)
        torch.cuda.synchronize()
        assert torch.equal(y[:375], ref[:375])


@pytest.mark.parametrize("rows", [5, 200])
def test_linear_nan_blocks_reach_their_outputs_only(B, rows):
    rng = np.random.default_rng(4)
    k, n_out = 256, 64
    xc, xs = mx_random(rng, rows, k)
    wc, ws = mx_random(rng, n_out, k)
    xs[3, 5] = 255                     # one row of x, one row of w
    ws[17, 0] = 255
    cu = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    y = torch.zeros(rows, n_out, dtype=torch.bfloat16, device="cuda")
    B.grouped_linear_mxfp4(cu(oracle.pack_mxfp4(xc)), cu(xs), cu(np.array([0, rows], dtype=np.int32)),
                           cu(oracle.pack_mxfp4(wc))[None], cu(ws)[None], y)
    torch.cuda.synchronize()
    nan = torch.zeros(rows, n_out, dtype=torch.bool)
    nan[3, :] = True
    nan[:, 17] = True
    assert torch.equal(y.isnan().cpu(), nan)


def test_quantize_then_two_linears_is_the_expert_ffn(B):
    """Quantise rows and weights, first Linear with SiLU through the row index,
    quantise the hidden rows, second Linear: the float64 FFN of what each step
    was given."""
    g = torch.Generator(device="cuda").manual_seed(3)
    T, d, f, counts = 40, 256, 384, [30, 0, 44, 6]
    G, rows = len(counts), sum(counts)
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")
    idx = torch.randint(0, T, (rows,), dtype=torch.int32, device="cuda", generator=g)
    x = torch.randn(T, d, device="cuda", generator=g).bfloat16()
    w1 = (torch.randn(G, f, d, device="cuda", generator=g) * d ** -0.5).bfloat16()
    w2 = (torch.randn(G, d, f, device="cuda", generator=g) * f ** -0.5).bfloat16()
    xc, xs, xw = quantize(B, x)
    c1, s1, v1 = quantize(B, w1.view(-1, d))
    c2, s2, v2 = quantize(B, w2.view(-1, f))
    h = torch.empty(rows, f, dtype=torch.bfloat16, device="cuda")
    B.grouped_linear_mxfp4(xc, xs, off, c1.view(G, f, -1), s1.view(G, f, -1), h, row_index=idx, silu=True)
    hc, hs, hw = quantize(B, h)
    y = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda")
    B.grouped_linear_mxfp4(hc, hs, off, c2.view(G, d, -1), s2.view(G, d, -1), y)
    torch.cuda.synchronize()
    o = off.tolist()
    for e in range(G):
        a, b = o[e], o[e + 1]
        z = xw[idx[a:b].long()].double() @ v1.view(G, f, d)[e].double().t()
        ref = z * torch.sigmoid(z)
        # half a bf16 step, and float32 sums of values of order one
        assert torch.all((h[a:b].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-4)
        ref = hw[a:b].double() @ v2.view(G, d, f)[e].double().t()
        assert torch.all((y[a:b].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-4)
    # against the unquantised FFN: each of the three quantisations is off by at
    # most half a step of a one-bit mantissa (1/4 relative for the smallest
    # codes, a tenth in the mean square), so the result keeps its direction
    for e in (0, 2):
        a, b = o[e], o[e + 1]
        z = x[idx[a:b].long()].double() @ w1[e].double().t()
        full = (z * torch.sigmoid(z)) @ w2[e].double().t()
        cos = torch.nn.functional.cosine_similarity(full.flatten(), y[a:b].double().flatten(), dim=0)
        assert cos > 0.9


@pytest.fixture(scope="module")
def long_codes():
    """2^20 - 1 rows of 8192 elements: just below the 4 GiB that the calls take."""
    g = torch.Generator(device="cuda").manual_seed(21)
    rows = (1 << 20) - 1
    codes = torch.randint(0, 256, (rows, 4096), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.randint(118, 124, (rows, 256), dtype=torch.uint8, device="cuda", generator=g)
    return codes, scales


def linear_reference(xc, xs, wc, ws):
    X = oracle.dequantize_mxfp4(oracle.unpack_mxfp4(xc.cpu().numpy()), xs.cpu().numpy())
    W = oracle.dequantize_mxfp4(oracle.unpack_mxfp4(wc.cpu().numpy()), ws.cpu().numpy())
    return X @ W.T, np.abs(X) @ np.abs(W).T


@pytest.mark.parametrize("rows", [5, 70])
def test_linear_rows_far_into_the_tokens(B, long_codes, rows):
    print(f"[mxfp4] {rows} rows out of 4 GiB", flush=True)
    codes, scales = long_codes
    idx = torch.linspace(0, codes.shape[0] - 1, rows, device="cuda", dtype=torch.float64).round().int()
    w, ws = codes[-4000:-3936].clone(), scales[-4000:-3936].clone()
    y = torch.zeros(rows, 64, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    B.grouped_linear_mxfp4(codes, scales, off, w[None], ws[None], y, row_index=idx)
    torch.cuda.synchronize()
    ref, mag = linear_reference(codes[idx.long()], scales[idx.long()], w, ws)
    err = 8193 * 2.0 ** -24 * mag
    assert np.all(np.abs(y.double().cpu().numpy() - ref) <= err * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref))


@pytest.mark.parametrize("rows", [3, 70])
def test_linear_features_far_into_a_matrix(B, long_codes, rows):
    print(f"[mxfp4] {rows} rows on a matrix of 4 GiB", flush=True)
    codes, scales = long_codes
    n_out = codes.shape[0] // 8 * 8
    x, xs = codes[-rows:].clone(), scales[-rows:].clone()
    y = torch.zeros(rows, n_out, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    B.grouped_linear_mxfp4(x, xs, off, codes[None, :n_out], scales[None, :n_out], y)
    torch.cuda.synchronize()
    for a in (0, (1 << 19) - 32, n_out - 64):
        ref, mag = linear_reference(x, xs, codes[a:a + 64], scales[a:a + 64])
        err = 8193 * 2.0 ** -24 * mag
        got = y[:, a:a + 64].double().cpu().numpy()
        assert np.all(np.abs(got - ref) <= err * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)), a


def test_quantise_and_linear_captured_beside_another_call(B):
    """Quantise and multiply, captured on one stream and replayed while another
    stream runs the same product eagerly: neither keeps anything between calls."""
    g = torch.Generator(device="cuda").manual_seed(5)
    counts, n_out, k = [70, 0, 3, 129, 20], 520, 768
    rows = sum(counts)
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")
    x = torch.randn(rows, k, device="cuda", generator=g).bfloat16()
    wc = torch.randint(0, 256, (5, n_out, k // 2), dtype=torch.uint8, device="cuda", generator=g)
    ws = torch.randint(118, 124, (5, n_out, k // 32), dtype=torch.uint8, device="cuda", generator=g)

    def buffers():
        return (torch.zeros(rows, k // 2, dtype=torch.uint8, device="cuda"),
                torch.zeros(rows, k // 32, dtype=torch.uint8, device="cuda"),
                torch.zeros(rows, n_out, dtype=torch.bfloat16, device="cuda"))

    def both(c, s, y, stream=None):
        B.quantize_mxfp4(x, c, s, stream=stream)
        B.grouped_linear_mxfp4(c, s, off, wc, ws, y, silu=True, stream=stream)

    one, two = buffers(), buffers()
    both(*one)
    torch.cuda.synchronize()
    ref = one[2].clone()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(*one)
    for _ in range(4):
        one[2].zero_()
        two[2].zero_()
        torch.cuda.synchronize()
        graph.replay()
        both(*two, stream=side)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(one[2], ref) and torch.equal(two[2], ref)
