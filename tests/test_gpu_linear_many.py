"""The single Linears and their gradients where a workgroup takes several tiles, where sums
are split, and where offsets pass 32 bits, against float64 products on the GPU.

Bounds as for the small cases: float32 sums of n products are off by at most
(n + 4) 2^-24 times the sum of magnitudes (parts of split sums hold 256 terms or more
each, so that adding them rounds less often than n), and a store to bf16 rounds by
2^-8 relative, one to float32 by 2^-24.  The SiLU's slope is at most 1.1 and within
2^-19 (1 + |z|) of its own size (for z that normal rows reach)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
U = 2.0 ** -24


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sparse_mixture_experts_renormalised_amd import binding
    binding.lib()
    return binding


def close(got, ref, bound, what):
    g = got.double()
    assert g.isfinite().all(), what
    over = (g - ref).abs() - (bound + HALF[got.dtype] * (ref.abs() + bound))
    assert not over.numel() or over.max() <= 0, f"{what}: beyond its bound by {over.max().item():.3e}"


class Data:
    def __init__(self, B, counts, n_out, k, seed, tokens=0, dtype=BF16):
        """tokens: rows of a gathered x (0: x has the groups' rows)."""
        g = torch.Generator(device="cuda").manual_seed(seed)
        off = [0]
        for c in counts:
            off.append(off[-1] + c)
        self.off, self.n_out, self.k, self.G, rows = off, n_out, k, len(counts), off[-1]

        def normal(*shape, std=1.0):
            return torch.randn(*shape, generator=g, device="cuda").mul_(std).to(dtype)

        self.rows, room = rows, rows + 3
        self.x, self.dy, self.z = normal(tokens or room, k), normal(room, n_out), normal(room, k)
        self.w = normal(self.G, n_out, k, std=k ** -0.5)
        self.index = None
        if tokens:
            self.index = torch.randint(0, tokens, (room,), generator=g, dtype=torch.int32, device="cuda")
            self.index[:min(2, rows)] = tokens - 1           # the last row, and it twice
        else:
            self.x[rows:] = float("nan")
        self.dy[rows:] = float("nan")
        self.z[rows:] = float("nan")
        self.offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
        n = B.grouped_linear_workspace_size("bf16" if dtype == BF16 else "f32", self.G, n_out, k, room)
        self.ws = torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda") if n else None

    def source(self, g):
        a, b = self.off[g], self.off[g + 1]
        return self.x[a:b] if self.index is None else self.x[self.index[a:b].long()]


def check_weight_grad(B, d, out, accumulate=False, columns=None):
    old = 3.0 if accumulate else float("nan")
    dw = torch.full((d.G, d.n_out, d.k), old, dtype=out, device="cuda")
    db = torch.full((d.G, d.n_out), old, dtype=out, device="cuda")
    B.grouped_linear_weight_grad(d.dy, d.offsets, d.x, dw, row_index=d.index, dbias=db, accumulate=accumulate, ws=d.ws)
    torch.cuda.synchronize()
    add = 3.0 if accumulate else 0.0
    for g in range(d.G):
        dy, x = d.dy[d.off[g]:d.off[g + 1]].double(), d.source(g).double()
        n = dy.shape[0]
        ref, mag = dy.t().contiguous() @ x, dy.abs().t().contiguous() @ x.abs()
        extra = U * (ref.abs() + add) if accumulate else 0.0
        close(dw[g], ref + add, (n + 4) * U * mag + extra, f"dw of group {g}")
        rb = dy.sum(0)
        extra = U * (rb.abs() + add) if accumulate else 0.0
        close(db[g], rb + add, (n + 4) * U * dy.abs().sum(0) + extra, f"dbias of group {g}")


def check_input_grad(B, d, pre):
    dx = torch.full((d.rows + 3, d.k), 0.5, dtype=d.w.dtype, device="cuda")
    B.grouped_linear_input_grad(d.dy, d.offsets, d.w, dx, pre=d.z if pre else None, ws=d.ws)
    torch.cuda.synchronize()
    assert (dx[d.rows:] == 0.5).all()
    for g in range(d.G):
        a, b = d.off[g], d.off[g + 1]
        dy, w = d.dy[a:b].double(), d.w[g].double()
        ref, bound = dy @ w, (d.n_out + 4) * U * (dy.abs() @ w.abs())
        if pre:
            z = d.z[a:b].double()
            s = torch.sigmoid(z)
            slope = s + z * s * (1 - s)
            # the slope's own error is absolute where its two terms cancel
            bound = 1.1 * bound + 2.0 ** -19 * (1 + z.abs()) * ref.abs() * (s + (z * s * (1 - s)).abs())
            ref = ref * slope
        close(dx[a:b], ref, bound, f"dx of group {g}")


def check_forward(B, d, bias, silu, pre):
    dt = d.w.dtype
    y, z = (torch.full((d.rows + 3, d.n_out), 0.5, dtype=dt, device="cuda") for _ in range(2))
    b = torch.randn(d.G, d.n_out, device="cuda").to(dt) if bias else None
    B.grouped_linear(d.x, d.offsets, d.w, y, row_index=d.index, bias=b, silu=silu, pre=z if pre else None, ws=d.ws)
    torch.cuda.synchronize()
    assert (y[d.rows:] == 0.5).all() and (z[d.rows:] == 0.5).all()
    for g in range(d.G):
        a, e = d.off[g], d.off[g + 1]
        x, w = d.source(g).double(), d.w[g].double().t().contiguous()
        add = b[g].double() if bias else torch.zeros(d.n_out, dtype=torch.float64, device="cuda")
        ref, bound = x @ w + add, (d.k + 4) * U * (x.abs() @ w.abs() + add.abs())
        if pre:
            close(z[a:e], ref, bound, f"pre of group {g}")
        if silu:
            ref = ref * torch.sigmoid(ref)
            bound = 1.1 * bound + 2.0 ** -19 * (1 + (x @ w + add).abs()) * ref.abs()
        close(y[a:e], ref, bound, f"y of group {g}")


SHORT = [0, 1, 31, 32, 33, 64, 97, 128, 130, 5]
WEIGHT = [
    # counts, n_out, k: short tiles after another, long ones, groups of very different lengths
    (SHORT * 20, 320, 320),
    ([900, 0, 1700], 2560, 2560),
    ([1] * 70 + [4000] + [0] * 30 + [33] * 90, 256, 832),
    ([511, 513] * 40 + [0, 2], 576, 448),
    ([9000, 700, 0, 1300, 64, 5000, 33, 1], 1088, 832),   # lengths far apart
    ([40] * 60 + [3000] + [20] * 100, 320, 320),
]
SPLIT = [([5000], 128, 192), ([4000, 3, 0, 900], 256, 320), ([2600, 2601], 448, 64)]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("out,accumulate", [(BF16, False), (F32, False), (BF16, True), (F32, True)])
@pytest.mark.parametrize("n", range(len(WEIGHT) + len(SPLIT)))
def test_weight_grad(B, n, out, accumulate, gather):
    counts, n_out, k = (WEIGHT + SPLIT)[n]
    print(f"[linear] weight gradient {n} {out} {accumulate} {gather}", flush=True)
    check_weight_grad(B, Data(B, counts, n_out, k, 40 + n, sum(counts) // 2 if gather else 0), out, accumulate)


INPUT = [
    (SHORT * 20, 64, 512),
    ([700, 0, 256, 257, 3, 511] * 6, 576, 1088),
    ([5, 300, 0, 1], 4096, 256),
    ([256 * 30], 2048, 320),
    ([1] * 1088, 64, 64),
]


@pytest.mark.parametrize("pre", [False, True])
@pytest.mark.parametrize("n", range(len(INPUT)))
def test_input_grad(B, n, pre):
    counts, n_out, k = INPUT[n]
    print(f"[linear] input gradient {n} {pre}", flush=True)
    check_input_grad(B, Data(B, counts, n_out, k, 60 + n), pre)


FORWARD = [
    ([700, 0, 256, 257, 3, 511] * 6, 576, 1088),
    ([138], 128, 5376),                      # split along the sum
    ([1221, 0, 900], 320, 2048),
    ([512] * 60 + [0, 1, 513], 256, 448),
    ([65] * 90 + [0, 200], 192, 64),         # two steps
    ([640, 641, 639], 2304, 128),
]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("bias,silu,pre", [(False, False, False), (True, False, False), (False, True, False), (True, True, True)])
@pytest.mark.parametrize("n", range(len(FORWARD)))
def test_forward(B, n, bias, silu, pre, gather):
    counts, n_out, k = FORWARD[n]
    print(f"[linear] forward {n} {bias} {silu} {pre} {gather}", flush=True)
    check_forward(B, Data(B, counts, n_out, k, 90 + n, sum(counts) // 2 if gather else 0), bias, silu, pre)


# few tiles and long sums in float32: counts, n_out, k
LONG = [([2967], 80, 208), ([700, 0, 3, 5000, 12], 48, 112), ([1988], 1808, 80), ([5, 0, 70, 130], 2048, 2032),
        ([1], 64, 16384), ([64, 1], 16400, 16)]


@pytest.mark.parametrize("n", range(len(LONG)))
def test_float32_split(B, n):
    counts, n_out, k = LONG[n]
    print(f"[linear] float32 split {n}", flush=True)
    d = Data(B, counts, n_out, k, 80 + n, sum(counts) // 2 + 1 if n % 2 else 0, F32)
    assert d.ws is not None
    check_weight_grad(B, d, F32)
    check_weight_grad(B, d, F32, True)
    check_input_grad(B, d, n % 2 == 0)
    check_forward(B, d, True, True, True)


def test_widths_beyond_the_tiles(B):
    """A width of 2^20, which the float32 kernel takes."""
    d = Data(B, [3, 0, 2], 64, 1 << 20, 71)
    check_weight_grad(B, d, BF16)
    check_input_grad(B, d, True)


def test_gathered_rows_beyond_4_gib(B):
    d = Data(B, [40, 0, 3], 64, 65536, 72, tokens=33000)
    check_weight_grad(B, d, F32)
    y = torch.full((d.rows + 3, 64), 0.5, dtype=BF16, device="cuda")
    B.grouped_linear(d.x, d.offsets, d.w, y, row_index=d.index, ws=d.ws)
    torch.cuda.synchronize()
    assert (y[d.rows:] == 0.5).all()
    for g in range(3):
        x, w = d.source(g).double(), d.w[g].double().t().contiguous()
        close(y[d.off[g]:d.off[g + 1]], x @ w, (d.k + 4) * U * (x.abs() @ w.abs()), f"y of group {g}")


def test_rows_beyond_4_gib(B):
    """Weight gradients, input gradients and outputs whose arrays pass 4 GiB: the last
    group's rows lie there."""
    k, n_out, rows = 2048, 64, (1 << 20) + 70000
    x = torch.zeros(rows, k, dtype=BF16, device="cuda")
    dy = torch.zeros(rows, n_out, dtype=BF16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(73)
    last = 300
    x[-last:] = torch.randn(last, k, generator=g, device="cuda").to(BF16)
    dy[-last:] = torch.randn(last, n_out, generator=g, device="cuda").to(BF16)
    w = torch.randn(2, n_out, k, generator=g, device="cuda").to(BF16)
    off = torch.tensor([0, rows - last, rows], dtype=torch.int32, device="cuda")
    n = B.grouped_linear_workspace_size("bf16", 2, n_out, k, rows)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    dw = torch.full((2, n_out, k), float("nan"), dtype=F32, device="cuda")
    B.grouped_linear_weight_grad(dy, off, x, dw, ws=ws)
    xs, ds, ww = x[-last:].double(), dy[-last:].double(), w[1].double()
    assert (dw[0] == 0).all()
    close(dw[1], ds.t().contiguous() @ xs, (last + 4) * U * (ds.abs().t().contiguous() @ xs.abs()), "dw")
    dx = x.fill_(0.5)
    B.grouped_linear_input_grad(dy, off, w, dx, ws=ws)
    torch.cuda.synchronize()
    assert (dx[:1000] == 0).all() and (dx[-last - 1000:-last] == 0).all()
    close(dx[-last:], ds @ ww, (n_out + 4) * U * (ds.abs() @ ww.abs()), "dx")


def test_long_sums_of_gathered_rows_beyond_4_gib(B):
    """Thousands of gathered rows from an x of more than 4 GiB, few tiles: the sums are split,
    here as well as where x is smaller."""
    d = Data(B, [5000, 0, 700], 64, 8192, 74, tokens=262144 + 5)
    assert d.x.numel() * 2 > 1 << 32
    check_weight_grad(B, d, F32)
    check_weight_grad(B, d, BF16, True)


def one_large(n, device="cuda"):
    """2^26 and then ones: beside the first, a one is below half a step of float32 (8), so that
    a sum in order loses every one, and a split sum those of its first part alone."""
    v = torch.ones(n, dtype=BF16, device=device)
    v[0] = 2.0 ** 26
    return v


def test_parts_of_sums_of_gathered_rows_beyond_4_gib(B):
    rows, n_out, k, tokens = 8000, 64, 8192, 262144 + 5
    x = torch.zeros(tokens, k, dtype=BF16, device="cuda")
    x[-rows:] = one_large(rows)[:, None]
    index = torch.arange(tokens - rows, tokens, dtype=torch.int32, device="cuda")
    dy = torch.ones(rows, n_out, dtype=BF16, device="cuda")
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    dw = torch.empty(1, n_out, k, dtype=F32, device="cuda")
    ws = torch.empty(B.grouped_linear_workspace_size("bf16", 1, n_out, k, rows), dtype=torch.uint8, device="cuda")
    B.grouped_linear_weight_grad(dy, off, x, dw, row_index=index, ws=ws)
    torch.cuda.synchronize()
    lost = 2.0 ** 26 + rows - 1 - dw.double()
    # the ones of the first part, of a quarter of the rows at most, and half a step of each sum of parts
    assert lost.abs().max() <= rows / 4 + 4 * 64


def test_parts_of_sums_over_a_wide_output(B):
    """A sum over 2^20 output features in one tile of the input gradient."""
    rows, n_out, k = 3, 1 << 20, 64
    dy = one_large(n_out).expand(rows, n_out).contiguous()
    w = torch.ones(1, n_out, k, dtype=BF16, device="cuda")
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    dx = torch.empty(rows, k, dtype=BF16, device="cuda")
    ws = torch.empty(B.grouped_linear_workspace_size("bf16", 1, n_out, k, rows), dtype=torch.uint8, device="cuda")
    B.grouped_linear_input_grad(dy, off, w, dx, ws=ws)
    torch.cuda.synchronize()
    # what is exact rounds to bf16, in steps of 2^19: 2^26 + 2^20 - 1 to 2^26 + 2^20
    assert (dx.double() == 2.0 ** 26 + 2.0 ** 20).all()


# forward calls that go through the layer's kernels: counts, n_out, k, rows of a gathered x
LAYER = [
    # more than 512 rows a group and many tiles: ends of 128 and of 64 rows and less, a last
    # round in halves, and (from 4096 terms on) along the sum
    ([600, 700, 513, 0, 900, 1025, 640, 1000], 2880, 192, 2500),
    ([600, 700, 513, 0, 900, 1025, 640, 1000], 2880, 4096, 2500),
    # few rows a group on average, and some groups with many
    ([5] * 60 + [200, 300, 129, 128], 320, 256, 700),
    ([5] * 60 + [200, 300, 129, 128], 1024, 4096, 700),
    # few rows, a last round along the sum
    ([20] * 290 + [0] * 10 + [40], 512, 1024, 3000),
    # an x of more than 4 GiB
    ([600] * 8, 2880, 8192, 262144 + 9),
]


@pytest.mark.parametrize("bias,silu,pre", [(False, True, True), (True, True, True), (True, True, False), (True, False, False)])
@pytest.mark.parametrize("n,gather", [(n, g) for n in range(len(LAYER)) for g in (False, True) if g or LAYER[n][3] < 1 << 18])
def test_forward_through_the_layers_kernels(B, n, gather, bias, silu, pre):
    counts, n_out, k, tokens = LAYER[n]
    print(f"[linear] layer's kernels {n} {gather} {bias} {silu} {pre}", flush=True)
    check_forward(B, Data(B, counts, n_out, k, 110 + n, tokens if gather else 0), bias, silu, pre)


@pytest.mark.parametrize("counts,n_out,k", [([3, 0, 2], 64, 1 << 20), ([3, 0, 2], 1 << 20, 64), ([2, 130], 1 << 20, 64)])
def test_forward_of_wide_rows(B, counts, n_out, k):
    print(f"[linear] forward {counts} {k}->{n_out}", flush=True)
    check_forward(B, Data(B, counts, n_out, k, 75), True, True, True)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("long", [3, 400])
def test_as_many_groups_as_there_may_be(B, dtype, long):
    """1088 groups: the last of them with rows, most of one row or none, the first one long."""
    counts = [long] + [g % 3 % 2 for g in range(1085)] + [0, 5]
    print(f"[linear] 1088 groups {dtype} {long}", flush=True)
    d = Data(B, counts, 64, 128, 120, sum(counts) // 2, dtype)
    check_weight_grad(B, d, F32)
    check_weight_grad(B, d, dtype, True)
    check_input_grad(B, d, True)
    check_forward(B, d, True, True, True)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("gather", [False, True])
def test_no_rows_of_wide_weights(B, gather, out):
    """Weight gradients without a row, of more tiles than the CUs take at once: zeros."""
    none = torch.empty(0, 2048, dtype=BF16, device="cuda")
    x = torch.full((3, 1408), float("nan"), dtype=BF16, device="cuda")
    off = torch.zeros(10, dtype=torch.int32, device="cuda")
    index = torch.empty(0, dtype=torch.int32, device="cuda") if gather else None
    dw = torch.full((9, 2048, 1408), float("nan"), dtype=out, device="cuda")
    db = torch.full((9, 2048), float("nan"), dtype=out, device="cuda")
    ws = torch.empty(B.grouped_linear_workspace_size("bf16", 9, 2048, 1408, 0), dtype=torch.uint8, device="cuda")
    B.grouped_linear_weight_grad(none, off, x, dw, row_index=index, dbias=db, ws=ws)
    torch.cuda.synchronize()
    assert (dw == 0).all() and (db == 0).all()
