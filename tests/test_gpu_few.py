"""The few-token layer (moe_layer_forward_few, _few_mxfp4) against the oracle's
layer in float64, against moe_layer_forward, and where it can go wrong: every
token count, capacity drops, all tokens on one expert, equal logits, garbage in
the workspace, two calls at once, captured graphs.

Bound of an output, with A the sum over the paths of |gate| |W2| (|h| + 1.1
|W1||x|) (how far errors of hidden values and of the sums reach): the hidden
values keep 16 bits (2^-16), float32 sums of n = d + f terms are off by at most
n * 2^-24 of their magnitudes, a gate by 1e-6, and the store to bf16 rounds by
2^-8 relative (float32: 2^-24)."""
import numpy as np
import pytest
import torch

import oracle
import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sparse_mixture_experts_renormalised_amd import binding
    binding.lib()
    return binding


class Few:
    """A layer on the GPU with its outputs and workspace."""

    def __init__(self, B, T, d, N, K, Ks, f, kind="bf16", cap=0.0, bias=False, router="none", seed=0,
                 scale=1.0, spread=0):
        self.B, self.kind = B, kind
        self.cfg = B.config(T, d, N, K, Ks, f, "f32" if kind == "f32" else "bf16", cap,
                            selection_only_bias=router == "select")
        dt = torch.float32 if kind == "f32" else torch.bfloat16
        self.act, self.shape, self.cap, self.router = dt, (T, d, N, K, Ks, f), cap, router
        g = torch.Generator(device="cuda").manual_seed(seed)
        rn = lambda *s, std=1.0: torch.randn(*s, device="cuda", generator=g) * std  # noqa: E731
        self.wr = rn(N, d, std=d ** -0.5)
        self.rb = None if router == "none" else rn(N, std=0.7)
        # tokens whose kept logits are further apart than their rounding
        x = rn(40 * T + 40, d, std=scale)
        if spread:                          # elements of very different size within a block
            x = x * torch.exp2(-torch.randint(0, spread, x.shape, device="cuda", generator=g).float())
        x = x.to(dt)
        key = x.double() @ self.wr.double().t() + (0 if self.rb is None else self.rb.double())
        top = key.sort(dim=1, descending=True).values[:, : K + 1]
        far = ((top[:, :-1] - top[:, 1:]) > 1e-5).all(dim=1) if N > 1 else torch.ones(len(x), dtype=torch.bool, device="cuda")
        self.x = x[far][:T].contiguous()
        assert len(self.x) == T
        self.w = {}
        for p, n in (("", N), ("s", Ks)):
            for lin, rows, cols in (("1", f, d), ("2", d, f)):
                m = rn(n, rows, cols, std=cols ** -0.5).to(dt) if n else None
                b = rn(n, rows, std=cols ** -0.5).to(dt) if n and bias else None
                if kind == "mxfp4" and n:
                    c = torch.empty(n * rows, cols // 2, dtype=torch.uint8, device="cuda")
                    s = torch.empty(n * rows, cols // 32, dtype=torch.uint8, device="cuda")
                    v = torch.empty(n * rows, cols, dtype=dt, device="cuda")
                    B.quantize_mxfp4(m.view(-1, cols), c, s, v)
                    self.w["c" + p + lin], self.w["k" + p + lin] = c, s
                    m = v.view(n, rows, cols)
                self.w["w" + p + lin], self.w["b" + p + lin] = m, b
        w = self.w
        if kind == "mxfp4":
            flat = []
            for p in ("", "s"):
                for lin in "12":
                    flat += [w.get("c" + p + lin), w.get("k" + p + lin), w["b" + p + lin]]
            self.table = B.weights_mxfp4(self.wr, self.rb, *flat)
            self.fn = B.layer_forward_few_mxfp4
        else:
            self.table = B.weights(self.wr, self.rb, *[w[a + p + lin] for p in ("", "s") for lin in "12"
                                                       for a in ("w", "b")])
            self.fn = B.layer_forward_few
        self.y = torch.full((T, d), float("nan"), dtype=dt, device="cuda")
        self.idx = torch.full((T, K), -1, dtype=torch.int32, device="cuda")
        self.gate = torch.full((T, K), float("nan"), device="cuda")
        self.counts = torch.full((N,), -1, dtype=torch.int32, device="cuda")
        self.ws = torch.full((B.few_workspace_size(self.cfg),), 0xFF, dtype=torch.uint8, device="cuda")

    def __call__(self, stream=None):
        self.fn(self.cfg, self.table, self.x, self.y, self.idx, self.gate, self.counts, self.ws, stream)

    def outputs(self):
        return [t.clone() for t in (self.y, self.idx, self.gate, self.counts)]

    def spoil(self):
        self.y.fill_(float("nan"))
        self.idx.fill_(-1)
        self.gate.fill_(float("nan"))
        self.counts.fill_(-1)
        self.ws.fill_(0xFF)

    def reference(self):
        T, d, N, K, Ks, f = self.shape
        h = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
        w = self.w

        def ex(p, e):
            return tuple(None if w[a + p + lin] is None else h(w[a + p + lin][e])
                         for lin in "12" for a in ("w", "b"))

        ref = oracle.layer_forward(self.x.float().cpu().numpy(), self.wr.cpu().numpy(),
                                   None if self.rb is None else self.rb.cpu().numpy(),
                                   lambda e: ex("", e), lambda i: ex("s", i), top_k=K, n_shared=Ks,
                                   capacity_factor=self.cap, selection_only_bias=self.router == "select")
        x, A = h(self.x), np.zeros((T, d))

        def reach(t, e4, g):
            w1, b1, w2, b2 = e4
            hid = np.abs(oracle.silu(w1 @ x[t] + (0 if b1 is None else b1)))
            hid = hid + 1.1 * (np.abs(w1) @ np.abs(x[t]) + (0 if b1 is None else np.abs(b1)))
            return g * (np.abs(w2) @ hid + (0 if b2 is None else np.abs(b2)))

        for t in range(T):
            for i in range(Ks):
                A[t] += reach(t, ex("s", i), 1.0)
            for k in range(K):
                if ref["slot_row"][t, k] >= 0:
                    A[t] += reach(t, ex("", int(ref["topk_idx"][t, k])), ref["gates"][t, k])
        return ref, A

    def bound(self, ref, A):
        T, d, N, K, Ks, f = self.shape
        last = 2.0 ** -24 if self.kind == "f32" else 2.0 ** -8
        # hidden rows: two bf16 parts leave 2^-8 of 2^-8, three E4M3 parts 2^-4 of
        # 2^-4 of 2^-4 (half a step of four significant bits each)
        hidden = {"f32": 0, "bf16": 2.0 ** -16, "mxfp4": 2.0 ** -12}[self.kind]
        return last * np.abs(ref["y"]) + (hidden + (d + f) * 2.0 ** -24 + 2e-6) * A * (1 + last)

    def check(self, label=""):
        ref, A = self.reference()
        assert np.array_equal(self.idx.cpu().numpy(), ref["topk_idx"]), label
        assert np.array_equal(self.counts.cpu().numpy(), ref["counts"]), label
        assert np.abs(self.gate.double().cpu().numpy() - ref["gates"]).max() <= 2e-6, label
        tol = self.bound(ref, A)
        diff = np.abs(self.y.double().cpu().numpy() - ref["y"])
        assert np.all(diff <= tol), (label, float(np.max(diff / np.maximum(tol, 1e-300))))
        if np.linalg.norm(ref["y"]):
            rel = np.linalg.norm(diff) / np.linalg.norm(ref["y"])
            print(f"[few] {label} rel_l2={rel:.2e}", flush=True)
            # no more than one rounding to the output's type, and float32 sums
            assert rel <= (2e-6 if self.kind == "f32" else 2.0 ** -8)


LAYERS = [
    # T, d, N, K, Ks, f, kind, cap, bias, router
    (1, 64, 1, 1, 0, 64, "bf16", 0.0, False, "none"),
    (1, 128, 4, 2, 0, 128, "mxfp4", 0.0, False, "none"),
    (1, 16, 3, 1, 0, 16, "f32", 0.0, True, "gauss"),
    (2, 64, 8, 2, 1, 192, "bf16", 0.0, True, "none"),
    (3, 256, 8, 3, 2, 384, "mxfp4", 0.0, True, "select"),
    (5, 144, 6, 2, 1, 80, "f32", 1.0, True, "select"),
    (7, 320, 16, 4, 1, 64, "bf16", 1.25, False, "gauss"),
    (8, 2048, 64, 8, 2, 1408, "bf16", 0.0, False, "none"),
    (11, 640, 32, 8, 1, 256, "mxfp4", 1.25, False, "gauss"),
    (16, 64, 4, 4, 0, 64, "bf16", 0.0, False, "none"),
    (16, 128, 2, 1, 1, 640, "mxfp4", 1.0, True, "gauss"),
    (16, 1024, 8, 2, 0, 2048, "mxfp4", 0.0, False, "none"),
    (16, 512, 300, 8, 1, 128, "bf16", 0.5, True, "select"),
    (16, 64, 1024, 64, 1, 64, "bf16", 0.0, False, "none"),
    (4, 1008, 20, 5, 3, 400, "f32", 0.0, False, "none"),
    (16, 128, 64, 2, 64, 64, "bf16", 0.0, False, "none"),
]


@pytest.mark.parametrize("case", LAYERS, ids=lambda c: f"{c[6]}-T{c[0]}-d{c[1]}-N{c[2]}-K{c[3]}-s{c[4]}-f{c[5]}")
def test_few_layers(B, case):
    print(f"[few] {case}", flush=True)
    L = Few(B, *case, seed=case[0] + case[1])
    L()
    torch.cuda.synchronize()
    L.check(str(case))
    first = L.outputs()
    L.spoil()
    L()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, L.outputs()))


@pytest.mark.parametrize("kind", ["bf16", "mxfp4", "f32"])
@pytest.mark.parametrize("T", range(1, 17))
def test_every_token_count(B, T, kind):
    print(f"[few] T={T} {kind}", flush=True)
    L = Few(B, T, 256, 10, 3, 1, 384, kind, seed=T)
    L()
    torch.cuda.synchronize()
    L.check(f"T={T} {kind}")


@pytest.mark.parametrize("seed", range(12))
def test_random_few_layers(B, seed):
    rng = np.random.default_rng(700 + seed)
    kind = ["bf16", "mxfp4", "f32"][seed % 3]
    step = {"bf16": 64, "mxfp4": 128, "f32": 16}[kind]
    N = int(np.exp(rng.uniform(0, np.log(200))))
    case = (int(rng.integers(1, 17)), step * int(rng.integers(1, 12)), N, int(rng.integers(1, min(N, 8) + 1)),
            int(rng.integers(0, 3)), step * int(rng.integers(1, 12)), kind,
            float(rng.choice([0.0, 0.5, 1.25])), bool(rng.integers(0, 2)),
            ["none", "gauss", "select"][int(rng.integers(0, 3))])
    print(f"[few] random {seed}: {case}", flush=True)
    L = Few(B, *case, seed=seed)
    L()
    torch.cuda.synchronize()
    L.check(f"random {seed}")


def test_no_capacity_leaves_the_shared_experts(B):
    for Ks in (0, 1):
        L = Few(B, 6, 128, 8, 2, Ks, 128, "bf16", seed=5)
        L.cfg.capacity = 0
        L()
        torch.cuda.synchronize()
        assert not L.counts.any()
        x = L.x.double()
        ref = torch.zeros_like(x)
        if Ks:
            z = x @ L.w["ws1"][0].double().t()
            ref = (z * torch.sigmoid(z)) @ L.w["ws2"][0].double().t()
        assert torch.all((L.y.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-4)


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
def test_all_tokens_on_one_expert_and_equal_logits(B, kind):
    # zero router weights: every logit equal, the lowest ids win with equal gates
    L = Few(B, 16, 128, 12, 3, 0, 128, kind, seed=6)
    L.wr.zero_()
    L()
    torch.cuda.synchronize()
    assert torch.equal(L.idx.cpu(), torch.arange(3, dtype=torch.int32).expand(16, 3))
    assert torch.all((L.gate - 1.0 / 3.0).abs() <= 1e-7)
    assert L.counts.tolist() == [16, 16, 16] + [0] * 9
    L.check(f"equal logits {kind}")
    # one expert far above the others, and a limit of five rows
    L = Few(B, 16, 128, 12, 1, 0, 128, kind, router="gauss", seed=7)
    L.rb[9] = 100.0
    L.cfg.capacity = 5
    L()
    torch.cuda.synchronize()
    assert L.idx.flatten().tolist() == [9] * 16 and int(L.counts[9]) == 5
    assert not L.y[5:].any() and L.y[:5].float().abs().sum(dim=1).min() > 0


def test_logits_that_are_not_numbers_keep_the_selection_in_range(B):
    L = Few(B, 4, 128, 10, 4, 1, 128, "bf16", router="gauss", seed=8)
    L.rb[3] = float("nan")
    L.rb[5] = -float("inf")
    L.x[2] = float("nan")
    L.x[1, 7] = float("inf")
    L()
    torch.cuda.synchronize()
    ids = L.idx.cpu().numpy()
    assert ((ids >= 0) & (ids < 10)).all()
    assert all(len(set(r)) == 4 for r in ids.tolist())


def test_optional_outputs(B):
    L = Few(B, 5, 256, 8, 2, 1, 128, "bf16", seed=9)
    L()
    torch.cuda.synchronize()
    y = L.y.clone()
    L.spoil()
    B.layer_forward_few(L.cfg, L.table, L.x, L.y, ws=L.ws)
    torch.cuda.synchronize()
    assert torch.equal(L.y, y) and (L.idx == -1).all() and (L.counts == -1).all()


def test_against_the_general_layer(B):
    wl = W.custom_workload("few_general", T=12, d_model=512, n_routed=32, top_k=4, n_shared=1, d_ff=256,
                           dtype="bf16", router_bias="zipf", zipf_s=1.1, capacity_factor=1.25)
    import workloads.device
    dl = workloads.device.DeviceLayer(wl)
    dl.forward()
    y = torch.empty_like(dl.y)
    idx, counts = torch.empty_like(dl.topk_idx), torch.empty_like(dl.counts)
    ws = torch.empty(B.few_workspace_size(dl.cfg), dtype=torch.uint8, device="cuda")
    B.layer_forward_few(dl.cfg, dl.weights, dl.x, y, idx, None, counts, ws)
    torch.cuda.synchronize()
    assert torch.equal(idx, dl.topk_idx) and torch.equal(counts, dl.counts)
    # the general layer rounds hidden rows and expert outputs to bf16 as well
    assert float((y.double() - dl.y.double()).norm() / dl.y.double().norm()) <= 2.0 ** -7


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
def test_captured_calls_replay_equal(B, kind):
    L = Few(B, 9, 512, 16, 4, 1, 640, kind, seed=10)
    L()
    torch.cuda.synchronize()
    ref = L.outputs()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L(torch.cuda.current_stream())
        L(torch.cuda.current_stream())      # twice in a row in one workspace
    for _ in range(3):
        L.spoil()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, L.outputs()))
        L()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, L.outputs()))


def test_two_layers_on_two_streams(B):
    # both larger than half the chip, so that neither is fully resident beside the other
    a = Few(B, 8, 2048, 64, 8, 2, 1408, "bf16", seed=11)
    b = Few(B, 16, 2048, 32, 4, 1, 2048, "mxfp4", seed=12)
    refs = []
    for L in (a, b):
        L()
        torch.cuda.synchronize()
        refs.append(L.outputs())
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        a.spoil()
        b.spoil()
        torch.cuda.synchronize()
        for _ in range(4):
            a(s1)
            b(s2)
        torch.cuda.synchronize()
        for L, ref in ((a, refs[0]), (b, refs[1])):
            assert all(torch.equal(p, q) for p, q in zip(ref, L.outputs()))


def test_repeats_bit_exact(B):
    L = Few(B, 3, 2048, 64, 8, 2, 1408, "mxfp4", seed=13)
    L()
    torch.cuda.synchronize()
    ref = L.outputs()
    for i in range(200):
        L()
        if i % 50 == 49:
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(ref, L.outputs())), i


@pytest.mark.parametrize("kind", ["bf16", "mxfp4", "f32"])
@pytest.mark.parametrize("T", [2, 7, 16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_weights_reach_their_experts_tokens_only(B, kind, T, bad):
    """One element of W1 of one expert and of W2 of another is not finite: outputs
    of tokens that neither expert computes are those of finite weights, and the
    W2 row's output of a token that it computes is not finite."""
    print(f"[few] non-finite weights {kind} T={T} {bad}", flush=True)
    L = Few(B, T, 256, 10, 2, 1, 384, kind, seed=40 + T)
    ref, A = L.reference()
    tol, idx = L.bound(ref, A), torch.from_numpy(ref["topk_idx"])
    met = sorted(set(idx.flatten().tolist()))
    e1, e2 = met[0], met[-1]
    if kind == "mxfp4":
        L.w["k1"].view(10, 384, 8)[e1, 77, 3] = 255
        L.w["k2"].view(10, 256, 12)[e2, 130, 7] = 255
    else:
        L.w["w1"][e1, 77, 100] = bad
        L.w["w2"][e2, 130, 250] = bad
    first = None
    for _ in range(2):
        L.spoil()
        L()
        torch.cuda.synchronize()
        assert np.array_equal(L.idx.cpu().numpy(), ref["topk_idx"])
        y, on1, on2 = L.y.double().cpu().numpy(), (idx == e1).any(1), (idx == e2).any(1)
        for t in range(T):
            if on1[t]:
                assert not np.isfinite(y[t]).any(), t
                continue
            fine = np.ones(y.shape[1], dtype=bool)
            fine[130] = not on2[t]
            assert np.all(np.abs(y[t] - ref["y"][t])[fine] <= tol[t][fine]), t
            assert fine[130] or not np.isfinite(y[t, 130]), t
        assert first is None or torch.equal(L.y.nan_to_num(), first)
        first = L.y.nan_to_num()


@pytest.mark.parametrize("T", [1, 6, 16])
def test_mxfp4_tokens_of_wide_range(B, T):
    print(f"[few] wide range T={T}", flush=True)
    L = Few(B, T, 512, 8, 2, 1, 256, "mxfp4", seed=60 + T, spread=24)
    L()
    torch.cuda.synchronize()
    x = L.x.clone()
    ref, A = L.reference()
    # a token's element is off by at most 2^-21 of its block's largest: the reach of
    # tokens whose elements all are that large, which bounds A too
    L.x = x.view(T, -1, 32).abs().amax(2, keepdim=True).expand(T, 16, 32).reshape(T, 512).contiguous()
    wide = np.zeros_like(A)
    h = lambda t: t.double().cpu().numpy()  # noqa: E731
    m = h(L.x)
    for t in range(T):
        pairs = [("", int(e), ref["gates"][t, k]) for k, e in enumerate(ref["topk_idx"][t])] + [("s", 0, 1.0)]
        for p, e, g in pairs:
            w1, w2 = np.abs(h(L.w["w" + p + "1"][e])), np.abs(h(L.w["w" + p + "2"][e]))
            wide[t] += g * (w2 @ (1.1 * (w1 @ m[t])))
    L.x = x
    tol = L.bound(ref, A) + 2.0 ** -21 * wide * (1 + 2.0 ** -8)
    assert np.array_equal(L.idx.cpu().numpy(), ref["topk_idx"])
    assert np.all(np.abs(L.y.double().cpu().numpy() - ref["y"]) <= tol)


@pytest.mark.parametrize("kind", ["bf16", "mxfp4", "f32"])
def test_non_finite_tokens_keep_to_themselves(B, kind):
    L = Few(B, 12, 256, 10, 2, 1, 384, kind, seed=70)
    ref, A = L.reference()
    tol = L.bound(ref, A)
    L.x[3, 40], L.x[8, 255] = float("nan"), float("inf")
    L()
    torch.cuda.synchronize()
    y = L.y.double().cpu().numpy()
    for t in range(12):
        if t in (3, 8):
            assert not np.isfinite(y[t]).any(), t
        else:
            assert np.array_equal(L.idx[t].cpu().numpy(), ref["topk_idx"][t])
            assert np.all(np.abs(y[t] - ref["y"][t]) <= tol[t]), t
    ids = L.idx.cpu()
    assert ids.min() >= 0 and ids.max() < 10 and all(len(set(r)) == 2 for r in ids.tolist())
