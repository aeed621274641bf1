"""The block around the layer and its gradients against float64.

Bounds, with u = 2^-24: a statistic of a row is a sum of at most 32 terms a thread,
six adds of a wave and four of waves, and a root and a quotient, so that r and the
means are within 2^-18 of the magnitudes that they are made of; the combined rows
are sums of K + n_shared + 1 terms.  Every bound below is 2^-16 times the
magnitudes that enter an output (gradients of a norm: r max|g| (1 + max v^2) of the
row), which leaves a factor of two for the second norm behind the first; a store to
bf16 rounds by 2^-8 relative, one to float32 by 2^-24."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
REL = 2.0 ** -16
EPS = 1e-5


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sparse_mixture_experts_renormalised_amd import binding
    binding.lib()
    return binding


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def close(got, ref, bound, what):
    g = f64(got)
    assert np.isfinite(g).all(), what
    over = np.abs(g - ref) - (bound + HALF[got.dtype] * (np.abs(ref) + bound))
    i = np.unravel_index(np.argmax(over), over.shape)
    assert over[i] <= 0, f"{what}: {g[i]} for {ref[i]} at {i}, off by {abs(g[i] - ref[i]):.3e}"


def top(v):
    return np.abs(v).max(axis=1, keepdims=True)


# T, d, K, shared, norm_out, norm_in, affine, gate, p
CASES = [
    (1, 8, 0, 0, "none", "rms", False, False, 0.0),
    (3, 64, 2, 0, "rms", "layer", True, True, 0.25),
    (33, 512, 4, 1, "layer", "rms", False, True, 0.1),
    (9, 520, 1, 2, "rms", "none", True, False, 0.0),
    (70, 2048, 8, 2, "none", "rms", False, False, 0.5),
    (5, 2056, 0, 0, "layer", "layer", True, True, 0.3),
    (6, 4096, 5, 0, "rms", "rms", False, True, 0.0),
    (7, 7168, 8, 1, "rms", "rms", True, True, 0.1),
    (4, 8200, 3, 1, "layer", "none", False, False, 0.2),
    (3, 16384, 2, 0, "rms", "layer", True, True, 0.0),
    (2100, 72, 2, 0, "layer", "rms", True, True, 0.1),
    (600, 2304, 2, 1, "rms", "layer", True, True, 0.0),
    (301, 136, 3, 1, "layer", "rms", True, True, 0.2),
    (1030, 512, 0, 0, "rms", "layer", True, False, 0.0),
]


def make(case, act, res, seed):
    T, d, K, ks, norm_out, norm_in, affine, gate, p = case
    g = torch.Generator().manual_seed(seed)

    def normal(shape, dtype, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=g) * std + mean).to(dtype).cuda()

    f32 = torch.float32
    t = {"residual": normal((T, d), DT[res], 2.0), "w_out": normal((d,), f32, 0.3, 1.0), "w_in": normal((d,), f32, 0.3, 1.0),
         "b_out": normal((d,), f32) if affine else None, "b_in": normal((d,), f32) if affine else None,
         "gate": normal((T,), f32) if gate else None,
         "rng": torch.tensor([seed, 77], dtype=torch.int64, device="cuda") if p else None,
         "branch": None, "y_rows": None, "slot_row": None, "topk_gate": None, "shared_out": None}
    if not affine:
        t["w_out"] = None
    if K:
        slot = torch.randperm(T * K, generator=g).view(T, K)
        slot[torch.rand(T, K, generator=g) < 0.15] = -1
        slot[T // 2] = -1                                   # a token without experts
        t["slot_row"] = slot.int().cuda()
        t["topk_gate"] = torch.rand(T, K, generator=g).cuda()
        t["y_rows"] = normal((T * K + 2, d), DT[act])
        # rows that no slot names reach nothing
        lost = torch.ones(T * K + 2, dtype=torch.bool)
        lost[slot[slot >= 0]] = False
        t["y_rows"][lost.cuda()] = float("nan")
        if ks:
            t["shared_out"] = normal((ks, T, d), DT[act])
    else:
        t["branch"] = normal((T, d), DT[act])
    return t


def mask_of(case, t, seed):
    T, d, p = case[0], case[1], case[8]
    if not p:
        return None
    # the generator in Python is slow: rows are checked up to this many elements
    keep = oracle.dropout_keep(T * d, p, seed, 77).reshape(T, d)
    return keep * (65536.0 / (65536 - oracle.dropout_cut(p)))


def run(B, case, act, res, t, scale, stream=None, outs=None):
    T, d, K, ks, norm_out, norm_in = case[:6]
    cfg = B.block(T, d, act, res, norm_out=norm_out, norm_in=norm_in, eps=EPS, scale=scale, dropout_p=case[8],
                  top_k=K, n_shared=ks if K else 0)
    o = outs or {"out": torch.full((T, d), 9.0, dtype=DT[res], device="cuda"),
                 "next": torch.full((T, d), 9.0, dtype=DT[act], device="cuda"),
                 "branch_out": torch.full((T, d), 9.0, dtype=DT[act], device="cuda") if K else None}
    B.block_join(cfg, **{**t, **o}, stream=stream)
    return cfg, o


TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]


def branch_of(t):
    if t["y_rows"] is None:
        return f64(t["branch"]), np.abs(f64(t["branch"]))
    y = np.nan_to_num(f64(t["y_rows"]))
    slot, w, sh = t["slot_row"].cpu().numpy(), f64(t["topk_gate"]), f64(t["shared_out"])
    return oracle.combine_rows(y, slot, w, sh), \
        oracle.combine_rows(np.abs(y), slot, np.abs(w), None if sh is None else np.abs(sh))


@pytest.mark.parametrize("act,res", TYPES)
@pytest.mark.parametrize("n", range(len(CASES)))
def test_join(B, n, act, res):
    case = CASES[n]
    print(f"[block] join {act}/{res} {case}", flush=True)
    t, scale = make(case, act, res, 50 + n), 0.7
    _, o = run(B, case, act, res, t, scale)
    torch.cuda.synchronize()
    b, mag = branch_of(t)
    mask = mask_of(case, t, 50 + n)
    out, nxt = oracle.block_join(f64(t["residual"]), b, case[4], case[5], EPS, scale, f64(t["gate"]), mask,
                                 f64(t["w_out"]), f64(t["b_out"]), f64(t["w_in"]), f64(t["b_in"]))
    if o["branch_out"] is not None:
        close(o["branch_out"], b, REL * mag, "branch_out")
    hat, r = oracle.norm_rows(b, case[4], EPS)
    w = 1.0 if t["w_out"] is None else np.abs(f64(t["w_out"]))
    f = scale * (1.0 if t["gate"] is None else np.abs(f64(t["gate"]))[:, None]) * (1.0 if mask is None else mask)
    bias = 0.0 if t["b_out"] is None else np.abs(f64(t["b_out"]))
    bound = REL * (np.abs(f64(t["residual"])) + f * (w * r * top(mag) * (1 + top(hat)) + bias))
    close(o["out"], out, bound, "out")
    hat, r = oracle.norm_rows(out, case[5], EPS)
    bound = r * (top(bound) + REL * top(out)) * (1 + top(hat) ** 2) * np.abs(f64(t["w_in"]))
    bound = bound + (0.0 if t["b_in"] is None else REL * np.abs(f64(t["b_in"])))
    close(o["next"], nxt, bound, "next")
    # the residual's own memory as the output
    again = {**o, "out": t["residual"], "next": torch.empty_like(o["next"])}
    run(B, case, act, res, t, scale, outs=again)
    assert torch.equal(again["out"], o["out"]) and torch.equal(again["next"], o["next"])


GRADS = ("d_residual", "d_branch", "d_gate", "d_w_out", "d_b_out", "d_w_in", "d_b_in", "d_y_rows", "d_topk_gate")


def grads_of(case, act, res, t, only=GRADS):
    T, d, K = case[:3]
    f32 = torch.float32
    g = {"d_residual": ((T, d), DT[res]), "d_branch": ((T, d), DT[act]), "d_gate": ((T,), f32), "d_w_out": ((d,), f32),
         "d_b_out": ((d,), f32), "d_w_in": ((d,), f32), "d_b_in": ((d,), f32)}
    if K:
        g.update({"d_y_rows": (tuple(t["y_rows"].shape), DT[act]), "d_topk_gate": ((T, K), f32)})
    return {n: torch.full(s, 9.0, dtype=dt, device="cuda") for n, (s, dt) in g.items() if n in only}


def run_grad(B, case, act, res, t, scale, saved, c, e, grads, ws, stream=None):
    T, d, K, ks, norm_out, norm_in = case[:6]
    cfg = B.block(T, d, act, res, norm_out=norm_out, norm_in=norm_in, eps=EPS, scale=scale, dropout_p=case[8], top_k=K)
    names = ("y_rows", "slot_row", "topk_gate", "gate", "w_out", "b_out", "w_in", "rng")
    if ws is None:
        n = B.block_join_grad_workspace_size(cfg)
        ws = torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda")
    B.block_join_grad(cfg, c, e, saved["out"], branch=saved["branch"], **{n: t[n] for n in names}, **grads, ws=ws,
                      stream=stream)
    return grads


def inputs_back(case, act, res, t, seed):
    T, d = case[:2]
    g = torch.Generator().manual_seed(seed)
    saved = {"out": (torch.randn(T, d, generator=g) * 2).to(DT[res]).cuda(),
             "branch": torch.randn(T, d, generator=g).to(DT[act]).cuda()}
    return saved, torch.randn(T, d, generator=g).to(DT[res]).cuda(), torch.randn(T, d, generator=g).to(DT[act]).cuda()


@pytest.mark.parametrize("act,res", TYPES)
@pytest.mark.parametrize("n", range(len(CASES)))
def test_join_grad(B, n, act, res):
    case = CASES[n]
    print(f"[block] gradients {act}/{res} {case}", flush=True)
    T, d, K, _, norm_out, norm_in = case[:6]
    t, scale = make(case, act, res, 90 + n), 0.7
    saved, c, e = inputs_back(case, act, res, t, n)
    # cases 0, 4, 8 ask for no sums of biases: another variant of the kernel
    only = [v for v in GRADS if n % 4 or not v.startswith("d_b_")]
    got = run_grad(B, case, act, res, t, scale, saved, c, e, grads_of(case, act, res, t, only), None)
    torch.cuda.synchronize()
    mask = mask_of(case, t, 90 + n)
    y = None if not K else np.nan_to_num(f64(t["y_rows"]))
    slot = None if not K else t["slot_row"].cpu().numpy()
    kw = dict(norm_out=norm_out, norm_in=norm_in, eps=EPS, scale=scale, gate=f64(t["gate"]), mask=mask,
              w_out=f64(t["w_out"]), b_out=f64(t["b_out"]), w_in=f64(t["w_in"]), slot_row=slot,
              topk_gate=f64(t["topk_gate"]), y_rows=y)
    ref = oracle.block_join_grad(f64(c), f64(e), f64(saved["out"]), f64(saved["branch"]), **kw)

    hat, r = oracle.norm_rows(f64(saved["out"]), norm_in, EPS)
    w = np.abs(f64(t["w_in"]))
    dn = np.abs(f64(e))
    e_dh = REL * (np.abs(f64(c)) + r * top(dn * w) * (1 + top(hat) ** 2))
    close(got["d_residual"], ref["d_residual"], e_dh, "d_residual")
    close(got["d_w_in"], ref["d_w_in"], REL * (dn * (1 + top(hat))).sum(axis=0), "d_w_in")
    if "d_b_in" in got:
        close(got["d_b_in"], ref["d_b_in"], REL * dn.sum(axis=0), "d_b_in")
    vhat, vr = oracle.norm_rows(f64(saved["branch"]), norm_out, EPS)
    wo = 1.0 if t["w_out"] is None else np.abs(f64(t["w_out"]))
    bo = 0.0 if t["b_out"] is None else np.abs(f64(t["b_out"]))
    m = scale * (1.0 if mask is None else mask)
    gate = 1.0 if t["gate"] is None else np.abs(f64(t["gate"]))[:, None]
    dh = np.abs(ref["d_residual"])
    e_u = m * (e_dh + REL * dh)                             # of the dropped, scaled stream gradient
    n_mag = (1 + top(vhat)) * wo + bo
    close(got["d_gate"], ref["d_gate"], ((e_u + REL * m * dh) * n_mag).sum(axis=1), "d_gate")
    close(got["d_w_out"], ref["d_w_out"], (gate * (e_u + REL * m * dh) * (1 + top(vhat))).sum(axis=0), "d_w_out")
    if "d_b_out" in got:
        close(got["d_b_out"], ref["d_b_out"], (gate * (e_u + REL * m * dh)).sum(axis=0), "d_b_out")
    g_top = top(gate * (e_u + REL * m * dh) * wo)
    e_db = vr * g_top * (1 + top(vhat) ** 2)
    close(got["d_branch"], ref["d_branch"], e_db, "d_branch")
    if K:
        w = f64(t["topk_gate"])
        hit = slot >= 0
        yabs = np.abs(y)
        bound = np.zeros((T, K))
        for i, k in zip(*np.nonzero(hit)):
            bound[i, k] = ((e_db[i] + REL * np.abs(ref["d_branch"][i])) * yabs[slot[i, k]]).sum()
        close(got["d_topk_gate"], ref["d_topk_gate"], bound, "d_topk_gate")
        assert (got["d_topk_gate"].cpu().numpy()[~hit] == 0).all()
        rows = got["d_y_rows"]
        named = np.zeros(len(rows), dtype=bool)
        named[slot[hit]] = True
        assert (rows[torch.from_numpy(~named).cuda()] == 9.0).all()
        i, k = np.nonzero(hit)
        want = w[i, k][:, None] * ref["d_branch"][i]
        close(rows[torch.from_numpy(slot[i, k]).long().cuda()], want,
              w[i, k][:, None] * (e_db[i] + REL * np.abs(ref["d_branch"][i])), "d_y_rows")
    # in place, and only some of the gradients: the same bits
    some = [v for v in ("d_residual", "d_y_rows") if v in got]
    part = grads_of(case, act, res, t, some)
    part["d_residual"] = c
    run_grad(B, case, act, res, t, scale, saved, c, e, part, None)
    for v in some:
        assert torch.equal(part[v], got[v]), v


def test_first_norm_and_its_gradient(B):
    """No branch: the norm before a model's first block."""
    T, d = 37, 1408
    g = torch.Generator().manual_seed(4)
    x = torch.randn(T, d, generator=g).cuda()
    w, e = torch.rand(d, generator=g).cuda(), torch.randn(T, d, generator=g).cuda()
    cfg = B.block(T, d, "f32", norm_out="rms", norm_in="rms", eps=EPS, dropout_p=0.5)
    nxt, out = torch.empty_like(x), torch.empty_like(x)
    B.block_join(cfg, x, out=out, next=nxt, w_in=w)
    hat, r = oracle.norm_rows(f64(x), "rms", EPS)
    assert torch.equal(out, x)
    close(nxt, hat * f64(w), REL * top(hat) * f64(w), "next")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ws = torch.empty(B.block_join_grad_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    dwo = torch.full_like(w, 5.0)
    B.block_join_grad(cfg, None, e, out, w_in=w, d_residual=dx, d_w_in=dw, d_w_out=dwo, ws=ws)
    ref = oracle.block_join_grad(0.0, f64(e), f64(x), None, "none", "rms", EPS, w_in=f64(w))
    close(dx, ref["d_residual"], REL * r * top(f64(e) * f64(w)) * (1 + top(hat) ** 2), "d_residual")
    close(dw, ref["d_w_in"], REL * (np.abs(f64(e)) * top(hat)).sum(axis=0), "d_w_in")
    assert (dwo == 0).all()
    # no gradient of next: the stream's passes through
    B.block_join_grad(cfg, e, None, None, d_residual=dx, d_w_in=dw, ws=ws)
    assert torch.equal(dx, e) and (dw == 0).all()


def test_no_tokens(B):
    cfg = B.block(0, 64, "bf16")
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    B.block_join(cfg, x, out=x, next=x)
    dw = torch.full((64,), 5.0, device="cuda")
    B.block_join_grad(cfg, x, x, x, d_residual=x, d_w_in=dw)
    torch.cuda.synchronize()
    assert (dw == 0).all()


def test_what_is_not_finite_stays_in_its_token(B):
    case = (40, 1024, 3, 1, "layer", "rms", True, True, 0.2)
    t = make(case, "bf16", "bf16", 5)
    _, clean = run(B, case, "bf16", "bf16", t, 0.5)
    t["residual"][3] = float("nan")
    t["shared_out"][:, 8] = float("inf")
    _, dirty = run(B, case, "bf16", "bf16", t, 0.5)
    ok = torch.ones(40, dtype=torch.bool, device="cuda")
    ok[[3, 8]] = False
    for n in ("out", "next", "branch_out"):
        assert torch.equal(clean[n][ok], dirty[n][ok]), n
    assert dirty["next"][3].isnan().all() and not dirty["next"][8].isfinite().any()


def test_other_streams_and_graphs(B):
    case, act, res = (65, 2048, 4, 1, "rms", "rms", True, True, 0.3), "bf16", "f32"
    t = make(case, act, res, 6)
    saved, c, e = inputs_back(case, act, res, t, 1)
    cfg, ref = run(B, case, act, res, t, 0.5)
    n = B.block_join_grad_workspace_size(cfg)
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(3)]
    gref = run_grad(B, case, act, res, t, 0.5, saved, c, e, grads_of(case, act, res, t), ws[0])
    got, side = ({k: torch.empty_like(v) for k, v in ref.items()} for _ in range(2))
    ggot, gside = grads_of(case, act, res, t), grads_of(case, act, res, t)
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(B, case, act, res, t, 0.5, outs=got)
        run_grad(B, case, act, res, t, 0.5, saved, c, e, ggot, ws[1])
    for _ in range(3):
        for v in [*got.values(), *ggot.values(), *side.values(), *gside.values()]:
            v.fill_(9.0)
        torch.cuda.synchronize()
        graph.replay()
        run(B, case, act, res, t, 0.5, stream=s, outs=side)
        run_grad(B, case, act, res, t, 0.5, saved, c, e, gside, ws[2], stream=s)
        torch.cuda.synchronize()
        for k in ref:
            assert torch.equal(ref[k], got[k]) and torch.equal(ref[k], side[k]), k
        for k in gref:
            assert torch.equal(gref[k], ggot[k]) and torch.equal(gref[k], gside[k]), k
        run(B, case, act, res, t, 0.5, outs=ref)


def test_a_dropped_element_takes_no_part(B):
    """Without a norm of the branch, what a dropped element holds reaches no output."""
    case = (9, 264, 0, 0, "none", "none", False, True, 0.4)
    t = make(case, "bf16", "f32", 12)
    t["w_out"] = torch.rand(264, device="cuda") + 0.5
    keep = torch.from_numpy(oracle.dropout_keep(9 * 264, 0.4, 12, 77).reshape(9, 264)).cuda()
    got = []
    for value in (0.0, float("inf"), float("nan")):
        t["branch"] = t["branch"].masked_fill(~keep.bool(), value)
        cfg, o = run(B, case, "bf16", "f32", t, 0.5)
        g = {"d_residual": torch.empty(9, 264, device="cuda"), "d_gate": torch.empty(9, device="cuda"),
             "d_branch": torch.empty(9, 264, dtype=torch.bfloat16, device="cuda"), "d_w_out": torch.empty(264, device="cuda")}
        ws = torch.empty(B.block_join_grad_workspace_size(cfg), dtype=torch.uint8, device="cuda")
        B.block_join_grad(cfg, t["residual"], o["next"], o["out"], branch=t["branch"], gate=t["gate"], w_out=t["w_out"],
                          w_in=t["w_in"], rng=t["rng"], ws=ws, **g)
        torch.cuda.synchronize()
        got.append([o["out"], o["next"], *g.values()])
    assert all(v.isfinite().all() for v in got[0])
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert torch.equal(a, b)


def test_no_tokens_with_expert_rows(B):
    """Empty slot arrays beside expert rows with room: nothing is written but the sums over
    tokens, which are zeros."""
    d, k = 64, 3
    cfg = B.block(0, d, "bf16", norm_out="rms", top_k=k, n_shared=1)
    x = torch.empty(0, d, dtype=torch.bfloat16, device="cuda")
    slots, gates = torch.empty(0, k, dtype=torch.int32, device="cuda"), torch.empty(0, k, device="cuda")
    y, dy = (torch.full((4, d), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    shared = torch.empty(1, 0, d, dtype=torch.bfloat16, device="cuda")
    B.block_join(cfg, x, out=x, next=x, y_rows=y, slot_row=slots, topk_gate=gates, shared_out=shared, branch_out=x)
    sums = {n: torch.full((d,), 5.0, device="cuda") for n in ("d_w_out", "d_b_out", "d_w_in", "d_b_in")}
    B.block_join_grad(cfg, x, x, x, branch=x, y_rows=y, slot_row=slots, topk_gate=gates, d_residual=x, d_branch=x,
                      d_y_rows=dy, d_topk_gate=torch.empty_like(gates), **sums)
    torch.cuda.synchronize()
    for n, v in sums.items():
        assert (v == 0).all(), n
    assert (y == 5).all() and (dy == 5).all()


@pytest.mark.parametrize("act,res", TYPES)
@pytest.mark.parametrize("T,d", [(8201, 64), (4103, 520), (2055, 2048), (2050, 2056), (2051, 4104), (1031, 8200)])
def test_join_of_more_tokens_than_workgroups(B, T, d, act, res):
    """A workgroup that takes several tokens gives each the bits that it gets in a batch of
    few."""
    print(f"[block] {T} tokens of {d} {act}/{res}", flush=True)
    t = make((T, d, 3, 1, "layer", "layer", True, True, 0.0), act, res, 13)
    names = [n for n in ("residual", "slot_row", "topk_gate", "gate") if t[n] is not None]
    case = (T, d, 3, 1, "layer", "layer", True, True, 0.0)
    _, o = run(B, case, act, res, t, 0.7)
    few = 500
    for a in range(0, T, few):
        e = min(T, a + few)
        part = {**t, **{n: t[n][a:e].contiguous() for n in names}, "shared_out": t["shared_out"][:, a:e].contiguous()}
        _, p = run(B, (e - a, *case[1:]), act, res, part, 0.7)
        for n in p:
            assert torch.equal(o[n][a:e], p[n]), (n, a)


def test_dropout_of_more_tokens_than_workgroups(B):
    """The same elements as moe_dropout drops, up to the last token.  Roundings: of the
    factor, of its product and of the sum, in float32."""
    T, d, p = 8201, 24, 0.3
    case = (T, d, 0, 0, "none", "none", False, False, p)
    t = make(case, "f32", "f32", 14)
    _, o = run(B, case, "f32", "f32", t, 0.7)
    dropped = torch.empty_like(t["branch"])
    B.dropout(t["branch"], dropped, p, t["rng"])
    b = 0.7 * f64(dropped)
    close(o["out"], f64(t["residual"]) + b, 4 * 2.0 ** -24 * (np.abs(b) + np.abs(f64(t["residual"]))), "out")


@pytest.mark.parametrize("act,res", TYPES)
def test_as_many_slots_and_shared_experts_as_there_may_be(B, act, res):
    """64 slots and 64 shared experts a token, and the gradients of the slots' rows and gates
    (no norms and no weights: sums of products alone)."""
    T, d, K = 3, 520, 64
    case = (T, d, K, 64, "none", "none", False, False, 0.0)
    t = make(case, act, res, 15)
    t["w_in"] = None
    _, o = run(B, case, act, res, t, 0.5)
    b, mag = branch_of(t)
    close(o["branch_out"], b, REL * mag, "branch_out")
    out = f64(t["residual"]) + 0.5 * b
    bound = REL * (np.abs(f64(t["residual"])) + mag)
    close(o["out"], out, bound, "out")
    saved, c, e = inputs_back(case, act, res, t, 2)
    got = run_grad(B, case, act, res, t, 0.5, saved, c, e, grads_of(case, act, res, t), None)
    torch.cuda.synchronize()
    dh = f64(c) + f64(e)
    close(got["d_residual"], dh, REL * np.abs(dh), "d_residual")
    slot, w, y = t["slot_row"].cpu().numpy(), f64(t["topk_gate"]), np.nan_to_num(f64(t["y_rows"]))
    for i in range(T):
        for k in range(K):
            r = slot[i, k]
            if r < 0:
                assert got["d_topk_gate"][i, k] == 0
                continue
            close(got["d_y_rows"][r], w[i, k] * 0.5 * dh[i], REL * np.abs(dh[i]), f"row of slot {k}")
            close(got["d_topk_gate"][i, k], np.array(0.5 * (dh[i] * y[r]).sum()), np.array(REL * np.abs(dh[i] * y[r]).sum()),
                  f"gate of slot {k}")
