"""One training step of a block around the layer, forward and back through the
library's calls in the order in which a program makes them, against automatic
differentiation in float64 on the CPU (with the same experts kept and the same
elements dropped), and against differences of its own forward.

Bounds, as relative L2 of a whole gradient: float32 steps are a dozen sums of at most
2^11 terms and norms, each within 2^-17 of what enters it, so 2^-13 together; bf16
steps round about sixteen intermediate tensors by 2^-9 (root mean square 0.6 of half a
step), which add up to 2^-9 sqrt(16) = 2^-7 in the stream and, with the two norms' and
the gates' factors on the way back, stay below 2^-4."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
TOL = {"bf16": 2.0 ** -4, "f32": 2.0 ** -13}
T, D, N, K, F = 96, 128, 8, 2, 192
EPS, SCALE, P_HID, P_OUT, CAP = 1e-5, 0.5, 0.2, 0.1, 1.25


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sparse_mixture_experts_renormalised_amd import binding
    binding.lib()
    return binding


class Step:
    def __init__(self, B, dtype, seed):
        g = torch.Generator().manual_seed(seed)
        act = self.act = DT[dtype]

        def normal(*shape, std=1.0, dt=act, mean=0.0):
            return (torch.randn(*shape, generator=g) * std + mean).to(dt).cuda()

        self.B, self.dtype = B, dtype
        self.p = {"x": normal(T, D), "w_router": normal(N, D, std=D ** -0.5, dt=torch.float32),
                  "w1": normal(N, F, D, std=D ** -0.5), "b1": normal(N, F, std=0.1),
                  "w2": normal(N, D, F, std=F ** -0.5), "b2": normal(N, D, std=0.1),
                  "ws1": normal(1, F, D, std=D ** -0.5), "ws2": normal(1, D, F, std=F ** -0.5),
                  "n0": normal(D, std=0.2, dt=torch.float32, mean=1.0),
                  "n1": normal(D, std=0.2, dt=torch.float32, mean=1.0),
                  "n2": normal(D, std=0.2, dt=torch.float32, mean=1.0),
                  "gate": (torch.rand(T, generator=g) + 0.5).cuda()}
        self.c, self.e = normal(T, D), normal(T, D)
        self.rng_hid = torch.tensor([5, 1], dtype=torch.int64, device="cuda")
        self.rng_out = torch.tensor([5, 2], dtype=torch.int64, device="cuda")
        self.cfg = B.config(T, D, N, K, 1, F, dtype, CAP)
        self.first = B.block(T, D, dtype, norm_in="rms", eps=EPS)
        self.join = B.block(T, D, dtype, norm_out="layer", norm_in="rms", eps=EPS, scale=SCALE, dropout_p=P_OUT,
                            top_k=K, n_shared=1)
        n = max(B.grouped_linear_workspace_size(dtype, N, F, D, T * K), B.grouped_linear_workspace_size(dtype, N, D, F, T * K),
                B.block_join_grad_workspace_size(self.join), B.permute_workspace_size(self.cfg))
        self.ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        self.whole = torch.tensor([0, T], dtype=torch.int32, device="cuda")

    def new(self, *shape, dt=None):
        return torch.full(shape, 0.5, dtype=dt or self.act, device="cuda")

    def forward(self):
        B, p, ws = self.B, self.p, self.ws
        i32, f32 = torch.int32, torch.float32
        s = self.s = {"xn": self.new(T, D), "logits": self.new(T, N, dt=f32), "gates": self.new(T, K, dt=f32),
                      "idx": torch.zeros(T, K, dtype=i32, device="cuda"), "z": self.new(T * K, F), "h": self.new(T * K, F),
                      "y": self.new(T * K, D), "zs": self.new(T, F), "hs": self.new(T, F), "ys": self.new(1, T, D),
                      "branch": self.new(T, D), "out": self.new(T, D), "next": self.new(T, D)}
        for name, n in (("counts", N), ("offsets", N + 1), ("row_token", T * K), ("slot_row", T * K), ("dropped", 4)):
            s[name] = torch.zeros(n, dtype=i32, device="cuda")
        B.block_join(self.first, p["x"], next=s["xn"], w_in=p["n0"])
        B.route(self.cfg, s["xn"], p["w_router"], None, s["logits"], s["idx"], s["gates"])
        B.permute(self.cfg, s["idx"], None, s["counts"], s["offsets"], s["row_token"], s["slot_row"], s["dropped"],
                  None, ws)
        B.grouped_linear(s["xn"], s["offsets"], p["w1"], s["h"], row_index=s["row_token"], bias=p["b1"], silu=True,
                         pre=s["z"], ws=ws)
        s["rows"] = s["offsets"][N:]
        B.dropout(s["h"], s["h"], P_HID, self.rng_hid, n_rows=s["rows"])
        B.grouped_linear(s["h"], s["offsets"], p["w2"], s["y"], bias=p["b2"], ws=ws)
        B.grouped_linear(s["xn"], self.whole, p["ws1"], s["hs"], silu=True, pre=s["zs"], ws=ws)
        B.grouped_linear(s["hs"], self.whole, p["ws2"], s["ys"][0], ws=ws)
        s["slot_row"] = s["slot_row"].view(T, K)
        B.block_join(self.join, p["x"], out=s["out"], next=s["next"], y_rows=s["y"], slot_row=s["slot_row"],
                     topk_gate=s["gates"], shared_out=s["ys"], branch_out=s["branch"], gate=p["gate"], w_out=p["n1"],
                     w_in=p["n2"], rng=self.rng_out)
        return (s["out"].double() * self.c.double()).sum() + (s["next"].double() * self.e.double()).sum()

    def backward(self):
        B, p, s, ws = self.B, self.p, self.s, self.ws
        f32 = torch.float32
        g = {n: torch.full_like(p[n], 7.0) for n in ("w1", "b1", "w2", "b2", "ws1", "ws2", "n0", "n1", "n2", "gate", "x")}
        dres, dbr, dy, dgate = self.new(T, D), self.new(T, D), self.new(T * K, D), self.new(T, K, dt=f32)
        B.block_join_grad(self.join, self.c, self.e, s["out"], branch=s["branch"], y_rows=s["y"], slot_row=s["slot_row"],
                          topk_gate=s["gates"], gate=p["gate"], w_out=p["n1"], w_in=p["n2"], rng=self.rng_out,
                          d_residual=dres, d_branch=dbr, d_y_rows=dy, d_topk_gate=dgate, d_gate=g["gate"],
                          d_w_out=g["n1"], d_w_in=g["n2"], ws=ws)
        B.grouped_linear_weight_grad(dy, s["offsets"], s["h"], g["w2"], dbias=g["b2"], ws=ws)
        dz, dx = self.new(T * K, F), self.new(T * K, D)
        # the mask is a factor, as the SiLU's slope is: either may come first
        B.grouped_linear_input_grad(dy, s["offsets"], p["w2"], dz, pre=s["z"], ws=ws)
        B.dropout(dz, dz, P_HID, self.rng_hid, n_rows=s["rows"])
        B.grouped_linear_weight_grad(dz, s["offsets"], s["xn"], g["w1"], row_index=s["row_token"], dbias=g["b1"], ws=ws)
        B.grouped_linear_input_grad(dz, s["offsets"], p["w1"], dx, ws=ws)
        dzs, dxs = self.new(T, F), self.new(1, T, D)
        B.grouped_linear_weight_grad(dbr, self.whole, s["hs"], g["ws2"], ws=ws)
        B.grouped_linear_input_grad(dbr, self.whole, p["ws2"], dzs, pre=s["zs"], ws=ws)
        B.grouped_linear_weight_grad(dzs, self.whole, s["xn"], g["ws1"], ws=ws)
        B.grouped_linear_input_grad(dzs, self.whole, p["ws1"], dxs[0], ws=ws)
        # a token's rows, its shared expert's, and the router's
        dxn, ones = self.new(T, D), torch.ones(T, K, device="cuda")
        B.combine(self.cfg, dx, s["slot_row"], ones, dxs, dxn)
        gates = s["gates"].double()
        dl = gates * (dgate.double() - (gates * dgate.double()).sum(dim=1, keepdim=True))
        dlogits = torch.zeros(T, N, dtype=torch.float64, device="cuda").scatter_(1, s["idx"].long(), dl)
        g["w_router"] = dlogits.t() @ s["xn"].double()
        dxn = (dxn.double() + dlogits @ p["w_router"].double()).to(self.act)
        B.block_join_grad(self.first, dres, dxn, p["x"], w_in=p["n0"], d_residual=g["x"], d_w_in=g["n0"], ws=ws)
        torch.cuda.synchronize()
        return g


def reference(st):
    """The step in float64 with automatic differentiation; experts, slots and masks as given."""
    s = st.s
    p = {n: v.double().cpu().requires_grad_() for n, v in st.p.items()}
    idx, slot = s["idx"].long().cpu(), s["slot_row"].long().cpu()

    def rms(v, w):
        return v * torch.rsqrt(v.square().mean(dim=1, keepdim=True) + EPS) * w

    xn = rms(p["x"], p["n0"])
    logits = xn @ p["w_router"].t()
    gates = torch.softmax(logits.gather(1, idx), dim=1)
    rows = int(s["rows"].item())
    keep = torch.from_numpy(oracle.dropout_keep(rows * F, P_HID, 5, 1).reshape(rows, F))
    k_hid, k_out = (65536.0 / (65536 - oracle.dropout_cut(q)) for q in (P_HID, P_OUT))
    branch = torch.zeros(T, D, dtype=torch.float64)
    for t in range(T):
        for j in range(K):
            r = int(slot[t, j])
            if r < 0:
                continue
            e = int(idx[t, j])
            z = p["w1"][e] @ xn[t] + p["b1"][e]
            h = z * torch.sigmoid(z) * keep[r] * k_hid
            branch[t] = branch[t] + gates[t, j] * (p["w2"][e] @ h + p["b2"][e])
    zs = xn @ p["ws1"][0].t()
    branch = branch + (zs * torch.sigmoid(zs)) @ p["ws2"][0].t()
    v = branch - branch.mean(dim=1, keepdim=True)
    n = v * torch.rsqrt(v.square().mean(dim=1, keepdim=True) + EPS) * p["n1"]
    mask = torch.from_numpy(oracle.dropout_keep(T * D, P_OUT, 5, 2).reshape(T, D)) * k_out
    out = p["x"] + SCALE * p["gate"].unsqueeze(1) * mask * n
    loss = (out * st.c.double().cpu()).sum() + (rms(out, p["n2"]) * st.e.double().cpu()).sum()
    loss.backward()
    return float(loss.detach()), {n: v.grad for n, v in p.items()}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_step_against_differentiation(B, dtype):
    st = Step(B, dtype, 3)
    loss = float(st.forward())
    g = st.backward()
    assert (st.s["slot_row"] < 0).any(), "the capacity drops some assignments"
    want, ref = reference(st)
    assert abs(loss - want) <= TOL[dtype] * (st.c.double().norm() + st.e.double().norm()).item() * np.sqrt(T * D) / 16
    for name, r in ref.items():
        err = float((g[name].double().cpu() - r).norm() / r.norm())
        print(f"[step] {dtype} {name}: {err:.2e}", flush=True)
        assert err <= TOL[dtype], name


@pytest.mark.parametrize("name", ["w1", "w2", "ws1", "n0", "n1", "gate", "x"])
def test_step_against_differences(B, name):
    """float32: (L(p + h v) - L(p - h v)) / 2 h against <gradient, v>, along the gradient
    itself, so that the difference is large beside the rounding of L (2^-20 of its terms'
    magnitudes) and beside the third order in h."""
    st = Step(B, "f32", 4)
    st.forward()
    idx = st.s["idx"].clone()
    v = st.backward()[name].double()
    v = v / v.norm()
    slope = (st.backward()[name].double() * v).sum().item()
    p0, h, side = st.p[name].clone(), 1e-2, []
    for sign in (1.0, -1.0):
        st.p[name] = (p0.double() + sign * h * v).to(p0.dtype)
        side.append(float(st.forward()))
        assert torch.equal(st.s["idx"], idx), "the same experts"
    assert (side[0] - side[1]) / (2 * h) == pytest.approx(slope, rel=2.0 ** -7)


def test_step_twice_gives_equal_bits(B):
    a, b = Step(B, "bf16", 5), Step(B, "bf16", 5)
    a.forward(), b.forward()
    ga, gb = a.backward(), b.backward()
    for n in ga:
        assert torch.equal(ga[n], gb[n]), n
