"""The few-token layer just below its size limits: expert matrices near 4 GiB, and hidden
rows near 4 GiB together.

The second matrices are zero but for the first and the last 64 hidden elements, so that
the sums have few terms that are not zero and are compared closely: an offset that wraps
takes weights or hidden values of other rows.  Bound as in test_gpu_few, with n the terms
of a sum that are not zero."""
import pytest
import torch

from test_gpu_few import B, Few  # noqa: F401  (B: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", [(5, 64, 2, 1, 0, (1 << 25) - 64, "bf16"), (16, 16, 65, 64, 8, 931200, "f32")],
                         ids=["matrices", "hidden-rows"])
def test_sizes_just_below_the_limits(B, case):  # noqa: F811
    T, d, N, K, Ks, f, kind = case
    size = 2 if kind == "bf16" else 4
    assert max(d * f, (T * (K + Ks) + 1) * f) * size > (1 << 32) - (1 << 15) * T
    print(f"[few] sizes just below the limits {case}", flush=True)
    L = Few(B, *case, seed=50)
    cols = torch.cat([torch.arange(64), torch.arange(f - 64, f)]).cuda()
    for w in ("w2", "ws2"):
        if L.w[w] is not None:
            L.w[w][:, :, 64:f - 64] = 0
    L()
    torch.cuda.synchronize()
    x = L.x.double()
    logit = x @ L.wr.double().t()
    top = logit.sort(dim=1, descending=True, stable=True)
    idx, kept = top.indices[:, :K], top.values[:, :K]
    gate = torch.softmax(kept, dim=1)
    assert torch.equal(L.idx.long(), idx)
    assert (L.gate.double() - gate).abs().max() <= 2e-6
    ref, A = torch.zeros_like(x), torch.zeros_like(x)
    for p, n in (("", N), ("s", Ks)):
        for e in range(n):
            w1, w2 = L.w["w" + p + "1"][e][cols].double(), L.w["w" + p + "2"][e][:, cols].double()
            g = torch.ones(T, dtype=torch.float64, device="cuda") if p else (gate * (idx == e)).sum(1)
            z = x @ w1.t().contiguous()
            h = z * torch.sigmoid(z)
            ref += g[:, None] * (h @ w2.t().contiguous())
            reach = h.abs() + 1.1 * (x.abs() @ w1.abs().t().contiguous())
            A += g[:, None] * (reach @ w2.abs().t().contiguous())
    last, hidden = (2.0 ** -8, 2.0 ** -16) if kind == "bf16" else (2.0 ** -24, 0.0)
    n = d + 128 * (K + Ks)
    tol = last * ref.abs() + (hidden + n * 2.0 ** -24 + 2e-6) * A * (1 + last)
    err = (L.y.double() - ref).abs()
    assert torch.all(err <= tol), float((err / tol).max())
