"""The MXFP4 product on the last rows and features below 4 GiB where the width does not
divide it and the last step of the reduction axis is a half one.  Bounds as in
test_gpu_mxfp4."""
import numpy as np
import pytest
import torch

from test_gpu_mxfp4 import B, linear_reference  # noqa: F401  (B: the fixture)

pytestmark = pytest.mark.gpu

K, ROWS = 384, 22369621                      # 192 bytes a row, 64 bytes below 2^32


@pytest.fixture(scope="module")
def long_rows():
    g = torch.Generator(device="cuda").manual_seed(22)
    codes = torch.randint(0, 256, (ROWS, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.randint(118, 124, (ROWS, K // 32), dtype=torch.uint8, device="cuda", generator=g)
    return codes, scales


def close(y, ref, mag):
    err = (K + 1) * 2.0 ** -24 * mag
    return np.all(np.abs(y.double().cpu().numpy() - ref) <= err * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref))


@pytest.mark.parametrize("rows", [5, 70, 300])
def test_the_last_rows_below_4_gib(B, long_rows, rows):  # noqa: F811
    print(f"[mxfp4] the last {rows} rows of 4 GiB", flush=True)
    codes, scales = long_rows
    idx = torch.arange(ROWS - rows, ROWS, device="cuda").int()
    w, ws = codes[:64].clone(), scales[:64].clone()
    y = torch.zeros(rows, 64, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    B.grouped_linear_mxfp4(codes, scales, off, w[None], ws[None], y, row_index=idx)
    torch.cuda.synchronize()
    assert close(y, *linear_reference(codes[idx.long()], scales[idx.long()], w, ws))


@pytest.mark.parametrize("rows", [3, 70])
def test_the_last_features_below_4_gib(B, long_rows, rows):  # noqa: F811
    print(f"[mxfp4] {rows} rows on a matrix of 4 GiB", flush=True)
    codes, scales = long_rows
    n_out = ROWS // 8 * 8
    x, xs = codes[:rows].clone(), scales[:rows].clone()
    y = torch.zeros(rows, n_out, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    B.grouped_linear_mxfp4(x, xs, off, codes[None, :n_out], scales[None, :n_out], y)
    torch.cuda.synchronize()
    for a in (0, n_out // 2, n_out - 64):
        assert close(y[:, a:a + 64], *linear_reference(x, xs, codes[a:a + 64], scales[a:a + 64])), a
