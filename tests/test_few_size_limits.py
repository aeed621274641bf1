"""Size limits of the few-token layer and the MXFP4 calls, at their borders: what is
refused, and that the largest sizes below are not (no GPU needed; the accepted sizes
are handed over with an argument missing, so that nothing is launched)."""
from test_mxfp4_few_args import B, few, linear, quant  # noqa: F401  (B: the fixture)


def test_few_hidden_rows_are_bounded_with_their_padding(B):  # noqa: F811
    """16 tokens of 72 paths have 1152 hidden rows and one of zeros.  931248 float32
    elements a row would end below 2^32 bytes, but rows are padded to chunks of 64,
    931264, and end behind."""
    w = B.Weights(w_router=4096, w1=4096, w2=4096, ws1=4096, ws2=4096)
    assert 1153 * 931248 < 1 << 30 <= 1153 * 931264

    def cfg(f):
        return B.config(16, 16, 65, 64, 8, f, "f32")

    assert B.few_workspace_size(cfg(931248)) == 0
    assert few(B, cfg(931248), w, ws=None) == -2
    assert B.few_workspace_size(cfg(931200)) > 1153 * 931200 * 4
    assert few(B, cfg(931200), w, ws=None) == -3
    assert B.few_workspace_size(B.config(16, 64, 65, 64, 8, 931200, "bf16")) > 0


def test_the_largest_matrices_below_4_gib_are_taken(B):  # noqa: F811
    """"Less than 4 GiB" holds for sizes that do not divide it, too."""
    # one expert matrix of the few-token layer: 2^32 is 368 * 2917776 * 4 + 1024
    w = B.Weights(w_router=4096, w1=4096, w2=4096)
    assert 368 * 2917776 * 4 < 1 << 32 <= 368 * (2917776 + 16) * 4
    assert few(B, B.config(1, 368, 2, 1, 0, 2917776, "f32"), w, ws=None) == -3
    assert few(B, B.config(1, 368, 2, 1, 0, 2917792, "f32"), w, ws=None) == -2
    # codes of a group's matrix (k / 2 = 1472 bytes a row) and of the token rows (192)
    assert 2917776 * 1472 < 1 << 32 <= (2917776 + 8) * 1472
    assert linear(B, n=2917776, k=2944, xc=None) == -1
    assert linear(B, n=2917784, k=2944, xc=None) == -2
    assert 22369621 * 192 < 1 << 32 <= 22369622 * 192
    assert linear(B, k=384, xr=22369621, xc=None) == -1
    assert linear(B, k=384, xr=22369622, xc=None) == -2
    # rows * d < 2^42
    assert 45812984490 * 96 < 1 << 42 <= 45812984491 * 96
    assert quant(B, d=96, stride=96, rows=45812984490, x=None) == -1
    assert quant(B, d=96, stride=96, rows=45812984491, x=None) == -2
