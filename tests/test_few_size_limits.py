"""Size limits of the few-token layer and the MXFP4 calls, at their borders: what is
refused, and that the largest sizes below are not (no GPU needed; the accepted sizes
are handed over with an argument missing, so that nothing is launched)."""
import ctypes

from test_mxfp4_few_args import B, few  # noqa: F401  (B: the fixture)


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
