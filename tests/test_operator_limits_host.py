"""What the operators take and refuse at the ends of their ranges
(no GPU: workspace sizes and refusals; a refused call enqueues nothing)."""
import pytest

from helpers import ensure_built

ensure_built()
import cnn_convolution_conv2d_amd as c2  # noqa: E402

P = 0x1000
TOP = 2 ** 31 - 1


def product(M, K, N):
    return c2.lib.conv2d_int8_matmul(P, P, P, P, None, P, P, 1 << 40, M, K, N, K, K, N, c2.BF16, 0, None)


@pytest.mark.parametrize("M,K,N", [(16, 16, TOP), (16, 17, 2 ** 27 + 1), (TOP, 16, 2 ** 27), (TOP, 17, 1 << 20),
                                   (2 ** 29, 16, 1 << 12), (TOP, 17, TOP), (2 ** 29 + 1, 1040, 2 ** 26)])
def test_products_whose_tiles_cannot_be_counted_are_refused(M, K, N):
    # (16 rows of short k in the aligned case stream the weights; every plan must hold for a size)
    code = product(M, K, N)
    assert code == c2.ERR_UNSUPPORTED, code
    assert c2.last_error()


@pytest.mark.parametrize("M", [2 ** 29, 2 ** 29 + 1, TOP - 500, TOP])
@pytest.mark.parametrize("K,N", [(16, 16), (17, 16), (8192, 64), (16, 300)])
def test_many_rows_need_no_workspace(M, K, N):
    assert c2.conv2d_int8_matmul_workspace_bytes(M, K, N) == 0


def test_eight_bits_over_their_input_are_refused():
    """Written in another place than they are read from: other rows would be lost."""
    for dtype in (c2.F32, c2.BF16):
        assert c2.lib.conv2d_quantize_rows(P, P, P, 8, 64, 64, 64, dtype, None) == c2.ERR_ARG
        assert c2.lib.conv2d_group_norm_quant_nhwc(P, None, None, P, P, None, None, P, 1 << 40, 2, 32, 5, 7, 4, 32, 32,
                                                   1e-5, dtype, 0, None) == c2.ERR_ARG
