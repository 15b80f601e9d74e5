"""The weight gradient's workspace and its single-row results on the host (no GPU): refusals come
before any CUDA call."""
import ctypes

import pytest

import sparsified_gradient_compression_gb300 as dgc

FAKE = 1 << 40  # aligned non-null address that is never dereferenced


@pytest.fixture(scope="module")
def L():
    dgc.build()
    return dgc.lib()


def mat(rows, cols, ld=None, dtype=dgc.BF16):
    return ctypes.byref(dgc.dgc_matrix(FAKE, rows, cols, -(-cols // 8) * 8 if ld is None else ld,
                                       dtype, 0))


@pytest.mark.parametrize("cols", [64, 61, 8, 1])
@pytest.mark.parametrize("rows", [1, 100, 121, 128])
def test_narrow_parts_ask_for_their_tiles_alone(L, rows, cols):
    """One tile of 128 rows: a part of the sum (512 tokens at least) is 128 rows of the workspace."""
    tokens = 1 << 16
    part = 128 * (-(-cols // 4) * 4) * 4
    need = dgc.dgc_ffn_weight_grad_workspace(rows, cols, tokens)
    assert need % part == 0 and 2 <= need // part <= tokens // 512


@pytest.mark.parametrize("rows", [300, 511, 512])
def test_wide_parts_ask_for_their_tiles_alone(L, rows):
    """Two tiles of 256 rows: a part (2048 tokens at least) is 512 rows of the workspace."""
    tokens, cols = 1 << 16, 500
    part = 512 * cols * 4
    need = dgc.dgc_ffn_weight_grad_workspace(rows, cols, tokens)
    assert need % part == 0 and 2 <= need // part <= tokens // 2048


@pytest.mark.parametrize("ld", [0, -5, 24, 2**37, 2**62])
def test_a_single_row_has_no_row_to_row_distance(L, ld):
    """dw's ld is not read where it has one row: what is missing is the workspace alone."""
    tokens, cols = 1 << 16, 24
    assert dgc.dgc_ffn_weight_grad_workspace(1, cols, tokens) > 0
    rc = L.dgc_ffn_weight_grad(mat(tokens, 1), mat(tokens, cols), 0, mat(1, cols, ld, dgc.F32),
                               FAKE, None, 0, None)
    assert rc == dgc.EINVAL
