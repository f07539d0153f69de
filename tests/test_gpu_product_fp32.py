"""The experts' products with fp32 outputs, in every form that a size may take.

Bounds and checks are those of test_gpu_products.py.  An fp32 output is turned
through twice the LDS that a 16-bit one takes, so each block shape is met with
it: the streams of 16, 32 and 64 rows, tiles of 64 x 64, 128 x 128 (for gradients
of matrices in half steps) and 256 x 256; rows of whole 16-byte pieces and not."""
import pytest

from test_gpu_products import BF16, F16, F32, Case, _run_gated, _run_linear, oproducts

pytestmark = pytest.mark.gpu


# y | dw: 128 x 128 of one matrix and of experts, aligned and odd; 256 x 256 of
# one matrix (y, dw) and of experts (y, dw); streams beside them
@pytest.mark.parametrize("N,n_in,n_out,E", [
    (300, 2048, 2048, 0), (120, 1536, 2048, 0), (90, 2048, 5632, 0), (300, 1408, 2048, 8), (90, 2056, 1032, 12),
    (1100, 1000, 4104, 0), (5000, 264, 520, 40), (200, 2001, 1999, 0), (5000, 265, 521, 40), (300, 521, 263, 100),
    (700, 331, 515, 512),
    (600, 72, 13208, 0), (770, 136, 13320, 0), (70, 13208, 1000, 0), (3000, 40, 8200, 4), (700, 2048, 512, 512),
    (1000, 201, 4103, 0), (17, 264, 200, 0), (32, 131, 77, 0), (33, 136, 200, 0), (64, 133, 201, 0), (20, 72, 8208, 0),
    (50, 71, 8209, 0)])
def test_linear_forms(N, n_in, n_out, E):
    _run_linear(Case(BF16 if N % 3 else F16, N, n_in, n_out, E, N // 50 if E else 0), n_in, n_out, F32)


@pytest.mark.parametrize("N,d,I,E", [
    (200, 2048, 1408, 0), (100, 1536, 2048, 0), (300, 768, 1024, 16), (5000, 136, 264, 40), (200, 2047, 1025, 0),
    (5000, 137, 263, 40), (600, 1024, 136, 300), (500, 512, 256, 64), (530, 6608, 264, 0)])
def test_gated_forms(N, d, I, E):
    _run_gated(Case(BF16 if N % 3 else F16, N, d, I, E, N // 50 if E else 0, mats=2), d, I, oproducts.ACTS[d % 3], F32)
