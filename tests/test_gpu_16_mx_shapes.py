"""GPU tests of the MX products at sizes whose workgroups do not come out even.

Bars as in test_gpu_13_mx_products.py, whose helpers these are."""
import pytest

from gpu_helpers import log
from test_gpu_13_mx_products import dense

pytestmark = pytest.mark.gpu


# row tiles of 32 that do not divide the CUs, at widths where a column tile's even share is more than the 32
# columns of a workgroup (on 256 CUs 33 to 41): every column has to be written
@pytest.mark.parametrize("a_format", ["E2M1", "E4M3"])
@pytest.mark.parametrize("M,N,K", [(96, 2730, 512), (200, 1168, 256), (400, 624, 96), (640, 400, 1024), (900, 280, 256),
                                   (3200, 81, 96), (160, 1638, 544), (96, 5456, 4640), (1365, 547, 4128)])
def test_row_tiles_that_do_not_divide_the_cus(M, N, K, a_format):
    log("uneven row tiles", M, N, K, a_format)
    dense(M, N, K, a_format, "BF16")
    dense(M, N, K, a_format, "F32", alpha=0.5, beta=2.0, with_bias=True, pitch=N + 5)
