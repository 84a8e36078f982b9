"""CPU tests of what the mixture-of-experts entry points decide on the host:
the kernel of a call at the limits of its sizes."""
import os

import pytest

import gguf_quantized_matvec_amd as g

pytestmark = pytest.mark.skipif(not os.path.exists(g.LIB_PATH), reason="libqmv.so not built")


@pytest.mark.parametrize("top,K,most", [
    # a row a wave, 6 waves of 64 a workgroup: 384 N threads below 2^32
    (6, 8224, ((1 << 32) - 1) // 384),
    # two rows a wave, 8 waves: 512 threads for two rows; 2^24 rows are 2^32 threads
    (8, 5632, (1 << 24) - 2),
    # a row a wave, two units of 4 waves: the same
    (4, 8224, (1 << 24) - 2),
    # a row a wave, two units of 3 waves: 192 threads a row are never as many
    (3, 8224, 1 << 24),
])
def test_no_grid_beyond_its_dimension(top, K, most):
    """The down products of a token whose matrix-vector launch would pass 2^32 threads go to the rows kernel."""
    assert g.qmv_moe_rows(g.Q4_0, 1, 1, top, 1, most, K) == 1
    if most < 1 << 24:
        assert g.qmv_moe_rows(g.Q4_0, 1, 1, top, 1, most + 1, K) == 4
        assert g.qmv_moe_rows(g.Q4_0, 1, 1, top, 1, 1 << 24, K) == 4
