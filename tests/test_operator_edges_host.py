"""Arguments of the operators around the quantizer at the edges of what they
take, on the host: every check runs before a device is touched."""
import pytest

import nvfp4_adaptive_block_amd as fos
from test_operators_host import O, P, SHAPE, linear


@pytest.mark.parametrize("G,M,N,K,fits", [
    (0, 16, 2 ** 29 - 64, 16, True), (0, 16, 2 ** 29, 16, False), (0, 64, 2 ** 30, 16, False),
    (0, 2 ** 16, 2 ** 21, 16, True), (0, 2 ** 20, 2 ** 20, 16, False),
    (2 ** 20, 2 ** 20, 256, 16, True), (2 ** 20, 2 ** 20, 1024, 16, False),
])
def test_products_past_a_launch_are_refused_for_their_shape(G, M, N, K, fits):
    """A launch has fewer than 2^32 threads, 256 to 1024 of them in a workgroup."""
    assert (fos.load_library().fos_linear_workspace(M, N, K, G) >= 0) == fits
    if not fits:
        assert linear(M=M, N=N, K=K, **(dict(G=G, offs=P(O)) if G else {})) == SHAPE
