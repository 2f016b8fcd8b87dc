"""Arguments of the operators around the quantizer at the edges of what they
take, on the host: every check runs before a device is touched."""
import pytest
import torch

import nvfp4_adaptive_block_amd as fos
from test_operators_host import C, INVALID, O, P, SHAPE, linear, operand

DEVICE = 6  # where there is no GPU, what a call that passes every check ends with


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


@pytest.mark.parametrize("kw", [
    dict(x=operand(0, type=3, gran=1, scale=0), M=0, y=0), dict(x=operand(0, 0, 0, 4, 1), M=0, y=0),
    dict(x=operand(0, type=3, gran=1, scale=0), M=0, y=0, G=2, offs=P(O)),
    dict(w=operand(0, 0, 0, 4, 1), N=0, y=0), dict(w=operand(0, 0, 0, 4, 1), N=0, y=0, G=2, offs=P(O)),
])
def test_operands_without_rows_need_no_row_scales(kw):
    """A tensor without elements has no address."""
    assert linear(**kw) in (0, DEVICE)


@pytest.mark.parametrize("kw", [dict(x=operand(type=3, gran=1, scale=0)), dict(x=operand(0, 0, 0, 4, 0), M=0, y=0),
                                dict(x=operand(0, type=3, scale=0), M=0, y=0), dict(w=operand(C, scale=0, gran=1)),
                                dict(w=operand(0, 0, 0, 4, 2), N=0, y=0, G=2, offs=P(O))])
def test_scales_that_there_are_are_needed(kw):
    assert linear(**kw) == INVALID


def test_a_status_without_elements_is_refused():
    host = torch.device("cpu")  # the checks are the same for any device
    word = torch.zeros(1, dtype=torch.int32)
    assert fos._status_pointer(word, host) == word.data_ptr()
    for bad in (torch.zeros(0, dtype=torch.int32), torch.zeros(3, 0, dtype=torch.int32), word[:0]):
        with pytest.raises(ValueError, match="must hold a value"):
            fos._status_pointer(bad, host)
