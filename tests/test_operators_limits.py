"""The language-model operators' binding at sizes of zero, without a GPU."""
import os

import pytest
import torch


@pytest.fixture(scope="module")
def ibp():
    import bit_packing_amd

    if not os.path.exists(bit_packing_amd.LIB_PATH):
        from bit_packing_amd.build import build_library
        build_library()
    bit_packing_amd.load_library()
    return bit_packing_amd


@pytest.mark.parametrize("shape,rows,cols", [((5, 0), 5, 0), ((2, 3, 0), 6, 0), ((0, 7), 0, 7), ((2, 0, 7), 0, 7), ((0, 0), 0, 0),
                                             ((4, 64), 4, 64), ((2, 3, 5), 6, 5), ((9,), 1, 9), ((0,), 1, 0)])
def test_rows_of_a_tensor(ibp, shape, rows, cols):
    assert ibp._matrix(torch.zeros(shape)) == (rows, cols)


def test_a_backward_pass_of_another_shape_is_refused(ibp):
    gate8 = ibp.make_mx(4, 64, ibp.IBP_MX_E4M3, "cpu")
    for shape in ((0, 64), (4, 0), (4, 32), (5, 64)):
        with pytest.raises(ValueError):
            ibp.ibp_mx_swiglu_backward(torch.zeros(shape), gate8, gate8)
