"""The language-model operators without a GPU: the binding at sizes of zero, and which
outputs may lie where an input does."""
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


# ---------------------------------------------------------------- outputs that overlap inputs

def apart(cols):
    """The rule, from how the kernels lay rows on lanes: lane i of a row writes its elements
    from 8 i on and reads them too, the last lane of a row that is no multiple of 8 reads the
    last eight elements of the row.  Wavefronts are 64 lanes; one reads before it writes."""
    lanes = -(-cols // 8)
    reads = [range(8 * i, 8 * i + 8) if 8 * i + 8 <= cols else range(max(cols - 8, 0), cols) for i in range(lanes)]
    writer = [e // 8 for e in range(cols)]
    return all(writer[e] // 64 == i // 64 or writer[e] == i for i in range(lanes) for e in reads[i])


def test_which_rows_may_be_written_in_place():
    """Where the rule allows it no lane reads what another wavefront writes, and it refuses
    rows of which one does."""
    assert all(apart(cols) for cols in range(1, 3000) if cols % 8 == 0 or cols <= 512)
    assert not any(apart(cols) for cols in (513, 519, 1025, 1031, 1537, 2049))
