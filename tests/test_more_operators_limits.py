"""8-bit integers without a GPU: the workspace of a product whose depth is cut."""
import ctypes
import os

import pytest

FAR = 0x40000000000  # never dereferenced: every call below fails its host checks first


@pytest.fixture(scope="module")
def ibp():
    import bit_packing_amd

    if not os.path.exists(bit_packing_amd.LIB_PATH):
        from bit_packing_amd.build import build_library
        build_library()
    bit_packing_amd.load_library()
    return bit_packing_amd


def test_a_cut_product_needs_its_workspace(ibp):
    lib = ibp.load_library()
    need = ibp.ibp_i8_matmul_workspace_bytes(128, 1024, 8192)
    assert need > 0 and need % (128 * 1024 * 4) == 0
    a, b = ibp.ibp_i8_t(128, 8192, FAR, 2 * FAR), ibp.ibp_i8_t(1024, 8192, 3 * FAR, 4 * FAR)
    call = lambda w, bytes: lib.ibp_i8_matmul(ctypes.byref(a), ctypes.byref(b), 5 * FAR, 0, w, bytes, None)  # noqa: E731
    assert call(8 * FAR, need - 1) == ibp.IBP_ERR_CAPACITY
    assert call(8 * FAR, 0) == ibp.IBP_ERR_CAPACITY
    assert call(None, need) == ibp.IBP_ERR_INVALID_ARG
    assert call(8 * FAR + 8, need) == ibp.IBP_ERR_INVALID_ARG
    for over in (FAR, 2 * FAR, 3 * FAR, 4 * FAR, 5 * FAR):  # over the operands, over the output
        assert call(over, need) == ibp.IBP_ERR_INVALID_ARG
