"""8-bit integer rows and layers of experts on the GPU where test_gpu_more_operators.py does
not reach: what two roundings make of a border, and every form of the kernels."""
import numpy as np
import pytest
import torch

import i8_ref

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def ibp():
    import bit_packing_amd

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    bit_packing_amd.load_library()
    return bit_packing_amd


def host(x):
    return x.double().cpu().numpy()


def rounded(x, t):
    """float32 values rounded to a type, as float64."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(DT[t]).double().numpy()


def i8(ibp, codes, scales, cols):
    return ibp.I8Tensor(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), codes.shape[0], cols)


# ---------------------------------------------------------------- two roundings

def next_to_borders(n, seed):
    """n codes and scales between 1 and 2 whose products, rounded to 32 bits, lie on a border
    between two half-precision numbers that the products themselves do not lie on: rounded at
    once they come out as the other one."""
    rng = np.random.default_rng(seed)
    codes, scales = [], []
    while len(codes) < n:
        q = rng.integers(3, 128, 1 << 18)
        s = (1 + rng.random(1 << 18)).astype(np.float32)
        p = q * s.astype(np.float64)  # exact: 31 bits
        pick = np.flatnonzero(p.astype(np.float16) != p.astype(np.float32).astype(np.float16))
        codes += list(q[pick])
        scales += list(s[pick])
    return np.int8(codes[:n]), np.float32(scales[:n])


@pytest.mark.parametrize("cols", [1, 2, 3, 5, 8, 9, 15, 16, 100, 2001, 2048])
def test_i8_unpack_rounds_to_32_bits_first(ibp, cols):
    q, s = next_to_borders(60, cols)
    codes = np.zeros((60, i8_ref.pitch(cols)), np.int8)
    codes[:, :cols] = q[:, None]
    codes[1::2] *= -1
    want = rounded(codes[:, :cols].astype(np.float32) * s[:, None], "f16")
    assert np.array_equal(host(ibp.ibp_i8_unpack(i8(ibp, codes, s, cols), dtype=torch.float16)), want)


# the direct kernel; small tiles, and with k cut; middle and large tiles
@pytest.mark.parametrize("m,n,k", [(3, 5, 40), (17, 35, 200), (20, 66, 64), (1030, 1001, 100), (300, 201, 5000), (130, 1003, 4200),
                                   (2050, 2049, 100), (3500, 3601, 64)])
def test_i8_matmul_rounds_to_32_bits_first(ibp, m, n, k):
    """Every output is one code times one scale, also at the rows' ends."""
    q, s = next_to_borders(50, m + n)
    for turned in (False, True):
        rows, others = (m, n) if turned else (n, m)
        pick = np.arange(rows) % 50
        a, b = np.zeros((others, i8_ref.pitch(k)), np.int8), np.zeros((rows, i8_ref.pitch(k)), np.int8)
        a[:, k - 1], b[:, k - 1] = 1, q[pick]
        a8, b8 = i8(ibp, a, np.ones(others, np.float32), k), i8(ibp, b, s[pick], k)
        want = np.broadcast_to(rounded(q[pick].astype(np.float32) * s[pick], "f16"), (others, rows))
        got = ibp.ibp_i8_matmul(b8, a8, dtype=torch.float16) if turned else ibp.ibp_i8_matmul(a8, b8, dtype=torch.float16)
        assert np.array_equal(host(got), want.T if turned else want)
