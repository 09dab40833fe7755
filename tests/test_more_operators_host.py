"""8-bit integer rows and experts without a GPU: size queries, refusals of the C entry points
before any HIP call, refusals of the binding, and the plain definitions of the GPU tests."""
import ctypes
import fractions
import os

import numpy as np
import pytest
import torch

import i8_ref

FAKE = 0x10000  # never dereferenced: every call below fails its host checks first
FAR = 0x40000000000
F32, F16, BF16 = 0, 1, 2


@pytest.fixture(scope="module")
def ibp():
    import bit_packing_amd

    if not os.path.exists(bit_packing_amd.LIB_PATH):
        from bit_packing_amd.build import build_library
        build_library()
    bit_packing_amd.load_library()
    return bit_packing_amd


def i8(ibp, rows=4, cols=64, codes=FAKE, scales=2 * FAKE):
    return ibp.ibp_i8_t(rows, cols, codes, scales)


def mx(ibp, fmt=0, rows=4, cols=64, codes=FAKE, scales=2 * FAKE, reserved=0):
    return ibp.ibp_mx_t(fmt, reserved, rows, cols, codes, scales)


def ref(t):
    return ctypes.byref(t)


def test_queries(ibp):
    for cols in (0, 1, 15, 16, 17, 4001):
        assert ibp.ibp_i8_codes_pitch(cols) == i8_ref.pitch(cols)
    assert ibp.ibp_i8_codes_pitch(ibp.IBP_MAX_COLS + 1) == 0
    assert ibp.ibp_i8_matmul_workspace_bytes(0, 5, 64) == 0
    assert ibp.ibp_i8_matmul_workspace_bytes(5, 5, ibp.IBP_I8_MAX_DEPTH + 1) == 0
    assert ibp.ibp_expert_order_workspace_bytes(64, 64) == 0
    assert ibp.ibp_expert_order_workspace_bytes(1 << 20, 64) > 0
    assert ibp.ibp_expert_order_workspace_bytes(ibp.IBP_MAX_TOKENS, 64) == 0
    assert ibp.ibp_expert_order_workspace_bytes(1 << 20, ibp.IBP_MAX_EXPERTS + 1) == 0
    assert ibp.ibp_mx_grouped_wgrad_workspace_bytes(10, 0, 8, 32) == 0
    assert ibp.ibp_mx_grouped_wgrad_workspace_bytes(10, 2, 8, 32, torch.float32) >= 3 * 10 * 8 * 2
    lib = ibp.load_library()
    assert lib.ibp_mx_grouped_wgrad_workspace_bytes(10, 2, 8, 32, BF16, FAKE) == 0  # taken as it lies
    assert lib.ibp_mx_grouped_wgrad_workspace_bytes(10, 2, 8, 32, BF16, FAKE + 2) == 10 * 8 * 2
    assert lib.ibp_mx_grouped_wgrad_workspace_bytes(10, 2, 9, 32, BF16, FAKE) == 10 * 16 * 2
    assert lib.ibp_mx_grouped_wgrad_workspace_bytes(10, 2, 8, 32, BF16, None) == 10 * 8 * 2


def test_i8_refusals(ibp):
    lib = ibp.load_library()
    bad = [(dict(cols=ibp.IBP_MAX_COLS + 1), ibp.IBP_ERR_SIZE), (dict(rows=1 << 62), ibp.IBP_ERR_SIZE),
           (dict(codes=FAKE + 8), ibp.IBP_ERR_INVALID_ARG), (dict(scales=FAKE + 2), ibp.IBP_ERR_INVALID_ARG),
           (dict(codes=None), ibp.IBP_ERR_INVALID_ARG), (dict(scales=None), ibp.IBP_ERR_INVALID_ARG)]
    good = i8(ibp)
    for kw, want in bad:
        t = i8(ibp, **kw)
        assert lib.ibp_i8_pack(FAR, F32, ref(t), None) == want, kw
        assert lib.ibp_i8_unpack(ref(t), FAR, F32, None) == want, kw
        assert lib.ibp_i8_matmul(ref(t), ref(good), FAR, F32, None, 0, None) == want, kw
        assert lib.ibp_i8_matmul(ref(good), ref(t), FAR, F32, None, 0, None) == want, kw
    no = ibp.IBP_ERR_INVALID_ARG
    assert lib.ibp_i8_pack(FAR, 3, ref(good), None) == no
    assert lib.ibp_i8_pack(None, F32, ref(good), None) == no
    assert lib.ibp_i8_pack(FAR + 2, F32, ref(good), None) == no
    assert lib.ibp_i8_pack(FAR, F32, None, None) == no
    assert lib.ibp_i8_pack(FAKE + 64, F32, ref(good), None) == no  # the input is what is written
    assert lib.ibp_i8_unpack(ref(good), None, F32, None) == no
    assert lib.ibp_i8_unpack(ref(good), FAR + 1, BF16, None) == no
    assert lib.ibp_i8_unpack(ref(good), 2 * FAKE - 16, F32, None) == no  # the output lies over the scales
    assert lib.ibp_i8_matmul(ref(good), ref(good), FAKE, F32, None, 0, None) == no
    assert lib.ibp_i8_matmul(ref(good), ref(good), FAR, 5, None, 0, None) == no
    assert lib.ibp_i8_matmul(ref(good), ref(good), None, F32, None, 0, None) == no
    assert lib.ibp_i8_matmul(ref(good), ref(good), FAR, F32, FAR + 4, 0, None) == no
    assert lib.ibp_i8_matmul(ref(good), ref(i8(ibp, cols=65)), FAR, F32, None, 0, None) == ibp.IBP_ERR_SIZE
    deep = i8(ibp, cols=ibp.IBP_I8_MAX_DEPTH + 1)
    assert lib.ibp_i8_matmul(ref(deep), ref(deep), FAR, F32, None, 0, None) == ibp.IBP_ERR_SIZE
    many = i8(ibp, rows=(1 << 30) + 1)
    assert lib.ibp_i8_matmul(ref(many), ref(good), FAR, F32, None, 0, None) == ibp.IBP_ERR_SIZE
    assert lib.ibp_i8_pack(None, F32, ref(i8(ibp, rows=0)), None) == ibp.IBP_OK
    assert lib.ibp_i8_unpack(ref(i8(ibp, cols=0)), None, F32, None) == ibp.IBP_OK
    assert lib.ibp_i8_matmul(ref(i8(ibp, rows=0)), ref(good), None, F32, None, 0, None) == ibp.IBP_OK


def test_i8_workspace_refusals(ibp):
    lib = ibp.load_library()
    a, b = i8(ibp, rows=128, cols=8192), i8(ibp, rows=1024, cols=8192, codes=FAR, scales=2 * FAR)
    need = ibp.ibp_i8_matmul_workspace_bytes(128, 1024, 8192)
    if need:
        assert lib.ibp_i8_matmul(ref(a), ref(b), 4 * FAR, F32, 8 * FAR, need - 1, None) == ibp.IBP_ERR_CAPACITY
        assert lib.ibp_i8_matmul(ref(a), ref(b), 4 * FAR, F32, None, need, None) == ibp.IBP_ERR_INVALID_ARG
        assert lib.ibp_i8_matmul(ref(a), ref(b), 4 * FAR, F32, 4 * FAR, need, None) == ibp.IBP_ERR_INVALID_ARG


def test_order_refusals(ibp):
    f = ibp.load_library().ibp_expert_order
    call = lambda ids=FAKE, n=100, e=8, order=2 * FAKE, offsets=3 * FAKE, w=None, wb=0, err=None: f(  # noqa: E731
        ids, n, e, order, offsets, w, wb, err, None)
    no = ibp.IBP_ERR_INVALID_ARG
    assert call(e=0) == ibp.IBP_ERR_SIZE
    assert call(e=ibp.IBP_MAX_EXPERTS + 1) == ibp.IBP_ERR_SIZE
    assert call(n=ibp.IBP_MAX_TOKENS) == ibp.IBP_ERR_SIZE
    assert call(ids=None) == no and call(order=None) == no and call(offsets=None) == no
    assert call(offsets=None, n=0) == no
    assert call(ids=FAKE + 4) == no and call(order=FAR + 4) == no and call(offsets=FAR + 4) == no and call(err=FAKE + 1) == no
    assert call(order=FAKE + 8) == no and call(offsets=FAKE) == no and call(offsets=2 * FAKE + 80) == no  # overlaps
    n = 1 << 20
    need = ibp.ibp_expert_order_workspace_bytes(n, 8)
    far = dict(n=n, ids=FAR, order=2 * FAR, offsets=3 * FAR, w=4 * FAR)
    assert call(**far, wb=need - 1) == ibp.IBP_ERR_CAPACITY
    assert call(**{**far, "w": None}, wb=need) == no
    assert call(**{**far, "w": 4 * FAR + 8}, wb=need) == no
    assert call(**{**far, "w": 2 * FAR}, wb=need) == no


def test_grouped_refusals(ibp):
    lib = ibp.load_library()
    a, b, no = mx(ibp), mx(ibp, fmt=1, rows=24, codes=3 * FAKE, scales=4 * FAKE), ibp.IBP_ERR_INVALID_ARG
    call = lambda a=a, b=b, off=5 * FAKE, n=8, y=FAR, t=F32, err=None: lib.ibp_mx_grouped_matmul(  # noqa: E731
        ref(a), ref(b), off, n, y, t, err, None)
    assert call(t=7) == no and call(b=mx(ibp, rows=24)) == no and call(a=mx(ibp, reserved=1)) == no
    assert call(n=0) == ibp.IBP_ERR_SIZE and call(n=ibp.IBP_MAX_EXPERTS + 1) == ibp.IBP_ERR_SIZE
    assert call(n=7) == ibp.IBP_ERR_SIZE  # 24 rows of weights
    assert call(a=mx(ibp, cols=65)) == ibp.IBP_ERR_SIZE
    assert call(a=mx(ibp, rows=(1 << 30) + 1)) == ibp.IBP_ERR_SIZE
    assert call(off=None) == no and call(off=FAKE + 4) == no and call(y=None) == no and call(y=FAR + 2) == no
    assert call(err=FAKE + 2) == no
    assert call(y=FAKE) == no and call(y=5 * FAKE) == no  # over the rows, over the offsets
    assert call(a=mx(ibp, rows=0)) == ibp.IBP_OK and call(b=mx(ibp, fmt=1, rows=0)) == ibp.IBP_OK

    x8 = mx(ibp)
    need = ibp.ibp_mx_grouped_wgrad_workspace_bytes(4, 3, 8, 64, torch.bfloat16)
    call = lambda dy=FAR, t=BF16, outs=8, x=x8, off=5 * FAKE, n=3, dw=2 * FAR, to=F32, w=4 * FAR, wb=1 << 20, err=None: (  # noqa: E731
        lib.ibp_mx_grouped_wgrad(dy, t, outs, ref(x), off, n, dw, to, w, wb, err, None))
    assert call(t=3) == no and call(to=-1) == no and call(x=mx(ibp, fmt=1)) == no
    assert call(n=0) == ibp.IBP_ERR_SIZE and call(n=ibp.IBP_MAX_EXPERTS + 1) == ibp.IBP_ERR_SIZE
    assert call(outs=(1 << 30) + 1) == ibp.IBP_ERR_SIZE and call(x=mx(ibp, rows=ibp.IBP_MAX_TOKENS)) == ibp.IBP_ERR_SIZE
    assert call(dy=None) == no and call(dw=None) == no and call(off=None) == no and call(off=FAKE + 4) == no
    assert call(dy=FAR + 1) == no and call(dw=FAR + 2) == no and call(w=FAR + 8) == no and call(err=FAKE + 2) == no
    assert call(dw=FAR) == no and call(dw=4 * FAR) == no  # over dy, over the workspace
    assert need > 0 and call(dy=FAR + 2, wb=need - 1) == ibp.IBP_ERR_CAPACITY and call(dy=FAR + 2, w=None) == no
    assert call(t=F32, wb=0) == ibp.IBP_ERR_CAPACITY
    assert call(outs=0, dw=None) == ibp.IBP_OK


def test_binding_refusals(ibp):
    x = torch.zeros(4, 64)
    off = torch.zeros(3, dtype=torch.int64)
    m8 = ibp.MxTensor(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8), 4, 64, 0)
    m4 = ibp.MxTensor(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8), 4, 64, 1)
    with pytest.raises(ValueError):
        ibp.ibp_i8_pack(torch.zeros(()))
    with pytest.raises(ValueError):
        ibp.ibp_i8_pack(torch.zeros(4, 64, dtype=torch.int8))
    with pytest.raises(ValueError):
        ibp.ibp_i8_pack(x, out=ibp.make_i8(4, 65, "cpu"))
    with pytest.raises(ValueError):
        ibp.I8Tensor(torch.zeros(4, 48, dtype=torch.int8), torch.zeros(4), 4, 64).struct()
    with pytest.raises(ValueError):
        ibp.I8Tensor(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(3), 4, 64).struct()
    with pytest.raises(ValueError):
        ibp.I8Tensor(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4), 4, 64).struct()
    with pytest.raises(ValueError):
        ibp.ibp_expert_order(torch.zeros(4, dtype=torch.int32), 4)
    for bad in (off.int(), off[:1], off.view(1, 3)):
        with pytest.raises(ValueError):
            ibp.ibp_mx_grouped_matmul(m8, m4, bad)
        with pytest.raises(ValueError):
            ibp.ibp_mx_grouped_wgrad(torch.zeros(4, 8, dtype=torch.bfloat16), m8, bad)
    with pytest.raises(ValueError):
        ibp.ibp_mx_grouped_matmul(m8, m4, torch.zeros(4, dtype=torch.int64))  # 4 rows of weights, 3 experts
    with pytest.raises(ValueError):
        ibp.ibp_mx_grouped_wgrad(torch.zeros(5, 8, dtype=torch.bfloat16), m8, off)


# ---------------------------------------------------------------- the plain definitions

@pytest.mark.parametrize("t", [torch.float32, torch.float16, torch.bfloat16])
def test_plain_codes_are_the_nearest(t):
    """Against fractions, which round the quotient itself, at random values and next to borders."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((6, 60))
    x[1] = x[1, 0] * (rng.integers(-126, 126, 60) + 0.5) / 127  # near borders
    x[2, 1:] = x[2, 0] / 2
    x[3] *= 1e-7
    x[4] = 0
    x = torch.from_numpy(x).to(t).double().numpy()
    codes, scales = i8_ref.pack(x)
    for r in range(6):
        m = max(fractions.Fraction(float(abs(v))) for v in x[r])
        for c in range(60):
            want = round(fractions.Fraction(float(x[r, c])) * 127 / m) if m else 0
            assert codes[r, c] == want
    assert np.array_equal(scales, np.abs(x).max(1).astype(np.float32) / np.float32(127))


def test_plain_product_and_order():
    a, b = np.array([[1, -128], [127, 3]], np.int8), np.array([[2, 4], [-5, 127], [0, 1]], np.int8)
    y = i8_ref.product(a, np.float32([0.5, 2]), b, np.float32([1, 2, 0.25]))
    assert np.array_equal(y, np.float32([[-255, -16261, -16], [532, -1016, 1.5]]))
    order, off = i8_ref.order(np.array([2, 0, -1, 2, 5, 0]), 4)
    assert list(order) == [1, 5, 0, 3, 2, 4] and list(off) == [0, 2, 2, 4, 4]


def test_plain_grouped_gradient_is_the_derivative():
    rng = np.random.default_rng(4)
    off = [0, 3, 3, 7]
    x, w, dy = rng.standard_normal((7, 5)), rng.standard_normal((3, 4, 5)), rng.standard_normal((7, 4))
    loss = lambda w: (i8_ref.grouped_product(x, w, off, np.zeros((7, 4))) * dy).sum()  # noqa: E731
    g = i8_ref.grouped_wgrad(dy, x, off)
    for e in range(3):
        for o in range(4):
            for i in range(5):
                d = np.zeros_like(w)
                d[e, o, i] = 1e-4
                assert abs((loss(w + d) - loss(w - d)) / 2e-4 - g[e, o, i]) < 1e-8
