"""The language-model operators without a GPU: size queries, refusals of the C entry
points before any HIP call, and the plain definitions the GPU tests use."""
import ctypes
import os

import numpy as np
import pytest
import torch

import mx_ref

FAKE = 0x10000  # never dereferenced: every call below fails its host checks first
F32, F16, BF16 = 0, 1, 2


@pytest.fixture(scope="module")
def ibp():
    import bit_packing_amd

    if not os.path.exists(bit_packing_amd.LIB_PATH):
        from bit_packing_amd.build import build_library
        build_library()
    bit_packing_amd.load_library()
    return bit_packing_amd


def mx(ibp, fmt=0, rows=4, cols=64, codes=FAKE, scales=FAKE, reserved=0):
    return ibp.ibp_mx_t(fmt, reserved, rows, cols, codes, scales)


def ref(t):
    return ctypes.byref(t)


def test_pitches(ibp):
    for cols in (0, 1, 31, 32, 33, 128, 129, 4001):
        assert ibp.ibp_mx_codes_pitch(cols, ibp.IBP_MX_E4M3) == mx_ref.pitch(cols, mx_ref.E4M3)
        assert ibp.ibp_mx_codes_pitch(cols, ibp.IBP_MX_E2M1) == mx_ref.pitch(cols, mx_ref.E2M1)
        assert ibp.ibp_mx_scales_pitch(cols) == mx_ref.scale_pitch(cols)
    assert ibp.ibp_mx_codes_pitch(32, 2) == 0
    assert ibp.ibp_mx_codes_pitch(ibp.IBP_MAX_COLS + 1, 0) == 0
    assert ibp.ibp_mx_scales_pitch(ibp.IBP_MAX_COLS + 1) == 0


def test_workspace_queries(ibp):
    assert ibp.ibp_embedding_grad_workspace_bytes(1 << 32, 10, 8) == 0
    assert ibp.ibp_embedding_grad_workspace_bytes(100, 1 << 31, 8) == 0
    assert ibp.ibp_embedding_grad_workspace_bytes(100, 10, 8) > 0
    assert ibp.ibp_mx_matmul_workspace_bytes(0, 10, 32, 0) == 0
    assert ibp.ibp_mx_matmul_workspace_bytes(10, 10, 32, 7) == 0
    assert ibp.ibp_mx_linear_wgrad_workspace_bytes(10, 0, 32) == 0
    lib = ibp.load_library()
    assert lib.ibp_mx_linear_wgrad_workspace_bytes(10, 8, 32, 7) == 0
    assert lib.ibp_mx_linear_wgrad_workspace_bytes(10, 8, 32, BF16) == 0  # one range, written as it is
    assert lib.ibp_mx_linear_wgrad_workspace_bytes(10, 8, 32, F16) == 2 * 8 * 32 * 4
    assert lib.ibp_mx_linear_wgrad_workspace_bytes(10, 8, 32, F32) == 3 * 8 * 32 * 4


def test_lookup_refusals(ibp):
    f = ibp.load_library().ibp_embedding_lookup
    call = lambda table=FAKE, td=F32, rows=10, dim=8, ids=FAKE, n=4, out=FAKE, od=F32, err=None: f(  # noqa: E731
        table, td, rows, dim, ids, n, 1.0, out, od, err, None)
    assert call(td=3) == ibp.IBP_ERR_INVALID_ARG
    assert call(od=-1) == ibp.IBP_ERR_INVALID_ARG
    assert call(rows=0) == ibp.IBP_ERR_SIZE
    assert call(dim=ibp.IBP_MAX_COLS + 1) == ibp.IBP_ERR_SIZE
    assert call(rows=1 << 62) == ibp.IBP_ERR_SIZE
    assert call(n=1 << 62) == ibp.IBP_ERR_SIZE
    assert call(table=None) == ibp.IBP_ERR_INVALID_ARG
    assert call(ids=None) == ibp.IBP_ERR_INVALID_ARG
    assert call(out=None) == ibp.IBP_ERR_INVALID_ARG
    assert call(table=FAKE + 2) == ibp.IBP_ERR_INVALID_ARG
    assert call(ids=FAKE + 4) == ibp.IBP_ERR_INVALID_ARG
    assert call(out=FAKE + 1, od=F16) == ibp.IBP_ERR_INVALID_ARG
    assert call(err=FAKE + 1) == ibp.IBP_ERR_INVALID_ARG
    assert call(n=0) == ibp.IBP_OK and call(dim=0) == ibp.IBP_OK  # nothing to write


def test_grad_refusals(ibp):
    f = ibp.load_library().ibp_embedding_grad
    ws = ibp.ibp_embedding_grad_workspace_bytes(10, 4, 8)
    call = lambda dout=FAKE, dd=F32, ids=FAKE, n=4, rows=10, dim=8, pad=-1, grad=FAKE, gd=F32, w=FAKE, wb=ws, err=None: f(  # noqa: E731
        dout, dd, ids, n, rows, dim, 1.0, pad, grad, gd, w, wb, err, None)
    assert call(dd=5) == ibp.IBP_ERR_INVALID_ARG
    assert call(gd=5) == ibp.IBP_ERR_INVALID_ARG
    assert call(pad=-2) == ibp.IBP_ERR_INVALID_ARG
    assert call(rows=0) == ibp.IBP_ERR_SIZE
    assert call(rows=(1 << 32) - 1) == ibp.IBP_ERR_SIZE
    assert call(n=ibp.IBP_MAX_TOKENS) == ibp.IBP_ERR_SIZE
    assert call(dim=ibp.IBP_MAX_COLS + 1) == ibp.IBP_ERR_SIZE
    assert call(wb=ws - 1) == ibp.IBP_ERR_CAPACITY
    assert call(w=None) == ibp.IBP_ERR_INVALID_ARG
    assert call(w=FAKE + 8) == ibp.IBP_ERR_INVALID_ARG
    assert call(dout=None) == ibp.IBP_ERR_INVALID_ARG
    assert call(grad=None) == ibp.IBP_ERR_INVALID_ARG
    assert call(dout=FAKE + 1) == ibp.IBP_ERR_INVALID_ARG
    assert call(rows=0, n=0) == ibp.IBP_OK


def test_pack_refusals(ibp):
    lib = ibp.load_library()
    bad = [(dict(fmt=2), ibp.IBP_ERR_INVALID_ARG), (dict(reserved=1), ibp.IBP_ERR_INVALID_ARG),
           (dict(cols=ibp.IBP_MAX_COLS + 1), ibp.IBP_ERR_SIZE), (dict(rows=1 << 62), ibp.IBP_ERR_SIZE),
           (dict(codes=FAKE + 8), ibp.IBP_ERR_INVALID_ARG), (dict(scales=FAKE + 2), ibp.IBP_ERR_INVALID_ARG),
           (dict(codes=None), ibp.IBP_ERR_INVALID_ARG), (dict(scales=None), ibp.IBP_ERR_INVALID_ARG)]
    good = mx(ibp)
    for kw, want in bad:
        t = mx(ibp, **kw)
        assert lib.ibp_mx_pack(FAKE, F32, ref(t), None) == want, kw
        assert lib.ibp_mx_unpack(ref(t), FAKE, F32, None) == want, kw
        assert lib.ibp_mx_swiglu(FAKE, FAKE, F32, FAKE, ref(t), ref(good), None) == want, kw
        assert lib.ibp_mx_swiglu_backward(FAKE, F32, ref(good), ref(t), FAKE, FAKE, None) == want, kw
        assert lib.ibp_mx_linear_wgrad(FAKE, BF16, 8, ref(t), FAKE, F32, None, 0, None) == want, kw
        w = mx(ibp, fmt=1, cols=t.cols)
        assert lib.ibp_mx_matmul(ref(t), ref(w), FAKE, F32, None, 0, None) == want, kw
    assert lib.ibp_mx_pack(FAKE, 3, ref(good), None) == ibp.IBP_ERR_INVALID_ARG
    assert lib.ibp_mx_pack(None, F32, ref(good), None) == ibp.IBP_ERR_INVALID_ARG
    assert lib.ibp_mx_pack(FAKE + 2, F32, ref(good), None) == ibp.IBP_ERR_INVALID_ARG
    assert lib.ibp_mx_pack(FAKE, F32, None, None) == ibp.IBP_ERR_INVALID_ARG
    assert lib.ibp_mx_unpack(ref(good), FAKE + 1, BF16, None) == ibp.IBP_ERR_INVALID_ARG
    assert lib.ibp_mx_pack(FAKE, F32, ref(mx(ibp, rows=0)), None) == ibp.IBP_OK


def test_gated_refusals(ibp):
    lib = ibp.load_library()
    g, four, other = mx(ibp), mx(ibp, fmt=1), mx(ibp, cols=65)
    assert lib.ibp_mx_swiglu(FAKE, FAKE, F32, FAKE, ref(g), ref(four), None) == ibp.IBP_ERR_INVALID_ARG
    assert lib.ibp_mx_swiglu(FAKE, FAKE, F32, FAKE, ref(g), ref(other), None) == ibp.IBP_ERR_SIZE
    assert lib.ibp_mx_swiglu(FAKE, None, F32, FAKE, ref(g), ref(g), None) == ibp.IBP_ERR_INVALID_ARG
    assert lib.ibp_mx_swiglu_backward(FAKE, F32, ref(g), ref(g), FAKE, FAKE + 2, None) == ibp.IBP_ERR_INVALID_ARG
    assert lib.ibp_mx_swiglu_backward(FAKE, 9, ref(g), ref(g), FAKE, FAKE, None) == ibp.IBP_ERR_INVALID_ARG


def test_product_refusals(ibp):
    lib = ibp.load_library()
    a, w = mx(ibp), mx(ibp, fmt=1)
    assert lib.ibp_mx_matmul(ref(a), ref(a), FAKE, F32, None, 0, None) == ibp.IBP_ERR_INVALID_ARG  # b not e2m1
    assert lib.ibp_mx_matmul(ref(a), ref(mx(ibp, fmt=1, cols=96)), FAKE, F32, None, 0, None) == ibp.IBP_ERR_SIZE
    assert lib.ibp_mx_matmul(ref(a), ref(w), FAKE, 4, None, 0, None) == ibp.IBP_ERR_INVALID_ARG
    assert lib.ibp_mx_matmul(ref(a), ref(w), None, F32, None, 0, None) == ibp.IBP_ERR_INVALID_ARG
    assert lib.ibp_mx_matmul(ref(a), ref(w), FAKE, F32, FAKE + 4, 0, None) == ibp.IBP_ERR_INVALID_ARG
    assert lib.ibp_mx_matmul(ref(mx(ibp, rows=(1 << 30) + 1)), ref(w), FAKE, F32, None, 0, None) == ibp.IBP_ERR_SIZE
    assert lib.ibp_mx_linear_wgrad(FAKE, 3, 8, ref(a), FAKE, F32, None, 0, None) == ibp.IBP_ERR_INVALID_ARG
    assert lib.ibp_mx_linear_wgrad(FAKE, F32, 8, ref(a), FAKE, F32, None, 0, None) == ibp.IBP_ERR_CAPACITY  # its parts are joined
    assert lib.ibp_mx_linear_wgrad(FAKE + 1, BF16, 8, ref(a), FAKE, F32, None, 0, None) == ibp.IBP_ERR_INVALID_ARG
    assert lib.ibp_mx_linear_wgrad(FAKE, BF16, 8, ref(w), FAKE, F32, None, 0, None) == ibp.IBP_ERR_INVALID_ARG  # x8 not e4m3
    assert lib.ibp_mx_linear_wgrad(FAKE, BF16, (1 << 30) + 1, ref(a), FAKE, F32, None, 0, None) == ibp.IBP_ERR_SIZE
    assert lib.ibp_mx_linear_wgrad(None, BF16, 8, ref(a), FAKE, F32, None, 0, None) == ibp.IBP_ERR_INVALID_ARG
    big = mx(ibp, rows=1 << 20, cols=64)
    need = ibp.ibp_mx_linear_wgrad_workspace_bytes(1 << 20, 8, 64)
    assert need > 0
    assert lib.ibp_mx_linear_wgrad(FAKE, BF16, 8, ref(big), FAKE, F32, FAKE, need - 1, None) == ibp.IBP_ERR_CAPACITY


def test_binding_refusals(ibp):
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        ibp.ibp_embedding_lookup(torch.zeros(4), torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        ibp.ibp_embedding_lookup(x, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        ibp.ibp_embedding_grad(x, torch.zeros(3, dtype=torch.int64), 10)
    with pytest.raises(ValueError):
        ibp.ibp_mx_pack(x, 2)
    with pytest.raises(ValueError):
        ibp.ibp_mx_swiglu(x, torch.zeros(4, 32))
    short = ibp.MxTensor(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8), 4, 64, 0)
    with pytest.raises(ValueError):
        short.struct()  # codes hold fewer bytes than 4 x 64
    with pytest.raises(ValueError):
        ibp.ibp_mx_linear_wgrad(torch.zeros(5, 8, dtype=torch.bfloat16), ibp.MxTensor(
            torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8), 4, 64, 0))


# ---------------------------------------------------------------- the plain definitions

@pytest.mark.parametrize("fmt", [mx_ref.E4M3, mx_ref.E2M1])
def test_plain_packing_bounds(fmt):
    """No element clips and each is off by at most half the step of its size: relative
    2^-4 (e4m3) or 2^-2 (e2m1) in the normal range, half the smallest code below."""
    rng = np.random.default_rng(fmt)
    x = rng.standard_normal((50, 101)) * 2.0 ** rng.integers(-60, 60, (50, 1))
    c, s = mx_ref.pack(x, fmt)
    y = mx_ref.unpack(c, s, 101, fmt)
    step = mx_ref.TABLE[fmt][1]
    scale = np.repeat(2.0 ** (s[:, :4].astype(float) - 127), 32, axis=1)[:, :101]
    half = 2.0 ** (-4 if fmt == mx_ref.E4M3 else -2)
    assert np.all(np.abs(y - x) <= np.maximum(half * np.abs(x), step / 2 * scale))
    again = mx_ref.unpack(*mx_ref.pack(y, fmt), 101, fmt)
    assert np.array_equal(again, y)  # packed values pack to themselves


def test_plain_e4m3_table_is_the_type():
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, mx_ref.TABLE[mx_ref.E4M3])


def test_plain_backward_is_the_derivative():
    rng = np.random.default_rng(1)
    g, u, dh = (rng.standard_normal((5, 7)) * 3 for _ in range(3))
    dg, du = mx_ref.swiglu_backward(dh, g, u)
    e = 1e-6
    ng = dh * (mx_ref.swiglu(g + e, u) - mx_ref.swiglu(g - e, u)) / (2 * e)
    nu = dh * (mx_ref.swiglu(g, u + e) - mx_ref.swiglu(g, u - e)) / (2 * e)
    assert np.allclose(dg, ng, atol=1e-7) and np.allclose(du, nu, atol=1e-7)


def test_plain_embedding_grad_is_the_derivative():
    rng = np.random.default_rng(2)
    table, ids = rng.standard_normal((6, 3)), np.array([1, 4, 1, 0, 5, 1])
    dout = rng.standard_normal((6, 3))
    g, _, n = mx_ref.embedding_grad(dout, ids, 6, 2.5, padding=4)
    loss = lambda t: float((2.5 * t[ids] * dout)[ids != 4].sum())  # noqa: E731
    for v in range(6):
        for c in range(3):
            d = np.zeros_like(table)
            d[v, c] = 1e-4
            assert abs((loss(table + d) - loss(table - d)) / 2e-4 - g[v, c]) < 1e-8
    assert list(n) == [1, 3, 0, 0, 0, 1]
