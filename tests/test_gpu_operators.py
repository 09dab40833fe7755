"""The language-model operators on the GPU against plain 64-bit definitions (mx_ref).

Tolerances count roundings: a result rounded once to its type is off by at most half a
step, eps / 2 relative (and half the smallest subnormal); a 32-bit sum of n terms by at
most n 2^-24 of the terms' magnitudes; expf by 2 ulp.  Where all partial sums are whole
multiples of a power of two that 24 bits hold, products are compared for equality.
"""
import numpy as np
import pytest
import torch

import mx_ref

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TINY = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}
U = 2.0 ** -24


@pytest.fixture(scope="module")
def ibp():
    import bit_packing_amd

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    bit_packing_amd.load_library()
    return bit_packing_amd


def half(t):
    return torch.finfo(DT[t]).eps / 2


def gpu(x, t):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DT[t]).cuda()


def host(x):
    return x.double().cpu().numpy()


def within(got, want, bound):
    """|got - want| <= bound, elementwise; equal where want is not finite."""
    got, want = np.asarray(got), np.asarray(want)
    assert got.shape == want.shape
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    over = np.abs(got[fine] - want[fine]) - np.broadcast_to(bound, want.shape)[fine]
    assert over.size == 0 or over.max() <= 0, f"off by {over.max()} more than allowed at {np.argmax(over)} of {over.size}"


def packed(ibp, x, fmt):
    """A float64 matrix packed by the plain definition, as a device MxTensor."""
    c, s = mx_ref.pack(x, fmt)
    return ibp.MxTensor(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), x.shape[0], x.shape[1], fmt)


# ---------------------------------------------------------------- embedding lookup

@pytest.mark.parametrize("ti", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("to", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,dim,n", [(1, 1, 1), (7, 5, 3), (100, 64, 33), (50, 1000, 9), (33, 2049, 130), (300, 4096, 8)])
def test_lookup(ibp, ti, to, rows, dim, n):
    rng = np.random.default_rng(rows * dim + n)
    table = gpu(rng.standard_normal((rows, dim)), ti)
    ids = rng.integers(0, rows, n)
    scale = float(np.float32(dim ** 0.5))
    out = ibp.ibp_embedding_lookup(table, torch.from_numpy(ids).cuda(), scale=scale, out_dtype=DT[to])
    want = host(table)[ids] * scale
    within(host(out), want, np.abs(want) * (half(to) + 2 * U) + TINY[to])


def test_lookup_offset_rows_pinned_and_bad_ids(ibp):
    """A table and an output that start one element into their storage, a pinned table, and
    ids out of range: zero rows and the error bit."""
    rng = np.random.default_rng(5)
    rows, dim = 40, 129
    raw = torch.from_numpy(rng.standard_normal(rows * dim + 1)).to(torch.bfloat16)
    ids = torch.tensor([[3, 39, 0], [-1, 40, 7]])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = raw[1:].view(rows, dim).double().numpy()[ids.numpy().clip(0, 39)]
    want[1, 0] = want[1, 1] = 0
    for table in (raw.cuda()[1:].view(rows, dim), raw.pin_memory()[1:].view(rows, dim)):
        err.zero_()
        flat = torch.full((6 * dim + 2,), 7.0, dtype=torch.bfloat16, device="cuda")
        out = flat[1:-1].view(2, 3, dim)
        got = ibp.ibp_embedding_lookup(table, ids.cuda(), out=out, err=err)
        assert got.data_ptr() == out.data_ptr()
        assert np.array_equal(host(out), want)
        assert flat[0].item() == 7.0 and flat[-1].item() == 7.0
        assert err.item() == ibp.IBP_DEVERR_BAD_ID


def test_lookup_past_32_bit_offsets(ibp):
    """Rows whose element offset needs more than 32 bits."""
    rows, dim = (1 << 20) + 50, 4100
    table = torch.empty(rows, dim, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, rows - 1, 1 << 20, 1047500], device="cuda")
    table[at] = torch.randn(4, dim, device="cuda").to(torch.bfloat16)
    out = ibp.ibp_embedding_lookup(table, at.flip(0).contiguous())
    assert torch.equal(out, table[at.flip(0)])


def test_lookup_of_nothing(ibp):
    out = ibp.ibp_embedding_lookup(torch.zeros(4, 8, device="cuda"), torch.zeros(0, dtype=torch.int64, device="cuda"))
    assert out.shape == (0, 8)


# ---------------------------------------------------------------- embedding gradient

def check_grad(ibp, ids, rows, dim, ti="f32", to="f32", scale=1.0, padding=-1, seed=0):
    rng = np.random.default_rng(seed)
    dout = gpu(rng.standard_normal((len(ids), dim)), ti)
    print(f"embedding gradient: n={len(ids)} rows={rows} dim={dim} {ti}->{to}", flush=True)
    fill = torch.full((rows, dim), float("nan"), dtype=DT[to], device="cuda")
    dev = torch.from_numpy(np.asarray(ids, dtype=np.int64)).cuda()
    got = ibp.ibp_embedding_grad(dout, dev, rows, scale=scale, padding_id=padding, grad=fill)
    want, mag, n = mx_ref.embedding_grad(host(dout), np.asarray(ids), rows, scale, padding)
    within(host(got), want, mag * U * (n[:, None] + 2) + np.abs(want) * half(to) + TINY[to])
    again = ibp.ibp_embedding_grad(dout, dev, rows, scale=scale, padding_id=padding, grad_dtype=DT[to])
    assert torch.equal(got, again)  # the order of the sums is fixed


@pytest.mark.parametrize("n,rows,dim", [(1, 1, 1), (1, 500, 8), (63, 7, 5), (64, 64, 64), (65, 3, 130), (1000, 511, 24),
                                        (2047, 512, 40), (4096, 513, 16), (4097, 100000, 9), (5000, 1, 33),
                                        (8192, 100000, 96), (8191, 90000, 101), (8193, 90000, 101), (20000, 777, 65),
                                        (33000, 40, 17), (40000, 300000, 8), (3, 5, 4100)])
def test_grad_sizes(ibp, n, rows, dim):
    rng = np.random.default_rng(n + rows)
    check_grad(ibp, rng.integers(0, rows, n), rows, dim, seed=n)


@pytest.mark.parametrize("ti", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("to", ["f32", "f16", "bf16"])
def test_grad_types(ibp, ti, to):
    rng = np.random.default_rng(3)
    check_grad(ibp, rng.integers(0, 90, 700), 90, 37, ti, to, scale=6.5)


@pytest.mark.parametrize("n", [300, 9000, 70000])
def test_grad_frequent_tokens(ibp, n):
    """Few ids own most tokens, in runs that cross many chunks; the padding id owns a third."""
    rng = np.random.default_rng(n)
    ids = rng.choice([5, 6, 900, 17, 18], n, p=[0.35, 0.3, 0.3, 0.04, 0.01])
    check_grad(ibp, ids, 1000, 72, "bf16", "f32", scale=0.5, padding=6)
    check_grad(ibp, np.full(n, 3), 4, 24)          # one id for all
    check_grad(ibp, np.full(n, 3), 4, 24, padding=3)  # nothing left: all rows 0


def test_grad_without_tokens_and_bad_ids(ibp):
    got = ibp.ibp_embedding_grad(torch.zeros(0, 12, device="cuda"), torch.zeros(0, dtype=torch.int64, device="cuda"), 30,
                                 grad=torch.full((30, 12), 5.0, device="cuda"))
    assert not got.any()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    dout = torch.ones(5, 12, device="cuda")
    ids = torch.tensor([2, -1, 30, 1 << 40, 2], device="cuda")
    got = ibp.ibp_embedding_grad(dout, ids, 30, err=err)
    assert err.item() == ibp.IBP_DEVERR_BAD_ID
    assert got.sum().item() == 24 and (got[2] == 2).all()


def test_grad_infinities_stay_in_their_rows(ibp):
    dout = torch.ones(50, 20, device="cuda")
    dout[7, 3], dout[9, 4] = float("inf"), float("nan")
    ids = torch.arange(50, device="cuda") % 10
    got = ibp.ibp_embedding_grad(dout, ids, 11)
    bad = ~torch.isfinite(got)
    assert bad.sum().item() == 2 and bad[7, 3] and bad[9, 4] and got[10].eq(0).all()


# ---------------------------------------------------------------- packing

def special(rng, rows, cols):
    x = rng.standard_normal((rows, cols)) * 2.0 ** rng.integers(-20, 20, (rows, 1))
    x[0] = 0.0
    x[1, ::3] = -0.0
    if rows > 8:
        x[2] = rng.choice([448.0, 449, 464, 6, 6.5, 7, 0.25, 0.75, 2.5, 3.5, 5, 1.0625, 1.1875], cols)  # borders
        x[3] *= 2.0 ** -150
        x[4] *= 2.0 ** 90
        x[5, 0], x[6, -1], x[7, cols // 2] = np.inf, -np.inf, np.nan
    return x


@pytest.mark.parametrize("fmt", [mx_ref.E4M3, mx_ref.E2M1])
@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", [(2, 1), (3, 31), (9, 32), (9, 33), (17, 129), (40, 1000), (10, 2049), (9, 4001)])
def test_pack_and_unpack(ibp, fmt, t, rows, cols):
    x = gpu(special(np.random.default_rng(cols), rows, cols), t)
    m = ibp.ibp_mx_pack(x, fmt)
    c, s = mx_ref.pack(host(x), fmt)
    assert np.array_equal(m.scales.cpu().numpy(), s)
    assert np.array_equal(m.codes.cpu().numpy(), c)
    for to in DT:
        got = host(ibp.ibp_mx_unpack(m, dtype=DT[to]))
        want = torch.from_numpy(mx_ref.unpack(c, s, cols, fmt)).to(DT[to]).double().numpy()
        assert np.array_equal(got, want, equal_nan=True), to


@pytest.mark.parametrize("fmt", [mx_ref.E4M3, mx_ref.E2M1])
def test_pack_the_largest_values(ibp, fmt):
    """Magnitudes up to the type's largest: scales stop where their values stay finite."""
    big = torch.finfo(torch.float32).max
    x = torch.tensor([[big, -big, big / 2, 1.0], [2.0 ** 127, 1.75 * 2.0 ** 127, 1e38, -3e38]], device="cuda")
    m = ibp.ibp_mx_pack(x, fmt)
    c, s = mx_ref.pack(host(x), fmt)
    assert np.array_equal(m.codes.cpu().numpy(), c) and np.array_equal(m.scales.cpu().numpy(), s)
    assert torch.isfinite(ibp.ibp_mx_unpack(m, dtype=torch.float32)).all()


def test_unpack_every_code_and_scale(ibp):
    """Codes and scales that the packer never writes are read as they are."""
    for fmt in (mx_ref.E4M3, mx_ref.E2M1):
        rows = 256
        codes = np.tile(np.arange(256, dtype=np.uint8), (rows, 1))
        cols = 256 if fmt == mx_ref.E4M3 else 512
        scales = np.tile(np.arange(rows, dtype=np.uint8)[:, None], (1, cols // 32))
        m = ibp.MxTensor(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), rows, cols, fmt)
        got = host(ibp.ibp_mx_unpack(m, dtype=torch.float32))
        want = torch.from_numpy(mx_ref.unpack(codes, scales, cols, fmt)).float().double().numpy()
        assert np.array_equal(got, want, equal_nan=True)


def test_pack_past_32_bit_offsets(ibp):
    rows, cols = (1 << 20) + 9, 4128
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 1 << 19, rows - 1], device="cuda")
    x[at] = torch.randn(3, cols, device="cuda").to(torch.bfloat16)
    m = ibp.ibp_mx_pack(x, ibp.IBP_MX_E4M3)
    c, s = mx_ref.pack(host(x[at]), mx_ref.E4M3)
    assert np.array_equal(m.codes[at].cpu().numpy(), c) and np.array_equal(m.scales[at].cpu().numpy(), s)
    y = ibp.ibp_mx_unpack(m, out=x)
    assert np.array_equal(host(y[at]), mx_ref.unpack(c, s, cols, mx_ref.E4M3))


# ---------------------------------------------------------------- gated activation

@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 32), (5, 33), (70, 257), (9, 4100)])
def test_swiglu(ibp, t, rows, cols):
    rng = np.random.default_rng(rows + cols)
    g, u, dh = (gpu(rng.standard_normal((rows, cols)) * 4, t) for _ in range(3))
    h, g8, u8 = ibp.ibp_mx_swiglu(g, u)
    dg, du = ibp.ibp_mx_swiglu_backward(dh, g8, u8)
    xg, xu, xd = host(g), host(u), host(dh)
    want = mx_ref.swiglu(xg, xu)
    # exp, sum, quotient, product: two units and three half units of the last place
    within(host(h), want, np.abs(want) * (half(t) + 8 * U) + TINY[t])
    for m, x in ((g8, xg), (u8, xu)):
        c, s = mx_ref.pack(x, mx_ref.E4M3)
        assert np.array_equal(m.codes.cpu().numpy(), c) and np.array_equal(m.scales.cpu().numpy(), s)
    kg, ku = (mx_ref.unpack(*mx_ref.pack(x, mx_ref.E4M3), cols, mx_ref.E4M3) for x in (xg, xu))
    wg, wu = mx_ref.swiglu_backward(xd, kg, ku)
    s = 1 / (1 + np.exp(-kg))
    # 1 + g (1 - s) cancels near g = -1.28: its error is that of its terms
    within(host(dg), wg, np.abs(wg) * half(t) + np.abs(xd * ku * s) * (1 + np.abs(kg)) * 12 * U + TINY[t])
    within(host(du), wu, np.abs(wu) * (half(t) + 8 * U) + TINY[t])


def test_swiglu_far_values(ibp):
    """exp overflows for gates below -88: the activation and its gradients are zeros there,
    and a NaN or infinity in a block makes that block's gradients NaN and no others."""
    g = torch.tensor([[-300.0, -100, 100, 300, 0, -0.0, 1, -1]], device="cuda").repeat(1, 8)
    u = torch.ones_like(g) * 2
    h, g8, u8 = ibp.ibp_mx_swiglu(g, u)
    dg, du = ibp.ibp_mx_swiglu_backward(torch.ones_like(g), g8, u8)
    assert torch.isfinite(h).all() and torch.isfinite(dg).all() and torch.isfinite(du).all()
    assert h[0, 0] == 0 and h[0, 3] == 600 and dg[0, 0] == 0 and dg[0, 3] == 2
    u[0, 40] = float("inf")
    h, g8, u8 = ibp.ibp_mx_swiglu(g, u)
    dg, du = ibp.ibp_mx_swiglu_backward(torch.ones_like(g), g8, u8)
    assert torch.isfinite(dg[0, :32]).all() and torch.isnan(dg[0, 32:]).all() and torch.isfinite(du).all()


# ---------------------------------------------------------------- products

def codes_of(rng, rows, cols, fmt, lo, hi):
    """A packed tensor whose values are whole multiples of 1/4 (e4m3) or 1/2 (e2m1) times
    scales 2^lo..2^hi, its columns past the end zero."""
    v = mx_ref.TABLE[fmt]
    pick = np.flatnonzero((v * 4 == np.floor(v * 4)) & (v < 4)) if fmt == mx_ref.E4M3 else np.arange(8)
    w = mx_ref.blocks(cols) * 32
    k = rng.choice(pick, (rows, w)) + rng.integers(0, 2, (rows, w)) * (128 if fmt == mx_ref.E4M3 else 8)
    k[:, cols:] = 0
    k = k.astype(np.uint8)
    codes = k if fmt == mx_ref.E4M3 else k[:, 0::2] | (k[:, 1::2] << 4)
    s = np.zeros((rows, mx_ref.scale_pitch(cols)), np.uint8)
    s[:, : mx_ref.blocks(cols)] = rng.integers(127 + lo, 128 + hi, (rows, mx_ref.blocks(cols)))
    return codes, s


def device(ibp, codes, scales, cols, fmt):
    return ibp.MxTensor(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), codes.shape[0], cols, fmt)


PRODUCTS = [(1, 1, 1), (1, 16, 32), (2, 33, 31), (16, 17, 129), (17, 100, 512), (31, 64, 513), (64, 65, 1000),
            (65, 200, 96), (130, 129, 640), (257, 300, 1056), (1, 1000, 2080), (300, 20, 160), (512, 512, 256),
            (1000, 1100, 288), (1030, 1000, 33), (3500, 3600, 160), (3600, 3500, 545)]


@pytest.mark.parametrize("fmt", [mx_ref.E4M3, mx_ref.E2M1])
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_matmul_is_exact_where_32_bits_are(ibp, fmt, m, n, k):
    """Values whose sums 24 bits hold (at most 2080 terms of up to 4 * 2 * 6 * 2 in steps of
    2^-5: below 2^24 steps): every output equals the 64-bit product."""
    rng = np.random.default_rng(m * 7 + n * 3 + k)
    a, b = codes_of(rng, m, k, fmt, -1, 1), codes_of(rng, n, k, mx_ref.E2M1, -1, 1)
    print(f"product: m={m} n={n} k={k} format={fmt}", flush=True)
    want = mx_ref.unpack(*a, k, fmt) @ mx_ref.unpack(*b, k, mx_ref.E2M1).T
    y = torch.full((m, n), float("nan"), device="cuda")
    ibp.ibp_mx_matmul(device(ibp, *a, k, fmt), device(ibp, *b, k, mx_ref.E2M1), dtype=torch.float32, out=y)
    assert np.array_equal(host(y), want)


@pytest.mark.parametrize("to", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("fmt", [mx_ref.E4M3, mx_ref.E2M1])
@pytest.mark.parametrize("m,n,k", [(1, 40, 700), (70, 90, 333), (260, 270, 900)])
def test_matmul(ibp, fmt, to, m, n, k):
    rng = np.random.default_rng(k)
    xa, xb = rng.standard_normal((m, k)) * 2.0 ** rng.integers(-6, 6, (m, 1)), rng.standard_normal((n, k)) * 0.1
    a, b = packed(ibp, xa, fmt), packed(ibp, xb, mx_ref.E2M1)
    va = mx_ref.unpack(a.codes.cpu().numpy(), a.scales.cpu().numpy(), k, fmt)
    vb = mx_ref.unpack(b.codes.cpu().numpy(), b.scales.cpu().numpy(), k, mx_ref.E2M1)
    want, mag = va @ vb.T, np.abs(va) @ np.abs(vb).T
    y = ibp.ibp_mx_matmul(a, b, dtype=DT[to])
    within(host(y), want, np.abs(want) * half(to) + mag * k * U + TINY[to])


@pytest.mark.parametrize("fmt", [mx_ref.E4M3, mx_ref.E2M1])
@pytest.mark.parametrize("m", [3, 300])
def test_matmul_nan_blocks_reach_their_rows_only(ibp, fmt, m):
    rng = np.random.default_rng(11)
    a, b = codes_of(rng, m, 320, fmt, 0, 0), codes_of(rng, 50, 320, mx_ref.E2M1, 0, 0)
    a[1][2, 3] = 255
    b[1][7, 9] = 255
    y = host(ibp.ibp_mx_matmul(device(ibp, *a, 320, fmt), device(ibp, *b, 320, mx_ref.E2M1), dtype=torch.float32))
    bad = np.zeros((m, 50), bool)
    bad[2], bad[:, 7] = True, True
    assert np.array_equal(np.isnan(y), bad)


@pytest.mark.parametrize("m", [3, 300, 4000])
def test_matmul_in_32_bits_keeps_small_products(ibp, m):
    """One product of 256 and one of 2^(8 - k) in the same block: both fit 32 bits."""
    cols, n = 160, 4000 if m == 4000 else 40
    code = {v: c for c, v in enumerate(mx_ref.TABLE[mx_ref.E4M3])}
    a = np.zeros((m, cols), np.uint8), np.zeros((m, mx_ref.scale_pitch(cols)), np.uint8)
    b = np.zeros((n, cols // 2), np.uint8), np.zeros((n, mx_ref.scale_pitch(cols)), np.uint8)
    a[1][:, :5], b[1][:, :5] = 127, 127
    k = np.arange(m) % 18
    a[0][:, 33] = code[256.0]
    a[0][np.arange(m), 40 + k] = [code[2.0 ** (8 - j)] for j in k]
    b[0][:] = 0x22  # ones
    y = ibp.ibp_mx_matmul(device(ibp, *a, cols, mx_ref.E4M3), device(ibp, *b, cols, mx_ref.E2M1), dtype=torch.float32)
    want = np.repeat((256 + 2.0 ** (8 - k))[:, None], n, 1)
    assert np.array_equal(host(y), want)


def test_matmul_of_nothing(ibp):
    for m, n, k in ((0, 5, 64), (5, 0, 64), (3, 4, 0)):
        a, b = ibp.make_mx(m, k, ibp.IBP_MX_E4M3, "cuda"), ibp.make_mx(n, k, ibp.IBP_MX_E2M1, "cuda")
        y = ibp.ibp_mx_matmul(a, b, out=torch.full((m, n), 9.0, device="cuda"), dtype=torch.float32)
        assert y.shape == (m, n) and not y.any()


WGRADS = [(1, 1, 1), (31, 16, 32), (32, 33, 31), (33, 128, 129), (100, 130, 257), (999, 50, 100), (3000, 40, 64),
          (700, 300, 520), (5000, 129, 64), (64, 512, 512),
          (130, 3504, 3600), (97, 3601, 3500), (2100, 520, 500)]


@pytest.mark.parametrize("t,n,k", WGRADS)
def test_wgrad_is_exact_where_32_bits_are(ibp, t, n, k):
    """dy whole from -4 to 4, x in steps of 1/4 up to 3.75 * 2 (scales 1/2 to 2): sums of at
    most 5000 terms of 30 in steps of 1/8 stay below 2^24 steps."""
    rng = np.random.default_rng(t + n + k)
    dy = rng.integers(-4, 5, (t, n)).astype(float)
    x = codes_of(rng, t, k, mx_ref.E4M3, -1, 1)
    print(f"weight gradient: t={t} n={n} k={k}", flush=True)
    want = dy.T @ mx_ref.unpack(*x, k, mx_ref.E4M3)
    dw = torch.full((n, k), float("nan"), device="cuda")
    ibp.ibp_mx_linear_wgrad(gpu(dy, "bf16"), device(ibp, *x, k, mx_ref.E4M3), dw=dw)
    assert np.array_equal(host(dw), want)


@pytest.mark.parametrize("ty", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("to", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("t,n,k", [(50, 70, 90), (2000, 130, 100), (37, 5, 64)])
def test_wgrad(ibp, ty, to, t, n, k):
    rng = np.random.default_rng(t)
    dy, x = gpu(rng.standard_normal((t, n)) * 0.1, ty), packed(ibp, rng.standard_normal((t, k)) * 3, mx_ref.E4M3)
    v = mx_ref.unpack(x.codes.cpu().numpy(), x.scales.cpu().numpy(), k, mx_ref.E4M3)
    want, mag = host(dy).T @ v, np.abs(host(dy)).T @ np.abs(v)
    got = ibp.ibp_mx_linear_wgrad(dy, x, dw_dtype=DT[to])
    within(host(got), want, np.abs(want) * half(to) + mag * t * U + TINY[to])


@pytest.mark.parametrize("ty,n,first", [("bf16", 3000, 0), ("bf16", 3000, 3), ("bf16", 3001, 0), ("bf16", 2999, 1), ("f16", 3000, 0),
                                        ("f32", 2999, 1)])
def test_wgrad_of_many_tokens_and_columns(ibp, ty, n, first):
    """The large tile: rows of whole pieces, rows that are laid out anew, tensors that begin
    anywhere.  Whole values, sums of 1100 terms up to 4 * 7.5 in steps of 1/8: exact."""
    t, k = 1100, 3300
    rng = np.random.default_rng(n + first)
    dy = rng.integers(-4, 5, (t, n)).astype(np.float32)
    x = codes_of(rng, t, k, mx_ref.E4M3, -1, 1)
    want = dy.T @ mx_ref.unpack(*x, k, mx_ref.E4M3).astype(np.float32)  # exact in 32 bits too
    print(f"weight gradient: ty={ty} n={n} first={first}", flush=True)
    flat = torch.zeros(first + t * n, dtype=DT[ty], device="cuda")
    flat[first:] = gpu(dy, ty).flatten()
    dw = torch.full((n, k), float("nan"), device="cuda")
    ibp.ibp_mx_linear_wgrad(flat[first:].view(t, n), device(ibp, *x, k, mx_ref.E4M3), dw=dw)
    assert np.array_equal(dw.cpu().numpy(), want)


def test_wgrad_takes_single_precision_whole(ibp):
    """One token: each output is one product of 24 and 4 bits, rounded to 32; the largest
    values, infinities and NaNs (whatever bits they carry) stay what they are."""
    x = packed(ibp, np.array([[1.0, 1.875, -0.5] + [0.0] * 29]), mx_ref.E4M3)
    dy = torch.tensor([[1 + 2.0 ** -23, 3.0e38, -torch.finfo(torch.float32).max, 2.0 ** -100, float("inf"), float("nan")]])
    dy = torch.cat([dy, torch.tensor([0x7F800001], dtype=torch.int32).view(torch.float32)[None]], 1).cuda()
    got = host(ibp.ibp_mx_linear_wgrad(dy, x))[:, :3]
    want = (dy[0, :, None] * torch.tensor([1.0, 1.875, -0.5], device="cuda")).double().cpu().numpy()
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[np.isinf(want)], want[np.isinf(want)])
    assert np.all(np.abs(got[fine] - want[fine]) <= 4 * U * np.abs(want[fine]))


def test_wgrad_of_small_and_nan_values(ibp):
    """The smallest packed values (2^-126) count, a NaN block reaches its columns only, and
    no tokens give zeros."""
    x = np.full((40, 70), 2.0 ** -126)
    m = packed(ibp, x, mx_ref.E4M3)
    dy = torch.ones(40, 9, dtype=torch.bfloat16, device="cuda") * 4
    got = ibp.ibp_mx_linear_wgrad(dy, m, dw_dtype=torch.float32)
    assert np.array_equal(host(got), np.full((9, 70), 160 * 2.0 ** -126))
    m.scales[5, 1] = 255
    got = host(ibp.ibp_mx_linear_wgrad(dy, m, dw_dtype=torch.float32))
    assert np.isnan(got[:, 32:64]).all() and np.isfinite(got[:, :32]).all() and np.isfinite(got[:, 64:]).all()
    got = ibp.ibp_mx_linear_wgrad(dy[:0], ibp.make_mx(0, 70, ibp.IBP_MX_E4M3, "cuda"), dw=torch.ones(9, 70, device="cuda"))
    assert not got.any()


# ---------------------------------------------------------------- gradients against differences

def test_embedding_grad_is_the_difference_of_lookups(ibp):
    """Whole values: sum(dout * lookup(table)) changes by exactly the gradient when an element
    of the table grows by one."""
    rng = np.random.default_rng(21)
    rows, dim, n = 7, 33, 200
    table, dout = rng.integers(-9, 10, (rows, dim)), rng.integers(-4, 5, (n, dim))
    ids = torch.from_numpy(rng.integers(0, rows - 1, n)).cuda()  # the last row has no token
    loss = lambda t: (host(ibp.ibp_embedding_lookup(gpu(t, "f32"), ids, scale=2.0)) * dout).sum()  # noqa: E731
    grad = host(ibp.ibp_embedding_grad(gpu(dout, "f32"), ids, rows, scale=2.0))
    base = loss(table)
    for v, c in ((0, 0), (1, 32), (3, 7), (5, 20), (rows - 1, 5)):
        more = table.copy()
        more[v, c] += 1
        assert loss(more) - base == grad[v, c]


def test_swiglu_backward_is_the_difference(ibp):
    """Central differences of the activation in 64 bits, at the checkpoints' values.  Step e:
    cut off after e^2 / 6 of a third derivative below 1, rounding 2^-52 of values below 2^8 over e."""
    rng = np.random.default_rng(22)
    g, u, dh = (gpu(rng.standard_normal((40, 200)) * 3, "f32") for _ in range(3))
    _, g8, u8 = ibp.ibp_mx_swiglu(g, u)
    dg, du = ibp.ibp_mx_swiglu_backward(dh, g8, u8)
    kg, ku, d, e = host(ibp.ibp_mx_unpack(g8, torch.float32)), host(ibp.ibp_mx_unpack(u8, torch.float32)), host(dh), 2.0 ** -15
    both = lambda f: (f(e) - f(-e)) / (2 * e)  # noqa: E731
    wg, wu = (both(f) * d for f in (lambda x: mx_ref.swiglu(kg + x, ku), lambda x: mx_ref.swiglu(kg, ku + x)))
    slack = np.abs(d) * (np.abs(ku) + 1) * (e * e / 6 + 2.0 ** -44 / e)
    within(host(dg), wg, np.abs(d * ku) * (1 + np.abs(kg)) * 13 * U + slack)
    within(host(du), wu, np.abs(wu) * 9 * U + slack)


def test_wgrad_is_the_difference_of_products(ibp):
    """Whole values: sum(dy * (x w^T)) changes by exactly the gradient when a weight grows by one."""
    rng = np.random.default_rng(23)
    t, o, i = 70, 40, 96
    x, w, dy = rng.integers(-8, 9, (t, i)).astype(float), rng.integers(0, 3, (o, i)).astype(float), rng.integers(-4, 5, (t, o)).astype(float)
    w[:, ::32] = 6  # every block keeps the scale 1, so 0 to 4 are codes
    x[:, ::32] = 256  # and of x, whose whole values up to 16 are codes then
    x8 = packed(ibp, x, mx_ref.E4M3)
    assert np.array_equal(host(ibp.ibp_mx_unpack(x8, torch.float32)), x)
    loss = lambda w: (host(ibp.ibp_mx_matmul(x8, packed(ibp, w, mx_ref.E2M1), torch.float32)) * dy).sum()  # noqa: E731
    dw = host(ibp.ibp_mx_linear_wgrad(gpu(dy, "bf16"), x8, dw_dtype=torch.float32))
    base = loss(w)
    for a, b in ((0, 1), (7, 33), (39, 95), (20, 50)):
        more = w.copy()
        more[a, b] += 1
        assert loss(more) - base == dw[a, b]


# ---------------------------------------------------------------- streams and graphs

def step(ibp, s):
    """Every operator once, as one training step uses them."""
    x = ibp.ibp_embedding_lookup(s["table"], s["ids"], scale=8.0)
    x8 = ibp.ibp_mx_pack(x, ibp.IBP_MX_E4M3)
    g, u = ibp.ibp_mx_matmul(x8, s["wg"]), ibp.ibp_mx_matmul(x8, s["wu"])
    h, g8, u8 = ibp.ibp_mx_swiglu(g, u)
    dg, du = ibp.ibp_mx_swiglu_backward(h, g8, u8)
    return [h, dg, du, ibp.ibp_mx_linear_wgrad(dg, x8, dw_dtype=torch.float32), ibp.ibp_mx_unpack(x8),
            ibp.ibp_embedding_grad(x, s["ids"], s["table"].shape[0], grad_dtype=torch.float32)]


def state(ibp, n, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    w = lambda: ibp.ibp_mx_pack(torch.randn(300, 200, generator=gen, device="cuda"), ibp.IBP_MX_E2M1)  # noqa: E731
    return {"table": torch.randn(500, 200, generator=gen, device="cuda").to(torch.bfloat16),
            "ids": torch.randint(500, (n,), generator=gen, device="cuda"), "wg": w(), "wu": w()}


@pytest.mark.parametrize("n", [5, 6000])
def test_side_stream_and_graph_replays(ibp, n):
    """The step on a stream of its own, and captured into a graph and replayed with new ids,
    equals the eager step bit for bit."""
    s = state(ibp, n, n)
    want = step(ibp, s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(ibp, s)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(ibp, s)
    for k in range(4):
        s["ids"].copy_(torch.randint(500, (n,), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        want = step(ibp, s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), k


def test_the_stream_argument(ibp):
    """A call given a stream runs there and its outputs belong there."""
    s = state(ibp, 700, 4)
    want = ibp.ibp_embedding_grad(ibp.ibp_embedding_lookup(s["table"], s["ids"]), s["ids"], 500)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        x = ibp.ibp_embedding_lookup(s["table"], s["ids"], stream=stream)
        got = ibp.ibp_embedding_grad(x, s["ids"], 500, stream=stream)
        m = ibp.ibp_mx_pack(x, ibp.IBP_MX_E2M1, stream=stream)
        y = ibp.ibp_mx_matmul(m, m, stream=stream)
        side.synchronize()
        assert torch.equal(got, want)
        assert torch.equal(y, ibp.ibp_mx_matmul(m, m))


def test_device_refusals(ibp):
    """Pointers that are not device memory, and ranges past their allocation, are refused."""
    x = torch.zeros(4, 64)
    with pytest.raises(ibp.IBPError):
        ibp.ibp_embedding_lookup(x, torch.zeros(2, dtype=torch.int64, device="cuda"))  # pageable host memory
    with pytest.raises(ibp.IBPError):
        ibp.ibp_mx_pack(x, ibp.IBP_MX_E4M3)
    with pytest.raises(ValueError):
        ibp.ibp_embedding_lookup(x.cuda().t(), torch.zeros(2, dtype=torch.int64, device="cuda"))  # not contiguous
    with pytest.raises(ValueError):
        ibp.ibp_embedding_lookup(x.cuda(), torch.zeros(2, dtype=torch.int64, device="cuda"), out=torch.zeros(3, 64, device="cuda"))
    with pytest.raises(ibp.IBPError):
        ibp.ibp_embedding_grad(torch.zeros(2, 64, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda"), 5,
                               workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
