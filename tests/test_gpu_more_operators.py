"""8-bit integer rows and layers of experts on the GPU against plain definitions (i8_ref,
mx_ref).

Packing, the integer product and the order are compared for equality: their definitions say
every rounding.  Only where a product is rounded to half precision the compiler may leave out
the rounding to 32 bits before it (one instruction does both), so there the result is within
half a step, and half a step of 32 bits, of the product.  The grouped products are exact where 32-bit sums are (whole multiples of a
power of two below 2^24 steps), and otherwise off by at most half a step of the result's type
and n 2^-24 of the terms' magnitudes for n terms.
"""
import numpy as np
import pytest
import torch

import i8_ref
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


def rounded(x, t):
    """float32 values rounded to a type, as float64."""
    return torch.from_numpy(np.ascontiguousarray(x)).to(DT[t]).double().numpy()


def within(got, want, bound):
    over = np.abs(got - want) - bound
    assert over.size == 0 or over.max() <= 0, f"off by {over.max()} more than allowed at {np.argmax(over)} of {over.size}"


def check_product(y, left, right, t):
    """y is the product of two float32 arrays, in t."""
    with np.errstate(over="ignore", invalid="ignore"):
        if t != "f16":
            assert np.array_equal(host(y), rounded(left * right, t), equal_nan=True)
            return
        want = left.astype(np.float64) * right.astype(np.float64)
    got, fits = host(y), np.abs(want) < 65504
    over = np.abs(want) >= 65520
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[over], np.sign(want[over]) * np.inf)
    within(got[fits], want[fits], np.abs(want[fits]) * (half(t) + U) + TINY[t])


def i8(ibp, codes, scales, cols):
    return ibp.I8Tensor(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), codes.shape[0], cols)


def mx(ibp, codes, scales, cols, fmt):
    return ibp.MxTensor(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), codes.shape[0], cols, fmt)


# ---------------------------------------------------------------- 8-bit integer rows

def special(rng, rows, cols):
    x = rng.standard_normal((rows, cols)) * 2.0 ** rng.integers(-20, 20, (rows, 1))
    x[0] = 0.0
    x[1, ::3] = -0.0
    if rows > 8:
        x[2, 1:] = x[2, 0] * rng.choice([0.5, -0.5, 0.25, 1.0, -1.0, 1.5 / 127, 2.5 / 127], cols - 1)  # borders and next to them
        x[3] *= 2.0 ** -140  # subnormal numbers of the wider types
        x[4] *= 2.0 ** 90
        x[5, 0], x[6, -1], x[7, cols // 2] = np.inf, -np.inf, np.nan
        x[8] = rng.integers(-254, 255, cols)
        x[8, 0] = 254  # codes are halves of these
    return x


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", [(2, 1), (3, 7), (9, 16), (20, 33), (70, 129), (17, 513), (40, 1000), (10, 2049),
                                       (9, 4001), (12, 9000), (9, 16385), (10, 40000)])
def test_i8_pack_and_unpack(ibp, t, rows, cols):
    x = gpu(special(np.random.default_rng(cols), rows, cols), t)
    out = ibp.make_i8(rows, cols, "cuda")
    out.codes.fill_(77)
    p = ibp.ibp_i8_pack(x, out=out)
    codes, scales = i8_ref.pack(host(x))
    assert np.array_equal(p.scales.cpu().numpy(), scales, equal_nan=True)
    assert np.array_equal(p.codes.cpu().numpy(), codes)
    for to in DT:
        check_product(ibp.ibp_i8_unpack(p, dtype=DT[to]), codes[:, :cols].astype(np.float32), scales[:, None], to)


@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
def test_i8_codes_of_every_size(ibp, t):
    """Rows whose largest magnitude takes every leading bits of a type, each with elements next
    to the borders between codes."""
    rng = np.random.default_rng(5)
    rows = 2048
    top = 1 + np.arange(rows) / rows if t != "bf16" else 1 + np.arange(rows) % 128 / 128
    border = (rng.integers(0, 127, (rows, 500)) + 0.5) / 127 * top[:, None] * rng.choice([-1, 1], (rows, 500))
    x = torch.from_numpy(np.concatenate([top[:, None], border], 1)).to(DT[t])
    p = ibp.ibp_i8_pack(x.cuda())
    codes, scales = i8_ref.pack(x.double().numpy())
    assert np.array_equal(p.codes.cpu().numpy(), codes) and np.array_equal(p.scales.cpu().numpy(), scales)


def test_i8_pack_the_largest_and_smallest(ibp):
    big, tiny = torch.finfo(torch.float32).max, 2.0 ** -149
    x = torch.tensor([[big, -big, big / 2, 1.0], [tiny, -tiny, 0, tiny], [tiny * 300, tiny * 150, -tiny * 3, tiny]])
    for t in ("f32", "bf16"):
        v = x.to(DT[t])
        if t == "bf16":
            v[0] = torch.tensor([3.0e38, -3.0e38, 1.5e38, 1.0])
            v[1:] = x[1:].mul(2.0 ** 20).to(DT[t])
        p = ibp.ibp_i8_pack(v.cuda())
        codes, scales = i8_ref.pack(v.double().numpy())
        assert np.array_equal(p.codes.cpu().numpy(), codes) and np.array_equal(p.scales.cpu().numpy(), scales)
        assert torch.isfinite(ibp.ibp_i8_unpack(p, dtype=torch.float32)).all()


def test_i8_empty_shapes(ibp):
    p = ibp.ibp_i8_pack(torch.zeros(0, 50, device="cuda"))
    assert p.rows == 0 and ibp.ibp_i8_unpack(p).shape == (0, 50)
    out = ibp.make_i8(5, 0, "cuda")
    out.scales.fill_(9)
    p = ibp.ibp_i8_pack(torch.zeros(5, 0, device="cuda"), out=out)
    assert not p.scales.any()
    y = ibp.ibp_i8_matmul(p, ibp.ibp_i8_pack(torch.zeros(40, 0, device="cuda")), out=torch.full((5, 40), 3.0, device="cuda"),
                          dtype=torch.float32)
    assert not y.any()
    for m, n in ((0, 7), (7, 0)):
        a, b = ibp.ibp_i8_pack(torch.ones(m, 20, device="cuda")), ibp.ibp_i8_pack(torch.ones(n, 20, device="cuda"))
        assert ibp.ibp_i8_matmul(a, b).shape == (m, n)


def test_i8_pack_takes_rows_of_any_alignment(ibp):
    flat = torch.randn(1 + 50 * 77, device="cuda").to(torch.bfloat16)
    x = flat[1:].view(50, 77)
    codes, scales = i8_ref.pack(host(x))
    p = ibp.ibp_i8_pack(x.view(5, 10, 77))
    assert np.array_equal(p.codes.cpu().numpy(), codes) and np.array_equal(p.scales.cpu().numpy(), scales)
    y = torch.zeros(1 + 50 * 77, dtype=torch.float16, device="cuda")
    ibp.ibp_i8_unpack(p, dtype=torch.float16, out=y[1:].view(50, 77))
    assert y[0] == 0
    check_product(y[1:].view(50, 77), codes[:, :77].astype(np.float32), scales[:, None], "f16")


def test_i8_pack_past_32_bit_offsets(ibp):
    rows, cols = (1 << 20) + 9, 4104
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 1 << 19, rows - 1], device="cuda")
    x[at] = torch.randn(3, cols, device="cuda").to(torch.bfloat16)
    p = ibp.ibp_i8_pack(x)
    codes, scales = i8_ref.pack(host(x[at]))
    assert np.array_equal(p.codes[at].cpu().numpy(), codes) and np.array_equal(p.scales[at].cpu().numpy(), scales)
    y = ibp.ibp_i8_unpack(p, out=x)
    assert np.array_equal(host(y[at]), rounded(i8_ref.unpack(codes, scales, cols), "bf16"))
    b = ibp.ibp_i8_pack(torch.randn(16, cols, device="cuda"))
    got = ibp.ibp_i8_matmul(p, b, dtype=torch.float32)[at]
    assert np.array_equal(host(got), i8_ref.product(codes, scales, b.codes.cpu().numpy(), b.scales.cpu().numpy()))


def test_i8_matmul_of_more_tiles_than_a_launch_has(ibp):
    """2^24 small tiles and some, of few rows and very many columns."""
    m, n, k = 10, (1 << 30) - 3, 16
    rng = np.random.default_rng(14)
    ac = rng.integers(-127, 128, (m, k)).astype(np.int8)
    a, b = ibp.make_i8(m, k, "cuda"), ibp.make_i8(n, k, "cuda")
    a.codes[:], a.scales[:] = torch.from_numpy(ac).cuda(), 0.5
    b.codes.random_(-128, 128)
    b.scales.fill_(2.0)
    y = ibp.ibp_i8_matmul(a, b, dtype=torch.float16)
    for c in (0, (1 << 28) - 500, (1 << 29) + 17, n - 1000):
        bc = b.codes[c : c + 1000].cpu().numpy()
        want = (ac.astype(np.int64) @ bc.T.astype(np.int64)).astype(np.float32)
        with np.errstate(over="ignore"):
            assert np.array_equal(host(y[:, c : c + 1000]), rounded(want, "f16"))


PRODUCTS = [(1, 1, 1), (1, 16, 64), (2, 33, 31), (16, 17, 129), (17, 100, 512), (31, 64, 513), (64, 65, 1000), (65, 200, 96),
            (130, 129, 640), (257, 300, 1056), (1, 1000, 2080), (300, 20, 160), (512, 512, 256), (1000, 1100, 288),
            (1030, 1000, 33), (3500, 3600, 160), (3600, 3500, 545), (128, 512, 4100), (1, 5000, 9000), (2050, 2049, 129),
            (4097, 300, 1000)]


@pytest.mark.parametrize("to", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_i8_matmul(ibp, to, m, n, k):
    """Any codes, -128 among them: the sums are exact, and every rounding after them is defined."""
    rng = np.random.default_rng(m * 7 + n * 3 + k)
    a, b = (np.zeros((r, i8_ref.pitch(k)), np.int8) for r in (m, n))
    a[:, :k], b[:, :k] = rng.integers(-128, 128, (m, k)), rng.integers(-128, 128, (n, k))
    sa, sb = (np.float32(rng.standard_normal(r) * 1e-3) for r in (m, n))
    print(f"product of 8-bit integers: m={m} n={n} k={k} to={to}", flush=True)
    # sums below 2^53 are exact in float64 products, which are quicker than integer ones
    sums = (a.astype(np.float64) @ b.T.astype(np.float64)).astype(np.int64).astype(np.float32)
    less = np.abs(sa)[:, None] < np.abs(sb)[None]
    y = torch.full((m, n), float("nan"), dtype=DT[to], device="cuda")
    ibp.ibp_i8_matmul(i8(ibp, a, sa, k), i8(ibp, b, sb, k), dtype=DT[to], out=y)
    check_product(y, sums * np.where(less, sa[:, None], sb[None]), np.where(less, sb[None], sa[:, None]), to)


@pytest.mark.parametrize("m,n", [(1, 20), (300, 200), (1100, 1100)])
def test_i8_matmul_of_the_largest_sums(ibp, m, n):
    """The deepest product of the largest codes: 131071 * 128^2 is below 2^31."""
    k = ibp.IBP_I8_MAX_DEPTH
    a, b = (torch.zeros(r, i8_ref.pitch(k), dtype=torch.int8, device="cuda") for r in (m, n))
    a[:, :k], b[:, :k] = -128, -128
    b[n // 2:, :k] = 127
    one = lambda r: torch.ones(r, device="cuda")  # noqa: E731
    y = ibp.ibp_i8_matmul(ibp.I8Tensor(a, one(m), m, k), ibp.I8Tensor(b, one(n), n, k), dtype=torch.float32)
    assert (y[:, : n // 2] == float(np.float32(k * 16384))).all() and (y[:, n // 2:] == float(np.float32(-k * 128 * 127))).all()


@pytest.mark.parametrize("m,n", [(3, 50), (300, 200)])
def test_i8_matmul_scales_of_any_size(ibp, m, n):
    """Scales far apart, zero, NaN and infinite: a result overflows only by itself, and a row
    that is NaN reaches its outputs only."""
    k = 200
    rng = np.random.default_rng(6)
    a, b = (np.zeros((r, i8_ref.pitch(k)), np.int8) for r in (m, n))
    a[:, :k], b[:, :k] = rng.integers(-128, 128, (m, k)), rng.integers(-128, 128, (n, k))
    b[9] = 0
    sa, sb = np.ones(m, np.float32), np.ones(n, np.float32)
    sa[0], sa[1], sa[2] = 2e36, 1e-36, np.nan
    sb[0], sb[1], sb[2], sb[3], sb[4], sb[5], sb[9] = 1e-30, 1e30, 0, np.inf, -1e-40, np.nan, 1e38
    want = i8_ref.product(a, sa, b, sb)
    y = ibp.ibp_i8_matmul(i8(ibp, a, sa, k), i8(ibp, b, sb, k), dtype=torch.float32).cpu().numpy()
    assert np.array_equal(y, want, equal_nan=True)
    assert np.isnan(y[2]).all() and np.isnan(y[:, 5]).all() and np.isfinite(y[0, 0]) and y[0, 9] == 0


# ---------------------------------------------------------------- order by expert

@pytest.mark.parametrize("n,experts", [(0, 4), (1, 1), (5, 3), (63, 64), (64, 64), (1000, 7), (8192, 256), (8193, 256), (8192, 1024),
                                       (20000, 1), (20000, 1000), (131072, 1024), (131073, 128), (700000, 60), (3000001, 17)])
def test_expert_order(ibp, n, experts):
    rng = np.random.default_rng(n + experts)
    p = rng.random(experts) ** 3 + 1e-9
    ids = rng.choice(experts, n, p=p / p.sum())
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    order, off = ibp.ibp_expert_order(torch.from_numpy(ids).cuda(), experts, err=err)
    want, woff = i8_ref.order(ids, experts)
    assert np.array_equal(off.cpu().numpy(), woff) and np.array_equal(order.cpu().numpy(), want) and err.item() == 0


@pytest.mark.parametrize("n", [50, 9000, 40000])
def test_expert_order_of_bad_ids(ibp, n):
    rng = np.random.default_rng(n)
    ids = rng.choice([-1, 0, 3, 4, 5, 1 << 40, -(1 << 62)], n)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    order, off = ibp.ibp_expert_order(torch.from_numpy(ids).cuda(), 5, err=err)
    want, woff = i8_ref.order(ids, 5)
    assert np.array_equal(off.cpu().numpy(), woff) and np.array_equal(order.cpu().numpy(), want)
    assert err.item() == ibp.IBP_DEVERR_BAD_ID
    order, off = ibp.ibp_expert_order(torch.full((n,), 7, device="cuda"), 5)
    assert not off.any() and np.array_equal(order.cpu().numpy(), np.arange(n))


# ---------------------------------------------------------------- products by expert

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


def offsets_of(rng, rows, experts, how):
    """Where the experts' rows begin, `rows` in all."""
    if how == "one":  # all with one expert
        e = rng.integers(experts)
        sizes = np.where(np.arange(experts) == e, rows, 0)
    elif how == "even":
        sizes = np.full(experts, rows // experts) + (np.arange(experts) < rows % experts)
    else:  # ragged, about a third of the experts without rows
        p = rng.random(experts) ** 2 * (rng.random(experts) < 0.67)
        p[rng.integers(experts)] += 0.1
        sizes = rng.multinomial(rows, p / p.sum())
    return np.concatenate([[0], np.cumsum(sizes)])


GROUPED = [(1, 1, 1, 1, "even"), (1, 3, 16, 32, "one"), (5, 8, 33, 31, "ragged"), (16, 4, 17, 129, "even"), (17, 2, 100, 512, "one"),
           (64, 64, 70, 700, "ragged"), (64, 300, 40, 96, "ragged"), (100, 1024, 9, 64, "ragged"), (300, 5, 129, 640, "ragged"),
           (700, 9, 200, 333, "ragged"), (1000, 3, 300, 288, "even"), (1500, 2, 256, 1056, "one"), (3000, 4, 520, 160, "ragged"),
           (2500, 20, 260, 545, "even"), (5000, 7, 500, 256, "ragged"), (600, 1, 257, 2080, "even"),
           (200, 100, 201, 320, "ragged"), (300, 10, 700, 160, "ragged"), (900, 20, 333, 2080, "ragged"), (130, 17, 2000, 96, "one"),
           (2100, 6, 1700, 160, "ragged"), (2200, 8, 2001, 545, "even"), (6500, 8, 3600, 96, "ragged"), (6600, 20, 3501, 160, "even")]


@pytest.mark.parametrize("fmt", [mx_ref.E4M3, mx_ref.E2M1])
@pytest.mark.parametrize("t,e,n,k,how", GROUPED)
def test_grouped_matmul_is_exact_where_32_bits_are(ibp, fmt, t, e, n, k, how):
    """At most 2080 terms of up to 4 * 2 * 6 * 2 in steps of 2^-5: below 2^24 steps."""
    rng = np.random.default_rng(t * 7 + e * 5 + n * 3 + k)
    a, b = codes_of(rng, t, k, fmt, -1, 1), codes_of(rng, e * n, k, mx_ref.E2M1, -1, 1)
    off = offsets_of(rng, t, e, how)
    print(f"grouped product: t={t} e={e} n={n} k={k} {how} format={fmt}", flush=True)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = torch.full((t, n), float("nan"), device="cuda")
    ibp.ibp_mx_grouped_matmul(mx(ibp, *a, k, fmt), mx(ibp, *b, k, mx_ref.E2M1), torch.from_numpy(off).cuda(), dtype=torch.float32,
                              out=y, err=err)
    want = i8_ref.grouped_product(mx_ref.unpack(*a, k, fmt), mx_ref.unpack(*b, k, mx_ref.E2M1).reshape(e, n, k), off, np.zeros((t, n)))
    assert np.array_equal(host(y), want) and err.item() == 0


@pytest.mark.parametrize("to", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("fmt", [mx_ref.E4M3, mx_ref.E2M1])
@pytest.mark.parametrize("t,e,n,k", [(7, 5, 40, 700), (400, 6, 90, 333), (1200, 4, 270, 900)])
def test_grouped_matmul(ibp, fmt, to, t, e, n, k):
    rng = np.random.default_rng(k)
    a = mx_ref.pack(rng.standard_normal((t, k)) * 2.0 ** rng.integers(-6, 6, (t, 1)), fmt)
    b = mx_ref.pack(rng.standard_normal((e * n, k)) * 0.1, mx_ref.E2M1)
    off = offsets_of(rng, t, e, "ragged")
    va, vb = mx_ref.unpack(*a, k, fmt), mx_ref.unpack(*b, k, mx_ref.E2M1).reshape(e, n, k)
    want = i8_ref.grouped_product(va, vb, off, np.zeros((t, n)))
    mag = i8_ref.grouped_product(np.abs(va), np.abs(vb), off, np.zeros((t, n)))
    y = ibp.ibp_mx_grouped_matmul(mx(ibp, *a, k, fmt), mx(ibp, *b, k, mx_ref.E2M1), torch.from_numpy(off).cuda(), dtype=DT[to])
    within(host(y), want, np.abs(want) * half(to) + mag * k * U + TINY[to])


@pytest.mark.parametrize("t", [40, 900, 3000])
def test_grouped_rows_of_no_expert_stay(ibp, t):
    """Rows before the first expert's and behind the last one's are left as they were, and
    so are the neighbours of an output inside a larger tensor."""
    rng = np.random.default_rng(t)
    e, n, k = 5, 70, 160
    a, b = codes_of(rng, t, k, mx_ref.E4M3, 0, 0), codes_of(rng, e * n, k, mx_ref.E2M1, 0, 0)
    off = offsets_of(rng, t - 20, e, "ragged") + 7
    whole = torch.full((t + 2, n), 5.0, device="cuda")
    ibp.ibp_mx_grouped_matmul(mx(ibp, *a, k, mx_ref.E4M3), mx(ibp, *b, k, mx_ref.E2M1), torch.from_numpy(off).cuda(),
                              dtype=torch.float32, out=whole[1:-1])
    want = i8_ref.grouped_product(mx_ref.unpack(*a, k, mx_ref.E4M3), mx_ref.unpack(*b, k, mx_ref.E2M1).reshape(e, n, k), off,
                                  np.full((t, n), 5.0))
    got = host(whole)
    assert np.array_equal(got[1:-1], want) and (got[0] == 5).all() and (got[-1] == 5).all()


@pytest.mark.parametrize("t", [40, 900, 3000])
def test_grouped_matmul_nan_blocks_reach_their_outputs_only(ibp, t):
    rng = np.random.default_rng(t + 1)
    e, n, k = 4, 50, 320
    a, b = codes_of(rng, t, k, mx_ref.E4M3, 0, 0), codes_of(rng, e * n, k, mx_ref.E2M1, 0, 0)
    off = offsets_of(rng, t, e, "even")
    a[1][off[1], 3] = 255  # the second expert's first row
    b[1][2 * n + 7, 9] = 255  # the third expert's column 7
    y = host(ibp.ibp_mx_grouped_matmul(mx(ibp, *a, k, mx_ref.E4M3), mx(ibp, *b, k, mx_ref.E2M1), torch.from_numpy(off).cuda(),
                                       dtype=torch.float32))
    bad = np.zeros((t, n), bool)
    bad[off[1]], bad[off[2]:off[3], 7] = True, True
    assert np.array_equal(np.isnan(y), bad)


BAD_OFFSETS = [[0, 50, 30, 90, 100], [0, 20, 40, 60, 1 << 40], [-5, 20, 40, 60, 100], [100, 100, 0, 100, 0], [0, 100, 0, 100, 100],
               [-(1 << 62), 1 << 62, -(1 << 62), 1 << 62, 7]]


@pytest.mark.parametrize("off", BAD_OFFSETS)
@pytest.mark.parametrize("scale", [1, 9, 30])
def test_bad_offsets_are_told_and_lead_nowhere(ibp, off, scale):
    """Offsets that fall or leave the rows: an error word, and nothing around the outputs changed."""
    rng = np.random.default_rng(9)
    t, e, n, k = 100 * scale, 4, 40, 96
    off = torch.tensor([o * scale if 0 < o <= 100 else o for o in off], device="cuda")
    a, b = codes_of(rng, t, k, mx_ref.E4M3, 0, 0), codes_of(rng, e * n, k, mx_ref.E2M1, 0, 0)
    a8 = mx(ibp, *a, k, mx_ref.E4M3)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    whole = torch.full((t + 2, n), 5.0, device="cuda")
    ibp.ibp_mx_grouped_matmul(a8, mx(ibp, *b, k, mx_ref.E2M1), off, dtype=torch.float32, out=whole[1:-1], err=err)
    assert err.item() == ibp.IBP_DEVERR_CORRUPT and (whole[0] == 5).all() and (whole[-1] == 5).all()
    err.zero_()
    dw = torch.full((e + 2, n, k), 5.0, device="cuda")
    ibp.ibp_mx_grouped_wgrad(torch.ones(t, n, dtype=torch.bfloat16, device="cuda"), a8, off, dw=dw[1:-1], err=err)
    assert err.item() == ibp.IBP_DEVERR_CORRUPT and (dw[0] == 5).all() and (dw[-1] == 5).all()


def test_grouped_of_nothing(ibp):
    off = torch.zeros(4, dtype=torch.int64, device="cuda")
    w = ibp.make_mx(15, 64, ibp.IBP_MX_E2M1, "cuda")
    assert ibp.ibp_mx_grouped_matmul(ibp.make_mx(0, 64, ibp.IBP_MX_E4M3, "cuda"), w, off).shape == (0, 5)
    a, none = ibp.make_mx(9, 0, ibp.IBP_MX_E4M3, "cuda"), ibp.make_mx(15, 0, ibp.IBP_MX_E2M1, "cuda")
    y = torch.full((9, 5), 3.0, device="cuda")
    ibp.ibp_mx_grouped_matmul(a, none, off, out=y, dtype=torch.float32)
    assert (y == 3).all()
    ibp.ibp_mx_grouped_matmul(a, none, off + torch.tensor([0, 2, 2, 9], device="cuda"), out=y, dtype=torch.float32)
    assert not y.any()
    for t in ("bf16", "f32"):
        dw = torch.ones(3, 6, 64, device="cuda")
        ibp.ibp_mx_grouped_wgrad(torch.zeros(0, 6, dtype=DT[t], device="cuda"), ibp.make_mx(0, 64, ibp.IBP_MX_E4M3, "cuda"), off, dw=dw)
        assert not dw.any()


def test_grouped_weights_past_32_bit_offsets(ibp):
    """The last expert's weights begin 5 GB into them, and its gradient lies 10 GB on."""
    e, n, k, t = 5, 1 << 19, 4096, 20
    w = ibp.make_mx(e * n, k, ibp.IBP_MX_E2M1, "cuda")
    rng = np.random.default_rng(12)
    a, b = codes_of(rng, t, k, mx_ref.E4M3, 0, 0), codes_of(rng, 64, k, mx_ref.E2M1, 0, 0)
    w.codes[-64:], w.scales[-64:] = torch.from_numpy(b[0]).cuda(), torch.from_numpy(b[1]).cuda()
    off = torch.tensor([0, 3, 3, 3, 3, t], device="cuda")
    a8 = mx(ibp, *a, k, mx_ref.E4M3)
    y = ibp.ibp_mx_grouped_matmul(a8, w, off, dtype=torch.float32)[3:, -64:]
    va = mx_ref.unpack(*a, k, mx_ref.E4M3)
    assert np.array_equal(host(y), va[3:] @ mx_ref.unpack(*b, k, mx_ref.E2M1).T)
    del w, y
    dy = rng.integers(-4, 5, (t, 1 << 18)).astype(np.float32)
    dw = ibp.ibp_mx_grouped_wgrad(gpu(dy, "bf16"), a8, off, dw_dtype=torch.bfloat16)
    want = dy[3:, -64:].T @ va[3:]
    assert np.array_equal(host(dw[4, -64:]), rounded(want.astype(np.float32), "bf16")) and not dw[2].any()


def test_grouped_matmul_of_more_tiles_than_a_launch_has(ibp):
    """2^24 tiles of one expert's rows."""
    t, n, k = 36, 1 << 30, 32
    rng = np.random.default_rng(15)
    a = codes_of(rng, t, k, mx_ref.E4M3, 0, 0)
    w = ibp.make_mx(n, k, ibp.IBP_MX_E2M1, "cuda")
    w.codes.random_(0, 256)
    w.scales.fill_(127)
    y = ibp.ibp_mx_grouped_matmul(mx(ibp, *a, k, mx_ref.E4M3), w, torch.tensor([0, t], device="cuda"), dtype=torch.bfloat16)
    for c in (0, (1 << 29) - 500, n - 1000):
        b = w.codes[c : c + 1000].cpu().numpy(), w.scales[c : c + 1000].cpu().numpy()
        want = mx_ref.unpack(*a, k, mx_ref.E4M3) @ mx_ref.unpack(*b, k, mx_ref.E2M1).T
        assert np.array_equal(host(y[:, c : c + 1000]), rounded(want.astype(np.float32), "bf16"))


def test_grouped_tokens_past_32_bit_offsets(ibp):
    """The second expert's rows lie 8 GB into the checkpoint and 4 GB into dy; the first one's
    are not written and not looked at."""
    t, n, k = (1 << 28) + 40, 8, 32
    rng = np.random.default_rng(13)
    x = codes_of(rng, 40, k, mx_ref.E4M3, 0, 0)
    x8 = ibp.make_mx(t, k, ibp.IBP_MX_E4M3, "cuda")
    x8.codes[-40:], x8.scales[-40:] = torch.from_numpy(x[0]).cuda(), torch.from_numpy(x[1]).cuda()
    dy = torch.empty(t, n, dtype=torch.bfloat16, device="cuda")
    tail = rng.integers(-4, 5, (40, n)).astype(float)
    dy[-40:] = gpu(tail, "bf16")
    off = torch.tensor([0, t - 40, t], device="cuda")
    v = mx_ref.unpack(*x, k, mx_ref.E4M3)
    dw = ibp.ibp_mx_grouped_wgrad(dy, x8, off, dw_dtype=torch.float32)
    assert np.array_equal(host(dw[1]), tail.T @ v)
    b = codes_of(rng, 2 * n, k, mx_ref.E2M1, 0, 0)
    y = ibp.ibp_mx_grouped_matmul(x8, mx(ibp, *b, k, mx_ref.E2M1), off, dtype=torch.float32)
    assert np.array_equal(host(y[-40:]), v @ mx_ref.unpack(*b, k, mx_ref.E2M1)[n:].T)


WGRADS = [(1, 1, 1, 1, "even"), (31, 3, 16, 32, "ragged"), (32, 4, 33, 31, "one"), (33, 40, 128, 129, "ragged"), (100, 6, 130, 257, "ragged"),
          (999, 2, 50, 100, "even"), (3000, 9, 40, 64, "ragged"), (700, 3, 300, 520, "ragged"), (5000, 1, 129, 64, "even"),
          (64, 1024, 8, 40, "ragged"), (64, 5, 512, 512, "ragged"), (130, 33, 504, 600, "ragged"), (2100, 30, 520, 500, "one"),
          (6000, 4, 256, 264, "ragged"), (2500, 45, 500, 600, "ragged"), (3000, 64, 264, 520, "ragged"), (2000, 50, 264, 513, "one"),
          (2100, 64, 300, 300, "even")]


@pytest.mark.parametrize("ty", ["bf16", "f32"])
@pytest.mark.parametrize("t,e,n,k,how", WGRADS)
def test_grouped_wgrad_is_exact_where_32_bits_are(ibp, ty, t, e, n, k, how):
    """dy whole from -4 to 4, x in steps of 1/4 up to 3.75 * 2 (scales 1/2 to 2): sums of at
    most 6000 terms of 30 in steps of 1/8 stay below 2^24 steps."""
    rng = np.random.default_rng(t + e + n + k)
    dy = rng.integers(-4, 5, (t, n)).astype(float)
    x = codes_of(rng, t, k, mx_ref.E4M3, -1, 1)
    off = offsets_of(rng, t, e, how)
    print(f"grouped weight gradient: t={t} e={e} n={n} k={k} {how} ty={ty}", flush=True)
    dw = torch.full((e, n, k), float("nan"), device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ibp.ibp_mx_grouped_wgrad(gpu(dy, ty), mx(ibp, *x, k, mx_ref.E4M3), torch.from_numpy(off).cuda(), dw=dw, err=err)
    assert np.array_equal(host(dw), i8_ref.grouped_wgrad(dy, mx_ref.unpack(*x, k, mx_ref.E4M3), off)) and err.item() == 0


@pytest.mark.parametrize("ty", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("to", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("t,e,n,k,first", [(50, 3, 70, 90, 0), (2000, 5, 130, 100, 0), (37, 4, 8, 64, 3), (500, 2, 512, 300, 1)])
def test_grouped_wgrad(ibp, ty, to, t, e, n, k, first):
    rng = np.random.default_rng(t)
    flat = torch.zeros(first + t * n, dtype=DT[ty], device="cuda")
    flat[first:] = gpu(rng.standard_normal(t * n) * 0.1, ty)
    dy = flat[first:].view(t, n)
    x = mx_ref.pack(rng.standard_normal((t, k)) * 3, mx_ref.E4M3)
    off = offsets_of(rng, t - 5, e, "ragged") + 2
    v = mx_ref.unpack(*x, k, mx_ref.E4M3)
    want, mag = i8_ref.grouped_wgrad(host(dy), v, off), i8_ref.grouped_wgrad(np.abs(host(dy)), np.abs(v), off)
    got = ibp.ibp_mx_grouped_wgrad(dy, mx(ibp, *x, k, mx_ref.E4M3), torch.from_numpy(off).cuda(), dw_dtype=DT[to])
    within(host(got), want, np.abs(want) * half(to) + mag * t * U + TINY[to])


@pytest.mark.parametrize("t,n", [(60, 40), (900, 300)])
def test_grouped_wgrad_keeps_bad_values_with_their_expert(ibp, t, n):
    """An infinity of dy and a NaN block of x reach their expert's gradient only, also where
    the next expert's rows share a tile's tokens with them."""
    rng = np.random.default_rng(t)
    e, k = 4, 96
    dy, x = rng.integers(-4, 5, (t, n)).astype(float), codes_of(rng, t, k, mx_ref.E4M3, 0, 0)
    off = offsets_of(rng, t, e, "even")
    dy[off[1] - 1, 3] = np.inf
    x[1][off[2], 1] = 255
    for ty in ("bf16", "f32"):
        got = host(ibp.ibp_mx_grouped_wgrad(gpu(dy, ty), mx(ibp, *x, k, mx_ref.E4M3), torch.from_numpy(off).cuda(), dw_dtype=torch.float32))
        bad = np.zeros((e, n, k), bool)
        bad[0, 3], bad[2, :, 32:64] = True, True
        assert np.array_equal(~np.isfinite(got), bad)


def test_grouped_wgrad_is_the_difference_of_products(ibp):
    """Whole values: sum(dy * product(w)) changes by exactly the gradient when a weight grows by one."""
    rng = np.random.default_rng(23)
    t, e, o, i = 70, 3, 40, 96
    off = torch.tensor([0, 30, 30, 70], device="cuda")
    x, w = rng.integers(-8, 9, (t, i)).astype(float), rng.integers(0, 3, (e * o, i)).astype(float)
    dy = rng.integers(-4, 5, (t, o)).astype(float)
    w[:, ::32] = 6  # every block keeps the scale 1, so 0 to 4 are codes
    x[:, ::32] = 256  # and of x, whose whole values up to 16 are codes then
    x8 = mx(ibp, *mx_ref.pack(x, mx_ref.E4M3), i, mx_ref.E4M3)

    def loss(w):
        w4 = mx(ibp, *mx_ref.pack(w, mx_ref.E2M1), i, mx_ref.E2M1)
        return (host(ibp.ibp_mx_grouped_matmul(x8, w4, off, torch.float32)) * dy).sum()

    dw = host(ibp.ibp_mx_grouped_wgrad(gpu(dy, "bf16"), x8, off, dw_dtype=torch.float32)).reshape(e * o, i)
    base = loss(w)
    for a, b in ((0, 1), (7, 33), (39, 95), (60, 50), (100, 5)):
        more = w.copy()
        more[a, b] += 1
        assert loss(more) - base == dw[a, b]
    assert not dw[o:2 * o].any()


# ---------------------------------------------------------------- a layer of experts

class Layer:
    """Experts of a gated layer: token -> top experts, forward and backward, as a training step
    calls the operators."""

    def __init__(self, ibp, tokens, dim, hidden, experts, top, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
        self.ibp, self.n, self.experts, self.top, self.dim, self.hidden = ibp, tokens, experts, top, dim, hidden
        self.x = rand(tokens, dim).to(torch.bfloat16)
        self.ids = torch.randint(experts, (tokens, top), generator=gen, device="cuda")
        self.share = torch.rand(tokens, top, generator=gen, device="cuda")
        self.dy = (rand(tokens, dim) * 0.01).to(torch.bfloat16)
        self.w = {k: rand(experts, o, i) * i ** -0.5 for k, o, i in (("gate", hidden, dim), ("up", hidden, dim), ("down", dim, hidden))}
        pack = lambda w: ibp.ibp_mx_pack(w.reshape(-1, w.shape[2]), ibp.IBP_MX_E2M1)  # noqa: E731
        self.w4 = {k: pack(w) for k, w in self.w.items()}
        self.w4t = {k: pack(w.transpose(1, 2).contiguous()) for k, w in self.w.items()}

    def step(self):
        """Everything that one step makes, by name."""
        ibp, s = self.ibp, {}
        s["order"], s["offsets"] = ibp.ibp_expert_order(self.ids, self.experts)
        s["token"] = s["order"] // self.top
        product = lambda a8, w: ibp.ibp_mx_grouped_matmul(a8, w, s["offsets"])  # noqa: E731
        e4m3 = lambda x: ibp.ibp_mx_pack(x, ibp.IBP_MX_E4M3)  # noqa: E731
        s["rows"] = ibp.ibp_embedding_lookup(self.x, s["token"])
        s["x8"] = e4m3(s["rows"])
        s["gate"], s["up"] = product(s["x8"], self.w4["gate"]), product(s["x8"], self.w4["up"])
        s["h"], s["gate8"], s["up8"] = ibp.ibp_mx_swiglu(s["gate"], s["up"])
        s["h8"] = e4m3(s["h"])
        s["out"] = product(s["h8"], self.w4["down"])
        s["part"] = self.share.flatten()[s["order"], None]
        s["weighted"] = s["out"] * s["part"]  # 32 bits
        s["y"] = ibp.ibp_embedding_grad(s["weighted"], s["token"], self.n, grad_dtype=torch.bfloat16)
        s["dout"] = (ibp.ibp_embedding_lookup(self.dy, s["token"], out_dtype=torch.float32) * s["part"]).to(torch.bfloat16)
        s["dout8"] = e4m3(s["dout"])
        s["dh"] = product(s["dout8"], self.w4t["down"])
        s["dgate"], s["dup"] = ibp.ibp_mx_swiglu_backward(s["dh"], s["gate8"], s["up8"])
        s["dgate8"], s["dup8"] = e4m3(s["dgate"]), e4m3(s["dup"])
        s["dx_gate"], s["dx_up"] = product(s["dgate8"], self.w4t["gate"]), product(s["dup8"], self.w4t["up"])
        s["dx"] = ibp.ibp_embedding_grad(s["dx_gate"] + s["dx_up"], s["token"], self.n, grad_dtype=torch.float32)
        for k, dy, x8 in (("gate", "dgate", "x8"), ("up", "dup", "x8"), ("down", "dout", "h8")):
            s["dw_" + k] = ibp.ibp_mx_grouped_wgrad(s[dy], s[x8], s["offsets"], dw_dtype=torch.float32)
        return s


@pytest.mark.parametrize("tokens,dim,hidden,experts,top", [(3, 64, 96, 8, 2), (500, 160, 264, 6, 2), (3000, 256, 512, 12, 3)])
def test_a_layer_of_experts(ibp, tokens, dim, hidden, experts, top):
    """Every step of the layer from what the step before gave, in 64 bits."""
    layer = Layer(ibp, tokens, dim, hidden, experts, top, tokens)
    s = layer.step()
    order, off = i8_ref.order(layer.ids.cpu().numpy().ravel(), experts)
    assert np.array_equal(s["order"].cpu().numpy(), order) and np.array_equal(s["offsets"].cpu().numpy(), off)
    value = lambda m: host(ibp.ibp_mx_unpack(m, torch.float32))  # noqa: E731
    for a, w, y in (("x8", layer.w4["gate"], "gate"), ("x8", layer.w4["up"], "up"), ("h8", layer.w4["down"], "out"),
                    ("dout8", layer.w4t["down"], "dh"), ("dgate8", layer.w4t["gate"], "dx_gate"), ("dup8", layer.w4t["up"], "dx_up")):
        va, vw = value(s[a]), value(w).reshape(experts, -1, w.cols)
        zero = np.zeros(s[y].shape)
        want, mag = i8_ref.grouped_product(va, vw, off, zero), i8_ref.grouped_product(np.abs(va), np.abs(vw), off, zero)
        within(host(s[y]), want, np.abs(want) * half("bf16") + mag * w.cols * U + TINY["bf16"])
    for k, dy, x8 in (("gate", "dgate", "x8"), ("up", "dup", "x8"), ("down", "dout", "h8")):
        d, x = host(s[dy]), value(s[x8])
        want, mag = i8_ref.grouped_wgrad(d, x, off), i8_ref.grouped_wgrad(np.abs(d), np.abs(x), off)
        within(host(s["dw_" + k]), want, np.abs(want) * half("f32") + mag * len(order) * U)
    token = order // top
    for rows, got, t in (("weighted", "y", "bf16"), (None, "dx", "f32")):
        r = host(s[rows]) if rows else host(s["dx_gate"] + s["dx_up"])
        want, mag, _ = mx_ref.embedding_grad(r, token, tokens, 1.0, -1)
        within(host(s[got]), want, np.abs(want) * half(t) + mag * top * U + TINY[t])


def same(a, b):
    for k in a:
        x, y = a[k], b[k]
        if not torch.is_tensor(x):
            x, y = x.codes, y.codes
        assert torch.equal(x, y), k


@pytest.mark.parametrize("tokens", [4, 3000])
def test_side_stream_and_graph_replays(ibp, tokens):
    """The layer and an integer product on a stream of their own, and captured into a graph and
    replayed with other routes, equal the eager ones bit for bit; two graphs share nothing."""
    layer = Layer(ibp, tokens, 160, 264, 10, 2, 1)
    w8 = ibp.ibp_i8_pack(torch.randn(600, 160, device="cuda"))

    def step():
        s = layer.step()
        s["x_i8"] = ibp.ibp_i8_pack(layer.x)
        s["y_i8"] = ibp.ibp_i8_matmul(s["x_i8"], w8)
        s["back"] = ibp.ibp_i8_unpack(s["x_i8"])
        return s

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    same(got, want)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = step()
        graphs.append((g, got))
    for k in range(4):
        layer.ids.copy_(torch.randint(10 if k else 1, layer.ids.shape, device="cuda"))
        layer.x.copy_(torch.randn_like(layer.x))
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        for _, got in graphs:
            same(got, want)


def test_two_streams_at_once(ibp):
    """Calls that run beside each other share nothing."""
    layers = [Layer(ibp, n, 160, 264, 10, 2, n) for n in (900, 3000)]
    w8 = ibp.ibp_i8_pack(torch.randn(200, 160, device="cuda"))
    want = [(layer.step(), ibp.ibp_i8_matmul(ibp.ibp_i8_pack(layer.x), w8)) for layer in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    got = [[] for _ in layers]
    for _ in range(3):
        for layer, stream, g in zip(layers, streams, got):
            with torch.cuda.stream(stream):
                g.append((layer.step(), ibp.ibp_i8_matmul(ibp.ibp_i8_pack(layer.x), w8)))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for s, y in g:
            same(s, w[0])
            assert torch.equal(y, w[1])


def test_the_stream_argument(ibp):
    layer = Layer(ibp, 700, 96, 160, 5, 2, 4)
    want = layer.step()
    dy = want["dgate"].float()
    want_dw = ibp.ibp_mx_grouped_wgrad(dy, want["x8"], want["offsets"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        order, off = ibp.ibp_expert_order(layer.ids, 5, stream=stream)
        y = ibp.ibp_mx_grouped_matmul(want["x8"], layer.w4["gate"], off, stream=stream)
        dw = ibp.ibp_mx_grouped_wgrad(dy, want["x8"], off, stream=stream)
        p = ibp.ibp_i8_pack(layer.x, stream=stream)
        z = ibp.ibp_i8_matmul(p, p, stream=stream)
        back = ibp.ibp_i8_unpack(p, stream=stream)
        side.synchronize()
        assert torch.equal(order, want["order"]) and torch.equal(y, want["gate"]) and torch.equal(dw, want_dw)
        assert torch.equal(z, ibp.ibp_i8_matmul(p, p)) and torch.equal(back, ibp.ibp_i8_unpack(p))


def test_device_refusals(ibp):
    """Host memory, tensors that are too small, outputs over inputs and outputs of another
    shape are refused."""
    x = torch.zeros(4, 64)
    cuda = x.cuda()
    p = ibp.ibp_i8_pack(cuda)
    with pytest.raises(ibp.IBPError):
        ibp.ibp_i8_pack(x, out=p)
    with pytest.raises(ValueError):
        ibp.ibp_i8_pack(cuda.t())
    with pytest.raises(ibp.IBPError):
        ibp.ibp_i8_pack(p.codes.view(torch.float32)[:, :4].contiguous(), out=ibp.I8Tensor(torch.zeros(4, 16, dtype=torch.int8), p.scales, 4, 4))
    with pytest.raises(ibp.IBPError):
        ibp.ibp_i8_matmul(p, p, out=p.codes.view(torch.float32).view(-1)[:16].view(4, 4), dtype=torch.float32)
    with pytest.raises(ValueError):
        ibp.ibp_i8_matmul(p, p, out=torch.zeros(4, 5, device="cuda"), dtype=torch.float32)
    with pytest.raises(ibp.IBPError):
        ibp.ibp_expert_order(torch.zeros(4, dtype=torch.int64), 3, order=torch.zeros(4, dtype=torch.int64, device="cuda"))
    with pytest.raises(ibp.IBPError):
        ibp.ibp_expert_order(torch.zeros(4, dtype=torch.int64, device="cuda"), 2000)
    with pytest.raises(ibp.IBPError):
        ibp.ibp_expert_order(torch.zeros(40000, dtype=torch.int64, device="cuda"), 3, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    a, w = ibp.ibp_mx_pack(cuda, ibp.IBP_MX_E4M3), ibp.ibp_mx_pack(cuda, ibp.IBP_MX_E2M1)
    with pytest.raises(ibp.IBPError):
        ibp.ibp_mx_grouped_matmul(a, w, torch.tensor([0, 1, 4]))  # offsets on the host
    with pytest.raises(ibp.IBPError):
        ibp.ibp_mx_grouped_matmul(a, a, torch.tensor([0, 1, 4], device="cuda"))  # weights in 8 bits
    with pytest.raises(ibp.IBPError):
        ibp.ibp_mx_grouped_wgrad(cuda, w, torch.tensor([0, 1, 4], device="cuda"))  # a checkpoint in 4 bits


def test_ranges_that_leave_an_allocation_are_refused(ibp):
    """Also where another tensor of the call, seen before, lies inside the same one."""
    import ctypes

    x = torch.ones(4, 64, device="cuda")
    (begin, end), = [(s["address"], s["address"] + s["total_size"]) for s in torch.cuda.memory_snapshot()
                     if s["address"] <= x.data_ptr() < s["address"] + s["total_size"]]
    p = ibp.ibp_i8_pack(x)
    lib, stream = ibp.load_library(), torch.cuda.current_stream().cuda_stream
    for codes, scales in ((end - 128, p.scales.data_ptr()), (p.codes.data_ptr(), end - 8), (begin - 128, p.scales.data_ptr())):
        t = ibp.ibp_i8_t(4, 64, codes, scales)
        assert lib.ibp_i8_pack(x.data_ptr(), 0, ctypes.byref(t), stream) == ibp.IBP_ERR_INVALID_ARG
    t = ibp.ibp_i8_t(4, 64, p.codes.data_ptr(), p.scales.data_ptr())
    assert lib.ibp_i8_unpack(ctypes.byref(t), end - 64, 0, stream) == ibp.IBP_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert torch.equal(ibp.ibp_i8_unpack(p, torch.float32), x)
