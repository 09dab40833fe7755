"""8-bit integer rows and layers of experts on the GPU where test_gpu_more_operators.py does
not reach: what two roundings make of a border, and every form of the kernels."""
import numpy as np
import pytest
import torch

import i8_ref
import mx_ref

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


# ---------------------------------------------------------------- from tile to tile

# 256 x 256 tiles (more than 256 of them), then 128 x 128 (more than 512): workgroups take a
# second one, or a third.  Ragged and whole tiles, none to eight stages of k.
@pytest.mark.parametrize("m,n,k", [(4400, 4500, 545), (4352, 4352, 1024), (4352, 4400, 100), (4352, 4352, 0), (256, 66000, 400),
                                   (3000, 3001, 130), (256, 66048, 700)])
def test_i8_matmul_from_tile_to_tile(ibp, m, n, k):
    rng = np.random.default_rng(m + n + k)
    a, b = (np.zeros((r, i8_ref.pitch(k)), np.int8) for r in (m, n))
    a[:, :k], b[:, :k] = rng.integers(-128, 128, (m, k)), rng.integers(-128, 128, (n, k))
    sa, sb = (np.float32(rng.standard_normal(r) * 1e-2) for r in (m, n))
    # sums below 2^53 are exact in float64 products
    sums = (a.astype(np.float64) @ b.T.astype(np.float64)).astype(np.float32)
    less = np.abs(sa)[:, None] < np.abs(sb)[None]
    want = torch.from_numpy(sums * np.where(less, sa[:, None], sb[None]) * np.where(less, sb[None], sa[:, None])).cuda()
    a8, b8 = i8(ibp, a, sa, k), i8(ibp, b, sb, k)
    for to in DT:
        print(f"product of 8-bit integers: m={m} n={n} k={k} to={to}", flush=True)
        whole = torch.full((m + 2, n), float("nan"), dtype=DT[to], device="cuda")
        ibp.ibp_i8_matmul(a8, b8, dtype=DT[to], out=whole[1:-1])
        assert torch.equal(whole[1:-1], want.to(DT[to])) and whole[0].isnan().all() and whole[-1].isnan().all()


# ---------------------------------------------------------------- every form of the products by expert

half = lambda t: torch.finfo(DT[t]).eps / 2  # noqa: E731
TINY = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}
U = 2.0 ** -24


def mx(ibp, codes, scales, cols, fmt):
    return ibp.MxTensor(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), codes.shape[0], cols, fmt)


def gpu(x, t):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DT[t]).cuda()


def codes_of(rng, rows, cols, fmt):
    """A packed tensor of scale 1 whose values are whole multiples of 1/4 up to 3.75 (e4m3) or
    of 1/2 up to 6 (e2m1), its columns past the end zero."""
    v = mx_ref.TABLE[fmt]
    pick = np.flatnonzero((v * 4 == np.floor(v * 4)) & (v < 4)) if fmt == mx_ref.E4M3 else np.arange(8)
    k = rng.choice(pick, (rows, mx_ref.blocks(cols) * 32)) + rng.integers(0, 2, (rows, mx_ref.blocks(cols) * 32)) * (128 if fmt == mx_ref.E4M3 else 8)
    k[:, cols:] = 0
    k = k.astype(np.uint8)
    scales = np.zeros((rows, mx_ref.scale_pitch(cols)), np.uint8)
    scales[:, : mx_ref.blocks(cols)] = 127
    return (k if fmt == mx_ref.E4M3 else k[:, 0::2] | (k[:, 1::2] << 4)), scales


def offsets_of(rng, rows, experts, how):
    """Where the experts' rows begin, `rows` in all."""
    if how == "one":  # all with one expert
        sizes = np.where(np.arange(experts) == rng.integers(experts), rows, 0)
    elif how == "even":
        sizes = np.full(experts, rows // experts) + (np.arange(experts) < rows % experts)
    else:  # ragged, about a third of the experts without rows
        p = rng.random(experts) ** 2 * (rng.random(experts) < 0.67)
        p[rng.integers(experts)] += 0.1
        sizes = rng.multinomial(rows, p / p.sum())
    return np.concatenate([[0], np.cumsum(sizes)])


def bad_offsets(t, e):
    """Offsets that fall, or leave the rows."""
    rng = np.random.default_rng(t + e)
    yield [0] + [t if k % 2 else 0 for k in range(1, e + 1)]
    yield [t - k * (t // e) for k in range(e + 1)]
    yield list(rng.choice([-5, -(1 << 62), 1 << 62, 1 << 40, 0, 1, t, t + 1], e)) + [-1]
    yield [k * t // e for k in range(e)] + [1 << 40]
    yield [-(1 << 62)] + [1 << 62] * e


# rows, experts, outputs: of 16, 32 and 64 rows an expert and kernel (e4m3, or 32 and 64 for
# e2m1), 128 x 128 tiles, 256 x 256 tiles
FORMS = [(500, 100, 201), (300, 10, 700), (3000, 4, 200), (2200, 8, 2001), (6500, 8, 3600)]


@pytest.mark.parametrize("fmt", [mx_ref.E4M3, mx_ref.E2M1])
@pytest.mark.parametrize("t,e,n", FORMS)
def test_bad_offsets_lead_nowhere_in_any_product(ibp, fmt, t, e, n):
    rng = np.random.default_rng(t)
    k = 96
    a, b = mx(ibp, *codes_of(rng, t, k, fmt), k, fmt), mx(ibp, *codes_of(rng, e * n, k, mx_ref.E2M1), k, mx_ref.E2M1)
    for to in ("f32", "bf16"):
        for off in bad_offsets(t, e):
            print(f"bad offsets: t={t} e={e} n={n} format={fmt} to={to} {off[:4]}", flush=True)
            err = torch.zeros(1, dtype=torch.int32, device="cuda")
            whole = torch.full((t + 2, n), 5.0, dtype=DT[to], device="cuda")
            ibp.ibp_mx_grouped_matmul(a, b, torch.tensor(off, device="cuda"), dtype=DT[to], out=whole[1:-1], err=err)
            assert err.item() == ibp.IBP_DEVERR_CORRUPT and (whole[0] == 5).all() and (whole[-1] == 5).all()


@pytest.mark.parametrize("fmt", [mx_ref.E4M3, mx_ref.E2M1])
@pytest.mark.parametrize("t,e,n", FORMS)
@pytest.mark.parametrize("to", ["f32", "f16", "bf16"])
def test_every_product_by_expert(ibp, fmt, t, e, n, to):
    """Ragged rows that begin behind the first and end before the last, columns that end inside
    a store, NaN blocks of one row and of one weight: exact, as 160 terms of up to 22.5 in steps
    of 1/8 are, and the rows of no expert stay."""
    rng = np.random.default_rng(t + e + n)
    k = 160
    a, b = codes_of(rng, t, k, fmt), codes_of(rng, e * n, k, mx_ref.E2M1)
    off = offsets_of(rng, t - 20, e, "ragged" if e < 100 else "even") + 7
    big = int(np.argmax(np.diff(off)))
    a[1][off[big] + 1, 3] = 255
    b[1][big * n + n - 2, 4] = 255
    want = i8_ref.grouped_product(mx_ref.unpack(*a, k, fmt), mx_ref.unpack(*b, k, mx_ref.E2M1).reshape(e, n, k), off,
                                  np.full((t, n), 5.0))
    print(f"product by expert: t={t} e={e} n={n} format={fmt} to={to}", flush=True)
    whole = torch.full((t + 2, n), 5.0, dtype=DT[to], device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ibp.ibp_mx_grouped_matmul(mx(ibp, *a, k, fmt), mx(ibp, *b, k, mx_ref.E2M1), torch.from_numpy(off).cuda(), dtype=DT[to],
                              out=whole[1:-1], err=err)
    got = host(whole)
    assert np.isnan(want).sum() == n + off[big + 1] - off[big] - 1
    assert np.array_equal(got[1:-1], rounded(want, to), equal_nan=True) and err.item() == 0
    assert (got[0] == 5).all() and (got[-1] == 5).all()


# ---------------------------------------------------------------- every form of the gradients by expert

# tokens, experts, outputs, inputs: 128 x 128 tiles whole and in units, 256 x 256 tiles whole
# (the experts of many tokens first) and in units
GRADIENTS = [(900, 4, 300, 96), (6000, 4, 256, 264), (2500, 45, 500, 601), (20000, 24, 500, 1000)]


@pytest.mark.parametrize("ty", ["bf16", "f32"])
@pytest.mark.parametrize("t,e,n,k", GRADIENTS)
def test_bad_offsets_lead_nowhere_in_any_gradient(ibp, ty, t, e, n, k):
    rng = np.random.default_rng(t)
    x8 = mx(ibp, *codes_of(rng, t, k, mx_ref.E4M3), k, mx_ref.E4M3)
    dy = torch.ones(t, n, dtype=DT[ty], device="cuda")
    for to in ("f32", "bf16"):
        for off in bad_offsets(t, e):
            print(f"bad offsets: t={t} e={e} n={n} k={k} ty={ty} to={to} {off[:4]}", flush=True)
            err = torch.zeros(1, dtype=torch.int32, device="cuda")
            dw = torch.full((e + 2, n, k), 5.0, dtype=DT[to], device="cuda")
            ibp.ibp_mx_grouped_wgrad(dy, x8, torch.tensor(off, device="cuda"), dw=dw[1:-1], err=err)
            assert err.item() == ibp.IBP_DEVERR_CORRUPT and (dw[0] == 5).all() and (dw[-1] == 5).all()


@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("how", ["ragged", "one"])
@pytest.mark.parametrize("t,e,n,k", [*GRADIENTS, (30000, 24, 500, 1000)])
def test_every_gradient_by_expert(ibp, ty, how, t, e, n, k):
    """dy whole from -8 to 8, x up to 3.75 in steps of 1/4: at most 30000 terms of 30 in such
    steps, below 2^24 of them, so every result is exact and rounded once.  An infinity of dy and
    a NaN block of x reach their expert's gradient only."""
    rng = np.random.default_rng(t + e + n + k)
    dy, x = rng.integers(-8, 9, (t, n)).astype(float), codes_of(rng, t, k, mx_ref.E4M3)
    off = offsets_of(rng, t - 9, e, how) + 4
    big = int(np.argmax(np.diff(off)))
    dy[off[big + 1] - 1, 3] = np.inf
    x[1][off[big], 2] = 255
    with np.errstate(invalid="ignore"):
        want = i8_ref.grouped_wgrad(dy, mx_ref.unpack(*x, k, mx_ref.E4M3), off)
    bad = np.zeros((e, n, k), bool)
    bad[big, 3], bad[big, :, 64:96] = True, True
    assert np.array_equal(~np.isfinite(want), bad)
    dy, x8, off = gpu(dy, ty), mx(ibp, *x, k, mx_ref.E4M3), torch.from_numpy(off).cuda()
    for to in DT:
        print(f"gradient by expert: t={t} e={e} n={n} k={k} {how} ty={ty} to={to}", flush=True)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        dw = torch.full((e + 2, n, k), 5.0, dtype=DT[to], device="cuda")
        ibp.ibp_mx_grouped_wgrad(dy, x8, off, dw=dw[1:-1], err=err)
        got = host(dw)
        assert np.array_equal(~np.isfinite(got[1:-1]), bad) and err.item() == 0
        assert np.array_equal(got[1:-1][~bad], rounded(want[~bad], to))
        assert (got[0] == 5).all() and (got[-1] == 5).all()


@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("t,e,n,k", GRADIENTS[2:])
def test_large_gradients_of_any_values(ibp, ty, t, e, n, k):
    """dy of every bit its type has: off by at most half a step of the result and, for sums of
    each of dy's parts in 32 bits, 2^-24 a term of the terms' magnitudes."""
    rng = np.random.default_rng(t + 1)
    dy = gpu(rng.standard_normal((t, n)) * 0.1, ty)
    x = mx_ref.pack(rng.standard_normal((t, k)) * 3, mx_ref.E4M3)
    off = offsets_of(rng, t, e, "ragged")
    v, d = mx_ref.unpack(*x, k, mx_ref.E4M3), host(dy)
    want, mag = i8_ref.grouped_wgrad(d, v, off), i8_ref.grouped_wgrad(np.abs(d), np.abs(v), off)
    terms = {"bf16": 1, "f16": 2, "f32": 3}[ty] * np.diff(off)[:, None, None]
    for to in DT:
        got = host(ibp.ibp_mx_grouped_wgrad(dy, mx(ibp, *x, k, mx_ref.E4M3), torch.from_numpy(off).cuda(), dw_dtype=DT[to]))
        over = np.abs(got - want) - (np.abs(want) * half(to) + mag * terms * U + TINY[to])
        assert over.max() <= 0


@pytest.mark.parametrize("m,n", [(2050, 2050), (4400, 4300)])
def test_i8_matmul_of_the_largest_sums_in_larger_tiles(ibp, m, n):
    """The deepest product of the largest codes, in 128 x 128 and in 256 x 256 tiles."""
    k = ibp.IBP_I8_MAX_DEPTH
    a, b = (torch.zeros(r, i8_ref.pitch(k), dtype=torch.int8, device="cuda") for r in (m, n))
    a[:, :k], b[:, :k] = -128, -128
    b[n // 2:, :k] = 127
    one = lambda r: torch.ones(r, device="cuda")  # noqa: E731
    print(f"product of 8-bit integers: m={m} n={n} k={k}", flush=True)
    y = ibp.ibp_i8_matmul(ibp.I8Tensor(a, one(m), m, k), ibp.I8Tensor(b, one(n), n, k), dtype=torch.float32)
    assert (y[:, : n // 2] == float(np.float32(k * 16384))).all() and (y[:, n // 2:] == float(np.float32(-k * 128 * 127))).all()
