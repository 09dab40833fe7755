"""The language-model operators on the GPU at the ends of their ranges: what
test_gpu_operators.py does not reach."""
import numpy as np
import pytest
import torch

import mx_ref

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def ibp():
    import bit_packing_amd

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    bit_packing_amd.load_library()
    return bit_packing_amd


def device(ibp, codes, scales, cols, fmt):
    return ibp.MxTensor(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), codes.shape[0], cols, fmt)


def rounded(want, t):
    """A float64 matrix whose values 32 bits hold, rounded once to a type."""
    assert np.array_equal(want, want.astype(np.float32))
    return torch.from_numpy(want.astype(np.float32)).to(DT[t]).cuda()


# ---------------------------------------------------------------- products of far apart sizes

def nibbles(k):
    return k[:, 0::2] | (k[:, 1::2] << 4)


def limit_product(fmt, how, seed):
    """Every code v of A (rows) with every code w of B next to the largest product of the
    types, 448 * 6 or 6 * 6: in one block, cancelled in that block, in another block of the
    same 128 columns or behind them, or with v w in all other places of the block.  Sums of
    up to 33 terms are whole multiples of the step of v w, below 2^24 of them: any order of
    adding in 32 bits is exact."""
    rng = np.random.default_rng(seed)
    nv, cols = (126, 160) if fmt == mx_ref.E4M3 else (7, 160)
    a, b = np.zeros((nv, cols), np.uint8), np.zeros((7, cols), np.uint8)
    sign = 128 if fmt == mx_ref.E4M3 else 8
    v = np.arange(1, nv + 1) + sign * rng.integers(0, 2, nv)
    w = np.arange(1, 8)
    p = 32 + rng.permutation(32)
    a[:, p[0]], b[:, p[0]] = nv, 7
    places = p[1:] if how == "many" else p[1:2]
    a[:, places], b[:, places] = v[:, None], w[:, None]
    other = {"block": p[2], "instruction": 64 + 5, "later": 128 + 9}.get(how)
    if other:
        a[:, other], b[:, other] = nv, 7 + 8
    scales = lambda rows: np.where(np.arange(8) < 5, 127, 0).astype(np.uint8)[None].repeat(rows, 0)  # noqa: E731
    return (a if fmt == mx_ref.E4M3 else nibbles(a), scales(nv)), (nibbles(b), scales(7)), cols


@pytest.mark.parametrize("m,n", [(126, 7), (130, 1100), (3500, 3600)])  # one form of the product each
@pytest.mark.parametrize("how", ["beside", "block", "instruction", "later", "many"])
@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("fmt", [mx_ref.E4M3, mx_ref.E2M1])
def test_matmul_keeps_every_product(ibp, fmt, t, how, m, n):
    a, b, cols = limit_product(fmt, how, 1)
    want = mx_ref.unpack(*a, cols, fmt) @ mx_ref.unpack(*b, cols, mx_ref.E2M1).T
    ra, rb = np.arange(m) % len(want), np.arange(n) % 7
    print(f"product: m={m} n={n} format={fmt} {t} {how}", flush=True)
    y = ibp.ibp_mx_matmul(device(ibp, a[0][ra], a[1][ra], cols, fmt), device(ibp, b[0][rb], b[1][rb], cols, mx_ref.E2M1),
                          dtype=DT[t])
    want = rounded(want, t)[torch.from_numpy(ra).cuda()][:, torch.from_numpy(rb).cuda()]
    off = (y != want).nonzero()
    assert len(off) == 0, (len(off), off[0].tolist(), y[tuple(off[0])].item(), want[tuple(off[0])].item())


@pytest.mark.parametrize("m,n", [(24, 7), (130, 1100), (3500, 3600)])
@pytest.mark.parametrize("fmt", [mx_ref.E4M3, mx_ref.E2M1])
def test_matmul_blocks_of_far_apart_scales(ibp, fmt, m, n):
    """One block of 2^j, j up to 23, and one of 1 in the same 128 columns, another behind them."""
    cols, one = 160, {mx_ref.E4M3: 56, mx_ref.E2M1: 2}
    j = np.arange(m) % 24
    a, b = np.zeros((m, cols), np.uint8), np.zeros((n, cols), np.uint8)
    for c in (3, 70, 140):
        a[:, c], b[:, c] = one[fmt], one[mx_ref.E2M1]
    sa = np.where(np.arange(8) < 5, 127, 0).astype(np.uint8)[None].repeat(m, 0)
    sb = np.where(np.arange(8) < 5, 127, 0).astype(np.uint8)[None].repeat(n, 0)
    sa[:, 0] = 127 + j
    y = ibp.ibp_mx_matmul(device(ibp, a if fmt == mx_ref.E4M3 else nibbles(a), sa, cols, fmt),
                          device(ibp, nibbles(b), sb, cols, mx_ref.E2M1), dtype=torch.float32)
    want = torch.from_numpy((2.0 ** j + 2).astype(np.float32)).cuda()[:, None].expand(m, n)
    assert torch.equal(y, want)


# ---------------------------------------------------------------- sizes of zero

@pytest.mark.parametrize("ty,n,k", [("f32", 4096, 4096), ("f16", 4096, 4096), ("bf16", 4097, 4096), ("bf16", 4096, 4096),
                                    ("f32", 130, 70), ("bf16", 130, 70)])
@pytest.mark.parametrize("to", ["f32", "bf16"])
def test_wgrad_of_no_tokens(ibp, ty, to, n, k):
    """A layer without tokens, large or small, has the gradient 0."""
    x8 = ibp.make_mx(0, k, ibp.IBP_MX_E4M3, "cuda")
    dw = torch.full((n, k), float("nan"), dtype=DT[to], device="cuda")
    ibp.ibp_mx_linear_wgrad(torch.zeros(0, n, dtype=DT[ty], device="cuda"), x8, dw=dw)
    assert dw.eq(0).all()


def test_rows_of_no_columns_stay_rows(ibp):
    """Packing keeps the rows of a tensor without columns, and its product has them, as zeros."""
    for shape, rows in (((5, 0), 5), ((2, 3, 0), 6), ((0, 7), 0)):
        x = torch.zeros(shape, device="cuda")
        a = ibp.ibp_mx_pack(x, ibp.IBP_MX_E4M3)
        assert (a.rows, a.cols) == (rows, shape[-1])
        assert ibp.ibp_mx_unpack(a).shape == (rows, shape[-1])
        b = ibp.ibp_mx_pack(torch.zeros(9, shape[-1], device="cuda"), ibp.IBP_MX_E2M1)
        y = torch.full((rows, 9), float("nan"), device="cuda")
        ibp.ibp_mx_matmul(a, b, dtype=torch.float32, out=y)
        assert y.eq(0).all()
        h, gate8, up8 = ibp.ibp_mx_swiglu(x, x)
        assert h.shape == shape and gate8.rows == up8.rows == rows
        dgate, dup = ibp.ibp_mx_swiglu_backward(x, gate8, up8)
        assert dgate.shape == dup.shape == shape
        dw = ibp.ibp_mx_linear_wgrad(torch.ones(rows, 4, device="cuda"), a)
        assert dw.shape == (4, shape[-1]) and dw.eq(0).all()


# ---------------------------------------------------------------- the gated activation far from zero

@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("least", [-80, -1000])
def test_swiglu_of_far_gates(ibp, t, least):
    """Gates whose sigmoid is a subnormal number, or exp(-g) above the largest: the results are
    not (|u| up to 2^100, dh powers of two from 1 on).  The sigmoid is held in 32 bits: 6 units of
    2^-24, or four steps of the subnormal numbers (exp, its sum and quotient or product); two
    products and the last rounding as everywhere."""
    U, tiny = 2.0 ** -24, {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}[t]
    half = torch.finfo(DT[t]).eps / 2
    rng = np.random.default_rng(31)
    gates = -np.concatenate([np.arange(80, 112, 0.5), [64, 72, 120, 192, 200, 208, 1000]])
    gates = np.concatenate([gates[gates >= least], -gates, np.arange(-80, 0, 1.5), [0.0, -0.0, 1.0, -1.0]])
    rows, cols = 40, len(gates)
    power = (0, 15) if t == "f16" else (0, 100)
    g = torch.from_numpy(np.tile(gates, (rows, 1))).to(DT[t]).cuda()
    u = torch.from_numpy(rng.choice([-1.0, 1], (rows, cols)) * 2.0 ** rng.integers(*power, (rows, 1))).to(DT[t]).cuda()
    dh = torch.from_numpy(2.0 ** rng.integers(0, 10, (rows, cols))).to(DT[t]).cuda()
    h, g8, u8 = ibp.ibp_mx_swiglu(g, u)
    dg, du = ibp.ibp_mx_swiglu_backward(dh, g8, u8)
    host = lambda x: x.double().cpu().numpy()  # noqa: E731
    xg, xu, xd = host(g), host(u), host(dh)
    top = torch.finfo(DT[t]).max

    def near(got, want, bound, what):
        got, fine = host(got), np.abs(want) <= top
        assert np.array_equal(got[~fine], np.sign(want[~fine]) * np.inf)
        over = (np.abs(got - want) - bound)[fine]
        at = np.argmax(over)
        assert over[at] <= 0, (what, np.broadcast_to(xg, want.shape)[fine][at], got[fine][at], want[fine][at])

    sig = lambda x: np.exp(np.minimum(x, 0)) / (1 + np.exp(-np.abs(x)))  # noqa: E731
    want = xg * sig(xg) * xu
    near(h, want, np.abs(want) * (half + 8 * U) + np.abs(xg * xu) * 2.0 ** -147 + tiny, "h")
    kg, ku = (host(ibp.ibp_mx_unpack(m, torch.float32)) for m in (g8, u8))
    s = sig(kg)
    want = xd * ku * s * (1 + kg * sig(-kg))
    near(dg, want, np.abs(want) * half + np.abs(xd * ku) * (1 + np.abs(kg)) * (12 * U * s + 2.0 ** -147) + tiny, "dgate")
    want = xd * kg * s
    near(du, want, np.abs(want) * (half + 8 * U) + np.abs(xd * kg) * 2.0 ** -147 + tiny, "dup")


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(70, 1000), (300, 512), (41, 333), (9, 4096), (2000, 2048)])
def test_swiglu_in_place(ibp, t, rows, cols):
    """Outputs in the place of an input equal those of their own."""
    rng = np.random.default_rng(cols)
    g, u, d = (torch.from_numpy(rng.standard_normal((rows, cols))).to(DT[t]).cuda() for _ in range(3))
    h, g8, u8 = ibp.ibp_mx_swiglu(g, u)
    dg, du = ibp.ibp_mx_swiglu_backward(d, g8, u8)
    for first in (True, False):
        x, y, e = g.clone(), u.clone(), d.clone()
        got, p8, q8 = ibp.ibp_mx_swiglu(x, y, h=x if first else y)
        assert torch.equal(got, h) and got.data_ptr() == (x if first else y).data_ptr()
        assert torch.equal(p8.codes, g8.codes) and torch.equal(q8.codes, u8.codes)
        assert torch.equal(p8.scales, g8.scales) and torch.equal(q8.scales, u8.scales)
        a, b = ibp.ibp_mx_swiglu_backward(e, g8, u8, dgate=e if first else None, dup=None if first else e)
        assert torch.equal(a, dg) and torch.equal(b, du)


@pytest.mark.parametrize("cols,in_place", [(513, False), (1000, True), (509, True), (4097, False), (3, True)])
def test_gated_overlaps_are_refused(ibp, cols, in_place):
    """Outputs that overlap, and inputs in whose place another wavefront may still read."""
    import ctypes

    rows, step, ref = 4, 1 << 18, ctypes.byref  # each tensor somewhere in a quarter of a megabyte of its own
    flat = torch.zeros(8 * step, dtype=torch.uint8, device="cuda")
    at = lambda i, off=0: flat.data_ptr() + i * step + off  # noqa: E731
    mx = lambda i: ibp.ibp_mx_t(0, 0, rows, cols, at(i), at(i, step // 2))  # noqa: E731
    lib, end = ibp.load_library(), rows * cols * 4

    def forward(gate=at(0), up=at(1), h=at(2), g8=mx(4), u8=mx(5)):
        return lib.ibp_mx_swiglu(gate, up, ibp.IBP_F32, h, ref(g8), ref(u8), None)

    def back(dh=at(0), dg=at(1), du=at(2), g8=mx(4), u8=mx(5)):
        return lib.ibp_mx_swiglu_backward(dh, ibp.IBP_F32, ref(g8), ref(u8), dg, du, None)

    assert forward() == back() == ibp.IBP_OK
    some = [forward(h=at(0)), forward(h=at(1)), back(dg=at(0)), back(du=at(0))]
    assert some == [ibp.IBP_OK if in_place else ibp.IBP_ERR_INVALID_ARG] * 4
    bad = [forward(h=at(0, 4)), forward(h=at(0, end - 4)), forward(h=at(1, -4)), forward(h=at(4)), forward(h=at(4, step // 2)),
           forward(g8=mx(5)), forward(gate=at(4)), forward(up=at(5, step // 2)), back(dg=at(2)), back(dg=at(0, 4)),
           back(du=at(0, 4)), back(dg=at(4)), back(du=at(5, step // 2)), back(dg=at(2, -4))]
    assert bad == [ibp.IBP_ERR_INVALID_ARG] * len(bad)
    torch.cuda.synchronize()


# ---------------------------------------------------------------- long products, cut products

def codes_of(rng, rows, cols, fmt):
    """Whole multiples of 1/4 below 4 (e4m3) or all codes (e2m1) times scales of 1/2 to 2."""
    v = mx_ref.TABLE[fmt]
    pick = np.flatnonzero((v * 4 == np.floor(v * 4)) & (v < 4)) if fmt == mx_ref.E4M3 else np.arange(8)
    w = mx_ref.blocks(cols) * 32
    k = (rng.choice(pick, (rows, w)) + rng.integers(0, 2, (rows, w)) * (128 if fmt == mx_ref.E4M3 else 8)).astype(np.uint8)
    k[:, cols:] = 0
    s = np.zeros((rows, mx_ref.scale_pitch(cols)), np.uint8)
    s[:, : mx_ref.blocks(cols)] = rng.integers(126, 129, (rows, mx_ref.blocks(cols)))
    return k if fmt == mx_ref.E4M3 else nibbles(k), s


def exact_product(va, vb, step):
    """va vb^T in 64 bits on the GPU; every partial sum is a whole number of steps below 2^24."""
    a, b = (torch.from_numpy(x).cuda() for x in (va, vb))
    assert (a.abs() @ b.abs().t().contiguous()).max().item() < 2.0 ** 24 * step
    return a @ b.t().contiguous()


# k of several scale groups, without cuts and with two and eight ranges; both tiles
LONG = [(300, 600, 2080, 2), (257, 1000, 8190, 8), (520, 700, 1500, 1), (3500, 3601, 2100, 1), (1100, 1100, 4100, 3)]


@pytest.mark.parametrize("fmt", [mx_ref.E4M3, mx_ref.E2M1])
@pytest.mark.parametrize("m,n,k,cuts", LONG)
def test_long_products_are_exact(ibp, fmt, m, n, k, cuts):
    """Products below 90 in steps of 2^-5."""
    rng = np.random.default_rng(m + n + k)
    a, b = codes_of(rng, m, k, fmt), codes_of(rng, n, k, mx_ref.E2M1)
    want = exact_product(mx_ref.unpack(*a, k, fmt), mx_ref.unpack(*b, k, mx_ref.E2M1), 2.0 ** -5).float()
    assert ibp.ibp_mx_matmul_workspace_bytes(m, n, k, fmt) == (cuts * m * n * 4 if cuts > 1 else 0)
    da, db = device(ibp, *a, k, fmt), device(ibp, *b, k, mx_ref.E2M1)
    for t in DT:
        print(f"product: m={m} n={n} k={k} format={fmt} {t}", flush=True)
        y = torch.full((m, n), float("nan"), dtype=DT[t], device="cuda")
        assert torch.equal(ibp.ibp_mx_matmul(da, db, dtype=DT[t], out=y), want.to(DT[t])), t


@pytest.mark.parametrize("fmt", [mx_ref.E4M3, mx_ref.E2M1])
@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,k", [(300, 600, 2080), (520, 700, 1500), (3500, 3601, 700)])
def test_long_products_keep_nan_blocks_in_their_rows(ibp, fmt, t, m, n, k):
    rng = np.random.default_rng(k)
    a, b = codes_of(rng, m, k, fmt), codes_of(rng, n, k, mx_ref.E2M1)
    want = exact_product(mx_ref.unpack(*a, k, fmt), mx_ref.unpack(*b, k, mx_ref.E2M1), 2.0 ** -5).to(DT[t])
    last = mx_ref.blocks(k) - 1
    a[1][2, last], a[1][m - 1, 17], b[1][n - 1, last - 1], b[1][130, 0] = 255, 255, 255, 255
    y = ibp.ibp_mx_matmul(device(ibp, *a, k, fmt), device(ibp, *b, k, mx_ref.E2M1), dtype=DT[t])
    bad = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    bad[[2, m - 1]] = True
    bad[:, [130, n - 1]] = True
    assert torch.equal(torch.isnan(y), bad) and torch.equal(y[~bad], want[~bad])


# the large tile with 16, 5 and 8 ranges (of each part), and the small one with 7
CUT_WGRADS = [("bf16", 9000, 1000, 1000, 16), ("bf16", 9000, 1001, 1000, 16), ("f32", 9000, 1001, 1000, 5),
              ("f16", 9001, 1000, 1003, 8), ("bf16", 1700, 130, 260, 7)]


@pytest.mark.parametrize("ty,t,n,k,cuts", CUT_WGRADS)
def test_cut_wgrads_are_exact(ibp, ty, t, n, k, cuts):
    """dy whole from -4 to 4, x below 7.5 in steps of 1/8."""
    rng = np.random.default_rng(t + n + k)
    dy = rng.integers(-4, 5, (t, n)).astype(float)
    x = codes_of(rng, t, k, mx_ref.E4M3)
    v = mx_ref.unpack(*x, k, mx_ref.E4M3)
    want = exact_product(np.ascontiguousarray(dy.T), np.ascontiguousarray(v.T), 2.0 ** -3).float()
    parts = {"bf16": 1, "f16": 2, "f32": 3}[ty]
    sums = -(-cuts * parts * n * k * 4 // 16) * 16
    copy = parts * t * -(-n // 8) * 16 if t >= 9000 and (parts > 1 or n % 8) else 0  # the large tile's
    assert ibp.ibp_mx_linear_wgrad_workspace_bytes(t, n, k, DT[ty]) == sums + copy
    x8 = device(ibp, *x, k, mx_ref.E4M3)
    print(f"weight gradient: t={t} n={n} k={k} {ty}", flush=True)
    for to in ("f32", "bf16"):
        dw = torch.full((n, k), float("nan"), dtype=DT[to], device="cuda")
        got = ibp.ibp_mx_linear_wgrad(torch.from_numpy(dy).to(DT[ty]).cuda(), x8, dw=dw)
        assert torch.equal(got, want.to(DT[to])), to


@pytest.mark.parametrize("ty", ["f32", "f16"])
def test_cut_wgrads_add_their_parts(ibp, ty):
    """dY whose bits fill all its parts: within the 32-bit sums' own bound."""
    t, n, k = 9000, 1000, 1000
    gen = torch.Generator(device="cuda").manual_seed(5)
    dy = (torch.randn(t, n, generator=gen, device="cuda") * 0.1).to(DT[ty])
    x8 = ibp.ibp_mx_pack(torch.randn(t, k, generator=gen, device="cuda"), ibp.IBP_MX_E4M3)
    v, d = ibp.ibp_mx_unpack(x8, torch.float32).double(), dy.double().t().contiguous()
    want, mag = d @ v, d.abs() @ v.abs()
    got = ibp.ibp_mx_linear_wgrad(dy, x8, dw_dtype=torch.float32).double()
    assert ((got - want).abs() <= mag * t * 2.0 ** -24).all()
    # and far closer than without the last part, whose share is 2^-8 (half precision) or 2^-16
    assert (got - want).norm() < want.norm() * (2.0 ** -19 if ty == "f32" else 2.0 ** -12)


# ---------------------------------------------------------------- the training example

def test_gradients_of_the_example_have_the_right_size():
    """The factor that fits a gradient of the example best to the one that torch computes from
    the same packed values is 1 up to 4%: rounding to e2m1 (a quarter at most, a tenth in the
    mean square) and e4m3 adds errors that are as good as independent of the gradient, so it
    moves the factor by its square, 1% for each of the two 4-bit packings of a weight."""
    import os
    import sys

    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import bit_packing_amd as ibp
    import packed_training

    torch.manual_seed(3)
    model = packed_training.Model(500, 192, 384, 9)
    model.scale = 1.25
    ids = torch.randint(500, (1000,), device="cuda")
    y, kept = model.forward(ids)
    dy = (torch.randn_like(y.float()) * 0.01).to(torch.bfloat16)
    grads = model.backward(dy, kept)
    wg, wu, wd = (ibp.ibp_mx_unpack(layer.w4, dtype=torch.float32).requires_grad_() for layer in (model.gate, model.up, model.down))
    table = model.table.float().requires_grad_()
    x = table[ids] * model.scale
    h = torch.nn.functional.silu(x @ wg.t()) * (x @ wu.t())
    (h @ wd.t()).backward(dy.float())
    for name, want in (("down", wd.grad), ("gate", wg.grad), ("up", wu.grad), ("table", table.grad)):
        factor = ((grads[name].double() * want.double()).sum() / want.double().square().sum()).item()
        print(name, factor)
        assert abs(factor - 1) < 0.04, (name, factor)
