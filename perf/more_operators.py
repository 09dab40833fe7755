"""Further language-model operators of the library, as they are measured.

Two groups:

* 8-bit integers with a scale for each row (tokens of an activation, output channels of a
  weight): quantisation and reading back, and the product of two such tensors;
* a layer of experts on microscaled tensors: the order of tokens by expert, the product of
  packed activations with the 4-bit weights of each row's expert, and those weights'
  gradients from an 8-bit checkpoint.

8-bit integer rows (plain form and library alike): with m the largest magnitude of a row,
its scale is m / 127 rounded to 32 bits and its codes are 127 x / m rounded to the nearest
whole number, ties to even; a row of zeros has the scale 0.

Microscaled rows: blocks of 32 elements (the last one filled up with zeros) with the scale
2^s, s the smallest exponent with max|x| <= M * 2^s (M = 448 for e4m3, 6 for e2m1), at least
-117 and at most 119 (e4m3) or 125 (e2m1), stored as the byte s + 127; elements are x / 2^s
rounded to the nearest code, ties to even.  e4m3: one byte an element; e2m1: the even
element in the low nibble.  Scale rows are padded to a multiple of 4 bytes with zeros.

Rows are sorted by expert: rows offsets[e] to offsets[e + 1] are expert e's.

With `own` false everything is computed by elementary torch operations, in 32 bits but for
codes, whose borders take 64.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
# largest value, its fraction of the next power of two, the exponent of that power, largest
# scale exponent, smallest normal exponent and fraction bits of the element types
ELEM = {"e4m3": (448.0, 0.875, 9, 119, -6, 3), "e2m1": (6.0, 0.75, 3, 125, 0, 1)}
MIN_EXP = -117


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a small projection's weight, odd sizes, to 8 bits and back
        {"name": "int8-small", "op": "int8", "rows": 127, "cols": 4001, "type": "f32"},
        # a whole weight matrix to 8 bits and back
        {"name": "int8-weight", "op": "int8", "rows": 16384, "cols": 8192, "type": "bf16"},
        # one token of serving through a layer of 8-bit weights
        {"name": "int8-serve", "op": "product", "tokens": 1, "outs": 8192, "ins": 8192, "type": "bf16", "out": "bf16"},
        # a short prompt through a small layer, nothing a multiple of a tile
        {"name": "int8-short", "op": "product", "tokens": 333, "outs": 1000, "ins": 2001, "type": "f16", "out": "f32"},
        # a batch of prompts through a wide layer
        {"name": "int8-batch", "op": "product", "tokens": 8192, "outs": 8192, "ins": 4096, "type": "bf16", "out": "bf16"},
        # eight sequences' next tokens, eight experts each
        {"name": "order-serve", "op": "order", "tokens": 64, "experts": 64},
        # a training batch of 16384 tokens, eight experts each
        {"name": "order-batch", "op": "order", "tokens": 131072, "experts": 256},
        # the same few tokens through their experts' 4-bit weights
        {"name": "experts-serve", "op": "grouped", "tokens": 64, "experts": 64, "outs": 2048, "ins": 4096, "a": "e4m3", "out": "bf16"},
        # a short prompt, ragged sizes, activations in 4 bits too
        {"name": "experts-short", "op": "grouped", "tokens": 1501, "experts": 24, "outs": 1000, "ins": 1503, "a": "e2m1", "out": "f32"},
        # a training batch: forward, and with the transposed weights the activations' gradient
        {"name": "experts-batch", "op": "grouped", "tokens": 32768, "experts": 32, "outs": 2048, "ins": 4096, "a": "e4m3", "out": "bf16"},
        # weight gradients of small experts in single precision, ragged sizes
        {"name": "experts-grad-short", "op": "wgrad", "tokens": 1501, "experts": 24, "outs": 500, "ins": 1000, "type": "f32", "grad": "f32"},
        # weight gradients of the training batch
        {"name": "experts-grad-batch", "op": "wgrad", "tokens": 32768, "experts": 32, "outs": 2048, "ins": 4096, "type": "bf16", "grad": "bf16"},
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], spread over its logarithm; most are odd sizes."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["int8", "product", "order", "grouped", "wgrad"])
    kind = lambda: rng.choice(["f32", "f16", "bf16"])  # noqa: E731
    if op == "int8":
        cols = _spread(rng, 16, 16384)
        return {"op": op, "rows": _spread(rng, 1, min(16384, (1 << 26) // cols)), "cols": cols, "type": kind()}
    if op == "product":
        return {"op": op, "tokens": _spread(rng, 1, 8192), "outs": _spread(rng, 32, 8192), "ins": _spread(rng, 32, 4096),
                "type": kind(), "out": kind()}
    if op == "order":
        return {"op": op, "tokens": _spread(rng, 1, 131072), "experts": _spread(rng, 1, 1024)}
    experts = _spread(rng, 2, 128)
    outs = _spread(rng, 32, 2048)
    ins = _spread(rng, 32, min(4096, (1 << 28) // (experts * outs)))
    case = {"op": op, "tokens": _spread(rng, 1, 32768), "experts": experts, "outs": outs, "ins": ins}
    if op == "grouped":
        return {**case, "a": rng.choice(["e4m3", "e2m1"]), "out": kind()}
    case["type"] = kind()
    if case["type"] != "bf16":
        case["tokens"] = min(case["tokens"], 8192 + case["tokens"] % 1024)
    return {**case, "grad": rng.choice(["f32", "bf16"])}


def _share(experts):
    """How the tokens fall on the experts, most frequent first: p(rank) ~ rank^-1/2."""
    p = torch.arange(1, experts + 1, dtype=torch.float64) ** -0.5
    return p / p.sum()


def _packed(rows, cols, elem):
    return rows * (cols * (1.0 if elem == "e4m3" else 0.5) + math.ceil(cols / 32))


def work(case):
    op = case["op"]
    if op == "int8":
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * (n * SIZE[case["type"]] + n + 4 * case["rows"]), "flops": 4 * n}
    if op == "order":
        return {"bytes": 16 * case["tokens"] + 8 * (case["experts"] + 1), "flops": case["tokens"]}
    t, o, i = case["tokens"], case["outs"], case["ins"]
    if op == "product":
        return {"bytes": t * i * SIZE[case["type"]] + o * (i + 4) + t * o * SIZE[case["out"]], "flops": 2 * t * o * i}
    e = case["experts"]
    if op == "grouped":
        used = float((1 - (1 - _share(e)) ** t).sum())  # experts that have a token
        return {"bytes": t * i * 2 + used * _packed(o, i, "e2m1") + t * o * SIZE[case["out"]] + 8 * (e + 1), "flops": 2 * t * o * i}
    return {"bytes": t * o * SIZE[case["type"]] + _packed(t, i, "e4m3") + e * o * i * SIZE[case["grad"]] + 8 * (e + 1),
            "flops": 2 * t * o * i}


# ------------------------------------------------------------------ inputs

def _activations(rows, cols, dtype, g, sd=1.0):
    """Normal values whose rows and columns differ in size, a few columns far larger than the rest."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= sd * torch.exp2(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))
    x *= torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, 10.0, 1.0)
    return x.to(dtype)


def _routes(tokens, experts, seed):
    """An expert for each of the tokens, which expert is how frequent drawn anew."""
    g = torch.Generator()
    g.manual_seed(int(seed) + 1)
    p = _share(experts)[torch.randperm(experts, generator=g)]
    return torch.multinomial(p, tokens, replacement=True, generator=g)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, s = case["op"], {"case": case}
    if op == "int8":
        s["x"] = _activations(case["rows"], case["cols"], DTYPES[case["type"]], g, 0.02)
    elif op == "product":
        s["x"] = _activations(case["tokens"], case["ins"], DTYPES[case["type"]], g)
        w = torch.randn(case["outs"], case["ins"], generator=g, device="cuda") * 0.02
        s["codes"], s["scales"] = _quantise(w)
    elif op == "order":
        s["ids"] = _routes(case["tokens"], case["experts"], seed).cuda()
    else:
        sizes = torch.bincount(_routes(case["tokens"], case["experts"], seed), minlength=case["experts"])
        s["sizes"] = sizes.tolist()  # for the plain form, which takes one expert after another
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), sizes.cumsum(0)]).cuda()
        x = _activations(case["tokens"], case["ins"], torch.bfloat16, g)
        if op == "grouped":
            s["x"] = x
            w = torch.randn(case["experts"] * case["outs"], case["ins"], generator=g, device="cuda") * 0.02
            s["codes"], s["scales"] = _pack(w, "e2m1")
        else:
            s["codes"], s["scales"] = _pack(x, "e4m3")
            s["dy"] = _activations(case["tokens"], case["outs"], DTYPES[case["type"]], g, 0.01)
    return s


# ------------------------------------------------------------------ the formats, plainly

def _quantise(x):
    """Codes, in rows filled up with zeros to a multiple of 16, and scales of x."""
    m = x.abs().amax(1)
    q = torch.round(x.double() * 127 / m.double().clamp(min=1e-300)[:, None]).to(torch.int8)
    return torch.nn.functional.pad(q, (0, -x.shape[1] % 16)).contiguous(), m.float() / 127


def _pow2(e):
    """2^e in 32 bits, exactly, for whole -126 <= e <= 127."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _blocks(x):
    """Rows cut into blocks of 32, the last filled up with zeros."""
    x = torch.nn.functional.pad(x, (0, -x.shape[1] % 32))
    return x.reshape(x.shape[0], -1, 32)


def _rounded(x, elem):
    """Scale exponents of the blocks, and their elements over the scale rounded to the element type."""
    big, part, lead, most, low, frac = ELEM[elem]
    x = _blocks(x.float())
    amax = x.abs().amax(2)
    m, e = torch.frexp(amax)
    s = torch.where(amax > 0, e - lead + (m > part), MIN_EXP).clamp(MIN_EXP, most)
    y = x * _pow2(-s)[:, :, None]
    step = _pow2((torch.frexp(y)[1] - 1).clamp(min=low) - frac)
    return s, (torch.round(y / step) * step).clamp(-big, big)


def _pack(x, elem):
    """Codes and scale bytes of x."""
    s, y = _rounded(x, elem)
    y = y.reshape(y.shape[0], -1)
    if elem == "e4m3":
        codes = y.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        code = torch.bucketize(y.abs(), torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=y.device), out_int32=True)
        code = (code + torch.where(torch.signbit(y), 8, 0)).to(torch.uint8)
        codes = code[:, 0::2] + code[:, 1::2] * 16
    scales = torch.nn.functional.pad((s + 127).to(torch.uint8), (0, -s.shape[1] % 4))
    return codes.contiguous(), scales.contiguous()


def _unpack(codes, scales, cols, elem, dtype=torch.float32):
    """The values that codes and scales stand for."""
    if elem == "e4m3":
        y = codes.view(torch.float8_e4m3fn).to(dtype)
    else:
        value = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device, dtype=dtype)
        value = torch.cat([value, -value])
        y = torch.stack([value[(codes & 15).long()], value[(codes >> 4).long()]], 2).reshape(codes.shape[0], -1)
    y = y.reshape(y.shape[0], -1, 32)
    y = y * _pow2(scales[:, : y.shape[1], None].int() - 127).to(dtype)
    return y.reshape(y.shape[0], -1)[:, :cols]


def _kept(x, elem):
    """What x reads back as after packing, in 32 bits."""
    s, y = _rounded(x, elem)
    return (y * _pow2(s)[:, :, None]).reshape(x.shape[0], -1)[:, : x.shape[1]]


# ------------------------------------------------------------------ one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import bit_packing_amd as ibp

    c = s["case"]
    op = c["op"]
    if op == "int8":
        return ibp.ibp_i8_unpack(ibp.ibp_i8_pack(s["x"]), dtype=DTYPES[c["type"]])
    if op == "product":
        w8 = ibp.I8Tensor(s["codes"], s["scales"], c["outs"], c["ins"])
        return ibp.ibp_i8_matmul(ibp.ibp_i8_pack(s["x"]), w8, dtype=DTYPES[c["out"]])
    if op == "order":
        return ibp.ibp_expert_order(s["ids"], c["experts"])
    if op == "grouped":
        w4 = ibp.MxTensor(s["codes"], s["scales"], c["experts"] * c["outs"], c["ins"], ibp.IBP_MX_E2M1)
        a = ibp.ibp_mx_pack(s["x"], ibp.IBP_MX_E4M3 if c["a"] == "e4m3" else ibp.IBP_MX_E2M1)
        return ibp.ibp_mx_grouped_matmul(a, w4, s["offsets"], dtype=DTYPES[c["out"]])
    x8 = ibp.MxTensor(s["codes"], s["scales"], c["tokens"], c["ins"], ibp.IBP_MX_E4M3)
    return ibp.ibp_mx_grouped_wgrad(s["dy"], x8, s["offsets"], dw_dtype=DTYPES[c["grad"]])


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "int8":
        codes, scales = _quantise(s["x"])
        return (codes[:, : c["cols"]].float() * scales[:, None]).to(DTYPES[c["type"]])
    if op == "product":
        codes, scales = _quantise(s["x"])
        y = codes[:, : c["ins"]].float() @ s["codes"][:, : c["ins"]].float().t()
        return (y * scales[:, None] * s["scales"]).to(DTYPES[c["out"]])
    if op == "order":
        order = torch.argsort(s["ids"], stable=True)
        return order, torch.searchsorted(s["ids"][order], torch.arange(c["experts"] + 1, device="cuda"))
    outs, at = c["outs"], 0
    if op == "grouped":
        x = _kept(s["x"], c["a"])
        y = torch.empty(c["tokens"], outs, device=x.device, dtype=DTYPES[c["out"]])
        for e, n in enumerate(s["sizes"]):
            if n:
                rows = slice(e * outs, (e + 1) * outs)
                y[at : at + n] = x[at : at + n] @ _unpack(s["codes"][rows], s["scales"][rows], c["ins"], "e2m1").t()
                at += n
        return y
    x, dy = _unpack(s["codes"], s["scales"], c["ins"], "e4m3"), s["dy"].float()
    dw = torch.empty(c["experts"], outs, c["ins"], device=x.device, dtype=DTYPES[c["grad"]])
    for e, n in enumerate(s["sizes"]):
        dw[e] = dy[at : at + n].t() @ x[at : at + n]
        at += n
    return dw


# ------------------------------------------------------------------ the definition in 64 bits

def _nearest(x, elem):
    """What x reads back as: the nearest of the element type's values, found in a table of them."""
    if elem == "e4m3":
        v = [m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1]
        most = 119
    else:
        v, most = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], 125
    v = torch.tensor(v, device=x.device, dtype=torch.float64)
    b = torch.cat([x.double(), x.new_zeros(x.shape[0], -x.shape[1] % 32, dtype=torch.float64)], 1).unflatten(1, (-1, 32))
    # the first power of two from 2^-117 on that, times M, is not below the block's largest
    power = torch.tensor([2.0 ** e for e in range(MIN_EXP, most + 1)], device=x.device, dtype=torch.float64)
    at = torch.searchsorted(power * v[-1], b.abs().max(2).values).clamp(max=len(power) - 1)
    scale = power[at][..., None]
    y = b / scale
    mid = (v[1:] + v[:-1]) / 2
    a = y.abs().contiguous()
    k = torch.searchsorted(mid, a)  # codes whose upper border lies below the value; a value on a border stays below it
    up = (k < len(mid)) & (mid[k.clamp(max=len(mid) - 1)] == a) & (k % 2 == 1)
    return (torch.copysign(v[k + up.long()], y) * scale).flatten(1)[:, : x.shape[1]]


def _whole(x):
    """Whole numbers next to 127 x / m, and the steps m / 127 they count, with m the rows' largest magnitudes."""
    m = x.double().abs().max(1, keepdim=True).values
    y = x.double() * 127
    low = torch.floor(y / m)
    twice = 2 * (y - low * m)  # exact: fewer than 53 bits
    return torch.where(m > 0, low + ((twice > m) | ((twice == m) & (low % 2 != 0))), 0.0), m / 127


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "int8":
        q, step = _whole(s["x"])
        return q * step
    if op == "product":
        q, step = _whole(s["x"])
        w = s["codes"][:, : case["ins"]].double().mul_(s["scales"].double()[:, None])
        return torch.mm(q, w.t().contiguous()).mul_(step)
    if op == "order":
        n = case["tokens"]
        key = torch.sort(s["ids"] * n + torch.arange(n, device="cuda")).values
        count = torch.zeros(case["experts"] + 1, dtype=torch.int64, device="cuda")
        return key % n, count.index_add_(0, s["ids"] + 1, torch.ones_like(s["ids"])).cumsum(0)
    outs, ends = case["outs"], s["offsets"].tolist()
    if op == "grouped":
        x = _nearest(s["x"], case["a"])
        parts = []
        for e in range(case["experts"]):
            w = _unpack(s["codes"][e * outs : (e + 1) * outs], s["scales"][e * outs : (e + 1) * outs], case["ins"], "e2m1", torch.float64)
            parts.append(torch.mm(x[ends[e] : ends[e + 1]], w.t().contiguous()))
        return torch.cat(parts)
    x = _unpack(s["codes"], s["scales"], case["ins"], "e4m3", torch.float64)
    return torch.stack([torch.mm(s["dy"][ends[e] : ends[e + 1]].double().t().contiguous(), x[ends[e] : ends[e + 1]])
                        for e in range(case["experts"])])
