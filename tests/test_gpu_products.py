"""GPU parity of the MXFP4 quantiser and its inverse, the MXFP4 product, the product grouped by
expert and the prefill layer on chosen activations, against plain 64-bit arithmetic."""
import numpy as np
import pytest
import torch

import expert_cache_offloaded_amd as mc
from oracle import bf16_to_f64, decode_mxfp4, prefill_per_token, route, sort_routes
from oracle.formats import encode_mxfp4

pytestmark = pytest.mark.gpu

U8, BF, F16, F32, I32 = torch.uint8, torch.bfloat16, torch.float16, torch.float32, torch.int32
TYPES = {"bf16": BF, "f16": F16, "f32": F32}
# a rounding is off by at most half a step: this much of the value
ROUND = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def wide(t, pad, fill):
    """The same values in rows that lie `pad` elements apart, the gaps filled."""
    b = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device=t.device)
    b[:, :t.shape[1]] = t
    return b, b[:, :t.shape[1]]


# ---------------------------------------------------------------- quantiser

def special_rows(rng, rows, cols, ty):
    """Rows with the values that decide something: ties, block maxima around powers of two, zeros,
    signed zeros, subnormals, the type's largest values, infinities and NaN."""
    v = rng.standard_normal((rows, cols)) * 2.0 ** rng.integers(-12, 12, size=(rows, 1))
    blocks = v.reshape(-1, 32)
    n = blocks.shape[0]
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.75])
    for i in range(n):
        kind = i % 12
        if kind == 1:                                   # every tie, under a maximum in [4, 8)
            s = 2.0 ** rng.integers(-8, 8)
            blocks[i] = rng.choice(ties, 32) * rng.choice([-1, 1], 32) * s
            blocks[i, 0] = 5.0 * s
        elif kind == 2:
            blocks[i] = 0.0
            blocks[i, 3] = -0.0
        elif kind == 3:                                 # a maximum just under and at a power of two
            blocks[i] *= 1e-3
            blocks[i, 5] = 2.0 * (1 - 2.0 ** -8) if i % 24 == 3 else -2.0
        elif kind == 4:
            tiny = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}[ty]
            blocks[i] = tiny * rng.integers(-9, 10, 32)
        elif kind == 5:
            blocks[i] *= {"f32": 2.0 ** -124, "bf16": 2.0 ** -124, "f16": 2.0 ** -12}[ty]
        elif kind == 6:
            big = {"f32": 3.4e38, "bf16": 3.3e38, "f16": 65504.0}[ty]
            blocks[i] = big * rng.uniform(-1, 1, 32)
            blocks[i, 7] = big
        elif kind == 7 and i % 36 == 7:
            blocks[i, rng.integers(32)] = rng.choice([np.inf, -np.inf])
        elif kind == 8 and i % 36 == 8:
            blocks[i, rng.integers(32)] = np.nan
    return v


@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols,pad", [(1, 32, 0), (3, 2048, 0), (37, 96, 8), (5, 4128, 64), (1, 1 << 16, 0),
                                           (300, 32, 40), (0, 64, 0), (1025, 544, 0)])
def test_quantise_bit_exact(ty, rows, cols, pad):
    """Codes and scales equal the definition's bit for bit (the rounding of exact quotients by a
    power of two has one right answer), read back as exactly the values they stand for."""
    rng = np.random.default_rng(rows * 7 + cols)
    v = torch.from_numpy(special_rows(rng, rows, cols, ty)).to(TYPES[ty])
    src = wide(v.cuda(), pad, float("nan"))[1]
    codes = torch.full((rows, cols // 2), 0xA5, dtype=U8, device="cuda")
    # scales at an odd address: any alignment will do
    room = torch.full((rows * (cols // 32) + 2,), 0x5A, dtype=U8, device="cuda")
    scales = room[1:1 + rows * (cols // 32)].view(rows, cols // 32)
    mc.mxfp4_quantize(src, codes, scales)
    rc, rs = encode_mxfp4(v.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), rs)
    assert np.array_equal(codes.cpu().numpy(), rc)
    assert room[0].item() == 0x5A and room[-1].item() == 0x5A


@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols,pad", [(1, 32, 0), (3, 2048, 8), (129, 96, 8), (7, 4128, 0), (0, 32, 0)])
def test_dequantise_every_code_and_scale(ty, rows, cols, pad):
    rng = np.random.default_rng(cols + rows)
    codes = rng.integers(0, 256, size=(rows, cols // 2)).astype(np.uint8)
    scales = rng.integers(0, 255, size=(rows, cols // 32)).astype(np.uint8)
    if ty == "f16":
        scales = rng.integers(100, 145, size=scales.shape).astype(np.uint8)
    ref = torch.from_numpy(decode_mxfp4(codes, scales)).to(TYPES[ty])     # one rounding from 64 bits
    nan = rng.random(scales.shape) < 0.05
    scales[nan] = 255
    ref[torch.from_numpy(np.repeat(nan, 32, axis=1))] = float("nan")
    buf, dst = wide(torch.zeros((rows, cols), dtype=TYPES[ty], device="cuda"), pad, 7.0)
    mc.mxfp4_dequantize(dev(codes), dev(scales), dst)
    got = dst.cpu()
    assert torch.equal(got.isnan(), ref.isnan())
    assert torch.equal(got.nan_to_num(0.0, 1e30, -1e30), ref.nan_to_num(0.0, 1e30, -1e30))
    if pad:
        assert (buf[:, cols:] == 7.0).all()


# ---------------------------------------------------------------- products

def operand(rng, fmt, *shape, size=1.0):
    """A random operand: (tensor, scales or None, its float64 values)."""
    if fmt == "bf16":
        t = torch.from_numpy(rng.standard_normal(shape) * size).to(BF)
        return t.cuda(), None, t.double().numpy()
    codes = rng.integers(0, 256, size=shape[:-1] + (shape[-1] // 2,)).astype(np.uint8)
    e = int(np.log2(size))
    scales = rng.integers(124 + e, 128 + e, size=shape[:-1] + (shape[-1] // 32,)).astype(np.uint8)
    return dev(codes), dev(scales), decode_mxfp4(codes, scales)


def product_bound(x, w):
    """How far an fp32 sum of the exact products may be from the true one: each of the K additions
    (and the instruction's own internal ones) is off by at most one unit, 2^-23, of a partial sum
    that stays below S = sum |x| |w|."""
    K = x.shape[-1]
    return (K + 8) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T) + 1e-37


def silu64(g):
    return g / (1.0 + np.exp(-g))


def swiglu_bound(v, dv, n):
    """Error of silu(g) u from errors dv of g and u: |silu'| <= 1.1; the fp32 evaluation adds the
    exponential's relative error (its argument g log2 e rounded to fp32: |g| 2^-23, and a few units)
    and a few units more."""
    g, u, dg, du = v[:, :n], v[:, n:], dv[:, :n], dv[:, n:]
    s = silu64(g)
    return 1.1 * dg * (np.abs(u) + du) + (np.abs(s) + 1.1 * dg) * du + np.abs(s * u) * (np.abs(g) + 8) * 2.0 ** -22


def check(got, ref, err, ty, what):
    got = got.double().cpu().numpy()
    tol = err + ROUND[ty] * (np.abs(ref) + err)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3g times the bound" % (
        what, bad.sum(), bad.size, np.max(np.abs(got - ref) / tol))


def check_quantised(codes, scales, ref, err, what):
    """Quantised results of values that are only known to within err: the block's exponent belongs to
    a maximum within err of the true one, and every value is within half a code step (and err)."""
    got = decode_mxfp4(codes, scales).reshape(-1, 32)
    r, e = ref.reshape(-1, 32), err.reshape(-1, 32)
    amax, da = np.abs(r).max(1), e.max(1)
    X = scales.reshape(-1).astype(int) - 127

    def exponent(a):
        return np.clip(np.where(a > 0, np.frexp(np.maximum(a, 1e-300))[1] - 3, -127), -127, 127)

    assert ((X >= exponent(np.maximum(amax - da, 0))) & (X <= exponent(amax + da))).all(), what
    s = np.ldexp(1.0, X)[:, None]
    u = np.minimum(np.abs(r) / s, 6.0)
    # a value's two neighbours are 0.5, 1 or 2 steps of its binade apart
    step = np.where(u + e / s < 2, 0.5, np.where(u + e / s < 4, 1.0, 2.0))
    over = np.maximum(np.abs(r) - 6.0 * s, 0.0)
    assert (np.abs(got - r) <= 0.5 * step * s + e + over).all(), what


@pytest.mark.parametrize("xf", ["bf16", "mxfp4"])
@pytest.mark.parametrize("yt", [BF, F32])
@pytest.mark.parametrize("M,N,K", [(1, 1, 32), (1, 4096, 2048), (2, 7, 96), (5, 33, 64), (16, 64, 128), (17, 65, 160),
                                   (63, 130, 544), (64, 256, 512), (100, 100, 1024), (129, 255, 288), (256, 256, 256),
                                   (257, 513, 2080), (300, 1000, 96), (1024, 512, 640)])
def test_matmul(xf, yt, M, N, K):
    rng = np.random.default_rng(M * 31 + N * 7 + K)
    x, xs, x64 = operand(rng, xf, M, K)
    w, ws, w64 = operand(rng, "mxfp4", N, K, size=2.0 ** -5)
    y = torch.full((M, N), float("nan"), dtype=yt, device="cuda")
    mc.mxfp4_matmul(x, w, ws, y, x_scale=xs)
    check(y, x64 @ w64.T, product_bound(x64, w64), yt, (xf, M, N, K))
    again = torch.empty_like(y)
    mc.mxfp4_matmul(x, w, ws, again, x_scale=xs)
    assert torch.equal(y, again)


@pytest.mark.parametrize("M,N,K,px,py", [(5, 36, 64, 8, 4), (70, 129, 96, 32, 3), (300, 260, 512, 64, 12),
                                         (1, 64, 2048, 8, 1)])
def test_matmul_strided(M, N, K, px, py):
    """Rows of x and y that lie apart; what lies between y's rows stays."""
    rng = np.random.default_rng(M + N)
    x, _, x64 = operand(rng, "bf16", M, K)
    w, ws, w64 = operand(rng, "mxfp4", N, K, size=2.0 ** -5)
    _, x = wide(x, px, float("nan"))
    buf, y = wide(torch.zeros((M, N), dtype=F32, device="cuda"), py, 7.0)
    mc.mxfp4_matmul(x, w, ws, y)
    check(y, x64 @ w64.T, product_bound(x64, w64), F32, (M, N, K))
    assert (buf[:, N:] == 7.0).all()


@pytest.mark.parametrize("xf", ["bf16", "mxfp4"])
@pytest.mark.parametrize("M", [3, 300])
def test_matmul_scale_range(xf, M):
    """Operand scales over the whole e8m0 range (results kept in fp32's normal range), and NaN scales:
    exactly the results that read a NaN block are NaN."""
    rng = np.random.default_rng(M)
    N, K = 70, 256
    for ew, ex in ((0, 252), (1, 240), (250, 4), (127, 127), (60, 180)):
        codes = rng.integers(0, 256, size=(N, K // 2)).astype(np.uint8)
        sw = np.full((N, K // 32), ew, dtype=np.uint8)
        w64 = decode_mxfp4(codes, sw)
        if xf == "mxfp4":
            xc = rng.integers(0, 256, size=(M, K // 2)).astype(np.uint8)
            xsc = np.full((M, K // 32), ex, dtype=np.uint8)
            x64, x, xs = decode_mxfp4(xc, xsc), dev(xc), dev(xsc)
        else:
            if ew == 0:
                # an MXFP4 value below bf16's smallest normal times a large bf16 one
                ex = 250
            x = torch.from_numpy(rng.choice([1.0, -1.5, 1.25, -1.0], size=(M, K)) * 2.0 ** (ex - 127)).to(BF).cuda()
            x64, xs = x.double().cpu().numpy(), None
        y = torch.empty((M, N), dtype=F32, device="cuda")
        mc.mxfp4_matmul(x, dev(codes), dev(sw), y, x_scale=xs)
        check(y, x64 @ w64.T, product_bound(x64, w64), F32, (xf, ew, ex))
    sw = np.full((N, K // 32), 120, dtype=np.uint8)
    sw[11, 3] = sw[69, 7] = 255
    x, xs, _ = operand(rng, xf, M, K)
    if xf == "mxfp4":
        xs[M - 1, 0] = 255
    y = torch.empty((M, N), dtype=F32, device="cuda")
    mc.mxfp4_matmul(x, dev(codes), dev(sw), y, x_scale=xs)
    nan = torch.zeros((M, N), dtype=torch.bool)
    nan[:, 11] = nan[:, 69] = True
    if xf == "mxfp4":
        nan[M - 1] = True
    assert torch.equal(y.isnan().cpu(), nan)


def grouped_case(rng, counts, N, K, xf, wf, x_div=1, lead=0, tail=0):
    """Offsets for the counts (lead rows before the first group, tail rows behind the last), operands,
    and every sorted row's group (-1: none)."""
    E = len(counts)
    off = lead + np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    M = int(off[-1]) + tail
    e_of = np.full(M, -1)
    for e in range(E):
        e_of[off[e]:off[e + 1]] = e
    w, ws, w64 = operand(rng, wf, E, N, K, size=2.0 ** -5)
    return off, M, e_of, w, ws, w64


COUNTS = [[1], [0, 0, 3, 0], [5, 1, 0, 17, 64, 2], [130, 0, 65, 255, 1, 300], [0] * 70 + [40] + [0] * 60 + [9, 1],
          [2] * 129, [700, 3], [16, 32, 48, 64, 80, 96, 112, 128, 144, 160, 176, 192]]
FORMATS = [("bf16", "bf16"), ("bf16", "mxfp4"), ("mxfp4", "mxfp4")]


@pytest.mark.parametrize("xf,wf", FORMATS)
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("ci", range(len(COUNTS)))
@pytest.mark.parametrize("N,K", [(34, 96), (256, 512), (640, 288)])
def test_grouped(xf, wf, swiglu, ci, N, K):
    """Ragged groups, rows of x gathered through perm and x_div, gates; rows of y outside the groups
    stay as they are."""
    counts = COUNTS[ci]
    rng = np.random.default_rng(ci * 100 + N + K)
    lead, tail = (2, 3) if ci % 2 else (0, 0)
    off, M, e_of, w, ws, w64 = grouped_case(rng, counts, N, K, xf, wf, lead=lead, tail=tail)
    x_div = 3
    T = (M + x_div - 1) // x_div
    x, xs, x64 = operand(rng, xf, T, K)
    perm = rng.permutation(T * x_div)[:M].astype(np.int32)
    gate = rng.uniform(0.1, 1.0, T * x_div).astype(np.float32)
    n_out = N // 2 if swiglu else N
    yt = BF if ci % 2 else F32
    for scatter in (False, True):
        y = torch.full((T * x_div if scatter else M, n_out), 7.0, dtype=yt, device="cuda")
        mc.grouped_matmul(x, w, dev(off), y, x_scale=xs, w_scale=ws, swiglu=swiglu, perm=dev(perm), x_div=x_div,
                          y_perm=scatter, gate=dev(gate))
        untouched = np.ones(y.shape[0], dtype=bool)
        for e in range(len(counts)):
            rows = np.nonzero(e_of == e)[0]
            if not len(rows):
                continue
            r = perm[rows]
            v, dv = x64[r // x_div] @ w64[e].T, product_bound(x64[r // x_div], w64[e])
            if swiglu:
                v, dv = silu64(v[:, :n_out]) * v[:, n_out:], swiglu_bound(v, dv, n_out)
            gt = gate[r].astype(np.float64)[:, None]
            at = r if scatter else rows
            check(y[torch.from_numpy(at).cuda()], gt * v, gt * dv + 2.0 ** -24 * np.abs(gt * v), yt, (counts[e], e, scatter))
            untouched[at] = False
        assert (y[torch.from_numpy(np.nonzero(untouched)[0]).cuda()] == 7.0).all()


@pytest.mark.parametrize("xf,wf", FORMATS)
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("counts,K", [([3, 0, 40], 96), ([300, 129, 5], 512), ([1], 2048)])
def test_grouped_quantised_results(xf, wf, swiglu, counts, K):
    rng = np.random.default_rng(sum(counts) + K)
    n_out = 160
    N = 2 * n_out if swiglu else n_out
    off, M, e_of, w, ws, w64 = grouped_case(rng, counts, N, K, xf, wf)
    x, xs, x64 = operand(rng, xf, M, K)
    y = torch.full((M + 1, n_out // 2), 0xA5, dtype=U8, device="cuda")
    sc = torch.full((M + 1, n_out // 32), 0xA5, dtype=U8, device="cuda")
    mc.grouped_matmul(x, w, dev(off), y, x_scale=xs, w_scale=ws, y_scale=sc, swiglu=swiglu)
    for e in range(len(counts)):
        r = np.nonzero(e_of == e)[0]
        if len(r):
            v, dv = x64[r] @ w64[e].T, product_bound(x64[r], w64[e])
            if swiglu:
                v, dv = silu64(v[:, :n_out]) * v[:, n_out:], swiglu_bound(v, dv, n_out)
            check_quantised(y.cpu().numpy()[r], sc.cpu().numpy()[r], v, dv, (e, counts[e]))
    assert (y[M] == 0xA5).all() and (sc[M] == 0xA5).all()


def gpu_operand(g, fmt, *shape, size=1.0):
    """A random operand made on the GPU, and its float64 values."""
    if fmt == "bf16":
        t = (torch.randn(shape, generator=g, device="cuda") * size).to(BF)
        return t, None, t.double()
    codes = torch.randint(0, 256, shape[:-1] + (shape[-1] // 2,), dtype=U8, device="cuda", generator=g)
    e = int(np.log2(size))
    scales = torch.randint(124 + e, 128 + e, shape[:-1] + (shape[-1] // 32,), dtype=U8, device="cuda", generator=g)
    nib = torch.stack([codes & 15, codes >> 4], -1).reshape(shape)
    mag = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")[(nib & 7).long()]
    v = torch.where(nib >= 8, -mag, mag) * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)
    return codes, scales, v


def gpu_check(got, x, w, swiglu, ty, what):
    """product_bound, swiglu_bound and check, on the GPU."""
    K = x.shape[1]
    v = x @ w.t()
    d = (K + 8) * 2.0 ** -23 * (x.abs() @ w.abs().t()) + 1e-37
    if swiglu:
        n = v.shape[1] // 2
        g, u, dg, du = v[:, :n], v[:, n:], d[:, :n], d[:, n:]
        s = g * torch.sigmoid(g)
        v = s * u
        d = 1.1 * dg * (u.abs() + du) + (s.abs() + 1.1 * dg) * du + v.abs() * (g.abs() + 8) * 2.0 ** -22
    tol = d + ROUND[ty] * (v.abs() + d)
    bad = ~((got.double() - v).abs() <= tol)
    assert not bad.any(), "%s: %d of %d off" % (what, int(bad.sum()), bad.numel())


@pytest.mark.parametrize("xf,wf", FORMATS)
@pytest.mark.parametrize("M,N,K", [(8200, 4096, 96), (8200, 4100, 512), (3000, 4096, 1088), (2100, 1000, 288),
                                   (700, 2048, 1024), (17, 8192, 4096), (250, 333, 8192)])
def test_large_products(xf, wf, M, N, K):
    """Sizes where a workgroup takes several tiles, of every tile shape, and where K is shared out among
    waves; one group, so that all three operand formats run."""
    g = torch.Generator(device="cuda")
    g.manual_seed(M + N + K)
    x, xs, x64 = gpu_operand(g, xf, M, K)
    w, ws, w64 = gpu_operand(g, wf, 1, N, K, size=2.0 ** -5)
    y = torch.full((M, N), float("nan"), dtype=F32, device="cuda")
    mc.grouped_matmul(x, w, torch.tensor([0, M], dtype=I32, device="cuda"), y, x_scale=xs, w_scale=ws)
    gpu_check(y, x64, w64[0], False, F32, (xf, wf, M, N, K))
    if wf == "mxfp4":
        y2 = torch.empty_like(y)
        mc.mxfp4_matmul(x, w[0], ws[0], y2, x_scale=xs)
        assert torch.equal(y, y2)


@pytest.mark.parametrize("xf,wf", FORMATS)
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("E,rows,N,K", [(16, 400, 8192, 96), (64, 24, 4096, 512), (1024, 3, 256, 160), (300, 1, 512, 544),
                                        (40, 1, 128, 64)])
def test_many_groups(xf, wf, swiglu, E, rows, N, K):
    """Many tiles per workgroup over ragged groups (empty ones among them), rows gathered, results
    scattered with gates."""
    g = torch.Generator(device="cuda")
    g.manual_seed(E + rows + N + K)
    r = np.random.default_rng(E + K)
    counts = r.integers(0, 2 * rows + 1, size=E)
    counts[r.integers(E)] = 0
    M = int(counts.sum())
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    x, xs, x64 = gpu_operand(g, xf, M, K)
    w, ws, w64 = gpu_operand(g, wf, E, N, K, size=2.0 ** -5)
    perm = r.permutation(M).astype(np.int32)
    gate = torch.rand(M, device="cuda", generator=g)
    n_out = N // 2 if swiglu else N
    y = torch.full((M, n_out), float("nan"), dtype=F32, device="cuda")
    mc.grouped_matmul(x, w, dev(off), y, x_scale=xs, w_scale=ws, swiglu=swiglu, perm=dev(perm), y_perm=True, gate=gate)
    p = dev(perm).long()
    # the gate's product is one more rounding: divide it out in 64 bits and allow for it
    z = y.double() / gate.double()[:, None]
    for e in range(E):
        at = p[off[e]:off[e + 1]]
        if len(at):
            gpu_check(z[at], x64[at], w64[e], swiglu, F32, (e, int(counts[e])))


@pytest.mark.parametrize("xf,wf", FORMATS)
def test_rows_beyond_32_bit_offsets(xf, wf):
    """Rows of x more than 4 GiB behind its start."""
    K = 2048
    n = (1 << 32) // (2 * K if xf == "bf16" else K // 2) + 100
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    at = torch.tensor([0, 5, n - 1, n - 2, n - 50] + list(range(n - 40, n - 5)), device="cuda")
    part, ps, x64 = gpu_operand(g, xf, len(at), K)
    x = torch.zeros((n, part.shape[1]), dtype=part.dtype, device="cuda")
    x[at] = part
    xs = None
    if ps is not None:
        xs = torch.zeros((n, K // 32), dtype=U8, device="cuda")
        xs[at] = ps
    w, ws, w64 = gpu_operand(g, wf, 2, 160, K, size=2.0 ** -5)
    M = len(at)
    y = torch.empty((M, 160), dtype=F32, device="cuda")
    mc.grouped_matmul(x, w, torch.tensor([0, 7, M], dtype=I32, device="cuda"), y, x_scale=xs, w_scale=ws,
                      perm=at.to(I32))
    gpu_check(y[:7], x64[:7], w64[0], False, F32, xf)
    gpu_check(y[7:], x64[7:], w64[1], False, F32, xf)


@pytest.mark.parametrize("xf,wf", FORMATS)
def test_consecutive_rows_beyond_32_bit_offsets(xf, wf):
    """All rows of an x of more than 4 GiB, one behind the other."""
    K, N = 8192, 32
    M = (1 << 32) // (2 * K if xf == "bf16" else K // 2) + 300
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    at = torch.tensor([0, 5, 4000, M // 2] + list(range(M - 290, M - 10)) + [M - 1], device="cuda")
    part, ps, x64 = gpu_operand(g, xf, len(at), K)
    x = torch.zeros((M, part.shape[1]), dtype=part.dtype, device="cuda")
    x[at] = part
    xs = None
    if ps is not None:
        xs = torch.zeros((M, K // 32), dtype=U8, device="cuda")
        xs[at] = ps
    w, ws, w64 = gpu_operand(g, wf, 2, N, K, size=2.0 ** -5)
    y = torch.empty((M, N), dtype=F32, device="cuda")
    cut = M - 150
    mc.grouped_matmul(x, w, torch.tensor([0, cut, M], dtype=I32, device="cuda"), y, x_scale=xs, w_scale=ws)
    lo = at < cut
    gpu_check(y[at[lo]], x64[lo], w64[0], False, F32, xf)
    gpu_check(y[at[~lo]], x64[~lo], w64[1], False, F32, xf)
    if wf == "mxfp4":
        mc.mxfp4_matmul(x, w[0], ws[0], y, x_scale=xs)
        gpu_check(y[at], x64, w64[0], False, F32, xf)


def test_more_columns_than_a_launch_holds():
    """One token and so many columns that workgroups take several tiles."""
    N, K = (1 << 28) + 1100, 32
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x, _, x64 = gpu_operand(g, "bf16", 1, K)
    at = torch.tensor([0, 1, N // 2] + list(range((1 << 28) - 100, N)), device="cuda")
    part, ps, w64 = gpu_operand(g, "mxfp4", len(at), K)
    w = torch.zeros((N, K // 2), dtype=U8, device="cuda")
    ws = torch.full((N, 1), 127, dtype=U8, device="cuda")
    w[at], ws[at] = part, ps
    y = torch.full((1, N), float("nan"), dtype=F32, device="cuda")
    mc.mxfp4_matmul(x, w, ws, y)
    gpu_check(y[:, at], x64, w64, False, F32, "")
    assert int((y != 0).sum()) <= len(at)          # every other column was written with its 0


def test_grouped_entries_and_bad_rows():
    """entry_of leaves groups out or maps them to other matrices; entries, routes and offsets outside
    their ranges skip rows and touch nothing."""
    rng = np.random.default_rng(5)
    counts, N, K = [9, 70, 4, 33, 300], 64, 128
    off, M, e_of, w, ws, w64 = grouped_case(rng, counts, N, K, "bf16", "mxfp4")
    entry = np.array([2, -1, 5, 0, 4], dtype=np.int32)             # 5 is past the last matrix
    x, _, x64 = operand(rng, "bf16", M, K)
    perm = np.arange(M, dtype=np.int32)
    perm[[1, 80, 100, 200, 411]] = [-5, M, 2 ** 31 - 1, -2 ** 31, M + 1]
    gate = rng.uniform(0.5, 1.0, M).astype(np.float32)
    y = torch.full((M, N), 7.0, dtype=F32, device="cuda")
    mc.grouped_matmul(x, w, dev(off), y, w_scale=ws, perm=dev(perm), y_perm=True, gate=dev(gate), entry_of=dev(entry))
    got = y.cpu().numpy()
    for i in range(M):
        en = entry[e_of[i]]
        if perm[i] != i or not 0 <= en < 5:
            assert (got[i] == 7.0).all(), i
        else:
            ref, err = x64[i] @ w64[en].T, product_bound(x64[i:i + 1], w64[en])[0]
            tol = gate[i] * (err + 2.0 ** -22 * np.abs(ref))
            assert (np.abs(got[i] - gate[i] * ref) <= tol).all(), i
    # offsets beyond the rows are clamped
    y2 = torch.full((M, N), 7.0, dtype=F32, device="cuda")
    wild = off.copy()
    wild[0], wild[-1] = -4, 2 ** 31 - 1
    mc.grouped_matmul(x, w, dev(wild), y2, w_scale=ws)
    y3 = torch.full((M, N), 7.0, dtype=F32, device="cuda")
    mc.grouped_matmul(x, w, dev(off), y3, w_scale=ws)
    assert torch.equal(y2, y3)


def test_grouped_with_router_sort():
    """The token sort's own offsets and perm, a masked and partly filled batch among them."""
    rng = np.random.default_rng(8)
    T, k, E, N, K = 75, 3, 20, 96, 160
    ids = rng.integers(0, E, size=(T, k)).astype(np.int32)
    ids[rng.random(ids.shape) < 0.1] = -1
    n_tok = 61
    counts, perm = (torch.empty(n, dtype=I32, device="cuda") for n in (E, T * k))
    offsets = torch.empty(E + 1, dtype=I32, device="cuda")
    perm.fill_(-1)
    ws_ = torch.empty(E * 16 + (E + 1) * 4 + 64, dtype=U8, device="cuda")
    mc._lib.prefill_sort_routes(dev(ids), dev(np.array([n_tok], dtype=np.int32)), E, ws_, counts, offsets, perm)
    x, xs, x64 = operand(rng, "mxfp4", T, K)
    w, ws, w64 = operand(rng, "mxfp4", E, N, K, size=2.0 ** -5)
    y = torch.full((T * k, N), 7.0, dtype=F32, device="cuda")
    mc.grouped_matmul(x, w, offsets, y, x_scale=xs, w_scale=ws, perm=perm, x_div=k, y_perm=True)
    flat = ids.reshape(-1)
    for r in range(T * k):
        t = r // k
        if t >= n_tok or flat[r] < 0:
            assert (y[r] == 7.0).all()
        else:
            check(y[r:r + 1], x64[t:t + 1] @ w64[flat[r]].T, product_bound(x64[t:t + 1], w64[flat[r]]), F32, r)


def test_products_on_a_side_stream_and_in_a_graph():
    """A call on another stream, and a captured run of quantise -> grouped gate_up -> grouped down whose
    tokens and group sizes change between replays, eager work in between: each replay equals the eager
    calls bit for bit."""
    rng = np.random.default_rng(11)
    T, k, E, H, I = 24, 2, 8, 128, 64
    gu, gus, _ = operand(rng, "mxfp4", E, 2 * I, H, size=2.0 ** -4)
    dn, dns, _ = operand(rng, "mxfp4", E, H, I, size=2.0 ** -4)
    x = torch.zeros((T, H), dtype=BF, device="cuda")
    off, perm = torch.zeros(E + 1, dtype=I32, device="cuda"), torch.zeros(T * k, dtype=I32, device="cuda")
    gate = torch.rand(T * k, device="cuda")
    xq, xqs = torch.empty((T, H // 2), dtype=U8, device="cuda"), torch.empty((T, H // 32), dtype=U8, device="cuda")
    hq = torch.empty((T * k, I // 2), dtype=U8, device="cuda")
    hqs = torch.empty((T * k, I // 32), dtype=U8, device="cuda")

    def steps(y, stream=None):
        mc.mxfp4_quantize(x, xq, xqs, stream=stream)
        mc.grouped_matmul(xq, gu, off, hq, x_scale=xqs, w_scale=gus, y_scale=hqs, swiglu=True, perm=perm, x_div=k,
                          stream=stream)
        mc.grouped_matmul(hq, dn, off, y, x_scale=hqs, w_scale=dns, perm=perm, x_perm=False, y_perm=True, gate=gate,
                          stream=stream)

    def fill(seed):
        r = np.random.default_rng(seed)
        ids = r.integers(0, E, size=(T, k)).astype(np.int32)
        c, o, p = sort_routes(ids, E, None)
        x.copy_(torch.from_numpy(r.standard_normal((T, H))).to(BF))
        off.copy_(torch.from_numpy(np.asarray(o, dtype=np.int32)))
        perm.copy_(torch.from_numpy(np.asarray(p, dtype=np.int32)))

    y_graph = torch.empty((T * k, H), dtype=F32, device="cuda")
    y_eager = torch.empty_like(y_graph)
    fill(0)
    steps(y_eager)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        steps(y_graph)
    side = torch.cuda.Stream()
    y_side = torch.empty_like(y_graph)
    for seed in (0, 1, 2, 3):
        fill(seed)
        y_graph.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        steps(y_eager)
        assert torch.equal(y_graph, y_eager)
        side.wait_stream(torch.cuda.current_stream())
        steps(y_side, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(y_side, y_eager)
        assert not torch.isnan(y_eager).any()


# ---------------------------------------------------------------- the layer

def layer_inputs(rng, T, k, E, H, I, fmt):
    logits = rng.standard_normal((T, E)).astype(np.float32)
    ids, w = route(logits, k)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(BF)
    gu, gus, gu64 = operand(rng, fmt, E, 2 * I, H, size=2.0 ** -4)
    dn, dns, dn64 = operand(rng, fmt, E, H, I, size=2.0 ** -4)
    banks = {"gate_up": gu, "down": dn}
    if fmt == "mxfp4":
        banks.update(gate_up_scale=gus, down_scale=dns)
    return np.asarray(ids, dtype=np.int32), np.asarray(w, dtype=np.float32), x, banks, gu64, dn64


def run_layer(x, ids, w, n_tok, E, H, I, fmt, act, banks):
    T, k = ids.shape
    y = torch.full((T, H), 7.0, dtype=BF, device="cuda")
    ws = torch.full((mc.prefill_act_ws_bytes(T, k, E, H, I, act),), 0xFF, dtype=U8, device="cuda")
    nt = None if n_tok is None else dev(np.array([n_tok], dtype=np.int32))
    mc.moe_experts_prefill_act(x.cuda(), dev(ids), dev(w), nt, E, mc.make_banks(fmt, H, I, banks), act, ws, y)
    torch.cuda.synchronize()
    return y


@pytest.mark.parametrize("act,fmt", [("bf16", "bf16"), ("bf16", "mxfp4"), ("mxfp4", "mxfp4")])
@pytest.mark.parametrize("T,k,E,H,I,n_tok", [(1, 2, 8, 64, 128, None), (5, 3, 16, 320, 64, 3), (130, 2, 4, 128, 192, None),
                                             (64, 4, 32, 256, 128, 0), (700, 3, 8, 192, 320, 611), (2, 8, 256, 2048, 512, None)])
def test_layer(act, fmt, T, k, E, H, I, n_tok):
    """Against the layer's formula in 64 bits.  bf16: h is rounded to bf16, 2^-8 of itself at most, so
    with A_d = sum_n |W_down[d][n] h[n]| the outputs are off by 2^-8 A_d and their own rounding, and by
    the fp32 sums, which are far smaller.  MXFP4: the same inputs are quantised on both sides, and the
    routes' outputs rounded to bf16; a value of h that lies within the fp32 sums' error of a rounding
    border may take the neighbouring code, which moves an output by one code's share; such values are
    rare, so the outputs are held to the rms bound the bf16 rounding of y sets (2^-8 / sqrt 3, a
    uniform rounding error, plus a tenth)."""
    rng = np.random.default_rng(T + H + I)
    ids, w, x, banks, gu, dn = layer_inputs(rng, T, k, E, H, I, fmt)
    ids[rng.random(ids.shape) < 0.03] = -1
    y = run_layer(x, ids, w, n_tok, E, H, I, fmt, act, banks).double().cpu().numpy()
    nt = T if n_tok is None else n_tok
    assert (y[nt:] == 0).all()
    x64 = x.double().numpy()
    if act == "mxfp4":
        x64 = decode_mxfp4(*encode_mxfp4(x64))
    ref, mag = np.zeros((T, H)), np.zeros((T, H))
    for t in range(nt):
        for j in range(k):
            e = ids[t, j]
            if e < 0:
                continue
            v = gu[e] @ x64[t]
            h = silu64(v[:I]) * v[I:]
            if act == "mxfp4":
                h = decode_mxfp4(*encode_mxfp4(h[None]))[0]
            else:
                mag[t] += w[t, j] * (np.abs(dn[e]) @ np.abs(h))
            r = w[t, j] * (dn[e] @ h)
            ref[t] += torch.from_numpy(r).to(BF).double().numpy() if act == "mxfp4" else r
    if act == "bf16":
        tol = (2.0 ** -8 + (H + I) * 2.0 ** -22) * mag + 2.0 ** -8 * np.abs(ref) * 1.01
        assert (np.abs(y - ref) <= tol).all()
    elif nt:
        rms = np.sqrt(np.mean((y - ref) ** 2)) / np.sqrt(np.mean(ref ** 2))
        assert rms <= 1.1 * 2.0 ** -8 / np.sqrt(3.0), rms


def test_layer_is_its_parts():
    """The layer equals its parts called one by one: sort, quantise, grouped gate_up with SwiGLU,
    grouped down scattered to the routes with the gates, and the sum over each token's routes."""
    rng = np.random.default_rng(3)
    T, k, E, H, I = 190, 4, 16, 256, 192
    ids, w, x, banks, _, _ = layer_inputs(rng, T, k, E, H, I, "mxfp4")
    y = run_layer(x, ids, w, None, E, H, I, "mxfp4", "mxfp4", banks)
    x = x.cuda()
    c, o, p = sort_routes(ids, E, None)
    off, perm = dev(np.asarray(o, dtype=np.int32)), dev(np.asarray(p, dtype=np.int32))
    xq, xqs = torch.empty((T, H // 2), dtype=U8, device="cuda"), torch.empty((T, H // 32), dtype=U8, device="cuda")
    hq = torch.empty((T * k, I // 2), dtype=U8, device="cuda")
    hqs = torch.empty((T * k, I // 32), dtype=U8, device="cuda")
    yr = torch.empty((T * k, H), dtype=BF, device="cuda")
    mc.mxfp4_quantize(x, xq, xqs)
    mc.grouped_matmul(xq, banks["gate_up"], off, hq, x_scale=xqs, w_scale=banks["gate_up_scale"], y_scale=hqs,
                      swiglu=True, perm=perm, x_div=k)
    mc.grouped_matmul(hq, banks["down"], off, yr, x_scale=hqs, w_scale=banks["down_scale"], perm=perm, x_perm=False,
                      y_perm=True, gate=dev(w).reshape(-1))
    s = torch.zeros((T, H), device="cuda")
    for j in range(k):
        s += yr.view(T, k, H)[:, j]
    assert torch.equal(y, s.to(BF))


def test_layer_near_the_bf16_activation_layer():
    """bf16 activations on MXFP4 experts: the same experts through moe_experts_prefill (h in fp16), both
    within the rounding of h and y of each other."""
    rng = np.random.default_rng(4)
    T, k, E, H, I = 200, 3, 8, 512, 256
    ids, w, x, banks, _, _ = layer_inputs(rng, T, k, E, H, I, "mxfp4")
    y = run_layer(x, ids, w, None, E, H, I, "mxfp4", "bf16", banks).double()
    ws = torch.empty(mc._lib.prefill_ws_bytes(T, k, E, H, I), dtype=U8, device="cuda")
    y0 = torch.empty((T, H), dtype=BF, device="cuda")
    mc._lib.moe_experts_prefill(x.cuda(), dev(ids), dev(w), None, E, mc.make_banks("mxfp4", H, I, banks), ws, y0)
    # three independent roundings to bf16 (h, y, y0), each at most 2^-8 / sqrt 3 rms
    assert float((y - y0.double()).norm() / y0.double().norm()) <= 3 ** 0.5 * 2.0 ** -8 / 3 ** 0.5


# ---------------------------------------------------------------- in the framework's own paths

@pytest.mark.parametrize("where", ["cpu", "cuda"])
def test_quantize_banks(where):
    """bf16 experts to MXFP4 experts, from and to host or device memory: the oracle's codes and
    scales, and a layer that runs on them."""
    from expert_cache_offloaded_amd.runtime import BankSet, alloc_banks, quantize_banks
    n, H, I = 3, 128, 64
    src, dst = (alloc_banks(n, H, I, f, device=where, pin=where == "cpu") for f in ("bf16", "mxfp4"))
    r = np.random.default_rng(2)
    for v in src.values():
        v.copy_(torch.from_numpy(r.standard_normal(tuple(v.shape)) * 0.02).to(BF).view(torch.int16))
    a, b = BankSet(src, H, I, "bf16"), BankSet(dst, H, I, "mxfp4")
    quantize_banks(a, b)
    for name in ("gate_up", "down"):
        c, s = encode_mxfp4(bf16_to_f64(src[name].cpu().numpy().view(np.uint16)))
        assert np.array_equal(dst[name].cpu().numpy(), c)
        assert np.array_equal(dst[name + "_scale"].cpu().numpy(), s)
    with pytest.raises(ValueError):
        quantize_banks(b, a)
    with pytest.raises(ValueError):
        quantize_banks(a, BankSet(alloc_banks(n + 1, H, I, "mxfp4", device=where), H, I, "mxfp4"))


@pytest.mark.parametrize("fmt,act", [("bf16", None), ("bf16", "bf16"), ("mxfp4", "mxfp4"), ("mxfp4", "bf16")])
@pytest.mark.parametrize("S", [32, 9, 1])
def test_prefill_runner_on_chosen_activations(fmt, act, S):
    """PrefillRunner with bf16 experts and with quantised activations: two whole layers in the pool,
    a pool that loads the routed experts in groups, and a single slot all give moe_experts_prefill_act's
    outputs bit for bit, and leave the last layer's experts in the cache."""
    from expert_cache_offloaded_amd.runtime import BankSet, CacheState, PrefillRunner, alloc_banks
    Lc, E, T, k, H, I = 2, 12, 70, 3, 128, 192
    r = np.random.default_rng(S)
    host = alloc_banks(Lc * E, H, I, fmt, pin=True)
    for name, v in host.items():
        if name.endswith("scale"):
            v.copy_(torch.from_numpy(r.integers(118, 122, tuple(v.shape)).astype(np.uint8)))
        elif fmt == "mxfp4":
            v.copy_(torch.from_numpy(r.integers(0, 256, tuple(v.shape)).astype(np.uint8)))
        else:
            v.copy_(torch.from_numpy(r.standard_normal(tuple(v.shape)) * 0.02).to(BF).view(torch.int16))
    pool = BankSet(alloc_banks(S, H, I, fmt, device="cuda"), H, I, fmt)
    cache = CacheState(Lc, E, S)
    logits = [dev(r.standard_normal((T, E)).astype(np.float32)) for _ in range(Lc)]
    x = dev(r.standard_normal((T, H)).astype(np.float32)).to(BF).view(torch.int16)
    ys = [torch.empty((T, H), dtype=torch.int16, device="cuda") for _ in range(Lc)]
    run = PrefillRunner(cache, BankSet(host, H, I, fmt), pool, T, k, act=act)
    held = run.run(logits, x, ys)
    torch.cuda.synchronize()
    assert cache.t["id_of"].cpu().tolist()[:len(held)] == held
    a = act or "bf16"
    for layer in range(Lc):
        ids, w = torch.empty((T, k), dtype=I32, device="cuda"), torch.empty((T, k), device="cuda")
        mc.moe_route(logits[layer], k, 1, ids, w)
        banks = {n: v[layer * E:(layer + 1) * E].cuda() for n, v in host.items()}
        ws = torch.empty(mc.prefill_act_ws_bytes(T, k, E, H, I, a), dtype=U8, device="cuda")
        y = torch.empty_like(ys[layer])
        mc.moe_experts_prefill_act(x, ids, w, None, E, mc.make_banks(fmt, H, I, banks), a, ws, y)
        assert torch.equal(ys[layer], y), layer
    if fmt == "bf16":
        with pytest.raises(ValueError):
            PrefillRunner(cache, BankSet(host, H, I, fmt), pool, T, k, act="mxfp4")


def test_layer_graph_replay_with_changing_batches():
    """A captured quantised layer replayed with other tokens, routes and valid counts, eager layers and
    synchronisations in between: each replay equals the eager call."""
    T, k, E, H, I = 96, 2, 16, 128, 128
    rng = np.random.default_rng(12)
    gu, gus, _ = operand(rng, "mxfp4", E, 2 * I, H, size=2.0 ** -4)
    dn, dns, _ = operand(rng, "mxfp4", E, H, I, size=2.0 ** -4)
    banks = {"gate_up": gu, "gate_up_scale": gus, "down": dn, "down_scale": dns}
    desc = mc.make_banks("mxfp4", H, I, banks)
    x, y = (torch.zeros((T, H), dtype=BF, device="cuda") for _ in range(2))
    y2 = torch.empty_like(y)
    ids, w = torch.zeros((T, k), dtype=I32, device="cuda"), torch.zeros((T, k), device="cuda")
    nt = torch.tensor([T], dtype=I32, device="cuda")
    ws, ws2 = (torch.empty(mc.prefill_act_ws_bytes(T, k, E, H, I, "mxfp4"), dtype=U8, device="cuda") for _ in range(2))
    mc.moe_experts_prefill_act(x, ids, w, nt, E, desc, "mxfp4", ws, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mc.moe_experts_prefill_act(x, ids, w, nt, E, desc, "mxfp4", ws, y)
    for seed, n in enumerate((T, 17, 0, 50)):
        r = np.random.default_rng(seed)
        x.copy_(torch.from_numpy(r.standard_normal((T, H))).to(BF))
        ids.copy_(torch.from_numpy(np.stack([r.permutation(E)[:k] for _ in range(T)]).astype(np.int32)))
        w.copy_(torch.from_numpy(r.random((T, k)).astype(np.float32)))
        nt.fill_(n)
        y.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        mc.moe_experts_prefill_act(x, ids, w, nt, E, desc, "mxfp4", ws2, y2)
        assert torch.equal(y, y2)
        assert (y[n:] == 0).all() and (n == 0 or bool((y[:n] != 0).any()))
