"""The products on the tiles of 256 x 256, of 128 x 128 and of 128 x 128 with K in two parts, in every form
of operands and results, and prefill layers whose products run on the first.  Each case says which tile it
is meant for, and the library which one its sizes choose."""
import ctypes as C

import numpy as np
import pytest
import torch

import expert_cache_offloaded_amd as mc
from expert_cache_offloaded_amd import _lib as L
from test_gpu_products import BF, F32, FORMATS, I32, ROUND, U8, dev, gpu_operand, run_layer

pytestmark = pytest.mark.gpu

BIG, MEDIUM, MEDIUM2 = (256, 256, 1), (128, 128, 1), (128, 128, 2)


def tile_of(xf, wf, y, E, M, N, K, swiglu, x_rows=None, grouped=True):
    """The tile for a product of these sizes, from the library's own rule."""
    keep = (C.c_uint8 * 32)()
    p = (C.addressof(keep) + 15) & ~15
    n_out = N // 2 if swiglu else N
    g = L.Grouped(L.FMT[xf], L.FMT[wf], {F32: L.MC_F32, BF: L.MC_BF16, U8: L.MC_MXFP4}[y], int(swiglu), E, M, N, K,
                  x_rows or M, 1, M, int(x_rows is not None), 0, 0, K, n_out, E, p, p, p, p, p, p, p if grouped else None,
                  p, None, None)
    tile = (C.c_int32 * 3)()
    L._check("mc_grouped_tile", L.lib().mc_grouped_tile(C.byref(g), tile))
    return tuple(tile)


def product(x, w, swiglu):
    """x w^T (through SwiGLU) in 64 bits and how far an fp32 evaluation may be from it: (K + 8) units of
    2^-23 of the sum of magnitudes; for SwiGLU see swiglu_bound."""
    K = x.shape[1]
    wt = w.t().contiguous()
    v = x @ wt
    d = (K + 8) * 2.0 ** -23 * (x.abs() @ wt.abs()) + 1e-37
    if swiglu:
        n = v.shape[1] // 2
        g, u, dg, du = v[:, :n], v[:, n:], d[:, :n], d[:, n:]
        s = g * torch.sigmoid(g)
        v = s * u
        d = 1.1 * dg * (u.abs() + du) + (s.abs() + 1.1 * dg) * du + v.abs() * (g.abs() + 8) * 2.0 ** -22
    return v, d


def values(codes, scales):
    """MXFP4 rows in 64 bits."""
    nib = torch.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)
    mag = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")[(nib & 7).long()]
    return torch.where(nib >= 8, -mag, mag) * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def check(y, ys, v, d, ty, what):
    """Results of type ty that are known to within d."""
    if ty is not U8:
        off = (y.double() - v).abs() / (d + ROUND[ty] * (v.abs() + d))
        assert bool((off <= 1).all()), "%s: %d of %d off" % (what, int((~(off <= 1)).sum()), off.numel())
        return
    # quantised: the exponent belongs to a maximum within d of the true one, every value lies within half
    # a code step (and d) of the true one
    r, e = v.reshape(-1, 32), d.reshape(-1, 32)
    amax, da = r.abs().amax(1), e.amax(1)

    def exponent(a):
        return torch.where(a > 0, torch.frexp(a)[1] - 3, torch.full_like(a, -127, dtype=torch.int32)).clamp(-127, 127)

    X = ys.reshape(-1).int() - 127
    assert bool(((X >= exponent((amax - da).clamp_min(0))) & (X <= exponent(amax + da))).all()), what
    s = torch.exp2(X.double())[:, None]
    u = (r.abs() / s).clamp(max=6.0) + e / s
    step = torch.where(u < 2, 0.5, torch.where(u < 4, 1.0, 2.0)).double()
    over = (r.abs() - 6 * s).clamp_min(0)
    assert bool(((values(y, ys).reshape(-1, 32) - r).abs() <= 0.5 * step * s + e + over).all()), what


def run_case(tile, E, M, N, K, xf, wf, ty, swiglu, scatter, seed=0):
    """M routes in E uneven groups, two routes per row of x, gathered, gated, scattered if asked."""
    T = (M + 1) // 2
    assert tile_of(xf, wf, ty, E, M, N, K, swiglu, x_rows=T) == tile
    g = torch.Generator(device="cuda")
    g.manual_seed(M + N + K + seed)
    r = np.random.default_rng(M + K + seed)
    share = r.random(E) + 0.05
    if E > 2:
        share[r.integers(E)] = 0.0
    counts = r.multinomial(M, share / share.sum())
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    x, xs, x64 = gpu_operand(g, xf, T, K)
    w, ws, w64 = gpu_operand(g, wf, E, N, K, size=2.0 ** -5)
    perm = torch.randperm(2 * T, device="cuda", generator=g)[:M]
    gate = torch.rand(2 * T, device="cuda", generator=g) + 0.25
    n_out, rows = N // 2 if swiglu else N, 2 * T if scatter else M
    ys = None
    if ty is U8:
        y = torch.full((rows, n_out // 2), 0xA5, dtype=U8, device="cuda")
        ys = torch.full((rows, n_out // 32), 0xA5, dtype=U8, device="cuda")
    else:
        y = torch.full((rows, n_out), 7.0, dtype=ty, device="cuda")
    mc.grouped_matmul(x, w, dev(off), y, x_scale=xs, w_scale=ws, y_scale=ys, swiglu=swiglu, perm=perm.to(I32), x_div=2,
                      y_perm=scatter, gate=gate)
    left = torch.ones(rows, dtype=torch.bool, device="cuda")
    for e in range(E):
        p = perm[off[e]:off[e + 1]]
        if not len(p):
            continue
        v, d = product(x64[p // 2], w64[e], swiglu)
        gt = gate[p].double()[:, None]
        at = p if scatter else torch.arange(off[e], off[e + 1], device="cuda")
        check(y[at], ys[at] if ty is U8 else None, gt * v, gt * d + 2.0 ** -24 * (gt * v).abs(), ty, (e, int(counts[e])))
        left[at] = False
    assert bool((y[left] == (0xA5 if ty is U8 else 7.0)).all())
    if ty is U8:
        assert bool((ys[left] == 0xA5).all())


@pytest.mark.parametrize("xf,wf", FORMATS)
@pytest.mark.parametrize("ty", [BF, F32, U8])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("K", [1024, 1056, 2048])
def test_grouped_on_256_rows(xf, wf, ty, swiglu, K):
    """Tiles of 256 x 256, several per workgroup, with several chunks of scales per tile (K of 1056: scales
    that are not loaded straight into LDS)."""
    run_case(BIG, 16, 8192, 8192, K, xf, wf, ty, swiglu, scatter=ty is not BF)


@pytest.mark.parametrize("xf,wf", FORMATS)
@pytest.mark.parametrize("ty", [BF, F32, U8])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("K", [96, 1024, 1120, 2048])
def test_grouped_on_128_rows(xf, wf, ty, swiglu, K):
    run_case(MEDIUM, 40, 2400, 2048, K, xf, wf, ty, swiglu, scatter=ty is not F32)


@pytest.mark.parametrize("xf,wf", FORMATS)
@pytest.mark.parametrize("ty", [BF, F32, U8])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("K", [32, 96, 512, 1024, 2080])
def test_grouped_on_128_rows_with_k_in_two_parts(xf, wf, ty, swiglu, K):
    """K down to lengths of which the second part gets nothing."""
    run_case(MEDIUM2, 3, 700, 4096, K, xf, wf, ty, swiglu, scatter=ty is not U8)


@pytest.mark.parametrize("xf", ["bf16", "mxfp4"])
@pytest.mark.parametrize("ty", [BF, F32])
@pytest.mark.parametrize("tile,M,N,K", [(MEDIUM2, 1000, 4096, 32), (MEDIUM2, 1000, 4096, 96), (MEDIUM2, 1000, 4096, 2080),
                                        (MEDIUM2, 512, 8192, 4096), (BIG, 8200, 4096, 1024), (BIG, 8192, 4096, 4096)])
def test_matmul_on_large_tiles(xf, ty, tile, M, N, K):
    assert tile_of(xf, "mxfp4", ty, 1, M, N, K, False, grouped=False) == tile
    g = torch.Generator(device="cuda")
    g.manual_seed(M + K)
    x, xs, x64 = gpu_operand(g, xf, M, K)
    w, ws, w64 = gpu_operand(g, "mxfp4", N, K, size=2.0 ** -5)
    y = torch.full((M, N), float("nan"), dtype=ty, device="cuda")
    mc.mxfp4_matmul(x, w, ws, y, x_scale=xs)
    v, d = product(x64, w64, False)
    check(y, None, v, d, ty, (xf, M, N, K))
    again = torch.empty_like(y)
    mc.mxfp4_matmul(x, w, ws, again, x_scale=xs)
    assert torch.equal(y, again)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp4"])
def test_bf16_layer_on_256_rows(fmt):
    """A layer on bf16 activations whose two products run on tiles of 256 x 256, partly filled.  h is
    rounded to bf16, 2^-8 of itself at most, so with A = sum |W_down h| the outputs are off by 2^-8 A,
    by their own rounding and by the fp32 sums.  (On MXFP4 activations: test_gpu_layer_act.py, whose
    largest batch has these sizes.)"""
    T, k, E, H, I, n_tok = 8200, 4, 8, 2048, 1024, 8111
    for xf in {"bf16", fmt}:
        assert tile_of(xf, fmt, BF, E, T * k, 2 * I, H, True, x_rows=T) == BIG
        assert tile_of(xf, fmt, F32, E, T * k, H, I, False) == BIG
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    gu, gus, gu64 = gpu_operand(g, fmt, E, 2 * I, H, size=2.0 ** -4)
    dn, dns, dn64 = gpu_operand(g, fmt, E, H, I, size=2.0 ** -4)
    banks = {"gate_up": gu, "down": dn}
    if fmt == "mxfp4":
        banks.update(gate_up_scale=gus, down_scale=dns)
    x = torch.randn((T, H), generator=g, device="cuda").to(BF)
    w, ids = torch.topk(torch.softmax(torch.randn((T, E), generator=g, device="cuda"), 1), k, dim=1)
    w, ids = w.contiguous(), ids.to(I32)
    ids[torch.rand(ids.shape, generator=g, device="cuda") < 0.03] = -1
    y = run_layer(x, ids.cpu().numpy(), w.cpu().numpy(), n_tok, E, H, I, fmt, "bf16", banks).double()
    assert bool((y[n_tok:] == 0).all())
    ref, mag = (torch.zeros((T, H), dtype=torch.float64, device="cuda") for _ in range(2))
    for e in range(E):
        t, j = torch.nonzero(ids[:n_tok] == e, as_tuple=True)
        v = x[t].double() @ gu64[e].t().contiguous()
        h = v[:, :I] * torch.sigmoid(v[:, :I]) * v[:, I:]
        gt = w[t, j].double()[:, None]
        wt = dn64[e].t().contiguous()
        ref.index_add_(0, t, gt * (h @ wt))
        mag.index_add_(0, t, gt * (h.abs() @ wt.abs()))
    tol = (2.0 ** -8 + (H + I) * 2.0 ** -22) * mag + 2.0 ** -8 * ref.abs() * 1.01
    assert bool(((y - ref).abs()[:n_tok] <= tol[:n_tok]).all())
