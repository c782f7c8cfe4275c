"""Products at the edges of their inputs."""
import numpy as np
import pytest
import torch

import expert_cache_offloaded_amd as mc
from oracle import decode_mxfp4
from test_gpu_products import BF, F32, FORMATS, I32, U8, dev, product_bound, silu64, swiglu_bound

pytestmark = pytest.mark.gpu

MAGNITUDES = [6.0, 4.0, 3.0, 2.0, 1.5, 1.0, 0.5]      # e2m1 codes 7 .. 1


def codes_with_sum(total):
    """32 e2m1 codes whose values add up to `total` (a multiple of 0.5)."""
    codes, left = [], abs(total)
    for i, m in enumerate(MAGNITUDES):
        while left >= m and len(codes) < 32:
            codes.append(7 - i + (8 if total < 0 else 0))
            left -= m
    assert left == 0
    return codes + [0] * (32 - len(codes))


def pack(rows):
    c = np.array(rows, dtype=np.uint8)
    return c[:, 0::2] | (c[:, 1::2] << 4)


@pytest.mark.parametrize("xf,wf", FORMATS)
@pytest.mark.parametrize("M", [3, 70, 300])
def test_swiglu_of_large_gates(xf, wf, M):
    """Gates down to -88.5, where e^-g is near fp32's end and silu(g) = g / (1 + e^-g), about 1e-37,
    still a normal number, with up values that bring it back to size; and up to 100, where silu(g) = g."""
    gates = [-88.5, -88.0, -87.5, -87.0, -80.0, -60.0, -20.0, -1.0, 0.0, 1.0, 20.0, 100.0]
    n = 32
    g = [gates[i % len(gates)] for i in range(n)]
    up = [1.0 + 0.5 * (i % 5) for i in range(n)]
    codes = pack([codes_with_sum(v) for v in g + up])
    scales = np.full((2 * n, 1), 127, dtype=np.uint8)
    scales[n:] = 127 + 60
    w64 = decode_mxfp4(codes, scales)
    x64 = np.ones((M, 32))
    if xf == "bf16":
        x, xs = torch.ones((M, 32), dtype=BF, device="cuda"), None
    else:
        x = torch.full((M, 16), 0x22, dtype=U8, device="cuda")
        xs = torch.full((M, 1), 127, dtype=U8, device="cuda")
    if wf == "bf16":
        w, ws = torch.from_numpy(w64).to(BF).cuda()[None], None
    else:
        w, ws = dev(codes)[None], dev(scales)[None]
    y = torch.full((M, n), 7.0, dtype=F32, device="cuda")
    mc.grouped_matmul(x, w, torch.tensor([0, M], dtype=I32, device="cuda"), y, x_scale=xs, w_scale=ws, swiglu=True)
    # the sums are exact: multiples of half a unit below 2^24 of them
    v = x64 @ w64.T
    ref = silu64(v[:, :n]) * v[:, n:]
    tol = swiglu_bound(v, np.zeros_like(v), n) + 2.0 ** -24 * np.abs(ref)
    off = np.abs(y.double().cpu().numpy() - ref)
    bad = ~(off <= tol)
    assert not bad.any(), (sorted(set(np.array(g)[np.nonzero(bad)[1]])), np.max(off[bad] / np.abs(ref[bad])))


@pytest.mark.parametrize("wf", ["bf16", "mxfp4"])
@pytest.mark.parametrize("M", [5, 90])
def test_gates_of_no_rows_skip_every_row(wf, M):
    """Rows past the gates' end are skipped; where there is no gate at all that is every row, whichever
    way the empty tensor came about."""
    n, K = 64, 64
    x = torch.ones((M, K), dtype=BF, device="cuda")
    w = torch.ones((1, n, K), dtype=BF, device="cuda") if wf == "bf16" else torch.full((1, n, K // 2), 0x22, dtype=U8, device="cuda")
    ws = None if wf == "bf16" else torch.full((1, n, K // 32), 127, dtype=U8, device="cuda")
    off = torch.tensor([0, M], dtype=I32, device="cuda")
    for some, rows in ((torch.ones(M, device="cuda")[:0], 0), (torch.empty(0, device="cuda"), 0),
                       (torch.ones(3, device="cuda"), 3)):
        y = torch.full((M, n), 7.0, dtype=F32, device="cuda")
        mc.grouped_matmul(x, w, off, y, w_scale=ws, gate=some)
        assert (y[:rows] == K).all() and (y[rows:] == 7.0).all()


@pytest.mark.parametrize("M", [3, 70, 300])
def test_largest_scales(M):
    """Weights with the scale bytes 253 and 254, whose larger codes stand for 2^128 and more.  Times MXFP4
    rows they are applied inside the matrix instruction and the products come out; times bf16 rows
    the weight becomes a bf16 first, and those codes infinity."""
    rng = np.random.default_rng(M)
    N, K = 40, 64
    for X, largest in ((252, 6.0), (253, 3.0), (254, 1.5)):
        codes = rng.integers(0, 16, size=(N, K))
        codes[N // 2:] = rng.choice([c for c in range(16) if [0, .5, 1, 1.5, 2, 3, 4, 6][c & 7] <= largest], size=(N - N // 2, K))
        scales = np.full((N, K // 32), X, dtype=np.uint8)
        w, ws = dev(pack(codes)), dev(scales)
        w64 = decode_mxfp4(pack(codes), scales)
        y = torch.empty((M, N), dtype=F32, device="cuda")
        xc = rng.integers(0, 256, size=(M, K // 2)).astype(np.uint8)
        xs = np.full((M, K // 32), 60, dtype=np.uint8)
        x64 = decode_mxfp4(xc, xs)
        mc.mxfp4_matmul(dev(xc), w, ws, y, x_scale=dev(xs))
        assert (np.abs(y.double().cpu().numpy() - x64 @ w64.T)
                <= product_bound(x64, w64) + 2.0 ** -24 * np.abs(x64 @ w64.T)).all(), X
        x = torch.from_numpy(rng.choice([1.0, -1.5, 1.25], size=(M, K)) * 2.0 ** -70).to(BF)
        x64 = x.double().numpy()
        mc.mxfp4_matmul(x.cuda(), w, ws, y)
        got = y.double().cpu().numpy()
        over = (np.abs(w64) >= 2.0 ** 128).any(axis=1)
        assert not np.isfinite(got[:, over]).any(), X
        fits = ~over
        assert (np.abs(got[:, fits] - x64 @ w64[fits].T)
                <= product_bound(x64, w64[fits]) + 2.0 ** -24 * np.abs(x64 @ w64[fits].T)).all(), X
        # read back: what is beyond the type is an infinity
        for t in (BF, F32):
            d = torch.empty((N, K), dtype=t, device="cuda")
            mc.mxfp4_dequantize(w, ws, d)
            want = np.where(np.abs(w64) >= 2.0 ** 128, np.copysign(np.inf, w64), w64)
            assert np.array_equal(d.double().cpu().numpy(), want), (X, t)


@pytest.mark.parametrize("where", ["cpu", "cuda"])
def test_quantize_banks_of_no_experts(where):
    from expert_cache_offloaded_amd.runtime import BankSet, alloc_banks, quantize_banks
    a, b = (BankSet(alloc_banks(0, 128, 64, f, device=where), 128, 64, f) for f in ("bf16", "mxfp4"))
    quantize_banks(a, b)
