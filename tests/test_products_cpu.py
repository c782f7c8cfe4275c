"""The MXFP4 encoder of the oracle against its definition, and the refusals of the quantiser, the
MXFP4 product, the grouped product and the prefill layer on chosen activations: bad arguments are
refused on the host, so none of these tests needs a GPU."""
import ctypes as C

import numpy as np
import pytest
import torch

from oracle import decode_mxfp4, e2m1_value
from oracle.formats import encode_mxfp4


# ---------------------------------------------------------------- the oracle's encoder

def test_encoder_keeps_every_representable_value():
    """A block whose largest magnitude is in e2m1's top binade (4 or 6 times its scale) comes back
    as it is, at every scale the encoder can choose."""
    vals = [e2m1_value(c) for c in range(16)]
    for X in (0, 1, 60, 127, 200, 252):
        row = np.array([6.0] + (vals * 2)[:31]) * 2.0 ** (X - 127)
        codes, scales = encode_mxfp4(row[None])
        assert scales.tolist() == [[X]]
        assert np.array_equal(decode_mxfp4(codes, scales)[0], row)


def test_encoder_rounds_to_the_even_code_and_saturates():
    # scale 1 (the maximum is in [4, 8)); ties between neighbouring codes go to the even one
    row = np.zeros(32)
    row[:12] = [7.9, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.26, -0.25, -5.01, 0.74]
    codes, scales = encode_mxfp4(row[None])
    assert scales.tolist() == [[127]]
    want = [6.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 0.5, 0.0, -6.0, 0.5]
    assert decode_mxfp4(codes, scales)[0, :12].tolist() == want


def test_encoder_of_special_blocks():
    row = np.zeros((1, 128))
    row[0, 32] = np.inf
    row[0, 70] = np.nan
    row[0, 96] = 2.0 ** -149
    codes, scales = encode_mxfp4(row)
    assert scales.tolist() == [[0, 255, 255, 0]]
    assert not codes.any()


# ---------------------------------------------------------------- refusals

def _buf(n=4096):
    b = (C.c_uint8 * (n + 16))()
    return b, (C.addressof(b) + 15) & ~15


def test_quantiser_refusals():
    from expert_cache_offloaded_amd import _lib as L
    lib = L.lib()
    keep, p = _buf()
    bad = [(p, 1, 2, 64, 64, p, p),            # MXFP4 is no source type
           (p, 9, 2, 64, 64, p, p),
           (p, 0, -1, 64, 64, p, p),
           (p, 0, 2, 48, 48, p, p),            # not a multiple of 32
           (p, 0, 2, 64, 32, p, p),            # ld < cols
           (p, 0, 2, 64, 68, p, p),            # ld % 8
           (p, 0, 1 << 40, 64, 1 << 30, p, p),
           (p + 8, 0, 2, 64, 64, p, p),
           (p, 0, 2, 64, 64, p + 4, p),
           (None, 0, 2, 64, 64, p, p),
           (p, 0, 2, 64, 64, None, p),
           (p, 0, 2, 64, 64, p, None)]
    for src, ty, r, c, ld, codes, sc in bad:
        assert lib.mc_mxfp4_quantize(src, ty, r, c, ld, codes, sc, None) == L.MC_EINVAL, (ty, r, c, ld)
        assert "mc_mxfp4_quantize" in L.last_error()
        assert lib.mc_mxfp4_dequantize(codes, sc, r, c, src, ty, ld, None) == L.MC_EINVAL
        assert "mc_mxfp4_dequantize" in L.last_error()
    assert lib.mc_mxfp4_quantize(None, 0, 0, 64, 64, None, None, None) == L.MC_OK
    assert lib.mc_mxfp4_dequantize(None, None, 5, 0, None, 0, 0, None) == L.MC_OK


def test_matmul_refusals():
    from expert_cache_offloaded_amd import _lib as L
    lib = L.lib()
    keep, p = _buf()

    def call(x=p, xs=p, xf=1, ldx=64, w=p, ws=p, M=2, N=4, K=64, y=p, yf=0, ldy=4):
        return lib.mc_mxfp4_matmul(x, xs, xf, ldx, w, ws, M, N, K, y, yf, ldy, None)

    for kw in (dict(xf=2), dict(xf=3), dict(yf=1), dict(yf=3), dict(M=-1), dict(N=-1), dict(K=0), dict(K=48),
               dict(xf=0, ldx=32), dict(xf=0, ldx=68), dict(ldy=3), dict(x=None), dict(w=None), dict(y=None),
               dict(K=(1 << 28) + 32, ldx=1 << 29), dict(M=(1 << 31) - 1),
               dict(N=(1 << 31) - 1, ldy=1 << 31),
               dict(ws=None), dict(xs=None), dict(x=p + 8), dict(w=p + 1), dict(y=p + 2), dict(ldy=1 << 31)):
        assert call(**kw) == L.MC_EINVAL, kw
        assert "mc_mxfp4_matmul" in L.last_error()
    assert call(M=0, x=None, y=None) == L.MC_OK
    assert call(N=0, w=None, y=None, ldy=0) == L.MC_OK


def test_grouped_refusals():
    from expert_cache_offloaded_amd import _lib as L
    lib = L.lib()
    keep, p = _buf()

    def call(**kw):
        d = dict(x_fmt=0, w_fmt=1, y_fmt=0, swiglu=0, E=2, M=2, N=64, K=64, x_rows=2, x_div=1, y_rows=2, x_perm=0,
                 y_perm=0, n_gate=2, ldx=64, ldy=64, n=2, x=p, x_scale=p, w=p, w_scale=p, y=p, y_scale=p, offsets=p,
                 perm=None, entry_of=None, gate=None)
        d.update(kw)
        return lib.mc_grouped_matmul(C.byref(L.Grouped(**d)), None)

    for kw in (dict(x_fmt=1, w_fmt=0), dict(x_fmt=2), dict(w_fmt=2), dict(y_fmt=3), dict(swiglu=2),
               dict(swiglu=1, N=63), dict(E=0), dict(E=1025), dict(M=-1), dict(K=40), dict(K=0), dict(x_rows=-1),
               dict(x_div=0), dict(y_rows=-1), dict(x_perm=1), dict(y_perm=1), dict(x_perm=2, perm=p), dict(ldx=60),
               dict(ldx=70), dict(ldy=63), dict(n=-1), dict(n=1 << 31), dict(x=None), dict(w=None), dict(y=None),
               dict(offsets=None), dict(w_scale=None), dict(x_fmt=1, x_scale=None), dict(y_fmt=1, y_scale=None),
               dict(y_fmt=1, N=48), dict(y_fmt=1, swiglu=1, N=96), dict(x=p + 4), dict(offsets=p + 2),
               dict(gate=p + 1), dict(gate=p, n_gate=-1)):
        assert call(**kw) == L.MC_EINVAL, kw
        assert "mc_grouped_matmul" in L.last_error()
    assert lib.mc_grouped_matmul(None, None) == L.MC_EINVAL
    assert call(M=0, x=None, y=None, offsets=None) == L.MC_OK
    # nothing to multiply, or nowhere to write: nothing is enqueued
    assert call(n=0) == L.MC_OK and call(x_rows=0) == L.MC_OK and call(y_rows=0) == L.MC_OK


def test_prefill_act_refusals():
    from expert_cache_offloaded_amd import _lib as L
    lib = L.lib()
    keep, p = _buf()
    b = L.Banks()
    b.fmt, b.H, b.I, b.n = L.MC_MXFP4, 64, 64, 4
    b.gate_up = b.gate_up_scale = b.down = b.down_scale = p
    big = 1 << 30

    def call(banks=b, x=p, ids=p, w=p, T=2, k=2, E=4, act=1, ws=p, ws_bytes=big, y=p, nxt=None):
        return lib.moe_experts_prefill_act(x, ids, w, T, k, None, E, C.byref(banks), act, ws, ws_bytes, y, None, nxt)

    b16 = L.Banks()
    b16.fmt, b16.H, b16.I, b16.n, b16.gate_up, b16.down = L.MC_BF16, 64, 64, 4, p, p
    odd = L.Banks()
    odd.fmt, odd.H, odd.I, odd.n = L.MC_MXFP4, 96, 64, 4
    odd.gate_up = odd.gate_up_scale = odd.down = odd.down_scale = p
    empty_next = L.Prefetch()
    for kw in (dict(act=2), dict(act=-1), dict(banks=b16), dict(banks=odd), dict(T=-1), dict(k=0), dict(k=5),
               dict(E=0), dict(E=1025), dict(E=5), dict(T=1 << 30, k=4), dict(x=None), dict(ids=None), dict(w=None),
               dict(ws=None), dict(y=None), dict(x=p + 8), dict(ws=p + 8), dict(ws_bytes=1000),
               dict(nxt=C.byref(empty_next))):
        assert call(**kw) == L.MC_EINVAL, kw
    part = lambda steps, entry, y=p: lib.moe_experts_prefill_act_part(  # noqa: E731
        p, p, p, 2, 2, None, 4, C.byref(b), entry, 1, steps, p, big, None, y, None)
    assert part(0, p) == part(8, p) == part(L.PF_EXPERTS, None) == part(L.PF_COMBINE, p, None) == L.MC_EINVAL
    n = lib.moe_experts_prefill_act_ws_bytes
    assert n(2, 2, 4, 64, 64, 2) == 0 and n(-1, 2, 4, 64, 64, 1) == 0
    assert n(100, 2, 4, 64, 64, 1) < n(100, 2, 4, 64, 64, 0)
    assert call(T=0, x=None, ids=None, w=None, ws=None, ws_bytes=0, y=None) == L.MC_OK


def test_binding_refusals():
    """The binding refuses tensors whose shape, type or device does not fit before it takes an
    address of them: CPU tensors in place of GPU ones among them."""
    import expert_cache_offloaded_amd as mc
    u8, bf = torch.uint8, torch.bfloat16
    codes, scales = torch.zeros(3, 32, dtype=u8), torch.zeros(3, 2, dtype=u8)
    x = torch.zeros(3, 64, dtype=bf)
    for call in (lambda: mc.mxfp4_quantize(x, codes, scales),                       # CPU tensors
                 lambda: mc.mxfp4_quantize(x[:2], codes, scales),
                 lambda: mc.mxfp4_quantize(x.t(), codes, scales),
                 lambda: mc.mxfp4_quantize(x, codes, scales[:, :1]),
                 lambda: mc.mxfp4_dequantize(codes, scales, x[:, :32]),
                 lambda: mc.mxfp4_matmul(x, codes, scales, torch.zeros(3, 3)),      # CPU tensors
                 lambda: mc.mxfp4_matmul(x[:, :32], codes, scales, torch.zeros(3, 3)),
                 lambda: mc.mxfp4_matmul(codes, codes, scales, torch.zeros(3, 3)),  # codes without scales
                 lambda: mc.mxfp4_matmul(x, codes, scales, torch.zeros(3, 4)),
                 lambda: mc.mxfp4_matmul(x, codes, scales, torch.zeros(3, 3), x_scale=scales),
                 lambda: mc.mxfp4_matmul(x.double(), codes, scales, torch.zeros(3, 3))):
        with pytest.raises(ValueError):
            call()
    w, off = torch.zeros(2, 4, 64, dtype=bf), torch.zeros(3, dtype=torch.int32)
    y = torch.zeros(3, 4)
    for kw in (dict(), dict(w_scale=scales), dict(x_scale=scales), dict(y=torch.zeros(3, 5)),
               dict(swiglu=True), dict(offsets=off.long()), dict(perm=off.long()), dict(w=w[:, ::2]),
               dict(entry_of=off), dict(gate=torch.zeros(3, dtype=torch.float64)),
               dict(w=w[0]), dict(y_scale=scales)):
        d = dict(x=x, w=w, offsets=off, y=y)
        d.update(kw)
        with pytest.raises(ValueError):
            mc.grouped_matmul(d.pop("x"), d.pop("w"), d.pop("offsets"), d.pop("y"), **d)


@pytest.mark.parametrize("lead", [(), (2, 1)])
def test_binding_wants_codes_in_rows(lead):
    """Codes of one or three dimensions, whose first one is not their number of rows, are refused for
    their shape: as [16] codes of one row they would be taken for 16 rows."""
    import expert_cache_offloaded_amd as mc
    codes, scales = torch.zeros(*lead, 16, dtype=torch.uint8), torch.zeros(*lead, 1, dtype=torch.uint8)
    wide = torch.zeros(codes.shape[0], 32, dtype=torch.bfloat16)
    for call in (lambda: mc.mxfp4_quantize(wide, codes, scales), lambda: mc.mxfp4_dequantize(codes, scales, wide)):
        with pytest.raises(ValueError, match="2-D"):
            call()


def test_sizes_past_32_bit_sums_are_refused():
    """Sizes whose tile sums or row offsets would leave 32 bits (of the grouped product even where
    groups overlap) are refused for that, before anything is enqueued."""
    from expert_cache_offloaded_amd import _lib as L
    lib = L.lib()
    keep, p = _buf()
    d = dict(x_fmt=0, w_fmt=1, y_fmt=0, E=1024, M=(1 << 25) + 1, N=64, K=64, x_rows=2, x_div=1, y_rows=2, ldx=64, ldy=64,
             n=2, x=p, x_scale=p, w=p, w_scale=p, y=p, offsets=p)
    assert lib.mc_grouped_matmul(C.byref(L.Grouped(**d)), None) == L.MC_EINVAL
    assert "too many" in L.last_error()
    b = L.Banks()
    for T, H, I, word in (((1 << 31) - 1, 64, 64, "too many"), (2, 1 << 29, 64, "too large"), (2, 64, 1 << 29, "too large")):
        b.fmt, b.H, b.I, b.n = L.MC_MXFP4, H, I, 4
        b.gate_up = b.gate_up_scale = b.down = b.down_scale = p
        assert lib.moe_experts_prefill_act(p, p, p, T, 1, None, 4, C.byref(b), 1, p, 1 << 62, p, None, None) == L.MC_EINVAL
        assert word in L.last_error(), (T, H, I)
