"""The prefill layer on MXFP4 activations against its definition in 64 bits, with its route outputs
in bf16 ("mxfp4") and in fp32 ("mxfp4_f32"): how far each may be from the unrounded sum."""
import numpy as np
import pytest
import torch

import expert_cache_offloaded_amd as mc
from oracle import sort_routes
from test_gpu_products import BF, F32, U8, dev, gpu_operand, layer_inputs, run_layer
from test_gpu_products import test_prefill_runner_on_chosen_activations as runner_case

pytestmark = pytest.mark.gpu


def mxfp4_values(v):
    """float64 rows -> the values of their MXFP4 codes."""
    b = v.reshape(-1, 32)
    s = torch.ldexp(torch.ones((), dtype=v.dtype, device=v.device),
                    (torch.frexp(b.abs().amax(1, keepdim=True))[1] - 3).clamp(-127, 127))
    a = b.abs() / s
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(v.dtype)
    return (torch.copysign((torch.round(a / step) * step).clamp(max=6.0), b) * s).reshape(v.shape)


def bf16_rounding(v):
    """The mean square of a bf16 rounding of v: its error is spread evenly over half a step to either
    side, and 2^(x-1) <= |v| < 2^x has steps of 2^(x-8)."""
    half = torch.ldexp(torch.ones_like(v), torch.frexp(v)[1] - 9)
    return torch.where(v == 0, torch.zeros_like(v), half * half / 3)


@pytest.mark.parametrize("act", ["mxfp4", "mxfp4_f32"])
@pytest.mark.parametrize("T,k,E,H,I,n_tok", [(2, 8, 256, 2048, 512, None), (130, 2, 4, 128, 192, None),
                                             (700, 3, 8, 192, 320, 611), (8200, 4, 8, 2048, 1024, 8111)])
def test_layer_against_the_unrounded_sum(act, T, k, E, H, I, n_tok):
    """The reference quantises x and h as the format asks and rounds nothing else.  What is left is y's
    own rounding to bf16 and, with bf16 route outputs, one rounding per route: independent errors
    whose mean squares add up to `want`.  The mean square that is seen may exceed it by six standard
    deviations (an error's square varies by at most twice its mean's square) and by a fifth, for
    values of h that lie so near a border between two codes that the fp32 sums take the other one.
    They are off by 2^-21 of themselves at the most, the codes half a scale apart or more, so about
    one value in 2^20 of the size of a scale changes sides, and by half a scale or so: some 2^-23 of
    the output's square, against 2^-18.5 that y's rounding makes.  With bf16 route outputs the error's
    square is about twice as large as without, so the bounds tell the two apart."""
    g = torch.Generator(device="cuda")
    g.manual_seed(T + H + I)
    gu, gus, gu64 = gpu_operand(g, "mxfp4", E, 2 * I, H, size=2.0 ** -4)
    dn, dns, dn64 = gpu_operand(g, "mxfp4", E, H, I, size=2.0 ** -4)
    x = torch.randn((T, H), generator=g, device="cuda").to(BF)
    w, ids = torch.topk(torch.softmax(torch.randn((T, E), generator=g, device="cuda"), 1), k, dim=1)
    w, ids = (w / w.sum(1, keepdim=True)).contiguous(), ids.to(torch.int32)
    y = run_layer(x, ids.cpu().numpy(), w.cpu().numpy(), n_tok, E, H, I, "mxfp4", act,
                  {"gate_up": gu, "gate_up_scale": gus, "down": dn, "down_scale": dns})
    nt = T if n_tok is None else n_tok
    assert (y[nt:] == 0).all()
    xq = mxfp4_values(x.double())
    ref, want = (torch.zeros((T, H), dtype=torch.float64, device="cuda") for _ in range(2))
    for e in range(E):
        t, j = torch.nonzero(ids[:nt] == e, as_tuple=True)
        if not len(t):
            continue
        v = xq[t] @ gu64[e].t().contiguous()
        h = mxfp4_values(v[:, :I] * torch.sigmoid(v[:, :I]) * v[:, I:])
        r = w[t, j].double()[:, None] * (h @ dn64[e].t().contiguous())
        ref.index_add_(0, t, r)
        if act == "mxfp4":
            want.index_add_(0, t, bf16_rounding(r))
    want = (want + bf16_rounding(ref))[:nt]
    seen = float(((y.double() - ref)[:nt] ** 2).mean())
    spread = float((2 * want ** 2).mean()) ** 0.5 / want.numel() ** 0.5
    print("seen / want %.3f, six deviations %.3f" % (seen / float(want.mean()), 6 * spread / float(want.mean())))
    assert seen <= 1.2 * float(want.mean()) + 6 * spread


def test_layer_with_fp32_routes_is_its_parts():
    """With fp32 route outputs too the layer equals its parts called one by one, bit for bit."""
    rng = np.random.default_rng(3)
    T, k, E, H, I = 190, 4, 16, 256, 192
    ids, w, x, banks, _, _ = layer_inputs(rng, T, k, E, H, I, "mxfp4")
    y = run_layer(x, ids, w, None, E, H, I, "mxfp4", "mxfp4_f32", banks)
    x = x.cuda()
    c, o, p = sort_routes(ids, E, None)
    off, perm = dev(np.asarray(o, dtype=np.int32)), dev(np.asarray(p, dtype=np.int32))
    xq, xqs = torch.empty((T, H // 2), dtype=U8, device="cuda"), torch.empty((T, H // 32), dtype=U8, device="cuda")
    hq = torch.empty((T * k, I // 2), dtype=U8, device="cuda")
    hqs = torch.empty((T * k, I // 32), dtype=U8, device="cuda")
    yr = torch.empty((T * k, H), dtype=F32, device="cuda")
    mc.mxfp4_quantize(x, xq, xqs)
    mc.grouped_matmul(xq, banks["gate_up"], off, hq, x_scale=xqs, w_scale=banks["gate_up_scale"], y_scale=hqs,
                      swiglu=True, perm=perm, x_div=k)
    mc.grouped_matmul(hq, banks["down"], off, yr, x_scale=hqs, w_scale=banks["down_scale"], perm=perm, x_perm=False,
                      y_perm=True, gate=dev(w).reshape(-1))
    s = torch.zeros((T, H), device="cuda")
    for j in range(k):
        s += yr.view(T, k, H)[:, j]
    assert torch.equal(y, s.to(BF))


@pytest.mark.parametrize("S", [32, 9, 1])
def test_prefill_runner_with_fp32_routes(S):
    """PrefillRunner(act="mxfp4_f32"): whole layers and layers in parts give the layer's own outputs."""
    runner_case("mxfp4", "mxfp4_f32", S)
