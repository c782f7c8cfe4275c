"""Sizes beyond 32 bits: the binding refuses them for that.  Passed on as 32-bit arguments, 2^32 + 5 rows
would be taken for 5.  The tensors have no storage (torch's meta device), so no GPU is needed."""
import pytest
import torch

import expert_cache_offloaded_amd as mc

U8, BF, F32, I32 = torch.uint8, torch.bfloat16, torch.float32, torch.int32
BIG = (1 << 32) + 5


def meta(*shape, dtype):
    return torch.empty(shape, dtype=dtype, device="meta")


def test_matmul():
    for M, N, K in ((BIG, 4, 64), (3, BIG, 64), (3, 4, (1 << 32) + 64), (1 << 31, 4, 64)):
        with pytest.raises(ValueError, match="32 bits"):
            mc.mxfp4_matmul(meta(M, K, dtype=BF), meta(N, K // 2, dtype=U8), meta(N, K // 32, dtype=U8),
                            meta(M, N, dtype=F32))
        with pytest.raises(ValueError, match="32 bits"):
            mc.mxfp4_matmul(meta(M, K // 2, dtype=U8), meta(N, K // 2, dtype=U8), meta(N, K // 32, dtype=U8),
                            meta(M, N, dtype=F32), x_scale=meta(M, K // 32, dtype=U8))


def test_grouped_matmul():
    d = dict(M=8, N=4, K=64, E=2, rows=8, x_div=1, gates=8)
    for bad in (dict(M=BIG), dict(N=BIG), dict(K=(1 << 32) + 64), dict(E=1 << 32), dict(rows=BIG), dict(x_div=(1 << 32) + 1),
                dict(gates=BIG)):
        s = dict(d, **bad)
        with pytest.raises(ValueError, match="32 bits"):
            mc.grouped_matmul(meta(s["rows"], s["K"], dtype=BF), meta(2, s["N"], s["K"], dtype=BF),
                              meta(s["E"] + 1, dtype=I32), meta(s["M"], s["N"], dtype=F32), perm=meta(s["M"], dtype=I32),
                              x_div=s["x_div"], gate=meta(s["gates"], dtype=F32))


def test_layer():
    banks = mc.make_banks("bf16", 64, 64, {"gate_up": torch.zeros(4, 128, 64, dtype=BF), "down": torch.zeros(4, 64, 64, dtype=BF)})
    x, ids, w = torch.zeros(2, 64, dtype=BF), torch.zeros(2, 2, dtype=I32), torch.zeros(2, 2)
    ws = torch.zeros(1 << 16, dtype=U8)
    E = (1 << 32) + 4
    for call in (lambda: mc.prefill_act_ws_bytes(2, 2, E, 64, 64, "bf16"),
                 lambda: mc.moe_experts_prefill_act(x, ids, w, None, E, banks, "bf16", ws, x),
                 lambda: mc.moe_experts_prefill_act_part(x, ids, w, None, E, banks, None, "bf16", 1, ws),
                 lambda: mc.moe_experts_prefill_act_part(x, ids, w, None, 4, banks, None, "bf16", (1 << 32) + 1, ws)):
        with pytest.raises(ValueError, match="32 bits"):
            call()
