"""The activations that a prefill layer can be asked for: values, workspaces, refusals (no GPU)."""
import pytest


def test_acts_and_their_workspaces():
    from expert_cache_offloaded_amd import _lib as L
    assert L.ACT == {"bf16": L.MC_BF16, "mxfp4": L.MC_MXFP4, "mxfp4_f32": L.MC_MXFP4_F32}
    T, k, E, H, I = 128, 2, 4, 64, 128
    short, long = (L.prefill_act_ws_bytes(T, k, E, H, I, a) for a in ("mxfp4", "mxfp4_f32"))
    assert long - short == T * k * H * 2          # four bytes per route output for two
    raw = L.lib().moe_experts_prefill_act_ws_bytes
    assert raw(T, k, E, H, I, L.MC_MXFP4_F32) == long
    assert raw(T, k, E, H, I, L.MC_F32) == raw(T, k, E, H, I, L.MC_F16) == raw(T, k, E, H, I, 5) == 0


def test_fp32_routes_need_mxfp4_experts_and_their_workspace():
    import ctypes as C
    from expert_cache_offloaded_amd import _lib as L
    keep = (C.c_uint8 * 4112)()
    p = (C.addressof(keep) + 15) & ~15

    def call(fmt, act, ws_bytes=1 << 30):
        b = L.Banks()
        b.fmt, b.H, b.I, b.n = fmt, 64, 64, 4
        b.gate_up = b.gate_up_scale = b.down = b.down_scale = p
        return L.lib().moe_experts_prefill_act(p, p, p, 2, 2, None, 4, C.byref(b), act, p, ws_bytes, p, None, None)

    assert call(L.MC_BF16, L.MC_MXFP4_F32) == L.MC_EINVAL and "need MXFP4 experts" in L.last_error()
    short = L.prefill_act_ws_bytes(2, 2, 4, 64, 64, "mxfp4")
    assert call(L.MC_MXFP4, L.MC_MXFP4_F32, short) == L.MC_EINVAL and "workspace" in L.last_error()


def test_binding_refuses_other_acts():
    import torch
    import expert_cache_offloaded_amd as mc
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    ids, w = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2)
    banks = mc.make_banks("mxfp4", 64, 64, {"gate_up": torch.zeros(4, 128, 32, dtype=torch.uint8),
                                            "gate_up_scale": torch.zeros(4, 128, 2, dtype=torch.uint8),
                                            "down": torch.zeros(4, 64, 32, dtype=torch.uint8),
                                            "down_scale": torch.zeros(4, 64, 2, dtype=torch.uint8)})
    with pytest.raises(ValueError, match="mxfp4_f32"):
        mc.moe_experts_prefill_act(x, ids, w, None, 4, banks, "f32", torch.zeros(16, dtype=torch.uint8), x)
    with pytest.raises(KeyError):
        mc.make_banks("mxfp4_f32", 64, 64, {})
