"""Timed cases of the MXFP4 quantiser and its inverse, the MXFP4 product, the product grouped by
expert, and the prefill MoE layer on quantised or bf16 activations.

``run`` computes each of them in plain torch operations (fp32), or, with ``own`` set, through the
entry points of ``expert_cache_offloaded_amd``.  The sizes are those of the library's two model
shapes (256 experts: top-8, hidden 2048, intermediate 512; top-6, hidden 4096, intermediate 2048)
and odd ones between one row and a prefill chunk.

MXFP4: blocks of 32 elements along a row share a power-of-two scale 2^e and hold e2m1 codes
(0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives).  The quantiser takes e = floor(log2(max |v|)) - 2
and rounds v / 2^e to the nearest code, ties to the even one, magnitudes over 6 to 6.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "f16": torch.float16}


def listed():
    return [
        # four decode tokens' activations on their way into a product with quantised operands
        dict(name="quantize_tokens", op="quantize", type="bf16", rows=4, cols=2048, pad=0),
        # fp32 expert weights of a checkpoint turned into a gate_up bank
        dict(name="quantize_bank", op="quantize", type="f32", rows=65536, cols=4096, pad=0),
        # an odd number of token rows cut out of a wider buffer
        dict(name="dequantize_odd", op="dequantize", type="f32", rows=777, cols=2080, pad=32),
        # the down banks of a whole layer (256 experts) read back as bf16
        dict(name="dequantize_bank", op="dequantize", type="bf16", rows=256 * 2048, cols=512, pad=0),
        # one token through a quantised projection: latency and weight bytes
        dict(name="matmul_one_token", op="matmul", x="bf16", M=1, N=4096, K=2048, y="bf16", pad=0),
        # a ragged batch, output columns and contraction no tile divides
        dict(name="matmul_odd", op="matmul", x="bf16", M=333, N=4100, K=2080, y="f32", pad=32),
        # a prefill chunk, both operands quantised
        dict(name="matmul_chunk_a4", op="matmul", x="mxfp4", M=8192, N=4096, K=4096, y="bf16", pad=0),
        # one token's eight experts, gate and up with SwiGLU (a decode step's first half)
        dict(name="grouped_decode", op="grouped", x="bf16", w="mxfp4", T=1, k=8, E=256, N=1024, K=2048,
             swiglu=True, gate=False, skew=0.0, y="bf16"),
        # bf16 experts, token counts as uneven as a skewed router makes them
        dict(name="grouped_bf16_skewed", op="grouped", x="bf16", w="bf16", T=4001, k=4, E=64, N=2048, K=2048,
             swiglu=False, gate=False, skew=1.1, y="bf16"),
        # a small chunk of quantised rows over every expert, scattered to routes with their gates
        dict(name="grouped_a4_gated", op="grouped", x="mxfp4", w="mxfp4", T=1024, k=6, E=256, N=4096, K=2048,
             swiglu=False, gate=True, skew=0.0, y="f32"),
        # the whole layer of a prefill chunk, activations quantised (the shape of the chunk benchmark)
        dict(name="layer_chunk_a4", op="layer", act="mxfp4", T=8192, valid=8192, k=6, E=256, H=4096, I=2048),
        # an odd, partly filled chunk through bf16 experts
        dict(name="layer_odd_bf16", op="layer", act="bf16", T=1111, valid=1003, k=8, E=256, H=2048, I=512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "dequantize", "matmul", "grouped", "grouped", "layer"])
    if op in ("quantize", "dequantize"):
        cols = 32 * _log(rng, 1, 256)
        return dict(op=op, type=rng.choice(list(TYPES)), rows=_log(rng, 1, 200_000_000 // cols), cols=cols,
                    pad=rng.choice([0, 32, 64]))
    if op == "matmul":
        return dict(op=op, x=rng.choice(["bf16", "mxfp4"]), M=_log(rng, 1, 8192), N=_log(rng, 1, 8192),
                    K=32 * _log(rng, 1, 160), y=rng.choice(["bf16", "f32"]), pad=0)
    if op == "grouped":
        x, w = rng.choice([("bf16", "bf16"), ("bf16", "mxfp4"), ("mxfp4", "mxfp4")])
        E = _log(rng, 2, 256)
        k = rng.randint(1, min(E, 8))
        swiglu = rng.random() < 0.5
        n = _log(rng, 8, 2048)
        return dict(op=op, x=x, w=w, T=_log(rng, 1, 2048), k=k, E=E, N=2 * n if swiglu else n, K=32 * _log(rng, 1, 96),
                    swiglu=swiglu, gate=rng.random() < 0.5, skew=rng.choice([0.0, 1.1]), y=rng.choice(["bf16", "f32"]))
    E = _log(rng, 8, 256)
    T = _log(rng, 1, 2048)
    return dict(op="layer", act=rng.choice(["bf16", "mxfp4"]), T=T, valid=rng.randint(0, T) if rng.random() < 0.3 else T,
                k=rng.randint(1, min(E, 8)), E=E, H=64 * _log(rng, 1, 40), I=64 * _log(rng, 1, 20))


# ------------------------------------------------------------------ inputs

def _normal(g, *shape, std=1.0, dtype=torch.float32):
    return torch.empty(shape, dtype=torch.float32, device=DEV).normal_(0.0, std, generator=g).to(dtype)


def _codes(g, *shape):
    """Random codes and scales of MXFP4 rows with elements around 0.02 (a weight's size)."""
    *lead, cols = shape
    codes = torch.randint(0, 256, (*lead, cols // 2), dtype=torch.uint8, device=DEV, generator=g)
    scales = torch.randint(119, 122, (*lead, cols // 32), dtype=torch.uint8, device=DEV, generator=g)
    return codes, scales


def _act_codes(g, *shape):
    """Codes and scales of MXFP4 rows with elements around 1 (an activation's size)."""
    codes, scales = _codes(g, *shape)
    return codes, scales + 6


def _wide(t, pad):
    """The same values as a view of a buffer whose rows are `pad` elements longer."""
    if not pad:
        return t
    b = torch.zeros((t.shape[0], t.shape[1] + pad), dtype=t.dtype, device=DEV)
    b[:, :t.shape[1]] = t
    return b[:, :t.shape[1]]


def _routes(g, T, k, E, skew):
    """ids int32 [T][k] of a router whose experts are about as popular as rank^-skew, and its gates."""
    order = torch.randperm(E, device=DEV, generator=g)
    base = -skew * torch.log(order.float() + 1.0)
    noise = -torch.log(-torch.log(torch.rand((T, E), device=DEV, generator=g).clamp_(1e-6, 1 - 1e-6)))
    top, ids = torch.topk(base + noise, k, dim=1)
    e = torch.exp(top - top[:, :1])
    return ids.to(torch.int32), (e / e.sum(1, keepdim=True)).contiguous()


def _sorted_routes(ids, E):
    """Routes grouped by expert: offsets int32 [E + 1] and perm int32 (route t*k + j of each row)."""
    flat = ids.reshape(-1).long()
    perm = torch.argsort(flat, stable=True).to(torch.int32)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.cumsum(torch.bincount(flat, minlength=E), 0).to(torch.int32)
    return offsets, perm


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c = dict(case)
    s = {"case": c}
    if c["op"] == "quantize":
        # rows of different sizes, as the channels of a layer have
        v = _normal(g, c["rows"], c["cols"]) * torch.exp(_normal(g, c["rows"], 1))
        s["src"] = _wide(v.to(TYPES[c["type"]]), c["pad"])
        s["codes"] = torch.empty((c["rows"], c["cols"] // 2), dtype=torch.uint8, device=DEV)
        s["scales"] = torch.empty((c["rows"], c["cols"] // 32), dtype=torch.uint8, device=DEV)
        s["y"] = torch.empty((c["rows"], c["cols"]), dtype=torch.bfloat16, device=DEV)
    elif c["op"] == "dequantize":
        s["codes"], s["scales"] = _codes(g, c["rows"], c["cols"])
        s["y"] = _wide(torch.empty((c["rows"], c["cols"]), dtype=TYPES[c["type"]], device=DEV), c["pad"])
    elif c["op"] == "matmul":
        if c["x"] == "mxfp4":
            s["x"], s["xs"] = _act_codes(g, c["M"], c["K"])
        else:
            s["x"], s["xs"] = _wide(_normal(g, c["M"], c["K"], dtype=torch.bfloat16), c["pad"]), None
        s["w"], s["ws"] = _codes(g, c["N"], c["K"])
        s["y"] = torch.empty((c["M"], c["N"]), dtype=TYPES[c["y"]], device=DEV)
    elif c["op"] == "grouped":
        ids, gates = _routes(g, c["T"], c["k"], c["E"], c["skew"])
        s["offsets"], s["perm"] = _sorted_routes(ids, c["E"])
        s["gates"] = gates.reshape(-1) if c["gate"] else None
        # the most rows an expert has: what the plain form pads every expert to
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        if c["x"] == "mxfp4":
            s["x"], s["xs"] = _act_codes(g, c["T"], c["K"])
        else:
            s["x"], s["xs"] = _normal(g, c["T"], c["K"], dtype=torch.bfloat16), None
        if c["w"] == "mxfp4":
            s["w"], s["ws"] = _codes(g, c["E"], c["N"], c["K"])
        else:
            s["w"], s["ws"] = _normal(g, c["E"], c["N"], c["K"], std=0.02, dtype=torch.bfloat16), None
        n_out = c["N"] // 2 if c["swiglu"] else c["N"]
        s["y"] = torch.empty((c["T"] * c["k"], n_out), dtype=TYPES[c["y"]], device=DEV)
    else:
        T, E, H, I = c["T"], c["E"], c["H"], c["I"]
        s["ids"], s["gates"] = _routes(g, T, c["k"], E, 0.0)
        s["n_tok"] = torch.tensor([c["valid"]], dtype=torch.int32, device=DEV) if c["valid"] < T else None
        most = torch.bincount(s["ids"][:c["valid"]].reshape(-1).long(), minlength=E).max()
        s["most"] = int(most)
        s["x"] = _normal(g, T, H, dtype=torch.bfloat16)
        if c["act"] == "mxfp4":
            gu, gus = _codes(g, E, 2 * I, H)
            dn, dns = _codes(g, E, H, I)
            s["banks"] = {"gate_up": gu, "gate_up_scale": gus, "down": dn, "down_scale": dns}
        else:
            s["banks"] = {"gate_up": _normal(g, E, 2 * I, H, std=0.02, dtype=torch.bfloat16),
                          "down": _normal(g, E, H, I, std=0.02, dtype=torch.bfloat16)}
        s["y"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    return s


# ------------------------------------------------------------------ the plain form

_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


_tables = {}


def _table(name, values):
    """A constant table on the GPU, made once."""
    if (name, DEV) not in _tables:
        _tables[name, DEV] = torch.tensor(values, device=DEV)
    return _tables[name, DEV]


def _decode(codes, scales):
    """MXFP4 rows -> fp32 (exact): both values of a byte from a table, times the block's scale."""
    table = _table("bytes", [[_E2M1[b & 15], _E2M1[b >> 4]] for b in range(256)])
    v = table.index_select(0, codes.reshape(-1).int())
    v = v.reshape(*codes.shape[:-1], codes.shape[-1] // 16, 32)
    v *= torch.exp2(scales.float() - 127.0).unsqueeze(-1)
    return v.reshape(*codes.shape[:-1], codes.shape[-1] * 2)


def _round_trip(v):
    """fp32 rows -> the fp32 values that their MXFP4 codes stand for."""
    b = v.reshape(*v.shape[:-1], v.shape[-1] // 32, 32)
    amax = b.abs().amax(-1, keepdim=True)
    e = (torch.frexp(amax)[1] - 3).clamp_(-127, 127)
    scale = torch.where(amax > 0, torch.exp2(e.float()), torch.ones_like(amax))
    a = (b / scale).abs()
    code = (a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    table = _table("magnitudes", _E2M1[:8])
    q = table.index_select(0, code.reshape(-1)).reshape(b.shape)
    return (torch.copysign(q, b) * scale).reshape(v.shape)


def _silu_mul(g, u):
    return g / (1.0 + torch.exp(-g)) * u


def _grouped_plain(x, w, offsets, most, swiglu):
    """Row i (fp32, sorted by group) times the transpose of its group's matrix.  Few rows take their
    matrices one by one; many are padded to the largest group and go through one batched product."""
    n_rows, E = x.shape[0], offsets.shape[0] - 1
    i = torch.arange(n_rows, device=x.device, dtype=torch.int32)
    e = torch.bucketize(i, offsets[1:], right=True)
    e = e.clamp_(max=E - 1)
    if n_rows <= 64 and n_rows < E:
        we = w(e)
        out = torch.bmm(we, x.unsqueeze(-1)).squeeze(-1)
    else:
        rows = offsets[:-1, None] + torch.arange(most, device=x.device, dtype=torch.int32)[None]
        batch = x[rows.clamp_(max=n_rows - 1).reshape(-1)].reshape(E, most, x.shape[1])
        full = torch.bmm(batch, w(None).transpose(1, 2))
        out = full.reshape(E * most, -1)[e * most + (i - offsets[e])]
    if swiglu:
        half = out.shape[1] // 2
        out = _silu_mul(out[:, :half], out[:, half:])
    return out


def _weights(codes, scales):
    if scales is None:
        return lambda e: (codes if e is None else codes[e]).float()
    return lambda e: _decode(codes, scales) if e is None else _decode(codes[e], scales[e])


def _rows_of(x, xs):
    return x.float() if xs is None else _decode(x, xs)


def _plain(s):
    c = s["case"]
    if c["op"] == "quantize":
        return _round_trip(s["src"].float()).to(torch.bfloat16)
    if c["op"] == "dequantize":
        return _decode(s["codes"], s["scales"]).to(TYPES[c["type"]])
    if c["op"] == "matmul":
        return torch.matmul(_rows_of(s["x"], s["xs"]), _decode(s["w"], s["ws"]).t()).to(TYPES[c["y"]])
    if c["op"] == "grouped":
        x = _rows_of(s["x"], s["xs"])[(s["perm"] // c["k"])]
        y = _grouped_plain(x, _weights(s["w"], s["ws"]), s["offsets"], s["most"], c["swiglu"])
        if c["gate"]:
            perm = s["perm"].long()
            y = torch.empty_like(y).index_copy_(0, perm, y * s["gates"][perm].unsqueeze(1))
        return y.to(TYPES[c["y"]])
    T, k, E, H = c["T"], c["k"], c["E"], c["H"]
    if c["valid"] == 0:
        return torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
    b = s["banks"]
    valid = c["valid"]
    offsets, perm = _sorted_routes(s["ids"][:valid], E)
    x = s["x"][:valid].float()
    if c["act"] == "mxfp4":
        x = _round_trip(x)
    h = _grouped_plain(x[perm // k], _weights(b["gate_up"], b.get("gate_up_scale")), offsets, s["most"], True)
    # the down product's input is held in the activations' type
    h = _round_trip(h) if c["act"] == "mxfp4" else h.to(torch.bfloat16).float()
    r = _grouped_plain(h, _weights(b["down"], b.get("down_scale")), offsets, s["most"], False)
    perm = perm.long()
    r = torch.empty_like(r).index_copy_(0, perm, r * s["gates"].reshape(-1)[perm].unsqueeze(1))
    y = torch.zeros((T, H), dtype=torch.float32, device=DEV)
    y[:valid] = r.reshape(valid, k, H).sum(1)
    return y.to(torch.bfloat16)


# ------------------------------------------------------------------ the library's operators

def _own(s):
    import expert_cache_offloaded_amd as mc

    c, y = s["case"], s["y"]
    if c["op"] == "quantize":
        mc.mxfp4_quantize(s["src"], s["codes"], s["scales"])
        mc.mxfp4_dequantize(s["codes"], s["scales"], y)
    elif c["op"] == "dequantize":
        mc.mxfp4_dequantize(s["codes"], s["scales"], y)
    elif c["op"] == "matmul":
        mc.mxfp4_matmul(s["x"], s["w"], s["ws"], y, x_scale=s["xs"])
    elif c["op"] == "grouped":
        mc.grouped_matmul(s["x"], s["w"], s["offsets"], y, x_scale=s["xs"], w_scale=s["ws"], perm=s["perm"],
                          x_div=c["k"], y_perm=c["gate"], gate=s["gates"], swiglu=c["swiglu"])
    else:
        banks = mc.make_banks("mxfp4" if c["act"] == "mxfp4" else "bf16", c["H"], c["I"], s["banks"])
        # the plain form's route outputs are not rounded before their sum
        act = "mxfp4_f32" if c["act"] == "mxfp4" else "bf16"
        ws = torch.empty(mc.prefill_act_ws_bytes(c["T"], c["k"], c["E"], c["H"], c["I"], act),
                         dtype=torch.uint8, device=DEV)
        mc.moe_experts_prefill_act(s["x"], s["ids"], s["gates"], s["n_tok"], c["E"], banks, act, ws, y)
    return y


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ work

def _distinct(E, rows):
    """Experts that `rows` uniform routes are expected to reach."""
    return E * (1.0 - (1.0 - 1.0 / E) ** rows)


def _bytes_of(fmt, n):
    return n * (0.53125 if fmt == "mxfp4" else 4 if fmt == "f32" else 2)


def work(case):
    c = case
    if c["op"] in ("quantize", "dequantize"):
        n = c["rows"] * c["cols"]
        if c["op"] == "dequantize":
            return {"bytes": _bytes_of("mxfp4", n) + _bytes_of(c["type"], n), "flops": n}
        # codes and scales are written and read back, the values written
        return {"bytes": _bytes_of(c["type"], n) + 2 * _bytes_of("mxfp4", n) + 2 * n, "flops": 4 * n}
    if c["op"] == "matmul":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": _bytes_of(c["x"], M * K) + _bytes_of("mxfp4", N * K) + _bytes_of(c["y"], M * N),
                "flops": 2 * M * N * K}
    if c["op"] == "grouped":
        rows = c["T"] * c["k"]
        n_out = c["N"] // 2 if c["swiglu"] else c["N"]
        return {"bytes": _bytes_of(c["x"], c["T"] * c["K"]) + _bytes_of(c["y"], rows * n_out)
                + _bytes_of(c["w"], _distinct(c["E"], rows) * c["N"] * c["K"]) + 8 * rows,
                "flops": 2 * rows * c["N"] * c["K"]}
    rows = c["valid"] * c["k"]
    fmt = "mxfp4" if c["act"] == "mxfp4" else "bf16"
    return {"bytes": 2 * c["valid"] * c["H"] + 2 * c["T"] * c["H"] + 8 * rows
            + _bytes_of(fmt, _distinct(c["E"], rows) * 3 * c["H"] * c["I"]) + 1,
            "flops": 6 * rows * c["H"] * c["I"]}


# ------------------------------------------------------------------ 64 bits

def _values64(codes, scales):
    """MXFP4 rows -> float64, from the fields of the code: sign, two exponent bits, one mantissa bit."""
    nib = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    ex, man = (nib >> 1) & 3, (nib & 1).double()
    mag = torch.where(ex == 0, 0.5 * man, (1.0 + 0.5 * man) * torch.exp2((ex.double() - 1.0)))
    mag = torch.where(nib >= 8, -mag, mag)
    return mag * torch.exp2(scales.double() - 127.0).repeat_interleave(32, dim=-1)


def _nearest64(v):
    """float64 rows -> the values of their MXFP4 codes: on each binade of e2m1 the codes are evenly
    spaced, so the nearest one is a rounding to that spacing (torch.round takes ties to even)."""
    b = v.reshape(-1, 32)
    amax = b.abs().amax(1, keepdim=True)
    top = torch.floor(torch.log2(torch.where(amax > 0, amax, torch.ones_like(amax))))
    # log2 of a value just under a power of two may round up to it
    top = torch.where(torch.exp2(top) > amax, top - 1, top)
    top = torch.where(torch.exp2(top + 1) <= amax, top + 1, top)
    scale = torch.exp2((top - 2).clamp(-127, 127))
    u = b / scale
    a = u.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    q = (torch.round(a / step) * step).clamp(max=6.0)
    return (torch.where(u < 0, -q, q) * scale).reshape(v.shape)


def _expert64(w, ws, e):
    return w[e].double() if ws is None else _values64(w[e], ws[e])


def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    if c["op"] == "quantize":
        out = torch.empty((c["rows"], c["cols"]), dtype=torch.float64, device=DEV)
        for r in range(0, c["rows"], 16384):
            out[r:r + 16384] = _nearest64(s["src"][r:r + 16384].double())
        return out
    if c["op"] == "dequantize":
        out = torch.empty((c["rows"], c["cols"]), dtype=torch.float64, device=DEV)
        for r in range(0, c["rows"], 65536):
            out[r:r + 65536] = _values64(s["codes"][r:r + 65536], s["scales"][r:r + 65536])
        return out
    if c["op"] == "matmul":
        x = s["x"].double() if s["xs"] is None else _values64(s["x"], s["xs"])
        return x @ _values64(s["w"], s["ws"]).t()
    if c["op"] == "grouped":
        x = s["x"].double() if s["xs"] is None else _values64(s["x"], s["xs"])
        off, perm = s["offsets"].tolist(), s["perm"].long()
        n_out = c["N"] // 2 if c["swiglu"] else c["N"]
        out = torch.empty((c["T"] * c["k"], n_out), dtype=torch.float64, device=DEV)
        for e in range(c["E"]):
            r = perm[off[e]:off[e + 1]]
            if not len(r):
                continue
            v = x[r // c["k"]] @ _expert64(s["w"], s["ws"], e).t()
            if c["swiglu"]:
                v = v[:, :n_out] * torch.sigmoid(v[:, :n_out]) * v[:, n_out:]
            if c["gate"]:
                out[r] = v * s["gates"][r].double()[:, None]
            else:
                out[off[e]:off[e + 1]] = v
        return out
    I, b, four = c["I"], s["banks"], c["act"] == "mxfp4"
    x = s["x"].double()
    x = _nearest64(x) if four else x
    y = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device=DEV)
    for e in range(c["E"]):
        t, j = torch.nonzero(s["ids"][:c["valid"]] == e, as_tuple=True)
        if not len(t):
            continue
        v = x[t] @ _expert64(b["gate_up"], b.get("gate_up_scale"), e).t()
        h = v[:, :I] * torch.sigmoid(v[:, :I]) * v[:, I:]
        h = _nearest64(h) if four else h.to(torch.float32).to(torch.bfloat16).double()
        y[t] += s["gates"][t, j].double()[:, None] * (h @ _expert64(b["down"], b.get("down_scale"), e).t())
    return y
