"""Timed cases of the norm that feeds the FP8 products, of the 4-bit casts and of the FP4 x FP4 GEMMs.

With `own` false, run() computes each operator in plain torch operations in 32 bits; with `own`
true it makes the library's calls. Formats as in include/moe.h: e4m3 codes and UE8M0 bytes
(value 2^(b-127)) in uint8 tensors, E2M1 pairs with element 2i in the low nibble. FP8 rows carry
one scale per 128 columns in rows of 4*ceil(K/512) bytes, FP4 rows one per 32 in rows of K/32.

Codes and scales are returned as the numbers that they are: e4m3 and UE8M0 bytes as torch's types
of the same bits, E2M1 codes through the cast back.
"""
import math

import torch

own = False

# Work of the largest listed GEMM (M*N*K), of the largest listed norm (elements) and of the largest
# listed cast (bytes read), which no drawn case passes.
_GEMM_MNK = 4096 * 7168 * 18432
_NORM_ELEMENTS = 8192 * 7168
_CAST_BYTES = 36864 * 7168 * 4
_EPS = 1e-6


def listed():
    return [
        # one decode step: sixteen sequences' hidden states in front of the expert layer; latency alone
        dict(name="norm_decode", op="norm", R=16, C=7168, residual=True, normed=False, wf32=False),
        # a prefill's hidden states, residual stream read and written
        dict(name="norm_prefill", op="norm", R=8192, C=7168, residual=True, normed=False, wf32=False),
        # a small model's first norm: no residual yet, the bf16 rows wanted too, FP32 weights, an odd number of rows
        dict(name="norm_ragged", op="norm", R=4099, C=640, residual=False, normed=True, wf32=True),
        # rows as wide as the widest intermediate, every output
        dict(name="norm_wide", op="norm", R=515, C=18432, residual=True, normed=True, wf32=False),
        # a decode batch's activations on their way to a 4-bit product and back
        dict(name="cast_decode", op="cast", R=33, C=2048, f32=False),
        # a prefill's activations
        dict(name="cast_prefill", op="cast", R=8192, C=7168, f32=False),
        # FP32 master weights: the gate and up rows of one wide expert
        dict(name="cast_weights", op="cast", R=36864, C=7168, f32=True),
        # one logit per expert, FP32 out
        dict(name="gemm_gate", op="gemm", layout="dense", M=128, N=32, K=7168, G=1, f32=True),
        # a down projection during decoding: an odd batch against a matrix read once
        dict(name="gemm_decode", op="gemm", layout="dense", M=33, N=7168, K=2048, G=1, f32=False),
        # a prefill's projection: matrix-core bound
        dict(name="gemm_prefill", op="gemm", layout="dense", M=4096, N=7168, K=18432, G=1, f32=False),
        # gate and up rows of 8 experts over sorted tokens, ragged groups with padding rows
        dict(name="gemm_contiguous", op="gemm", layout="contiguous", M=8192, N=4096, K=7168, G=8, f32=False),
        # the same product while decoding: counts on the device, about 32 rows for each of 32 experts
        dict(name="gemm_masked", op="gemm", layout="masked", M=64, N=4096, K=7168, G=32, f32=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _log_of(rng, unit, lo, hi):
    return unit * _log(rng, max(1, lo // unit), max(1, hi // unit))


def draw(rng):
    op = rng.choice(("norm", "cast", "gemm", "gemm"))
    if op == "norm":
        C = _log_of(rng, 128, 128, 18432)
        return dict(op=op, R=_log(rng, 1, min(32768, _NORM_ELEMENTS // C)), C=C, residual=rng.random() < 0.7,
                    normed=rng.random() < 0.5, wf32=rng.random() < 0.5)
    if op == "cast":
        f32 = rng.random() < 0.5
        C = _log_of(rng, 32, 32, 18432)
        return dict(op=op, R=_log(rng, 1, min(65536, _CAST_BYTES // (C * (4 if f32 else 2)))), C=C, f32=f32)
    layout = rng.choice(("dense", "contiguous", "masked"))
    K = _log_of(rng, 128, 128, 18432)
    f32 = rng.random() < 0.3
    if layout == "masked":
        G = _log(rng, 2, 32)
        return dict(op=op, layout=layout, M=rng.randint(1, 128), N=_log_of(rng, 16, 16, min(8192, 32 * 4096 * 7168 // (G * K))),
                    K=K, G=G, f32=f32)
    G = 1 if layout == "dense" else _log(rng, 2, 16)
    M = _log(rng, 1 if G == 1 else 2 * G, 8192)
    return dict(op=op, layout=layout, M=M, N=_log_of(rng, 16, 16, min(8192, _GEMM_MNK // (G * M * K))), K=K, G=G, f32=f32)


def work(case):
    c = case
    if c["op"] == "norm":
        each = 2 + 1 + (4 if c["residual"] else 0) + (2 if c["normed"] else 0)
        return {"bytes": c["R"] * c["C"] * each + c["R"] * (c["C"] // 128) + c["C"] * (4 if c["wf32"] else 2), "flops": 4 * c["R"] * c["C"]}
    if c["op"] == "cast":
        # rows read, codes and scales written, and read, rows written
        return {"bytes": c["R"] * (2 * c["C"] * (4 if c["f32"] else 2) + 2 * (c["C"] // 2 + c["C"] // 32)), "flops": 2 * c["R"] * c["C"]}
    rows = c["M"] * c["G"] // 2 if c["layout"] == "masked" else c["M"]
    return {"bytes": (rows + c["G"] * c["N"]) * (c["K"] // 2 + c["K"] // 32) + rows * c["N"] * (4 if c["f32"] else 2),
            "flops": 2 * rows * c["N"] * c["K"]}


# ---------------------------------------------------------------------------- inputs


def _exponent(amax, mantissa, exponent):
    """The least s with amax <= mantissa * 2^(exponent + s), mantissa in [1, 2); 0 for amax 0."""
    m, e = torch.frexp(amax)
    s = e - 1 - exponent + (2 * m > mantissa).to(e.dtype)
    return torch.where(amax == 0, torch.zeros_like(s), s)


def _e2m1(v):
    """v rounded to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 with v's sign, ties to even codes."""
    step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0)).to(v.dtype)
    return torch.round(v / step) * step


def _fp4_rows(x):
    """Rows as E2M1 pairs with one UE8M0 byte per 1x32 block."""
    R, K = x.shape
    b = x.view(R, K // 32, 32)
    s = _exponent(b.abs().amax(-1), 1.5, 2).clamp(min=-127)
    v = _e2m1(torch.ldexp(b, -s.unsqueeze(-1))).view(R, K)
    a = v.abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)
    return code[:, 0::2] | (code[:, 1::2] << 4), (s + 127).to(torch.uint8)


def _inputs(c, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    if c["op"] == "norm":
        # a residual stream a few times the layer's output, some of its channels much larger than the others
        s = dict(x=normal(c["R"], c["C"]).to(torch.bfloat16), weight=1 + 0.1 * normal(c["C"]))
        if not c["wf32"]:
            s["weight"] = s["weight"].to(torch.bfloat16)
        if c["residual"]:
            channel = torch.where(torch.rand(c["C"], generator=g, device=dev) < 0.01, 30.0, 3.0)
            s["residual"] = (normal(c["R"], c["C"]) * channel).to(torch.bfloat16)
        return s
    if c["op"] == "cast":
        if c["f32"]:
            return dict(x=normal(c["R"], c["C"]) * 0.02)
        return dict(x=normal(c["R"], c["C"]).to(torch.bfloat16))
    M, N, K, G = c["M"], c["N"], c["K"], c["G"]
    rows = G * M if c["layout"] == "masked" else M
    a, a_sf = _fp4_rows(normal(rows, K))
    b = torch.empty(G, N, K // 2, dtype=torch.uint8, device=dev)
    b_sf = torch.empty(G, N, K // 32, dtype=torch.uint8, device=dev)
    for i in range(G):
        b[i], b_sf[i] = _fp4_rows(normal(N, K) * 0.02)
    s = dict(a=a, a_sf=a_sf, b=b, b_sf=b_sf)
    if c["layout"] == "contiguous":
        # G sorted segments of random length, each followed by up to 127 padding rows
        cut = torch.randint(0, M + 1, (G - 1,), generator=g, device=dev).sort().values
        group = (torch.arange(M, device=dev)[:, None] >= cut[None, :]).sum(1)
        end = torch.cat((cut, torch.tensor([M], device=dev)))[group]
        pad = torch.randint(0, min(128, M // (2 * G) + 1), (G,), generator=g, device=dev)[group]
        s["group"] = torch.where(torch.arange(M, device=dev) < end - pad, group, -1).to(torch.int32)
    elif c["layout"] == "masked":
        # counts about half the capacity, from a quarter to three quarters
        s["count"] = torch.randint(M // 4, max(1, 3 * M // 4) + 1, (G,), generator=g, device=dev).to(torch.int32)
    return s


def prepare(case, seed):
    c = case
    s = _inputs(c, seed)
    s["case"] = c
    dev = "cuda"
    if c["op"] == "norm":
        s["q"] = torch.empty(c["R"], c["C"], dtype=torch.uint8, device=dev)
        s["sf"] = torch.empty(c["R"], 4 * ((c["C"] + 511) // 512), dtype=torch.uint8, device=dev)
        s["normed"] = torch.empty_like(s["x"]) if c["normed"] else None
        s["sum"] = torch.empty_like(s["x"]) if c["residual"] else None
    elif c["op"] == "cast":
        s["q"] = torch.empty(c["R"], c["C"] // 2, dtype=torch.uint8, device=dev)
        s["sf"] = torch.empty(c["R"], c["C"] // 32, dtype=torch.uint8, device=dev)
        s["back"] = torch.empty_like(s["x"])
    else:
        rows = s["a"].shape[0]
        # rows that belong to no group are not written: they keep these zeros
        s["d"] = torch.zeros(rows, c["N"], dtype=torch.float32 if c["f32"] else torch.bfloat16, device=dev)
        if own:
            # what a program sets up once: packed weights and a workspace
            import block_scaled_fp8_dispatch_amd as moe
            s["packed"] = torch.empty(moe.moe_gemm_packed_b_bytes(c["G"], c["N"], c["K"]), dtype=torch.uint8, device=dev)
            moe.moe_gemm_prepare_b(c["G"], c["N"], c["K"], s["b"], s["b_sf"], s["packed"])
            s["ws"] = torch.empty(moe.moe_fp4_gemm_workspace_bytes(rows, c["G"]), dtype=torch.uint8, device=dev)
    return s


# ---------------------------------------------------------------------------- the library's calls


def _own_run(s):
    import block_scaled_fp8_dispatch_amd as moe
    c = s["case"]
    if c["op"] == "norm":
        moe.moe_rmsnorm_to_fp8(s["q"], s["sf"], s["normed"], s["sum"], s["x"], s.get("residual"), s["weight"],
                               moe.MOE_F32 if c["wf32"] else moe.MOE_BF16, c["R"], c["C"], _EPS)
        out = {"codes": s["q"].view(torch.float8_e4m3fn), "scales": s["sf"].view(torch.float8_e8m0fnu)}
        if c["normed"]:
            out["normed"] = s["normed"]
        if c["residual"]:
            out["sum"] = s["sum"]
        return out
    if c["op"] == "cast":
        ty = moe.MOE_F32 if c["f32"] else moe.MOE_BF16
        moe.moe_cast_to_fp4(s["x"], ty, c["R"], c["C"], s["q"], s["sf"])
        moe.moe_cast_from_fp4(s["q"], s["sf"], c["R"], c["C"], s["back"], ty)
        return {"values": s["back"], "scales": s["sf"].view(torch.float8_e8m0fnu)}
    d_type = moe.MOE_F32 if c["f32"] else moe.MOE_BF16
    M, N, K, G = c["M"], c["N"], c["K"], c["G"]
    if c["layout"] == "dense":
        moe.moe_fp4_gemm(s["d"], d_type, s["a"], s["a_sf"], M, N, K, s["packed"], s["ws"])
    elif c["layout"] == "contiguous":
        moe.moe_m_grouped_fp4_gemm_contiguous(s["d"], d_type, s["a"], s["a_sf"], s["group"], M, G, N, K, s["packed"], s["ws"])
    else:
        moe.moe_m_grouped_fp4_gemm_masked(s["d"], d_type, s["a"], s["a_sf"], s["count"], G, M, (M + 1) // 2, N, K, s["packed"],
                                          s["ws"])
    return {"d": s["d"]}


# ---------------------------------------------------------------------------- plain forms


def _plain_norm(s):
    c = s["case"]
    R, C = c["R"], c["C"]
    h = s["x"].float()
    if c["residual"]:
        h = h + s["residual"].float()
    n = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + _EPS) * s["weight"].float()
    b = n.view(R, C // 128, 128)
    e = _exponent(b.abs().amax(-1), 1.75, 8).clamp(min=-127)
    codes = torch.ldexp(b, -e.unsqueeze(-1)).view(R, C).to(torch.float8_e4m3fn)
    sf = torch.zeros(R, 4 * ((C + 511) // 512), dtype=torch.uint8, device=h.device)
    sf[:, : C // 128] = (e + 127).to(torch.uint8)
    out = {"codes": codes, "scales": sf.view(torch.float8_e8m0fnu)}
    if c["normed"]:
        out["normed"] = n.to(torch.bfloat16)
    if c["residual"]:
        out["sum"] = h.to(torch.bfloat16)
    return out


def _plain_cast(s):
    c = s["case"]
    R, C = c["R"], c["C"]
    b = s["x"].float().view(R, C // 32, 32)
    e = _exponent(b.abs().amax(-1), 1.5, 2).clamp(min=-127)
    values = torch.ldexp(_e2m1(torch.ldexp(b, -e.unsqueeze(-1))), e.unsqueeze(-1)).view(R, C)
    return {"values": values.to(s["x"].dtype), "scales": (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)}


def _plain_fp4(packed, sf):
    """E2M1 pairs [..., K/2] times their 1x32 scales: [..., K]."""
    half = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=packed.device)
    value = torch.cat((half, -half))
    byte = torch.arange(256, device=packed.device)
    pairs = torch.stack((value[byte & 15], value[byte >> 4]), dim=-1)
    v = pairs[packed.int()].view(*packed.shape[:-1], sf.shape[-1], 32)
    return (v * torch.exp2(sf.float() - 127.0).unsqueeze(-1)).view(*packed.shape[:-1], -1)


def _plain_gemm(s):
    c = s["case"]
    G, M, N, K = c["G"], c["M"], c["N"], c["K"]
    a, b = _plain_fp4(s["a"], s["a_sf"]), _plain_fp4(s["b"], s["b_sf"])
    if c["layout"] == "dense":
        d = a @ b[0].t()
    elif c["layout"] == "contiguous":
        every = (a @ b.view(G * N, K).t()).view(M, G, N)
        d = every[torch.arange(M, device=a.device), s["group"].clamp(min=0).long()]
        d = torch.where(s["group"][:, None] >= 0, d, 0.0)
    else:
        d = torch.matmul(b, a.view(G, M, K).transpose(1, 2).contiguous()).transpose(1, 2)
        d = torch.where(torch.arange(M, device=a.device)[None, :, None] < s["count"][:, None, None], d, 0.0)
    return {"d": d.reshape(s["d"].shape).to(s["d"].dtype)}


def run(state):
    if own:
        return _own_run(state)
    return {"norm": _plain_norm, "cast": _plain_cast, "gemm": _plain_gemm}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------- 64-bit values


def _least_exponent(amax, largest):
    """The least integer s with amax <= largest * 2^s, 0 for amax 0, from logarithms; not below -127."""
    s = torch.ceil(torch.log2(amax / largest))
    s = s + (amax > largest * torch.exp2(s)).to(s.dtype) - (amax <= largest * torch.exp2(s - 1)).to(s.dtype)
    return torch.where(amax == 0, 0.0, s).clamp(min=-127)


def exact(case, seed):
    c = case
    s = _inputs(c, seed)
    f64 = torch.float64
    if c["op"] == "norm":
        R, C = c["R"], c["C"]
        h = s["x"].to(f64)
        if c["residual"]:
            h = h + s["residual"].to(f64)
        n = h / torch.sqrt((h * h).sum(-1, keepdim=True) / C + _EPS) * s["weight"].to(f64)
        e = _least_exponent(n.view(R, C // 128, 128).abs().amax(-1), 448.0)
        # the numbers before their last rounding: to e4m3 for the codes, to bf16 for the rows
        out = {"codes": n * torch.exp2(-e).repeat_interleave(128, dim=1),
               "scales": torch.nn.functional.pad(torch.exp2(e), (0, (-(C // 128)) % 4), value=2.0 ** -127)}
        if c["normed"]:
            out["normed"] = n
        if c["residual"]:
            out["sum"] = h
        return out
    if c["op"] == "cast":
        R, C = c["R"], c["C"]
        x = s["x"].to(f64).view(R, C // 32, 32)
        scale = torch.exp2(_least_exponent(x.abs().amax(-1, keepdim=True), 6.0))
        v = x / scale
        # the nearest of the eight magnitudes: how many midpoints lie below (a midpoint goes to the even code)
        a = v.abs()
        code = (a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int() + (a >= 3.5).int() + (a > 5.0).int()
        magnitude = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=f64, device=x.device)[code]
        return {"values": (torch.where(v < 0, -magnitude, magnitude) * scale).view(R, C), "scales": scale.view(R, C // 32)}
    # E2M1 values from their bit fields
    n4 = torch.arange(16, device="cuda")
    ex, man = ((n4 >> 1) & 3).to(f64), (n4 & 1).to(f64)
    e2m1 = torch.where(ex == 0, man / 2, (1 + man / 2) * torch.exp2(ex - 1))
    e2m1 = torch.where(n4 >= 8, -e2m1, e2m1)

    def fp4(packed, sf):
        v = torch.stack((e2m1[(packed & 15).int()], e2m1[(packed >> 4).int()]), dim=-1).flatten(-2)
        return v * torch.exp2(sf.to(f64) - 127).repeat_interleave(32, dim=-1)

    a = fp4(s["a"], s["a_sf"])
    d = torch.zeros(a.shape[0], c["N"], dtype=f64, device=a.device)
    for i in range(c["G"]):
        if c["layout"] == "dense":
            rows = torch.arange(c["M"], device=a.device)
        elif c["layout"] == "contiguous":
            rows = torch.nonzero(s["group"] == i)[:, 0]
        else:
            rows = i * c["M"] + torch.arange(int(s["count"][i]), device=a.device)
        d[rows] = a[rows] @ fp4(s["b"][i], s["b_sf"][i]).t()
    return {"d": d}
