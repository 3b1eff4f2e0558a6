"""The operators of the 4-bit floating-point and gated feed-forward paths: the
cases they are measured on, their plain forms and their values in 64 bits.

Formats (rows of e2m1 codes, two per byte, the even column in the low nibble):
  "mx"  blocks of 32 columns, scale 2^k, k = floor(log2(amax)) - 2 in -127..127,
        stored as the byte k + 127 (0 for a block of zeros);
  "nv"  blocks of 16 columns, scale s * g: g one fp32 number per matrix, s the
        e4m3 byte of fl(amax / fl(6 g)).
A code is v / d rounded to the nearest e2m1 value (ties to even, at most 6), d
the fp32 scale and the quotient rounded to fp32.  Scale bytes lie in tiles of
128 rows x 4 blocks: row r, block b at
  ((r // 128) * ceil(blocks / 4) + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4.
"""
import math

import torch

own = False

BLOCK = {"mx": 32, "nv": 16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a 7B attention weight taken to the MX grid, with its dequantized form for the loss
        {"name": "quantize_attn_weight", "op": "quantize", "fmt": "mx", "rows": 4096, "cols": 4096, "dtype": "f32", "pad": 0},
        # the activations into a down projection, an odd number of tokens, rows 8 elements apart
        {"name": "quantize_mlp_acts", "op": "quantize", "fmt": "nv", "rows": 2047, "cols": 11008, "dtype": "bf16", "pad": 8},
        # one token through a gate or up projection
        {"name": "matvec_token", "op": "matvec", "fmt": "mx", "batch": 1, "d_in": 4096, "d_out": 11008, "dtype": "bf16"},
        # eight sequences decoding through a down projection, fp32 vectors
        {"name": "matvec_batch8", "op": "matvec", "fmt": "nv", "batch": 8, "d_in": 11008, "d_out": 4096, "dtype": "f32"},
        # a short odd prompt through an attention projection, activations quantized in the call
        {"name": "linear_short", "op": "linear", "fmt": "nv", "tokens": 77, "d_in": 4096, "d_out": 4096},
        # a long prompt through a gate or up projection
        {"name": "linear_prompt", "op": "linear", "fmt": "mx", "tokens": 8192, "d_in": 4096, "d_out": 11008},
        # a small decode batch through the gated half of the MLP, 4-bit
        {"name": "gated_fp4_decode", "op": "gated_fp4", "fmt": "nv", "tokens": 16, "d": 4096, "f": 11008, "act": "silu"},
        # a prompt through it
        {"name": "gated_fp4_prompt", "op": "gated_fp4", "fmt": "mx", "tokens": 4096, "d": 4096, "f": 11008, "act": "silu"},
        # a few calibration tokens through the bf16 block
        {"name": "gated_few", "op": "gated", "tokens": 8, "d": 4096, "f": 11008, "act": "silu"},
        # a calibration batch through it
        {"name": "gated_calibration", "op": "gated", "tokens": 4096, "d": 4096, "f": 11008, "act": "silu"},
        # a ragged narrow block, its backward pass
        {"name": "backward_ragged", "op": "backward", "tokens": 333, "d": 1001, "f": 2730, "act": "gelu"},
        # the backward pass of a calibration batch
        {"name": "backward_calibration", "op": "backward", "tokens": 4096, "d": 4096, "f": 11008, "act": "silu"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantize", "matvec", "linear", "gated_fp4", "gated", "backward"))
    fmt, act = rng.choice(("mx", "nv")), rng.choice(("silu", "gelu"))
    if op == "quantize":
        return {"op": op, "fmt": fmt, "rows": _log(rng, 1, 4096), "cols": _log(rng, 40, 5500),
                "dtype": rng.choice(("f32", "bf16")), "pad": rng.choice((0, 1, 8))}
    if op == "matvec":
        return {"op": op, "fmt": fmt, "batch": rng.randint(1, 8), "d_in": _log(rng, 128, 11008),
                "d_out": _log(rng, 128, 11008), "dtype": rng.choice(("f32", "bf16"))}
    if op == "linear":
        return {"op": op, "fmt": fmt, "tokens": _log(rng, 1, 8192), "d_in": _log(rng, 128, 4096),
                "d_out": _log(rng, 128, 11008)}
    case = {"op": op, "tokens": _log(rng, 1, 4096), "d": _log(rng, 128, 4096), "f": _log(rng, 128, 11008), "act": act}
    if op == "gated_fp4":
        case["fmt"] = fmt
    return case


# ------------------------------------------------------------------ inputs

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _acts(gen, tokens, d):
    """Activations: normal values under per-channel gains, a few channels far above the others."""
    gain = torch.exp(0.5 * _normal(gen, d))
    gain = torch.where(torch.rand(d, generator=gen, device="cuda") < 0.01, 8 * gain, gain)
    return _normal(gen, tokens, d) * gain


def _padded(x, dtype, multiple, extra=0):
    """x as a view of rows `multiple` elements or a multiple of that apart (TMA wants 16 bytes)."""
    rows, cols = x.shape
    ld = -(-cols // multiple) * multiple + extra
    store = torch.zeros((rows, ld), dtype=dtype, device=x.device)
    store[:, :cols] = x
    return store[:, :cols]


def _round_e2m1(v):
    a = v.abs().clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign(torch.round(a / step) * step, v)


def _grid(m, fmt, g):
    """(e2m1 values, block scales fp32, scale bytes) of a matrix, in fp32."""
    rows, cols = m.shape
    bs = BLOCK[fmt]
    nb = -(-cols // bs)
    x = torch.nn.functional.pad(m.float(), (0, nb * bs - cols)).view(rows, nb, bs)
    amax = x.abs().amax(2)
    if fmt == "mx":
        k = (torch.frexp(amax)[1] - 3).clamp(-127, 127)
        k = torch.where(amax > 0, k, -127)
        byte = (k + 127).to(torch.uint8)
        scale = torch.ldexp(torch.ones_like(amax), k)
    else:
        s8 = torch.clamp(amax / (6.0 * g), max=448.0).to(torch.float8_e4m3fn)
        byte = s8.view(torch.uint8)
        scale = s8.float() * g
    q = torch.where(scale[..., None] > 0, x / scale[..., None], 0.0)
    return _round_e2m1(q), scale, byte


def _code_bytes(v, cols):
    """Packed codes of e2m1 values [rows, blocks, block]: rows padded to 32 codes."""
    rows = v.shape[0]
    v = v.reshape(rows, -1)
    v = torch.nn.functional.pad(v, (0, -(-cols // 32) * 32 - v.shape[1]))
    a = v.abs()
    mag = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4))
    code = mag.to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)
    return code[:, 0::2] | (code[:, 1::2] << 4)


def _tile_index(rows, nb, device):
    """Place of every scale byte [rows, nb] in the tiled layout."""
    r = torch.arange(rows, device=device)[:, None]
    b = torch.arange(nb, device=device)[None, :]
    return ((r // 128) * -(-nb // 4) + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4


def _tile_bytes(byte):
    rows, nb = byte.shape
    out = torch.zeros(-(-rows // 128) * -(-nb // 4) * 512, dtype=torch.uint8, device=byte.device)
    out[_tile_index(rows, nb, byte.device).reshape(-1)] = byte.reshape(-1)
    return out


def _weight(gen, rows, cols, fmt):
    """A quantized weight as a user's program holds it: codes, tiled scales, g."""
    w = 0.02 * _normal(gen, rows, cols)
    g = (w.abs().amax() / (6.0 * 448.0)).reshape(1) if fmt == "nv" else None
    v, _, byte = _grid(w, fmt, g)
    return {"rows": rows, "cols": cols, "codes": _code_bytes(v, cols), "scales": _tile_bytes(byte), "g": g}


def _bf16_weight(gen, rows, cols):
    return _padded(0.02 * _normal(gen, rows, cols), torch.bfloat16, 8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, fmt = case["op"], case.get("fmt")
    s = {"case": case, "info": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if op == "quantize":
        m = _acts(gen, case["rows"], case["cols"])
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        s["m"] = _padded(m, dt, 1, case["pad"])
        s["g"] = (s["m"].float().abs().amax() / (6.0 * 448.0)).reshape(1) if fmt == "nv" else None
        return s
    if op == "matvec":
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        s["x"] = _acts(gen, case["batch"], case["d_in"]).to(dt)
        s["w"] = _weight(gen, case["d_out"], case["d_in"], fmt)
        return s
    t, d = case["tokens"], case["d_in"] if op == "linear" else case["d"]
    s["x"] = _padded(_acts(gen, t, d), torch.bfloat16, 8)
    # the static scale of the activations, from calibration
    s["g"] = (s["x"].float().abs().amax() / (6.0 * 448.0)).reshape(1) if fmt == "nv" else None
    if op == "linear":
        s["w"] = _weight(gen, case["d_out"], d, fmt)
    elif op == "gated_fp4":
        s["w_gate"], s["w_up"] = _weight(gen, case["f"], d, fmt), _weight(gen, case["f"], d, fmt)
    else:
        s["w_gate"], s["w_up"] = _bf16_weight(gen, case["f"], d), _bf16_weight(gen, case["f"], d)
        if op == "backward":
            s["dh"] = _padded(0.01 * _normal(gen, t, case["f"]), torch.bfloat16, 8)
    return s


# ------------------------------------------------------------------ plain forms

def _unpacked(w, fmt):
    """The fp32 matrix that a quantized weight stands for."""
    rows, cols = w["rows"], w["cols"]
    code = torch.stack((w["codes"] & 15, w["codes"] >> 4), 2).reshape(rows, -1)[:, :cols].to(torch.int32)
    mag = code & 7
    v = torch.where(mag < 4, mag * 0.5, torch.where(mag < 6, mag - 2.0, mag * 2.0 - 8.0))
    v = torch.where(code > 7, -v, v)
    nb = -(-cols // BLOCK[fmt])
    byte = w["scales"][_tile_index(rows, nb, v.device)]
    if fmt == "mx":
        scale = torch.ldexp(torch.ones_like(byte, dtype=torch.float32), byte.to(torch.int32) - 127)
    else:
        scale = byte.view(torch.float8_e4m3fn).float() * w["g"]
    return v * scale.repeat_interleave(BLOCK[fmt], 1)[:, :cols]


def _quantized(m, fmt, g):
    """fp32 values of a matrix after quantization."""
    v, scale, _ = _grid(m, fmt, g)
    return (v * scale[..., None]).reshape(m.shape[0], -1)[:, :m.shape[1]]


_C = math.sqrt(2.0 / math.pi)


def _act(g, name):
    if name == "silu":
        return g / (1.0 + torch.exp(-g))
    return 0.5 * g * (1.0 + torch.tanh(_C * (g + 0.044715 * g * g * g)))


def _act_slope(g, name):
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return s * (1.0 + g * (1.0 - s))
    t = torch.tanh(_C * (g + 0.044715 * g * g * g))
    return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * _C * (1.0 + 3 * 0.044715 * g * g)


def _run_plain(s):
    case = s["case"]
    op, fmt, act = case["op"], case.get("fmt"), case.get("act")
    if op == "quantize":
        return _quantized(s["m"], fmt, s["g"])
    if op == "matvec":
        return (s["x"].float() @ _unpacked(s["w"], fmt).T).to(s["x"].dtype)
    if op == "linear":
        return (_quantized(s["x"], fmt, s["g"]) @ _unpacked(s["w"], fmt).T).bfloat16()
    if op == "gated_fp4":
        x = _quantized(s["x"], fmt, s["g"])
        g, u = x @ _unpacked(s["w_gate"], fmt).T, x @ _unpacked(s["w_up"], fmt).T
        return (_act(g, act) * u).bfloat16()
    x, wg, wu = s["x"].float(), s["w_gate"].float(), s["w_up"].float()
    g, u = x @ wg.T, x @ wu.T
    if op == "gated":
        return (_act(g, act) * u).bfloat16()
    dh = s["dh"].float()
    du, dg = dh * _act(g, act), dh * u * _act_slope(g, act)
    dx = dg @ wg + du @ wu
    return {k: v.bfloat16() for k, v in (("dG", dg), ("dU", du), ("dX", dx), ("dW_gate", dg.T @ x), ("dW_up", du.T @ x))}


# ------------------------------------------------------------------ the framework's calls

def _handle(P, w, fmt):
    """The weight's handle, made once as a program that serves it does."""
    if "handle" not in w:
        w["handle"] = P.Fp4Matrix(w["rows"], w["cols"], fmt, w["codes"], w["scales"], w["g"])
    return w["handle"]


def _run_own(s):
    import post_weight_quantization_syrk_b200 as P
    case = s["case"]
    op, fmt = case["op"], {"mx": P.KQ_FP4_MX, "nv": P.KQ_FP4_NV}.get(case.get("fmt"))
    act = {"silu": P.KQ_ACT_SILU, "gelu": P.KQ_ACT_GELU}.get(case.get("act"))
    info = s["info"]
    if op == "quantize":
        m = s["m"]
        m_hat = torch.empty(m.shape, dtype=torch.float32, device=m.device)
        P.kq_fp4_quantize(m, fmt, s["g"], M_hat=m_hat, info=info)
        return m_hat
    if op == "matvec":
        return P.kq_fp4_matvec(_handle(P, s["w"], fmt), s["x"])
    if op == "linear":
        return P.kq_fp4_gemm(P.kq_fp4_quantize(s["x"], fmt, s["g"], info=info), _handle(P, s["w"], fmt), info=info)
    if op == "gated_fp4":
        xq = P.kq_fp4_quantize(s["x"], fmt, s["g"], info=info)
        return P.kq_fp4_gated_ffn(xq, _handle(P, s["w_gate"], fmt), _handle(P, s["w_up"], fmt), act, info=info)
    if op == "gated":
        return P.kq_gated_ffn(s["x"], s["w_gate"], s["w_up"], act, info=info)
    dg, du, dx, dwg, dwu = P.kq_gated_ffn_backward(s["x"], s["w_gate"], s["w_up"], s["dh"], act, info=info)
    return {"dG": dg, "dU": du, "dX": dx, "dW_gate": dwg, "dW_up": dwu}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ work and 64-bit values

def _fp4_bytes(rows, cols, fmt):
    return rows * cols * (0.5 + 1.0 / BLOCK[fmt])


def work(case):
    op, fmt = case["op"], case.get("fmt")
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * ((4 if case["dtype"] == "f32" else 2) + 4) + _fp4_bytes(case["rows"], case["cols"], fmt),
                "flops": 0}
    if op == "matvec":
        e = 4 if case["dtype"] == "f32" else 2
        return {"bytes": _fp4_bytes(case["d_out"], case["d_in"], fmt) + e * case["batch"] * (case["d_in"] + case["d_out"]),
                "flops": 2.0 * case["batch"] * case["d_in"] * case["d_out"]}
    if op == "linear":
        t, k, n = case["tokens"], case["d_in"], case["d_out"]
        return {"bytes": 2 * t * (k + n) + _fp4_bytes(n, k, fmt), "flops": 2.0 * t * k * n}
    t, d, f = case["tokens"], case["d"], case["f"]
    if op == "gated_fp4":
        return {"bytes": 2 * t * (d + f) + 2 * _fp4_bytes(f, d, fmt), "flops": 4.0 * t * d * f}
    if op == "gated":
        return {"bytes": 2 * t * (d + f) + 4 * f * d, "flops": 4.0 * t * d * f}
    # X, dH and both weights read; dG, dU, dX and both weights' gradients written
    return {"bytes": 2 * t * (2 * d + 3 * f) + 8 * f * d, "flops": 12.0 * t * d * f}


_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# between two neighbours the tie goes to the even code: up at 0.75, 1.75 and 3.5
_TIES = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


def _nearest_e2m1(q):
    """Index 0..7 of the e2m1 magnitude nearest to |q| (fp64)."""
    n = torch.zeros(q.shape, dtype=torch.int64, device=q.device)
    a = q.abs()
    for i, t in enumerate(_TIES):
        n += (a >= t) if i % 2 else (a > t)
    return n


def _exact_values(m, fmt, g):
    """The quantized matrix in fp64; the roundings that the format defines (scale
    byte, fp32 scale, fp32 quotient) at their places."""
    rows, cols = m.shape
    bs = BLOCK[fmt]
    nb = -(-cols // bs)
    x = torch.zeros((rows, nb * bs), dtype=torch.float64, device=m.device)
    x[:, :cols] = m.double()
    x = x.view(rows, nb, bs)
    top = x.abs().max(dim=2, keepdim=True).values
    if fmt == "mx":
        k = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
        k = torch.where(torch.exp2(k) > top, k - 1, torch.where(torch.exp2(k + 1) <= top, k + 1, k)) - 2
        d = torch.where(top > 0, torch.exp2(k.clamp(-127, 127)), 1.0)
    else:
        r = (top / (6.0 * g.double()).float().double()).float().double().clamp(max=448.0)
        # e4m3: three mantissa bits down to 2^-6, steps of 2^-9 below
        step = torch.exp2(torch.floor(torch.log2(r.clamp(min=2.0 ** -6))) - 3)
        s = torch.round(r / step) * step
        d = (s * g.double()).float().double()
    q = torch.where(d > 0, (x / torch.where(d > 0, d, 1.0)).float().double(), 0.0)
    v = torch.tensor(_VALUES, dtype=torch.float64, device=m.device)[_nearest_e2m1(q)] * torch.sign(q)
    return (v * d).view(rows, -1)[:, :cols]


def _exact_weight(w, fmt):
    rows, cols = w["rows"], w["cols"]
    table = torch.tensor(_VALUES + tuple(-v for v in _VALUES), dtype=torch.float64, device=w["codes"].device)
    c = w["codes"].long()
    v = torch.empty((rows, 2 * c.shape[1]), dtype=torch.float64, device=c.device)
    v[:, 0::2], v[:, 1::2] = table[c % 16], table[c // 16]
    bs = BLOCK[fmt]
    nb = -(-cols // bs)
    tiles = w["scales"].view(-1, -(-nb // 4), 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, -(-nb // 4) * 4)[:rows, :nb].double()
    if fmt == "mx":
        scale = torch.exp2(tiles - 127)
    else:
        e, f = torch.floor(tiles / 8), tiles % 8
        s = torch.where(e > 0, torch.exp2(e - 7) * (1 + f / 8), torch.exp2(torch.full_like(e, -6.0)) * f / 8)
        scale = (s * w["g"].double()).float().double()
    return v[:, :cols] * scale.repeat_interleave(bs, dim=1)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    op, fmt, act = case["op"], case.get("fmt"), case.get("act")
    if op == "quantize":
        return _exact_values(s["m"], fmt, s["g"])
    if op == "matvec":
        return s["x"].double() @ _exact_weight(s["w"], fmt).T
    if op == "linear":
        return _exact_values(s["x"], fmt, s["g"]) @ _exact_weight(s["w"], fmt).T
    if op == "gated_fp4":
        x = _exact_values(s["x"], fmt, s["g"])
        a, b = x @ _exact_weight(s["w_gate"], fmt).T, x @ _exact_weight(s["w_up"], fmt).T
    else:
        x, wa, wb = s["x"].double(), s["w_gate"].double(), s["w_up"].double()
        a, b = x @ wa.T, x @ wb.T
    if act == "silu":
        sig = torch.sigmoid(a)
        val, slope = a * sig, sig + a * sig * (1 - sig)
    else:
        z = math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)
        val = a / 2 * (1 + torch.tanh(z))
        slope = (1 + torch.tanh(z)) / 2 + a / 2 / torch.cosh(z) ** 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * a ** 2)
    if op != "backward":
        return val * b
    dh = s["dh"].double()
    du, dg = dh * val, dh * b * slope
    return {"dG": dg, "dU": du, "dX": dg @ wa + du @ wb, "dW_gate": dg.T @ x, "dW_up": du.T @ x}
