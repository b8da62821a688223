"""Cases of the low-precision linear layer: RMS norm (forward, with the
residual's addition and a quantised output, and backward), microscaled
quantisation, and the product of microscaled operands.

``run`` computes a case in its plain form (elementary torch operations in 32
bits) or, where ``own`` is true, through the library's entry points.

Formats (codes along K, one scale per block):
  mxfp8  e4m3 codes, blocks of 32, power-of-two scales (one exponent byte)
  mxfp4  e2m1 codes, blocks of 32, power-of-two scales
  nvfp4  e2m1 codes, blocks of 16, e4m3 scales, and one fp32 scale a tensor
Two 4-bit codes share a byte, the earlier one in the low half.  A row of codes
is padded with zeros to a multiple of 32 values.  Scale (row r, block b) is byte
(r % 32) * 16 + (r % 128 // 32) * 4 + b % 4 of the 512-byte tile
[r // 128][b // 4]; the padding of the last tiles is zero.
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BLOCK = {"mxfp8": 32, "mxfp4": 32, "nvfp4": 16}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_EPS = 1e-6


# ------------------------------------------------------------------ cases

def _norm(name, rows, cols, dtype="bf16", out="mxfp8", residual=True):
    return {"name": name, "op": "norm", "rows": rows, "cols": cols, "dtype": dtype, "out": out,
            "residual": residual}


def _norm_bwd(name, rows, cols, dtype="bf16", residual=True):
    return {"name": name, "op": "norm_bwd", "rows": rows, "cols": cols, "dtype": dtype,
            "residual": residual}


def _quant(name, rows, cols, fmt, dtype="bf16", transposed=False):
    return {"name": name, "op": "quant", "rows": rows, "cols": cols, "fmt": fmt, "dtype": dtype,
            "transposed": transposed}


def _gemm(name, m, n, k, fmt, act="none", with_c=False, dtype="bf16"):
    return {"name": name, "op": "gemm", "m": m, "n": n, "k": k, "fmt": fmt, "act": act,
            "with_c": with_c, "dtype": dtype}


def listed():
    return [
        # one decoding step of a small batch: the residual stream's norm, latency only
        _norm("norm mxfp8 8x4096", 8, 4096),
        # the norm before a layer's first product, over a long prompt or a training batch
        _norm("norm mxfp8 16384x8192", 16384, 8192),
        # a first layer without a residual, 16-bit output, sizes that fill no vector evenly
        _norm("norm f16 4099x1999", 4099, 1999, dtype="f16", out="16", residual=False),
        # training: gradient of the norm and of the residual stream around it
        _norm_bwd("norm bwd 16384x4096", 16384, 4096),
        # the same for a short, ragged last batch
        _norm_bwd("norm bwd 257x1536", 257, 1536, dtype="f16", residual=False),
        # the weights (or a prompt's activations) of an 8192-wide layer to 4 bits
        _quant("quant nvfp4 8192x8192", 8192, 8192, "nvfp4"),
        # weight gradient: token-major activations quantised along the tokens
        _quant("quant mxfp8 t 4096x32768", 4096, 32768, "mxfp8", transposed=True),
        # a small batch's activations between two products
        _quant("quant mxfp4 64x1544", 64, 1544, "mxfp4"),
        # prefill / training of an 8192-wide layer in 4 bits: the tensor core's rate
        _gemm("gemm nvfp4 8192", 8192, 8192, 8192, "nvfp4"),
        # the 8-bit layer with its residual-like input and activation, both outputs
        _gemm("gemm mxfp8 4096 gelu", 4096, 4096, 4096, "mxfp8", act="gelu_tanh", with_c=True),
        # decoding: 16 tokens against 4-bit weights, bound by the weights' bytes
        _gemm("gemm nvfp4 16x8192x8192", 16, 8192, 8192, "nvfp4"),
        # a ragged batch and sizes that end inside tiles
        _gemm("gemm mxfp4 1000x1544x2080", 1000, 1544, 2080, "mxfp4", act="silu"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "norm_bwd", "quant", "gemm"))
    dtype = rng.choice(("bf16", "f16"))
    if op == "norm":
        c = _norm("", _log(rng, 1, 16384), _log(rng, 64, 8192), dtype, rng.choice(("mxfp8", "16")),
                  rng.random() < 0.7)
    elif op == "norm_bwd":
        c = _norm_bwd("", _log(rng, 1, 16384), _log(rng, 64, 8192), dtype, rng.random() < 0.7)
    elif op == "quant":
        cols = _log(rng, 32, 32768)
        c = _quant("", _log(rng, 1, min(8192, (1 << 27) // cols)), cols, rng.choice(tuple(_BLOCK)),
                   dtype, rng.random() < 0.4)
    else:
        c = _gemm("", _log(rng, 1, 8192), 8 * _log(rng, 8, 1024), _log(rng, 64, 8192),
                  rng.choice(tuple(_BLOCK)), rng.choice(("none", "gelu_tanh", "silu")),
                  rng.random() < 0.3, dtype)
    del c["name"]
    return c


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["rows"] * c["cols"]
        moved = 2 * n + (4 * n if c["residual"] else 0) + 2 * c["cols"] + 4 * c["rows"] + 2 * n
        if c["out"] == "mxfp8":
            moved += n + n / 32
        return {"bytes": moved, "flops": 8 * n}
    if c["op"] == "norm_bwd":
        n = c["rows"] * c["cols"]
        return {"bytes": (8 if c["residual"] else 6) * n + 6 * c["cols"] + 4 * c["rows"],
                "flops": 10 * n}
    if c["op"] == "quant":
        n = c["rows"] * c["cols"]
        return {"bytes": 4 * n + _code_bytes(c["fmt"]) * n, "flops": 3 * n}
    m, n, k = c["m"], c["n"], c["k"]
    outs = 2 * m * n * (1 + (c["act"] != "none") + c["with_c"])
    return {"bytes": _code_bytes(c["fmt"]) * (m + n) * k + outs, "flops": 2 * m * n * k}


def _code_bytes(fmt):
    return (1.0 if fmt == "mxfp8" else 0.5) + 1.0 / _BLOCK[fmt]


# ----------------------------------------------------------------- inputs

def _activations(gen, rows, cols, dtype):
    """A residual stream: normal values whose channels differ in size, a few by a lot."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    gain = torch.exp(0.5 * torch.randn(cols, generator=gen, device="cuda"))
    gain = torch.where(torch.rand(cols, generator=gen, device="cuda") < 0.002, gain * 20.0, gain)
    return (x * gain).to(_DT[dtype])


def _codes_and_scales(x, fmt):
    """Codes (rows, padded bytes), scale tiles and tensor scale of a matrix, in plain torch."""
    code, scale, t = _quantise(x.float(), fmt, _tensor_scale(x, fmt))
    rows, cols = x.shape
    pad = -cols % 32
    if fmt == "mxfp8":
        raw = code.to(torch.float8_e4m3fn).view(torch.uint8)
        raw = torch.nn.functional.pad(raw, (0, pad))
        s = (torch.frexp(scale)[1] - 1 + 127).to(torch.uint8)
    else:
        low = code.abs()
        raw = torch.zeros(rows, cols, dtype=torch.uint8, device=x.device)
        for i, v in enumerate(_E2M1):
            raw += (low == v).to(torch.uint8) * i
        raw += (code < 0).to(torch.uint8) * 8
        raw = torch.nn.functional.pad(raw, (0, pad))
        raw = raw[:, 0::2] | (raw[:, 1::2] << 4)
        if fmt == "mxfp4":
            s = (torch.frexp(scale)[1] - 1 + 127).to(torch.uint8)
        else:
            s = scale.to(torch.float8_e4m3fn).view(torch.uint8)
    s = torch.nn.functional.pad(s, (0, -s.shape[1] % 4, 0, -rows % 128))
    s = s.view(s.shape[0] // 128, 4, 32, s.shape[1] // 4, 4).permute(0, 3, 2, 1, 4)
    return {"codes": raw.contiguous(), "scales": s.contiguous().view(-1), "tensor_scale": t,
            "rows": rows, "cols": cols, "fmt": fmt}


def _tensor_scale(x, fmt):
    if fmt != "nvfp4":
        return None
    return (x.abs().max().float() / (448.0 * 6.0)).clamp_min(1e-30).reshape(1)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": c}
    if c["op"] == "norm":
        dt = _DT[c["dtype"]]
        s["x"] = _activations(gen, c["rows"], c["cols"], c["dtype"])
        s["residual"] = _activations(gen, c["rows"], c["cols"], c["dtype"]) if c["residual"] else None
        s["weight"] = (1.0 + 0.2 * torch.randn(c["cols"], generator=gen, device="cuda")).to(dt)
    elif c["op"] == "norm_bwd":
        dt = _DT[c["dtype"]]
        s["h"] = _activations(gen, c["rows"], c["cols"], c["dtype"])
        s["inv"] = torch.rsqrt(s["h"].float().square().mean(1) + _EPS)
        s["weight"] = (1.0 + 0.2 * torch.randn(c["cols"], generator=gen, device="cuda")).to(dt)
        g = torch.randn(c["rows"], c["cols"], generator=gen, device="cuda")
        s["dy"] = (g * 0.1).to(dt)
        s["dh"] = None
        if c["residual"]:
            s["dh"] = (torch.randn(c["rows"], c["cols"], generator=gen, device="cuda") * 0.1).to(dt)
    elif c["op"] == "quant":
        if c["transposed"]:   # stored token-major; the operand's K runs along the tokens
            s["x"] = _activations(gen, c["cols"], c["rows"], c["dtype"]).t()
        else:
            s["x"] = _activations(gen, c["rows"], c["cols"], c["dtype"])
        s["tensor_scale"] = _tensor_scale(s["x"], c["fmt"])
    else:
        m, n, k = c["m"], c["n"], c["k"]
        s["A"] = _codes_and_scales(_activations(gen, m, k, "bf16"), c["fmt"])
        w = torch.randn(n, k, generator=gen, device="cuda") / math.sqrt(k)
        s["B"] = _codes_and_scales(w.bfloat16(), c["fmt"])
        s["C"] = None
        if c["with_c"]:
            s["C"] = torch.randn(m, n, generator=gen, device="cuda").to(_DT[c["dtype"]])
    return s


# -------------------------------------------------------------- plain form

def _blocks(x, fmt):
    size = _BLOCK[fmt]
    x = torch.nn.functional.pad(x, (0, -x.shape[1] % size))
    return x.view(x.shape[0], -1, size)


def _pow2(e):
    """2^e in fp32 for whole e in [-127, 127], from its bits."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _quantise(x, fmt, t):
    """Code values (rows, cols) and scales (rows, blocks) of fp32 x, without the tensor scale t."""
    rows, cols = x.shape
    v = _blocks(x, fmt)
    amax = v.abs().amax(2)
    if fmt == "nvfp4":
        scale = (amax / (6.0 * t)).clamp(2.0 ** -9, 448.0).to(torch.float8_e4m3fn).float()
        v = v * (1.0 / (scale * t)).unsqueeze(2)
    else:
        mant, exp = torch.frexp(amax)
        if fmt == "mxfp8":       # 448 = 0.875 * 2^9
            exp = exp - 9 + (mant > 0.875)
        else:                    # 6 = 0.75 * 2^3
            exp = exp - 3 + (mant > 0.75)
        exp = torch.where(amax > 0, exp, -127).clamp(-127, 127)
        scale = _pow2(exp)
        v = v * _pow2(-exp).unsqueeze(2)
    if fmt == "mxfp8":
        code = v.to(torch.float8_e4m3fn).float()
    else:
        a = v.abs()
        code = 0.5 * ((a > 0.25).float() + (a >= 0.75).float() + (a > 1.25).float() +
                      (a >= 1.75).float()) + (a > 2.5).float() + (a >= 3.5).float() + \
            2.0 * (a > 5.0).float()
        code = torch.where(v < 0, -code, code)
    return code.reshape(rows, -1)[:, :cols], scale, t


def _values(x, fmt, t):
    code, scale, _ = _quantise(x, fmt, t)
    v = (_blocks(code, fmt) * scale.unsqueeze(2)).reshape(x.shape[0], -1)[:, :x.shape[1]]
    return v if t is None else v * t


def _untile(s, rows, blocks):
    tiles = s.view((rows + 127) // 128, (blocks + 3) // 4, 32, 4, 4).permute(0, 3, 2, 1, 4)
    return tiles.reshape(tiles.shape[0] * 128, -1)[:rows, :blocks]


def _decode(q, dtype=torch.float32):
    """The values of an operand without its tensor scale."""
    rows, cols, fmt = q["rows"], q["cols"], q["fmt"]
    size = _BLOCK[fmt]
    blocks = (cols + size - 1) // size
    if fmt == "mxfp8":
        code = q["codes"].view(torch.float8_e4m3fn).to(dtype)
    else:
        table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=dtype, device=q["codes"].device)
        raw = q["codes"].int()
        code = torch.stack((table[raw & 15], table[raw >> 4]), 2).reshape(rows, -1)
    s = _untile(q["scales"], rows, blocks)
    if fmt == "nvfp4":
        s = s.contiguous().view(torch.float8_e4m3fn).to(dtype)
    else:
        s = _pow2(s.int() - 127).to(dtype)
    return (_blocks(code[:, :cols], fmt) * s.unsqueeze(2)).reshape(rows, -1)[:, :cols]


def _act(v, act):
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    return v


def _run_plain(s):
    c = s["case"]
    if c["op"] == "norm":
        dt = s["x"].dtype
        out = {}
        h = s["x"].float()
        if s["residual"] is not None:
            out["h"] = (h + s["residual"].float()).to(dt)
            h = out["h"].float()
        inv = 1.0 / torch.sqrt((h * h).mean(1) + _EPS)
        y = h * inv.unsqueeze(1) * s["weight"].float()
        out["inv"] = inv
        if c["out"] == "mxfp8":
            out["y"] = _values(y, "mxfp8", None).to(torch.bfloat16)
        else:
            out["y"] = y.to(dt)
        return out
    if c["op"] == "norm_bwd":
        dt = s["h"].dtype
        h, dy, inv = s["h"].float(), s["dy"].float(), s["inv"].unsqueeze(1)
        g = dy * s["weight"].float()
        dh = inv * (g - h * ((g * h).mean(1, keepdim=True) * inv * inv))
        if s["dh"] is not None:
            dh = dh + s["dh"].float()
        return {"dx": dh.to(dt), "dw": (dy * (h * inv)).sum(0)}
    if c["op"] == "quant":
        return {"values": _values(s["x"].float(), c["fmt"], s["tensor_scale"]).to(torch.bfloat16)}
    A, B = s["A"], s["B"]
    v = _decode(A) @ _decode(B).t()
    if A["tensor_scale"] is not None:
        v = v * (A["tensor_scale"] * B["tensor_scale"])
    if s["C"] is not None:
        v = v + 0.5 * s["C"].float()
    dt = _DT[c["dtype"]]
    out = {"D": v.to(dt)}
    if c["act"] != "none":
        out["P"] = _act(v, c["act"]).to(dt)
    return out


# ------------------------------------------------------------ the library

def _run_own(s):
    from grouped_gemm_epilogues_gb300 import binding as gge

    c = s["case"]
    if c["op"] == "norm":
        x = s["x"]
        rows, cols = x.shape
        out = {"inv": torch.empty(rows, dtype=torch.float32, device=x.device)}
        if s["residual"] is not None:
            out["h"] = torch.empty_like(x)
        q = values = y = None
        if c["out"] == "mxfp8":
            q = gge.mx_empty(rows, cols, "mxfp8", device=x.device)
            out["y"] = values = torch.empty(rows, cols, dtype=torch.bfloat16, device=x.device)
        else:
            out["y"] = y = torch.empty_like(x)
        gge.gge_rmsnorm(x, s["weight"], residual=s["residual"], residual_out=out.get("h"), Y=y,
                        Q=q, values=values, inv_rms=out["inv"], eps=_EPS)
        return out
    if c["op"] == "norm_bwd":
        out = {"dx": torch.empty_like(s["h"]),
               "dw": torch.empty(c["cols"], dtype=torch.float32, device=s["h"].device)}
        gge.gge_rmsnorm_bwd(s["dy"], s["h"], s["weight"], s["inv"], out["dx"], dW=out["dw"],
                            dH=s["dh"])
        return out
    if c["op"] == "quant":
        x = s["x"]
        q = gge.mx_empty(c["rows"], c["cols"], c["fmt"], device=x.device,
                         tensor_scale=s["tensor_scale"])
        values = torch.empty(c["rows"], c["cols"], dtype=torch.bfloat16, device=x.device)
        gge.gge_mx_quantize(x, q, values=values)
        return {"values": values}
    ops = [gge.MxTensor(q["codes"], q["scales"], q["fmt"], q["rows"], q["cols"],
                        tensor_scale=q["tensor_scale"]) for q in (s["A"], s["B"])]
    out = {"D": torch.empty(c["m"], c["n"], dtype=_DT[c["dtype"]], device=ops[0].codes.device)}
    if c["act"] != "none":
        out["P"] = torch.empty_like(out["D"])
    gge.gge_gemm_mx(ops[0], ops[1], D=out["D"], PostAct=out.get("P"), act=c["act"], C=s["C"],
                    alpha=1.0, beta=0.5 if c["with_c"] else 0.0)
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------- 64-bit definition

def _nearest(v, levels):
    """v >= 0 to the nearest of the ascending levels; halfway goes to the even index."""
    lv = torch.tensor(levels, dtype=torch.float64, device=v.device)
    hi = torch.searchsorted(lv, v.contiguous()).clamp(1, len(levels) - 1)
    lo = hi - 1
    below, above = v - lv[lo], lv[hi] - v
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return lv[torch.where(up, hi, lo)]


def _e4m3_levels():
    return [m * 2.0 ** -9 for m in range(8)] + \
        [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)
         if not (e == 15 and m == 7)]


def _exact_values(x, fmt, t):
    rows, cols = x.shape
    size = _BLOCK[fmt]
    out = torch.zeros(rows, (cols + size - 1) // size * size, dtype=torch.float64, device=x.device)
    out[:, :cols] = x
    b = out.view(rows, -1, size)
    amax = b.abs().max(2).values
    if fmt == "nvfp4":
        unit = _nearest((amax / 6.0 / t).clamp(2.0 ** -9, 448.0), _e4m3_levels()) * t
    else:
        top = 448.0 if fmt == "mxfp8" else 6.0
        unit = torch.exp2(torch.ceil(torch.log2(amax / top)).clamp(-127, 127))
    unit = unit.unsqueeze(2)
    code = _nearest((b / unit).abs(), _e4m3_levels() if fmt == "mxfp8" else list(_E2M1))
    return (code * unit * torch.sign(b)).view(rows, -1)[:, :cols]


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "norm":
        h = s["x"].double()
        out = {}
        if s["residual"] is not None:
            out["h"] = (h + s["residual"].double()).to(s["x"].dtype).double()
            h = out["h"]
        ms = torch.einsum("tc,tc->t", h, h) / c["cols"]
        out["inv"] = (ms + _EPS) ** -0.5
        y = h * torch.outer(out["inv"], s["weight"].double())
        out["y"] = _exact_values(y, "mxfp8", None) if c["out"] == "mxfp8" else y
        return out
    if c["op"] == "norm_bwd":
        # through the Jacobian of h / rms(h): (I - n n^T / C) / rms, n = h inv
        n = s["h"].double() * s["inv"].double()[:, None]
        dy = s["dy"].double()
        u = dy * s["weight"].double()
        along = torch.einsum("tc,tc->t", u, n) / c["cols"]
        dx = (u - n * along[:, None]) * s["inv"].double()[:, None]
        if s["dh"] is not None:
            dx = dx + s["dh"].double()
        return {"dx": dx, "dw": torch.einsum("tc,tc->c", dy, n)}
    if c["op"] == "quant":
        t = s["tensor_scale"].double() if s["tensor_scale"] is not None else None
        return {"values": _exact_values(s["x"].double(), c["fmt"], t)}
    A, B = s["A"], s["B"]
    v = torch.einsum("mk,nk->mn", _decode(A, torch.float64), _decode(B, torch.float64))
    if A["tensor_scale"] is not None:
        v = v * A["tensor_scale"].double() * B["tensor_scale"].double()
    if s["C"] is not None:
        v = v + 0.5 * s["C"].double()
    out = {"D": v}
    if c["act"] == "gelu_tanh":
        out["P"] = v * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))
    elif c["act"] == "silu":
        out["P"] = v * torch.sigmoid(v)
    return out
