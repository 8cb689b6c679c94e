"""Cases, plain forms and exact values of the block-scaled training operators:
the FP8 matrix product with a scale for each block of 128, LayerNorm forward
and backward, and activations kept in 8 bits and read back in the backward
pass (the block quantiser, LayerNorm's and SwiGLU's).

``run`` computes a case by elementary torch operations, or, where ``own`` is
true, by the calls a user makes of fp8_mixed_precision_amax_gb300.

A block-scaled tensor is codes [rows, pitch] (FP8, one byte each; the pitch is
the columns rounded up to 16) and one scale per 128 columns of a row
(``block`` 1) or per 128 x 128 tile (``block`` 128): a byte b for 2^(b - 127),
or a float.  The quantiser takes the smallest power of two, not below 2^-127,
under which the block's largest finite magnitude still fits the format; an
infinity saturates, a NaN stays.  Outputs held in 8 bits come back as FP8
tensors beside their scales (float8_e8m0fnu: the powers of two themselves).
"""
import math

import torch

own = False

E4M3, E5M2 = 0, 1
F8 = {E4M3: torch.float8_e4m3fn, E5M2: torch.float8_e5m2}
FMAX = {E4M3: 448.0, E5M2: 57344.0}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5


def listed():
    return [
        # one new token through an attention projection: reads 17 MB of weights for one row
        {"name": "gemm_token", "op": "gemm", "M": 1, "N": 4096, "K": 4096, "scale": "e8m0", "fa": E4M3, "block_b": 128},
        # a batch of 48 sequences decoding through the up projection of the 7B layer, weights with float scales
        {"name": "gemm_batch_f32", "op": "gemm", "M": 48, "N": 11008, "K": 4096, "scale": "f32", "fa": E4M3, "block_b": 128},
        # forward product of the 7B layer in training: 8192 tokens
        {"name": "gemm_fprop", "op": "gemm", "M": 8192, "N": 11008, "K": 4096, "scale": "e8m0", "fa": E4M3, "block_b": 128},
        # weight gradient over 8192 tokens: both operands scaled along the tokens, the gradient in E5M2, float scales
        {"name": "gemm_wgrad_f32", "op": "gemm", "M": 4096, "N": 11008, "K": 8192, "scale": "f32", "fa": E5M2, "block_b": 1},
        # LayerNorm of one token while serving
        {"name": "ln_fwd_token", "op": "ln_fwd", "rows": 1, "cols": 4096, "type": "bf16", "wtype": "bf16", "save": False},
        # LayerNorm in front of the 7B layer in training: output as the product's operand, input kept in 8 bits
        {"name": "ln_fwd_save", "op": "ln_fwd", "rows": 8192, "cols": 4096, "type": "bf16", "wtype": "bf16", "save": True},
        # LayerNorm's backward pass at the 70B layer's width, with the weight's and the bias's gradient
        {"name": "ln_bwd", "op": "ln_bwd", "rows": 8192, "cols": 8192, "type": "bf16", "wtype": "bf16", "saved": False},
        # the same from the input kept in 8 bits, for a ragged pack of tokens and an odd width
        {"name": "ln_bwd_saved", "op": "ln_bwd", "rows": 5003, "cols": 4111, "type": "bf16", "wtype": "f32", "saved": True},
        # weights of a small odd matrix in tiles of 128 x 128, with the transposed copy
        {"name": "quantize_tile", "op": "quantize", "rows": 1000, "cols": 2731, "type": "f32", "fmt": E4M3, "block": 128, "way": "both"},
        # an output gradient of the 7B layer, for the two products of the backward pass
        {"name": "quantize_both", "op": "quantize", "rows": 8192, "cols": 4096, "type": "bf16", "fmt": E5M2, "block": 1, "way": "both"},
        # SwiGLU between the products of a narrow layer on 777 tokens, its input kept in 8 bits
        {"name": "swiglu_fwd", "op": "swiglu_fwd", "M": 777, "F": 2688, "type": "bf16"},
        # SwiGLU's backward pass in the 7B layer from the input kept in 8 bits: operands of four products
        {"name": "swiglu_bwd", "op": "swiglu_bwd", "M": 8192, "F": 11008, "type": "bf16", "fmt": E5M2},
    ]


def draw(rng):
    def size(lo, hi):
        n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return n if n < 64 or rng.random() < 0.5 else max(lo, n // 64 * 64)

    op = rng.choice(["gemm", "gemm", "gemm", "ln_fwd", "ln_fwd", "ln_bwd", "ln_bwd", "quantize", "quantize", "swiglu_fwd", "swiglu_bwd"])
    if op == "gemm":
        return {"op": op, "M": size(1, 8192), "N": size(64, 11008), "K": size(128, 4096), "scale": rng.choice(["e8m0", "f32"]),
                "fa": rng.choice([E4M3, E5M2]), "block_b": rng.choice([1, 128])}
    types = ["bf16", "bf16", "f16", "f32"]
    if op in ("ln_fwd", "ln_bwd"):
        cols = size(64, 16384)
        rows = size(1, min(16384, (1 << 26) // cols))
        return {"op": op, "rows": rows, "cols": cols, "type": rng.choice(types), "wtype": rng.choice(["bf16", "f32"]),
                "save" if op == "ln_fwd" else "saved": rng.random() < 0.5}
    if op == "quantize":
        cols = size(64, 16384)
        rows = size(1, min(16384, (1 << 25) // cols))
        return {"op": op, "rows": rows, "cols": cols, "type": rng.choice(types), "fmt": rng.choice([E4M3, E5M2]),
                "block": rng.choice([1, 1, 128]), "way": rng.choice(["rows", "both", "cols"])}
    case = {"op": op, "M": size(1, 8192), "F": 128 * size(1, 86), "type": rng.choice(["bf16", "f16"])}
    return case if op == "swiglu_fwd" else {**case, "fmt": rng.choice([E4M3, E5M2])}


# ------------------------------------------------------------- the inputs --

def up(n, m):
    return -(-n // m) * m


def codes_like(rows, cols, fmt, g):
    """Codes as a block's quantiser leaves them: normal values that reach up to the format's largest."""
    v = torch.randn(rows, cols, generator=g, device="cuda") * (FMAX[fmt] / 4)
    c = torch.zeros(rows, up(cols, 16), dtype=torch.uint8, device="cuda")
    c[:, :cols] = v.clamp(-FMAX[fmt], FMAX[fmt]).to(F8[fmt]).view(torch.uint8)
    return c


def scales_like(rows, cols, block, kind, size, g):
    """Scales around 2^size that vary from block to block; a row's scales fill whole 4-byte words."""
    shape = (-(-rows // block), up(-(-cols // 128), 4))
    if kind == "e8m0":
        return torch.randint(size + 125, size + 130, shape, generator=g, device="cuda", dtype=torch.uint8)
    return torch.exp2(size + torch.randn(shape, generator=g, device="cuda") * 0.7)


def kept(x, fmt=E4M3):
    """x in 8 bits, a scale for each 128 columns, in a user's buffers."""
    c, s = quantize(x.float(), fmt, 1)
    rows, cols = x.shape
    codes = torch.zeros(rows, up(cols, 16), dtype=torch.uint8, device="cuda")
    codes[:, :cols] = c.view(torch.uint8)
    scales = torch.zeros(rows, up(s.shape[1], 4), dtype=torch.uint8, device="cuda")
    scales[:, : s.shape[1]] = s.view(torch.uint8)
    return codes, scales


def room(rows, cols, block=1):
    """Buffers of a block-scaled tensor: codes and scale bytes."""
    return (torch.empty(rows, up(cols, 16), dtype=torch.uint8, device="cuda"),
            torch.empty(-(-rows // block), up(-(-cols // 128), 4), dtype=torch.uint8, device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c, op = dict(case), case["op"]
    s = {"case": c}

    def normal(rows, cols, std, kind):
        return (torch.randn(rows, cols, generator=g, device="cuda") * std).to(TYPES[kind])

    if op == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        s["A"], s["B"] = codes_like(M, K, c["fa"], g), codes_like(N, K, E4M3, g)
        s["sa"] = scales_like(M, K, 1, c["scale"], -7 if c["fa"] == E4M3 else -24, g)
        s["sb"] = scales_like(N, K, c["block_b"], c["scale"], -13, g)
        s["D"] = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    elif op in ("ln_fwd", "ln_bwd"):
        rows, cols, kind = c["rows"], c["cols"], c["type"]
        x = torch.randn(rows, cols, generator=g, device="cuda") * 2 + 0.5
        x[:, :: 97] *= 8  # a few channels are much larger than the rest
        x = x.to(TYPES[kind])
        s["gamma"] = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(TYPES[c["wtype"]])
        s["beta"] = (0.1 * torch.randn(cols, generator=g, device="cuda")).to(TYPES[c["wtype"]])
        if op == "ln_fwd":
            s["x"] = x
            s["mean"], s["rstd"] = torch.empty(2, rows, device="cuda")
            if c["save"]:
                s["y8"], s["x8"] = room(rows, cols), room(rows, cols)
            else:
                s["y"] = torch.empty_like(x)
        else:
            mean = x.float().mean(1, keepdim=True)
            var = (x.float() - mean).square().mean(1)
            s["mean"], s["rstd"] = mean[:, 0].contiguous(), torch.rsqrt(var + EPS)
            s["x"] = kept(x) if c["saved"] else x
            s["dy"] = normal(rows, cols, 0.01 if kind == "f16" else 1e-3, kind)
            s["dx"] = torch.empty_like(x)
            s["dgamma"], s["dbeta"] = torch.empty(2, cols, device="cuda")
    elif op == "quantize":
        rows, cols, block = c["rows"], c["cols"], c["block"]
        s["x"] = normal(rows, cols, 1e-2, c["type"])
        s["x"][rows // 2] = 0  # a masked token
        s["q"] = room(rows, cols, block) if c["way"] != "cols" else None
        s["qt"] = room(cols, rows, block) if c["way"] != "rows" else None
    elif op == "swiglu_fwd":
        M, F = c["M"], c["F"]
        s["h"] = normal(M, 2 * F, 1.5, c["type"])
        s["a8"], s["h8"] = room(M, F), room(M, 2 * F)
    else:
        M, F = c["M"], c["F"]
        s["h8"] = kept(normal(M, 2 * F, 1.5, c["type"]))
        s["da"] = normal(M, F, 1e-2, c["type"])
        s["dh8"], s["dh8t"], s["a8t"] = room(M, 2 * F), room(2 * F, M), room(F, M)
    return s


# --------------------------------------------------------- the plain forms --

def padded(x, rows, cols):
    return torch.nn.functional.pad(x, (0, cols - x.shape[1], 0, rows - x.shape[0]))


def quantize(x, fmt, block):
    """(codes, scales) of x (32 bits): FP8 [rows, cols] and powers of two [rows / block, cols / 128], rounded up."""
    rows, cols = x.shape
    R, C = up(rows, block), up(cols, 128)
    v = padded(x, R, C).view(R // block, block, C // 128, 128)
    amax = torch.where(v.isfinite(), v.abs(), 0.0).amax((1, 3))
    m, e = torch.frexp(amax)  # amax = m 2^e, 1/2 <= m < 1, and both formats' largest value is 7/8 of a power of two
    e = (e + (m > 0.875) - (9 if fmt == E4M3 else 16)).clamp(-127, 127)
    e = torch.where(amax == 0, -127, e).to(torch.int32)
    q = (v * ((127 - e) << 23).view(torch.float32)[:, None, :, None]).clamp(-FMAX[fmt], FMAX[fmt])
    return q.view(R, C)[:rows, :cols].to(F8[fmt]), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def transposed(x, fmt, block):
    """quantize() of the transpose, and for tiles the same tiles seen from the other side."""
    return quantize(x.t().contiguous(), fmt, block)


def values(codes, scales, fmt, rows, cols, block, kind=torch.float32):
    """What codes and scales stand for."""
    nb = -(-cols // 128)
    s = scales[:, :nb]
    s = s.view(torch.float8_e8m0fnu).to(kind) if s.dtype == torch.uint8 else s.to(kind)
    s = s.repeat_interleave(block, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
    return codes[:, :cols].view(F8[fmt]).to(kind) * s


def run(state):
    if own:
        return own_run(state)
    s, c = state, state["case"]
    op = c["op"]
    if op == "gemm":
        a = values(s["A"], s["sa"], c["fa"], c["M"], c["K"], 1)
        b = values(s["B"], s["sb"], E4M3, c["N"], c["K"], c["block_b"])
        return {"D": (a @ b.t()).to(torch.bfloat16)}
    if op == "ln_fwd":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        rstd = 1 / torch.sqrt((x - mean).square().mean(1, keepdim=True) + EPS)
        y = (x - mean) * rstd * s["gamma"].float() + s["beta"].float()
        out = {"mean": mean[:, 0], "rstd": rstd[:, 0]}
        if not c["save"]:
            return {**out, "y": y.to(s["x"].dtype)}
        return {**out, "y8": quantize(y, E4M3, 1), "x8": quantize(x, E4M3, 1)}
    if op == "ln_bwd":
        x = values(*s["x"], E4M3, c["rows"], c["cols"], 1) if c["saved"] else s["x"].float()
        dy = s["dy"].float()
        xhat = (x - s["mean"][:, None]) * s["rstd"][:, None]
        u = dy * s["gamma"].float()
        dx = s["rstd"][:, None] * (u - u.mean(1, keepdim=True) - xhat * (u * xhat).mean(1, keepdim=True))
        return {"dx": dx.to(s["dy"].dtype), "dgamma": (dy * xhat).sum(0), "dbeta": dy.sum(0)}
    if op == "quantize":
        x = s["x"].float()
        return {"q": quantize(x, c["fmt"], c["block"]) if s["q"] else None,
                "qt": transposed(x, c["fmt"], c["block"]) if s["qt"] else None}
    F = c["F"]
    if op == "swiglu_fwd":
        h = s["h"].float()
        gate, value = h[:, :F], h[:, F:]
        return {"a8": quantize(gate / (1 + torch.exp(-gate)) * value, E4M3, 1), "h8": quantize(h, E4M3, 1)}
    h = values(*s["h8"], E4M3, c["M"], 2 * F, 1)
    gate, value, da = h[:, :F], h[:, F:], s["da"].float()
    sig = 1 / (1 + torch.exp(-gate))
    dh = torch.cat([da * value * sig * (1 + gate * (1 - sig)), da * (gate * sig)], 1)
    return {"dh8": quantize(dh, c["fmt"], 1), "dh8t": transposed(dh, c["fmt"], 1),
            "a8t": transposed(gate * sig * value, E4M3, 1)}


# ---------------------------------------------------------- the own calls --

def own_run(s):
    import fp8_mixed_precision_amax_gb300 as f

    c = s["case"]
    op = c["op"]

    def block(buffers, cols, fmt, rows=1):
        return f.BlockFp8(buffers[0], buffers[1], cols, fmt, rows)

    def out(q):
        nb = -(-q.cols // 128)
        return q.codes[:, : q.cols].view(F8[q.fmt]), q.scales[:, :nb].view(torch.float8_e8m0fnu)

    if op == "gemm":
        a = block((s["A"], s["sa"]), c["K"], c["fa"])
        f.fp8_block_gemm_tn(a, block((s["B"], s["sb"]), c["K"], E4M3, c["block_b"]), s["D"])
        return {"D": s["D"]}
    if op == "ln_fwd":
        if not c["save"]:
            f.fp8_layernorm_fwd(s["x"], s["gamma"], s["beta"], EPS, s["mean"], s["rstd"], y=s["y"])
            return {"mean": s["mean"], "rstd": s["rstd"], "y": s["y"]}
        y8, x8 = block(s["y8"], c["cols"], E4M3), block(s["x8"], c["cols"], E4M3)
        f.fp8_layernorm_fwd(s["x"], s["gamma"], s["beta"], EPS, s["mean"], s["rstd"], y8=y8, x8=x8)
        return {"mean": s["mean"], "rstd": s["rstd"], "y8": out(y8), "x8": out(x8)}
    if op == "ln_bwd":
        x = block(s["x"], c["cols"], E4M3) if c["saved"] else s["x"]
        f.fp8_layernorm_bwd(s["dy"], x, s["gamma"], s["mean"], s["rstd"], s["dx"], s["dgamma"], s["dbeta"])
        return {"dx": s["dx"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}
    if op == "quantize":
        q = block(s["q"], c["cols"], c["fmt"], c["block"]) if s["q"] else None
        qt = block(s["qt"], c["rows"], c["fmt"], c["block"]) if s["qt"] else None
        f.fp8_block_quantize(s["x"], q, qt)
        return {"q": out(q) if q else None, "qt": out(qt) if qt else None}
    F = c["F"]
    if op == "swiglu_fwd":
        a8, h8 = block(s["a8"], F, E4M3), block(s["h8"], 2 * F, E4M3)
        f.fp8_swiglu_fwd(s["h"], a8, h8)
        return {"a8": out(a8), "h8": out(h8)}
    dh8, dh8t = block(s["dh8"], 2 * F, c["fmt"]), block(s["dh8t"], c["M"], c["fmt"])
    a8t = block(s["a8t"], c["M"], E4M3)
    f.fp8_swiglu_bwd(s["da"], block(s["h8"], 2 * F, E4M3), dh8, dh8t, a8t)
    return {"dh8": out(dh8), "dh8t": out(dh8t), "a8t": out(a8t)}


# ------------------------------------------------------- what they cost --

def work(case):
    c, op = case, case["op"]

    def kept_bytes(rows, cols, block=1):
        return rows * cols + -(-rows // block) * -(-cols // 128)

    if op == "gemm":
        M, N, K, one = c["M"], c["N"], c["K"], 1 if c["scale"] == "e8m0" else 4
        nb = -(-K // 128)
        return {"bytes": M * K + N * K + one * nb * (M + -(-N // c["block_b"])) + 2 * M * N, "flops": 2 * M * N * K}
    size = TYPES[c["type"]].itemsize
    if op in ("ln_fwd", "ln_bwd"):
        rows, cols = c["rows"], c["cols"]
        w = TYPES[c["wtype"]].itemsize * cols
        if op == "ln_fwd":
            return {"bytes": size * rows * cols + 2 * w + 8 * rows + (2 * kept_bytes(rows, cols) if c["save"] else size * rows * cols),
                    "flops": 9 * rows * cols}
        return {"bytes": 2 * size * rows * cols + (kept_bytes(rows, cols) if c["saved"] else size * rows * cols) + w + 8 * rows + 8 * cols,
                "flops": 14 * rows * cols}
    if op == "quantize":
        rows, cols = c["rows"], c["cols"]
        outs = (c["way"] != "cols") * kept_bytes(rows, cols, c["block"]) + (c["way"] != "rows") * kept_bytes(cols, rows, c["block"])
        return {"bytes": size * rows * cols + outs, "flops": 3 * rows * cols}
    M, F = c["M"], c["F"]
    if op == "swiglu_fwd":
        return {"bytes": 2 * size * M * F + kept_bytes(M, F) + kept_bytes(M, 2 * F), "flops": 12 * M * F}
    return {"bytes": size * M * F + 2 * kept_bytes(M, 2 * F) + kept_bytes(2 * F, M) + kept_bytes(F, M), "flops": 30 * M * F}


# ------------------------------------------------- the same in 64 bits --

def two_to(e):
    """2^e in 64 bits, exactly: from its bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def exact_block(x, fmt, block, flip=False):
    """Codes and scales of x (64 bits) by the definition: the scale by a search over its exponents' logarithm, the code by
    rounding to the nearest multiple of the step at its size, ties to the even one."""
    x = x.t() if flip else x
    rows, cols = x.shape
    br, bc = -(-rows // block), -(-cols // 128)
    v = torch.zeros(br * block, bc * 128, dtype=torch.float64, device=x.device)
    v[:rows, :cols] = x
    v = v.reshape(br, block, bc, 128).permute(0, 2, 1, 3).reshape(br, bc, -1)
    amax = torch.nan_to_num(v, nan=0.0, posinf=0.0, neginf=0.0).abs().max(-1).values
    e = torch.ceil(torch.log2(amax / FMAX[fmt])).clamp(-127, 127)  # -inf for a block of zeros
    e = torch.where(amax > FMAX[fmt] * two_to(e), e + 1, e)
    e = torch.where((amax <= FMAX[fmt] * two_to(e - 1)) & (e > -127), e - 1, e)
    s = two_to(e)
    q = (v / s[..., None]).clamp(-FMAX[fmt], FMAX[fmt])
    bits, least = (3, -6) if fmt == E4M3 else (2, -14)
    step = two_to((torch.frexp(q).exponent - 1).clamp(min=least) - bits)
    q = torch.round(q / step) * step
    q = q.reshape(br, bc, block, 128).permute(0, 2, 1, 3).reshape(br * block, bc * 128)[:rows, :cols]
    return q, s


def exact_values(codes, scales, fmt, rows, cols, block=1):
    at = torch.arange(cols, device=codes.device) // 128
    of = torch.arange(rows, device=codes.device) // block
    s = two_to(scales.to(torch.int64) - 127) if scales.dtype == torch.uint8 else scales.double()
    return codes[:, :cols].view(F8[fmt]).double() * s[of][:, at]


def exact(case, seed):
    s, c, op = prepare(case, seed), case, case["op"]
    if op == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        b = exact_values(s["B"], s["sb"], E4M3, N, K, c["block_b"])
        a = exact_values(s["A"], s["sa"], c["fa"], M, K)
        return {"D": torch.mm(a, b.t())}
    if op in ("ln_fwd", "ln_bwd"):
        rows, cols = c["rows"], c["cols"]
        gamma, beta = s["gamma"].double(), s["beta"].double()
        if op == "ln_fwd":
            x = s["x"].double()
            mean = x.sum(1) / cols
            rstd = (((x - mean[:, None]) ** 2).sum(1) / cols + EPS) ** -0.5
            y = torch.addcmul(beta, (x - mean[:, None]) * rstd[:, None], gamma)
            out = {"mean": mean, "rstd": rstd}
            if not c["save"]:
                return {**out, "y": y}
            return {**out, "y8": exact_block(y, E4M3, 1), "x8": exact_block(x, E4M3, 1)}
        x = exact_values(*s["x"], E4M3, rows, cols) if c["saved"] else s["x"].double()
        dy, r = s["dy"].double(), s["rstd"].double()[:, None]
        z = (x - s["mean"].double()[:, None]) * r
        u = dy * gamma
        dx = u * r - r / cols * u.sum(1, keepdim=True) - r / cols * z * (u * z).sum(1, keepdim=True)
        return {"dx": dx, "dgamma": torch.einsum("rc,rc->c", dy, z), "dbeta": dy.sum(0)}
    if op == "quantize":
        x = s["x"].double()
        return {"q": exact_block(x, c["fmt"], c["block"]) if s["q"] else None,
                "qt": exact_block(x, c["fmt"], c["block"], True) if s["qt"] else None}
    F = c["F"]
    h = s["h"].double() if op == "swiglu_fwd" else exact_values(*s["h8"], E4M3, c["M"], 2 * F)
    gate, value = h.split(F, 1)
    sig = torch.sigmoid(gate)
    if op == "swiglu_fwd":
        return {"a8": exact_block(gate * sig * value, E4M3, 1), "h8": exact_block(h, E4M3, 1)}
    da = s["da"].double()
    dh = torch.empty_like(h)
    dh[:, :F] = da * value * (sig + gate * sig * torch.sigmoid(-gate))
    dh[:, F:] = da * gate * sig
    return {"dh8": exact_block(dh, c["fmt"], 1), "dh8t": exact_block(dh, c["fmt"], 1, True),
            "a8t": exact_block(gate * sig * value, E4M3, 1, True)}
