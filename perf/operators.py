"""The 8-bit operators of the framework, case by case: what each computes, on which inputs, in which sizes.

``listed()`` and ``draw()`` give cases, ``prepare()`` the inputs of one, ``run()`` one pass through its operator:
in plain form (elementary torch operations in 32 bits, rounded once) where ``own`` is false, by the framework's
kernels where it is true.  ``exact()`` gives the same outputs from the definition in 64 bits, with 8-bit outputs
unrounded, and ``work()`` the bytes and operations that a pass cannot do without.

The operators are those of a pre-norm projection in 8-bit floating point, served and trained:

    gemm            D[m][n] = sum over blocks b of 128: sa[m][b] sb[n][b] sum_{k in b} a[m][k] b[n][k]
    quantize        8-bit codes with a power-of-two scale per block of 128, along rows, columns or both
    norm            h = x + residual; y = h / rms(h) * weight, quantised along the rows
    norm_backward   gradients of that norm with respect to h and to the weight

A quantised matrix is codes (e4m3, R x K) and scales (e8m0, ceil(K / 512) x R x 4): byte j of scales[i][r] is the
biased exponent of the scale of row r's block 4 i + j, 127 past the last block.
"""
import math

import torch

own = False

EPS = 1e-6


def listed():
    return [
        # one token of a decode loop against a square projection: streams the weights
        {"name": "gemm 1x8192x8192", "op": "gemm", "m": 1, "n": 8192, "k": 8192, "out": "bf16"},
        # a batch of 64 sequences decoding together
        {"name": "gemm 64x8192x8192", "op": "gemm", "m": 64, "n": 8192, "k": 8192, "out": "bf16"},
        # a prompt whose length, and a projection whose width, divide by nothing (the ragged workload)
        {"name": "gemm ragged", "op": "gemm", "m": 6143, "n": 5999, "k": 4104, "out": "bf16"},
        # a training step's forward product (the cube8192 workload)
        {"name": "gemm cube8192", "op": "gemm", "m": 8192, "n": 8192, "k": 8192, "out": "bf16"},
        # a weight gradient: the contraction runs over the tokens, the sums stay in 32 bits (the longk workload)
        {"name": "gemm longk fp32", "op": "gemm", "m": 2048, "n": 2048, "k": 32768, "out": "fp32"},
        # the activations of a decode batch, from 32 bits
        {"name": "quantize 64 rows", "op": "quantize", "r": 64, "c": 8192, "form": "rows", "tile": False, "dtype": "fp32"},
        # an output gradient of ragged size, for both backward products
        {"name": "quantize ragged both", "op": "quantize", "r": 6143, "c": 5999, "form": "both", "tile": False, "dtype": "bf16"},
        # a weight matrix after an optimiser step, for the forward product and the input gradient
        {"name": "quantize weights", "op": "quantize", "r": 8192, "c": 8192, "form": "both", "tile": True, "dtype": "bf16"},
        # one token of a decode loop
        {"name": "norm 1x8192", "op": "norm", "r": 1, "c": 8192, "residual": True, "wdtype": "bf16"},
        # a training step's tokens
        {"name": "norm 8192x8192", "op": "norm", "r": 8192, "c": 8192, "residual": True, "wdtype": "bf16"},
        # backward over a ragged number of tokens, the norm's weight held in 32 bits
        {"name": "norm_backward ragged", "op": "norm_backward", "r": 6143, "c": 4104, "residual": False, "wdtype": "fp32"},
        # backward of a training step's tokens, the residual stream's own gradient added
        {"name": "norm_backward 8192x8192", "op": "norm_backward", "r": 8192, "c": 8192, "residual": True, "wdtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "quantize", "norm", "norm_backward"])
    if op == "gemm":
        while True:
            m, n, k = _log(rng, 1, 8192), _log(rng, 64, 16384), _log(rng, 64, 32768)
            if m * n * k <= 8192**3 and m * k + n * k <= 2**28 and m * n <= 2**26:
                break
        return {"op": op, "m": m, "n": n, "k": k, "out": rng.choice(["bf16", "bf16", "fp32"])}
    r, c = _log(rng, 1, 8192), _log(rng, 64, 8192)
    if op == "quantize":
        form = rng.choice(["rows", "columns", "both", "normed columns"])
        tile = form in ("rows", "both") and rng.random() < 0.4
        dtype = "bf16" if form == "normed columns" else rng.choice(["bf16", "bf16", "fp32"])
        return {"op": op, "r": r, "c": c, "form": form, "tile": tile, "dtype": dtype}
    return {"op": op, "r": r, "c": c, "residual": rng.random() < 0.7, "wdtype": rng.choice(["bf16", "fp32"])}


# ---------------------------------------------------------------- inputs
def _activations(r, c, gen, scale=1.0):
    # hidden states: normal, with some channels far larger than the rest
    x = torch.randn(r, c, generator=gen, device="cuda")
    loud = 1.0 + 15.0 * (torch.rand(c, generator=gen, device="cuda") < 0.01).float()
    return x * loud * scale


def _quantized(x):
    """Codes (rows at a multiple of 128 bytes, as the framework's quantiser lays them out) and scales of x's rows."""
    codes, scales = _quantize_plain(x, False)
    held = torch.zeros(x.shape[0], -(-x.shape[1] // 128) * 128, dtype=torch.uint8, device=x.device)
    held[:, : x.shape[1]] = codes.view(torch.uint8)
    return held.view(torch.float8_e4m3fn)[:, : x.shape[1]], scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    op = case["op"]
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        if case["out"] == "fp32":  # a weight gradient: output gradients against activations
            s["a"], s["sa"] = _quantized(torch.randn(m, k, generator=gen, device="cuda") * 1e-3)
            s["b"], s["sb"] = _quantized(torch.randn(n, k, generator=gen, device="cuda"))
        else:
            s["a"], s["sa"] = _quantized(_activations(m, k, gen))
            s["b"], s["sb"] = _quantized(torch.randn(n, k, generator=gen, device="cuda") * 0.02)
        return s
    r, c = case["r"], case["c"]
    if op == "quantize":
        x = _activations(r, c, gen, 0.02 if case["tile"] else 1.0)
        s["x"] = x.to(torch.bfloat16) if case["dtype"] == "bf16" else x
        if case["form"] == "normed columns":
            s["rf"] = torch.rsqrt(s["x"].float().square().mean(1) + EPS)
            s["cf"] = (1.0 + 0.1 * torch.randn(c, generator=gen, device="cuda")).to(torch.bfloat16)
        return s
    w = 1.0 + 0.1 * torch.randn(c, generator=gen, device="cuda")
    s["w"] = w.to(torch.bfloat16) if case["wdtype"] == "bf16" else w
    if op == "norm":
        s["x"] = _activations(r, c, gen).to(torch.bfloat16)
        s["res"] = _activations(r, c, gen).to(torch.bfloat16) if case["residual"] else None
        return s
    s["h"] = _activations(r, c, gen).to(torch.bfloat16)
    s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + EPS)
    s["dy"] = (torch.randn(r, c, generator=gen, device="cuda") * 1e-3).to(torch.bfloat16)
    s["dres"] = (torch.randn(r, c, generator=gen, device="cuda") * 1e-3).to(torch.bfloat16) if case["residual"] else None
    return s


# ---------------------------------------------------------------- the plain form
def _bytes_of(amax):
    """The biased exponent of the least power of two s with amax / s <= 448 = 1.75 * 2^8."""
    bits = amax.view(torch.int32)
    return ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).int()).clamp_min(0)


def _quantize_plain(y, tile):
    """Codes and scales of the rows of y (32 bits)."""
    r, c = y.shape
    kb = -(-c // 128)
    y = torch.nn.functional.pad(y, (0, kb * 128 - c))
    amax = y.view(r, kb, 128).abs().amax(2)
    if tile:
        rb = -(-r // 128)
        amax = torch.nn.functional.pad(amax, (0, 0, 0, rb * 128 - r)).view(rb, 128, kb).amax(1)
        amax = amax.repeat_interleave(128, 0)[:r].contiguous()
    e = _bytes_of(amax)
    up = ((254 - e) << 23).view(torch.float32)  # 2^(127 - e)
    codes = (y.view(r, kb, 128) * up[:, :, None]).reshape(r, kb * 128)[:, :c].contiguous().to(torch.float8_e4m3fn)
    kt = -(-kb // 4)
    e = torch.nn.functional.pad(e, (0, kt * 4 - kb), value=127).to(torch.uint8)
    return codes, e.view(r, kt, 4).permute(1, 0, 2).contiguous().view(torch.float8_e8m0fnu)


def _values_plain(codes, scales):
    kt, r, _ = scales.shape
    s = scales.view(torch.uint8).permute(1, 0, 2).reshape(r, kt * 4).float() - 127.0
    s = torch.exp2(s).repeat_interleave(128, 1)[:, : codes.shape[1]]
    return codes.float() * s


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "gemm":
        d = _values_plain(s["a"], s["sa"]) @ _values_plain(s["b"], s["sb"]).t()
        return d.to(torch.bfloat16) if case["out"] == "bf16" else d
    if op == "quantize":
        x, form = s["x"].float(), case["form"]
        if form == "normed columns":
            x = x * s["rf"][:, None] * s["cf"].float()
        out = ()
        if form in ("rows", "both"):
            out += _quantize_plain(x, case["tile"])
        if form != "rows":
            out += _quantize_plain(x.t().contiguous(), case["tile"])
        return out
    w = s["w"].float()
    if op == "norm":
        h = s["x"].float()
        if s["res"] is not None:
            h = (h + s["res"].float()).to(torch.bfloat16).float()
        rstd = torch.rsqrt(h.square().mean(1) + EPS)
        codes, scales = _quantize_plain(h * rstd[:, None] * w, False)
        return (codes, scales, rstd) + ((h.to(torch.bfloat16),) if s["res"] is not None else ())
    xh = s["h"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy * w
    dx = s["rstd"][:, None] * (g - xh * (g * xh).mean(1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return dx.to(torch.bfloat16), (dy * xh).sum(0)


# ---------------------------------------------------------------- the framework's kernels
def _run_own(s):
    from warp_specialized_tma_gb300 import fp8

    case = s["case"]
    op = case["op"]
    if op == "gemm":
        return fp8.gemm(s["a"], s["sa"], s["b"], s["sb"], out_dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32)
    if op == "quantize":
        form = case["form"]
        if form == "rows":
            return fp8.quantize(s["x"], tile=case["tile"])
        if form == "columns":
            return fp8.quantize_columns(s["x"])
        if form == "normed columns":
            return fp8.quantize_columns(s["x"], row_factor=s["rf"], column_factor=s["cf"])
        return fp8.quantize_both(s["x"], tile=case["tile"])
    if op == "norm":
        codes, scales, h, rstd = fp8.rmsnorm(s["x"], s["w"], residual=s["res"], eps=EPS)
        return (codes, scales, rstd) + ((h,) if s["res"] is not None else ())
    return fp8.rmsnorm_backward(s["dy"], s["h"], s["w"], s["rstd"], dresidual=s["dres"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- the definition in 64 bits
def _exact_quantized(y, tile):
    # y / s before its rounding to 8 bits, and s
    r, c = y.shape
    kb, kt = -(-c // 128), -(-c // 512)
    full = torch.zeros(-(-r // 128) * 128, kt * 512, dtype=torch.float64, device=y.device)
    full[:r, :c] = y
    blocks = full.reshape(full.shape[0], kt * 4, 128)
    top = blocks.abs().max(2).values
    if tile:
        top = top.reshape(-1, 128, kt * 4).max(1).values.repeat_interleave(128, 0)
    e = torch.ceil(torch.log2(top.clamp_min(2.0**-126) / 448.0)).clamp_min(-127.0)
    e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)
    e = torch.where(top <= 448.0 * torch.exp2(e - 1), (e - 1).clamp_min(-127.0), e)
    e = torch.where(top == 0, torch.full_like(e, -127.0), e)
    codes = (blocks / torch.exp2(e)[:, :, None]).reshape(full.shape)[:r, :c]
    s = torch.exp2(e[:r])
    s[:, kb:] = 1.0
    return codes, s.reshape(r, kt, 4).transpose(0, 1)


def _exact_values(codes, scales):
    e = scales.view(torch.uint8).double() - 127.0
    each = torch.exp2(e).transpose(0, 1).reshape(codes.shape[0], -1)
    cols = torch.arange(codes.shape[1], device=codes.device) // 128
    return codes.double() * each[:, cols]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gemm":
        return _exact_values(s["a"], s["sa"]) @ _exact_values(s["b"], s["sb"]).T
    if op == "quantize":
        x, out = s["x"].double(), []
        if case["form"] == "normed columns":
            x = x * s["rf"].double().reshape(-1, 1) * s["cf"].double().reshape(1, -1)
        if case["form"] in ("rows", "both"):
            out += _exact_quantized(x, case["tile"])
        if case["form"] != "rows":
            out += _exact_quantized(x.T.contiguous(), case["tile"])
        return tuple(out)
    w = s["w"].double()
    if op == "norm":
        h = s["x"].double()
        if s["res"] is not None:
            h = h + s["res"].double()
        # the norm is that of the residual stream as it is stored
        kept = h.to(torch.bfloat16).double()
        rstd = 1.0 / torch.sqrt(torch.sum(kept * kept, 1) / case["c"] + EPS)
        out = _exact_quantized(kept * rstd.unsqueeze(1) * w, False) + (rstd,)
        return out + ((h,) if s["res"] is not None else ())
    rstd, h, dy = s["rstd"].double().unsqueeze(1), s["h"].double(), s["dy"].double()
    inner = torch.sum(dy * w * h, 1, keepdim=True) / case["c"]
    dx = rstd * dy * w - rstd**3 * h * inner
    if s["dres"] is not None:
        dx = dx + s["dres"].double()
    return dx, torch.einsum("rc,rc->c", dy, h * rstd)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        size = 2 if case["out"] == "bf16" else 4
        return {"bytes": (m + n) * (k + -(-k // 128)) + m * n * size, "flops": 2 * m * n * k}
    r, c = case["r"], case["c"]
    rows = r * (c + -(-c // 128))
    if op == "quantize":
        nbytes = r * c * (2 if case["dtype"] == "bf16" else 4)
        nbytes += rows if case["form"] in ("rows", "both") else 0
        nbytes += c * (r + -(-r // 128)) if case["form"] != "rows" else 0
        nbytes += 4 * r + 2 * c if case["form"] == "normed columns" else 0
        return {"bytes": nbytes, "flops": 4 * r * c}
    wsize = 2 if case["wdtype"] == "bf16" else 4
    if op == "norm":
        return {"bytes": r * c * (6 if case["residual"] else 2) + rows + 4 * r + wsize * c, "flops": 8 * r * c}
    return {"bytes": r * c * (8 if case["residual"] else 6) + 4 * r + (wsize + 4) * c, "flops": 12 * r * c}
