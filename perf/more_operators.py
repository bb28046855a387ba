"""The bf16 operators of a feed-forward block, case by case: what each computes, on which inputs, in which sizes.

``listed()`` and ``draw()`` give cases, ``prepare()`` the inputs of one, ``run()`` one pass through its operator:
in plain form (elementary torch operations in 32 bits, rounded once) where ``own`` is false, by the framework's
kernels where it is true.  ``exact()`` gives the same outputs from the definition in 64 bits, and ``work()`` the bytes
and operations that a pass cannot do without.

The operators, with M tokens of bf16:

    linear           z = x W^T + b; y = act(z) + r, and z where it is saved for the backward pass
    linear_backward  dz = dy act'(z) in bf16; dx = dz W; dW = dz^T x; db = the sum of dy act'(z) over the tokens
    gated            g = x Wg^T; u = x Wu^T; h = act(g) u, and g and u where they are saved
    gated_backward   dh = dy Wd; dg = dh u act'(g), du = dh act(g), h = act(g) u, each in bf16;
                     dx = dg Wg + du Wu; dWg = dg^T x; dWu = du^T x; dWd = dy^T h
    step             gated with g and u saved in 8 bits, y = h Wd^T + r, and gated_backward from what was saved

g and u saved in 8 bits are codes (e4m3, M x F) and scales (e8m0, ceil(F / 512) x M x 4): byte j of scales[i][m] is the
biased exponent of the least power of two s with |value| / s <= 448 in row m's block 4 i + j of 128 columns.
"""
import math

import torch

own = False


def listed():
    return [
        # one token of a decode loop through an up projection
        {"name": "linear 1x8192x8192", "op": "linear", "m": 1, "n": 8192, "k": 8192, "act": "gelu", "bias": True, "residual": False, "save": False, "out": "bf16"},
        # a batch of 64 sequences decoding together, back into the residual stream
        {"name": "linear 64x8192x8192", "op": "linear", "m": 64, "n": 8192, "k": 8192, "act": None, "bias": True, "residual": True, "save": False, "out": "bf16"},
        # a training step over a number of tokens and widths that divide by nothing large (the ragged workload)
        {"name": "linear ragged", "op": "linear", "m": 6143, "n": 5999, "k": 4104, "act": "gelu", "bias": True, "residual": False, "save": True, "out": "bf16"},
        # a prompt's tokens through a square projection back into the residual stream (the cube8192 workload)
        {"name": "linear cube8192", "op": "linear", "m": 8192, "n": 8192, "k": 8192, "act": "silu", "bias": True, "residual": True, "save": False, "out": "bf16"},
        # the backward pass of the ragged step
        {"name": "linear_backward ragged", "op": "linear_backward", "m": 6143, "n": 5999, "k": 4104, "act": "gelu", "bias": True},
        # the backward pass of a training step's tokens
        {"name": "linear_backward cube4096", "op": "linear_backward", "m": 4096, "n": 4096, "k": 4096, "act": "gelu_tanh", "bias": True},
        # one token of a decode loop through a gated block's first half
        {"name": "gated 1 token", "op": "gated", "m": 1, "c": 4096, "f": 16384, "act": "silu", "save": None},
        # a prompt of ragged length and widths
        {"name": "gated ragged", "op": "gated", "m": 6143, "c": 4104, "f": 5999, "act": "silu", "save": None},
        # a training step's tokens, g and u kept for the backward pass
        {"name": "gated 4096 tokens", "op": "gated", "m": 4096, "c": 4096, "f": 16384, "act": "silu", "save": "bf16"},
        # its backward pass
        {"name": "gated_backward 4096 tokens", "op": "gated_backward", "m": 4096, "c": 4096, "f": 16384, "act": "silu", "save": "bf16"},
        # a backward pass over a ragged batch whose checkpoints are 8 bits
        {"name": "gated_backward ragged", "op": "gated_backward", "m": 2047, "c": 2056, "f": 5999, "act": "gelu_tanh", "save": "e4m3"},
        # a whole training step through a block with 8-bit checkpoints
        {"name": "step 8192 tokens", "op": "step", "m": 8192, "c": 2048, "f": 8192, "act": "silu", "save": "e4m3"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    # most widths are multiples of 8 (a row of bf16 then starts on 16 bytes); some are anything
    w = _log(rng, lo, hi)
    return w if rng.random() < 0.3 else max(8, w // 8 * 8)


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "gated", "gated_backward", "step"])
    act = rng.choice(["silu", "gelu", "gelu_tanh", "relu"])
    while True:
        m, n, k = _log(rng, 1, 8192), _width(rng, 64, 16384), _width(rng, 64, 16384)
        products = {"linear": 1, "linear_backward": 2, "gated": 2, "gated_backward": 6, "step": 9}[op]
        if products * m * n * k <= 8192**3 and m * n <= 2**26 and m * k <= 2**26 and n * k <= 2**27:
            break
    if op == "linear":
        return {"op": op, "m": m, "n": n, "k": k, "act": rng.choice([None, act]), "bias": rng.random() < 0.6, "residual": rng.random() < 0.5,
                "save": rng.random() < 0.3, "out": rng.choice(["bf16", "bf16", "bf16", "fp32"])}
    if op == "linear_backward":
        return {"op": op, "m": m, "n": n, "k": k, "act": rng.choice([None, act, act]), "bias": rng.random() < 0.7}
    save = {"gated": rng.choice([None, None, "bf16"]), "gated_backward": rng.choice(["bf16", "e4m3"]), "step": "e4m3"}[op]
    return {"op": op, "m": m, "c": k, "f": n, "act": act, "save": save}


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    op = case["op"]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def activations(r, c):
        # normed hidden states: normal, with some channels larger than the rest
        loud = 1.0 + 7.0 * (torch.rand(c, generator=gen, device="cuda") < 0.01).float()
        return (randn(r, c) * loud).to(torch.bfloat16)

    def weight(n, k):
        return (randn(n, k) / math.sqrt(k)).to(torch.bfloat16)

    m = case["m"]
    if op in ("linear", "linear_backward"):
        n, k = case["n"], case["k"]
        s["x"], s["w"] = activations(m, k), weight(n, k)
        if op == "linear":
            s["b"] = (0.1 * randn(n)).to(torch.bfloat16) if case["bias"] else None
            s["r"] = randn(m, n).to(torch.bfloat16) if case["residual"] else None
            return s
        s["dy"] = (randn(m, n) * 1e-3).to(torch.bfloat16)
        s["z"] = randn(m, n).to(torch.bfloat16) if case["act"] else None
        return s
    c, f = case["c"], case["f"]
    s["x"], s["wg"], s["wu"] = activations(m, c), weight(f, c), weight(f, c)
    if op == "gated":
        return s
    s["wd"] = weight(c, f)
    s["dy"] = (randn(m, c) * 1e-3).to(torch.bfloat16)
    if op == "step":
        s["r"] = randn(m, c).to(torch.bfloat16)
        return s
    # what the forward pass saved
    g, u = s["x"].float() @ s["wg"].float().t(), s["x"].float() @ s["wu"].float().t()
    if case["save"] == "bf16":
        s["saved"] = g.to(torch.bfloat16), u.to(torch.bfloat16)
    else:
        s["saved"] = _codes(g) + _codes(u)
    return s


# ---------------------------------------------------------------- the plain form
def _codes(y):
    """Codes (rows at a multiple of 128 bytes, as the framework lays them out) and scales of y's rows (32 bits)."""
    r, c = y.shape
    kb = -(-c // 128)
    kt = -(-kb // 4)
    held = torch.zeros(r, kb * 128, device=y.device)
    held[:, :c] = y
    bits = held.view(r, kb, 128).abs().amax(2).view(torch.int32)
    e = ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).int()).clamp_min(0)
    up = ((254 - e) << 23).view(torch.float32)  # 2^(127 - e)
    codes = (held.view(r, kb, 128) * up[:, :, None]).view(r, kb * 128).to(torch.float8_e4m3fn)[:, :c]
    e = torch.nn.functional.pad(e, (0, kt * 4 - kb), value=127).to(torch.uint8)
    return codes, e.view(r, kt, 4).permute(1, 0, 2).contiguous().view(torch.float8_e8m0fnu)


def _values(codes, scales):
    e = scales.view(torch.uint8).permute(1, 0, 2).reshape(codes.shape[0], -1).float() - 127.0
    return codes.float() * torch.exp2(e).repeat_interleave(128, 1)[:, : codes.shape[1]]


def _act_plain(name, z):
    """act(z) and act'(z) of 32-bit values."""
    if name is None:
        return z, torch.ones_like(z)
    if name == "relu":
        on = (z > 0).float()
        return z * on, on
    if name == "gelu":
        cdf = 0.5 * torch.erfc(z * -(0.5**0.5))
        return z * cdf, cdf + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if name == "silu":
        sig = 1.0 / (1.0 + torch.exp(-z))
        return z * sig, sig * (1.0 + z * (1.0 - sig))
    a = 2.0 * math.sqrt(2.0 / math.pi)  # gelu by tanh: z / (1 + exp(-a (z + 0.044715 z^3)))
    sig = 1.0 / (1.0 + torch.exp(-a * (z + 0.044715 * z * z * z)))
    return z * sig, sig + z * sig * (1.0 - sig) * a * (1.0 + 3.0 * 0.044715 * z * z)


def _bf16(v):
    return v.to(torch.bfloat16)


def _gated_backward_plain(s, g, u):
    case = s["case"]
    x, wg, wu, wd, dy = (s[name].float() for name in ("x", "wg", "wu", "wd", "dy"))
    a, da = _act_plain(case["act"], g)
    dh = dy @ wd
    # held in bf16 between the products
    dg, du, h = _bf16(dh * u * da).float(), _bf16(dh * a).float(), _bf16(a * u).float()
    return _bf16(dg @ wg + du @ wu), _bf16(dg.t() @ x), _bf16(du.t() @ x), _bf16(dy.t() @ h)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "linear":
        z = s["x"].float() @ s["w"].float().t()
        if s["b"] is not None:
            z = z + s["b"].float()
        y = _act_plain(case["act"], z)[0]
        if s["r"] is not None:
            y = y + s["r"].float()
        y = _bf16(y) if case["out"] == "bf16" else y
        return (y, _bf16(z)) if case["save"] else y
    if op == "linear_backward":
        dz = s["dy"].float()
        if case["act"]:
            dz = dz * _act_plain(case["act"], s["z"].float())[1]
        held = _bf16(dz).float()  # held in bf16 for the products
        out = _bf16(held @ s["w"].float()), _bf16(held.t() @ s["x"].float())
        return out + (dz.sum(0),) if case["bias"] else out
    if op == "gated_backward":
        if case["save"] == "bf16":
            g, u = (v.float() for v in s["saved"])
        else:
            g, u = _values(*s["saved"][:2]), _values(*s["saved"][2:])
        return _gated_backward_plain(s, g, u)
    g, u = s["x"].float() @ s["wg"].float().t(), s["x"].float() @ s["wu"].float().t()
    h = _bf16(_act_plain(case["act"], g)[0] * u)
    if op == "gated":
        return (h, _bf16(g), _bf16(u)) if case["save"] else h
    y = _bf16(h.float() @ s["wd"].float().t() + s["r"].float())
    return (y,) + _gated_backward_plain(s, _values(*_codes(g)), _values(*_codes(u)))


# ---------------------------------------------------------------- the framework's kernels
def _run_own(s):
    from warp_specialized_tma_gb300 import ffn

    case = s["case"]
    op, act = case["op"], case["act"]
    if op == "linear":
        out = torch.bfloat16 if case["out"] == "bf16" else torch.float32
        return ffn.linear(s["x"], s["w"], bias=s["b"], activation=act, residual=s["r"], save=case["save"], out_dtype=out)
    if op == "linear_backward":
        dx, dw, db = ffn.linear_backward(s["dy"], s["x"], s["w"], z=s["z"], activation=act, bias=case["bias"])
        return (dx, dw, db) if case["bias"] else (dx, dw)
    if op == "gated":
        if case["save"] is None:
            return ffn.gated(s["x"], s["wg"], s["wu"], activation=act)
        h, saved = ffn.gated(s["x"], s["wg"], s["wu"], activation=act, save=case["save"])
        return (h,) + tuple(saved)
    if op == "gated_backward":
        return ffn.gated_backward(s["dy"], s["x"], s["saved"], s["wg"], s["wu"], s["wd"], activation=act)
    h, saved = ffn.gated(s["x"], s["wg"], s["wu"], activation=act, save=case["save"])
    y = ffn.linear(h, s["wd"], residual=s["r"])
    return (y,) + ffn.gated_backward(s["dy"], s["x"], saved, s["wg"], s["wu"], s["wd"], activation=act)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- the definition in 64 bits
def _exact_act(name, z):
    if name is None:
        return z
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "gelu":
        return z * torch.special.erfc(-z / 2**0.5) / 2
    if name == "silu":
        return z * torch.sigmoid(z)
    return z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z**3))) / 2


def _exact_slope(name, z):
    if name == "relu":
        return (z > 0).double()
    if name == "gelu":
        return torch.special.erfc(-z / 2**0.5) / 2 + z * torch.exp(-z * z / 2) / (2 * math.pi) ** 0.5
    if name == "silu":
        return torch.sigmoid(z) * (1 + z * torch.sigmoid(-z))
    t = torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z**3))
    return (1 + t) / 2 + z * (1 - t * t) / 2 * (2 / math.pi) ** 0.5 * (1 + 0.134145 * z * z)


def _exact_saved(v):
    # v as it stands for itself in 8 bits: the nearest of sign * j/8 * 2^e, ties to the even j, for each block's scale
    r, c = v.shape
    blocks = torch.nn.functional.pad(v, (0, -c % 128)).reshape(r, -1, 128)
    top = blocks.abs().max(2, keepdim=True).values
    e = torch.ceil(torch.log2(top.clamp_min(2.0**-118) / 448.0))
    e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)
    e = torch.where(top <= 448.0 * torch.exp2(e - 1), e - 1, e).clamp_min(-127.0)
    scaled = blocks / torch.exp2(e)
    step = torch.exp2(torch.floor(torch.log2(scaled.abs().clamp_min(2.0**-6))) - 3)
    return (torch.round(scaled / step) * step * torch.exp2(e)).reshape(r, -1)[:, :c]


def _exact_backward(case, s, g, u):
    x, wg, wu, wd, dy = (s[name].double() for name in ("x", "wg", "wu", "wd", "dy"))
    dh = torch.einsum("mn,nf->mf", dy, wd)
    dg = (dh * u * _exact_slope(case["act"], g)).to(torch.bfloat16).double()
    du = (dh * _exact_act(case["act"], g)).to(torch.bfloat16).double()
    h = (_exact_act(case["act"], g) * u).to(torch.bfloat16).double()
    del dh
    dx = torch.einsum("mf,fc->mc", dg, wg) + torch.einsum("mf,fc->mc", du, wu)
    return dx, torch.einsum("mf,mc->fc", dg, x), torch.einsum("mf,mc->fc", du, x), torch.einsum("mn,mf->nf", dy, h)


def exact(case, seed):
    s = prepare(case, seed)
    op, act = case["op"], case["act"]
    if op == "linear":
        z = torch.einsum("mk,nk->mn", s["x"].double(), s["w"].double())
        z = z if s["b"] is None else z + s["b"].double()
        y = _exact_act(act, z)
        y = y if s["r"] is None else y + s["r"].double()
        return (y, z) if case["save"] else y
    if op == "linear_backward":
        dz = s["dy"].double()
        if act:
            dz = dz * _exact_slope(act, s["z"].double())
        held = dz.to(torch.bfloat16).double()
        out = torch.einsum("mn,nk->mk", held, s["w"].double()), torch.einsum("mn,mk->nk", held, s["x"].double())
        return out + (torch.einsum("mn->n", dz),) if case["bias"] else out
    if op == "gated_backward":
        if case["save"] == "bf16":
            g, u = (v.double() for v in s["saved"])
        else:
            g, u = (_exact_codes(*s["saved"][i : i + 2]) for i in (0, 2))
        return _exact_backward(case, s, g, u)
    g = torch.einsum("mc,fc->mf", s["x"].double(), s["wg"].double())
    u = torch.einsum("mc,fc->mf", s["x"].double(), s["wu"].double())
    h = _exact_act(act, g) * u
    if op == "gated":
        return (h, g, u) if case["save"] else h
    y = torch.einsum("mf,nf->mn", h.to(torch.bfloat16).double(), s["wd"].double()) + s["r"].double()
    return (y,) + _exact_backward(case, s, _exact_saved(g), _exact_saved(u))


def _exact_codes(codes, scales):
    cols = torch.arange(codes.shape[1], device=codes.device)
    byte = scales.view(torch.uint8)[cols // 512, :, cols // 128 % 4].t()
    return codes.double() * torch.exp2(byte.double() - 127.0)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op, m = case["op"], case["m"]
    if op == "linear":
        n, k = case["n"], case["k"]
        nbytes = 2 * (m * k + n * k) + m * n * (2 if case["out"] == "bf16" else 4)
        nbytes += 2 * n * case["bias"] + 2 * m * n * case["residual"] + 2 * m * n * case["save"]
        return {"bytes": nbytes, "flops": 2 * m * n * k}
    if op == "linear_backward":
        n, k = case["n"], case["k"]
        return {"bytes": 2 * (2 * m * k + 2 * n * k + m * n * (2 if case["act"] else 1)) + 4 * n * case["bias"], "flops": 4 * m * n * k}
    c, f = case["c"], case["f"]
    saved = {None: 0, "bf16": 4 * m * f, "e4m3": 2 * m * (f + -(-f // 128))}[case["save"]]
    forward = 2 * m * c + 4 * f * c + 2 * m * f
    if op == "gated":
        return {"bytes": forward + saved, "flops": 4 * m * c * f}
    # dy, x, what was saved and three weights; dx and three gradients
    backward = 4 * m * c + saved + 6 * c * f + 2 * m * c + 6 * c * f
    if op == "gated_backward":
        return {"bytes": backward, "flops": 12 * m * c * f}
    # the step reads x and each weight once, and writes y, dx and the gradients; h and the checkpoints stay between
    return {"bytes": 2 * m * c * 5 + 12 * c * f, "flops": 18 * m * c * f}
