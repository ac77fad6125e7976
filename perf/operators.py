"""Cases for the microscaled 4-bit operators: quantisation, products, products grouped by expert.

A matrix in 4 bits holds e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) in blocks along its
depth (the dimension that a product sums over), with one scale a block:

* ``nv``: blocks of 16, the scale s in e4m3, and one fp32 scale g for the matrix; value = code * s * g;
* ``mx``: blocks of 32, the scale a power of two (e8m0); value = code * s.

``run`` takes a case through quantisation (and back), a linear layer, a linear layer's gradients, the
products of an expert layer, or their gradients.
"""
import math

import torch

own = False

BLOCK = {"nv": 16, "mx": 32}
DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TOP = 6.0 * 448.0  # the largest value of an nv block over its matrix's scale


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # a feed-forward weight put into 4 bits once and read back: the pruned weight's kept values only
        dict(name="round_weight", kind="round", fmt="nv", rows=11008, depth=4096, axis=1, dtype="bf16",
             scale="amax", mask=True),
        # a prompt's activations, stored channel by token, blocks down the channels
        dict(name="round_columns", kind="round", fmt="mx", rows=4096, depth=4096, axis=0, dtype="bf16",
             scale="none", mask=False),
        # a small matrix of odd sizes in 32 bits with a scale from calibration
        dict(name="round_odd", kind="round", fmt="nv", rows=77, depth=1003, axis=1, dtype="fp32",
             scale="given", mask=False),
        # one token through an attention projection: latency
        dict(name="linear_token", kind="linear", fmt="nv", M=4096, K=4096, N=1, axis=1, out="bf16",
             scale="given", act="none", bias=True),
        # a batch of decoded tokens through the down projection
        dict(name="linear_decode", kind="linear", fmt="mx", M=4096, K=11008, N=32, axis=1, out="bf16",
             scale="none", act="none", bias=False),
        # a prompt through the up projection, channel by token
        dict(name="linear_prompt", kind="linear", fmt="nv", M=11008, K=4096, N=4096, axis=0, out="bf16",
             scale="amax", act="silu", bias=False),
        # odd sizes everywhere, 32-bit output
        dict(name="linear_odd", kind="linear", fmt="mx", M=1000, K=1547, N=777, axis=0, out="fp32",
             scale="none", act="gelu", bias=True),
        # the gradients of a linear layer: W, dY and X quantised along the summed dimension of each product
        dict(name="linear_grad", kind="grad", fmt="nv", M=4096, K=4096, N=8192, scale="amax"),
        # decoded tokens over many experts, several without any
        dict(name="experts_decode", kind="experts", fmt="nv", E=32, M=2048, K=1024, tokens=96,
             capacity=128, scale="given"),
        # a prompt over the experts, tokens shared out unevenly
        dict(name="experts_prompt", kind="experts", fmt="mx", E=16, M=4096, K=2048, tokens=16001,
             capacity=16384, scale="none"),
        # a handful of tokens over small experts
        dict(name="experts_small", kind="experts", fmt="nv", E=4, M=257, K=272, tokens=7,
             capacity=8, scale="given"),
        # the gradients of an expert layer's product: the weight's sum over each expert's own tokens
        dict(name="experts_grad", kind="experts_grad", fmt="nv", E=16, M=2048, K=1024, tokens=8111,
             capacity=8192, scale="amax"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["round", "round", "linear", "linear", "linear", "grad", "experts", "experts",
                       "experts_grad"])
    fmt = rng.choice(["nv", "mx"])
    scale = rng.choice(["amax", "given"]) if fmt == "nv" else "none"
    if kind == "round":
        rows = _log(rng, 1, 11008)
        depth = _log(rng, 64, max(64, min(16384, 45_000_000 // rows)))
        return dict(kind=kind, fmt=fmt, rows=rows, depth=depth, axis=rng.choice([0, 1]),
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), scale=scale,
                    mask=rng.random() < 0.3)
    if kind == "linear":
        M, K = _log(rng, 64, 11008), _log(rng, 64, 11008)
        N = _log(rng, 1, max(1, min(4096, 180_000_000_000 // (M * K))))
        return dict(kind=kind, fmt=fmt, M=M, K=K, N=N, axis=rng.choice([0, 1]),
                    out=rng.choice(["bf16", "bf16", "fp16", "fp32"]), scale=scale,
                    act=rng.choice(["none", "relu", "silu", "gelu"]), bias=rng.random() < 0.5)
    if kind == "grad":
        M, K = _log(rng, 64, 4096), _log(rng, 64, 4096)
        return dict(kind=kind, fmt=fmt, M=M, K=K, N=_log(rng, 16, 8192), scale="amax" if fmt == "nv" else "none")
    E, tokens = _log(rng, 2, 64), _log(rng, 4, 8192 if kind == "experts_grad" else 16384)
    M, K = _log(rng, 64, 2048), _log(rng, 64, 2048)
    if kind == "experts_grad" and fmt == "nv":
        scale = "amax"
    return dict(kind=kind, fmt=fmt, E=E, M=M, K=K, tokens=tokens,
                capacity=tokens + rng.choice([0, 1, 64]), scale=scale)


# ----------------------------------------------------------------------------- inputs
def _pow2(e):
    """2 ** (e - 127) for whole e >= 0, from its bits (a power computed as such may be off by a bit)."""
    return torch.where(e > 0, e << 23, torch.full_like(e, 1 << 22)).view(torch.float32)


def _pow2_scale(amax):
    """The power of two g with amax / g <= 6 * 448 < 2 amax / g."""
    m, e = torch.frexp(amax.double() / TOP)
    e = torch.where(m > 0.5, e, e - 1).clamp(-126, 126)
    return _pow2(torch.where(amax > 0, e, torch.full_like(e, -126)).int() + 127)


def _pack(w, fmt):
    """Weights [E, R, D] in the packed form that a program keeps: codes [E * R, ceil(D / 128) * 64] with
    two to a byte (the lower nibble first), scales [E, ceil(R / 128), chunks, 512] (a chunk is 4 blocks of
    depth; the byte of row r and block b of it at 16 (r mod 32) + 4 (r / 32 mod 4) + b), g [E]."""
    E, R, D = w.shape
    B, Dp, Rp = BLOCK[fmt], (D + 127) // 128 * 128, (R + 127) // 128 * 128
    g = _pow2_scale(w.abs().amax((1, 2)).float()) if fmt == "nv" else torch.ones(E, device=w.device)
    x = torch.zeros(E, Rp, Dp, device=w.device)
    x[:, :R, :D] = w.float() / g[:, None, None]
    x = x.view(E, Rp, Dp // B, B)
    a = x.abs().amax(-1)
    if fmt == "nv":
        sb = (a / 6).clamp(max=448.0).to(torch.float8_e4m3fn)
        s, sb = sb.float(), sb.view(torch.uint8)
    else:
        sb = ((a.view(torch.int32) >> 23) - 2).clamp(min=0)
        s = _pow2(sb)
    q = torch.where(s[..., None] > 0, x / s[..., None], torch.zeros_like(x))
    n = q.abs()
    c = ((n > 0.25).int() + (n >= 0.75) + (n > 1.25) + (n >= 1.75) + (n > 2.5) + (n >= 3.5) + (n > 5))
    c = (c + 8 * torch.signbit(q)).view(E, Rp, Dp)[:, :R].to(torch.uint8)
    values = (c[..., 0::2] | (c[..., 1::2] << 4)).reshape(E * R, Dp // 2).contiguous()
    chunks = Dp // (4 * B)
    scales = sb.to(torch.uint8).view(E, Rp // 128, 4, 32, chunks, 4).permute(0, 1, 4, 3, 2, 5)
    return values, scales.reshape(E, Rp // 128, chunks, 512).contiguous(), g


def _counts(E, tokens, g):
    """How many of the tokens each expert gets: uneven shares, some experts none."""
    share = torch.rand(E, generator=g) ** 2 + 0.02
    share[torch.rand(E, generator=g) < 0.15] = 0
    share[int(torch.randint(E, (1,), generator=g))] += 0.5
    cut = (share.double().cumsum(0) / share.double().sum() * tokens).round().long()
    return torch.diff(cut, prepend=torch.zeros(1, dtype=torch.long))


def _activations(shape, g, dtype, channel_dim):
    """N(0, 1) with a few channels ten times as large, as activations of language models have them."""
    x = torch.randn(shape, generator=g, device="cuda")
    n = shape[channel_dim]
    big = torch.ones(n, device="cuda")
    big[torch.rand(n, generator=g, device="cuda") < 0.01] = 10.0
    view = [1] * len(shape)
    view[channel_dim] = n
    return (x * big.view(view)).to(dtype)


def _input_scale(c, like):
    """A given scale is one of calibration: what covers values up to about 60."""
    if c["fmt"] != "nv":
        return None
    return torch.full((1,), 0.0225, device="cuda") if c["scale"] == "given" else "amax"


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.Generator().manual_seed(seed)
    s = {"case": c}
    if c["kind"] == "round":
        shape = (c["rows"], c["depth"]) if c["axis"] == 1 else (c["depth"], c["rows"])
        x = torch.randn(shape, generator=g, device="cuda") * 0.02
        s["x"] = torch.where(torch.rand(shape, generator=g, device="cuda") < 0.002, x * 10, x).to(DTYPE[c["dtype"]])
        s["scale"] = None if c["fmt"] == "mx" else "amax" if c["scale"] == "amax" else torch.full((1,), 1.1e-4, device="cuda")
        s["bits"] = None
        if c["mask"]:  # kept elements, 32 to a word; whole blocks are pruned in places
            R, C = shape
            keep = torch.rand(R, (C + 31) // 32, 32, generator=g, device="cuda") < 0.5
            keep &= torch.rand(R, (C + 31) // 32, 1, generator=g, device="cuda") < 0.9
            w = (keep.long() << torch.arange(32, device="cuda")).sum(-1)
            s["bits"] = torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)
        s["out"] = torch.empty(shape, dtype=DTYPE[c["dtype"]], device="cuda")
    elif c["kind"] == "linear":
        M, K, N = c["M"], c["K"], c["N"]
        w = (torch.randn(1, M, K, generator=g, device="cuda") * 0.02).bfloat16()
        s["w"] = _pack(w, c["fmt"])
        s["x"] = _activations((N, K) if c["axis"] == 1 else (K, N), g, torch.bfloat16, c["axis"])
        s["scale"] = _input_scale(c, s["x"])
        s["bias"] = torch.randn(M, generator=g, device="cuda") * 0.1 if c["bias"] else None
        s["out"] = torch.empty((N, M) if c["axis"] == 1 else (M, N), dtype=DTYPE[c["out"]], device="cuda")
    elif c["kind"] == "grad":
        M, K, N = c["M"], c["K"], c["N"]
        s["w"] = (torch.randn(M, K, generator=g, device="cuda") * 0.02).bfloat16()
        s["x"] = _activations((K, N), g, torch.bfloat16, 0)
        s["dy"] = (torch.randn(M, N, generator=g, device="cuda") * 1e-3).bfloat16()
        s["scale"] = "amax" if c["fmt"] == "nv" else None
        s["dx"] = torch.empty((K, N), dtype=torch.bfloat16, device="cuda")
        s["dw"] = torch.empty((M, K), dtype=torch.float32, device="cuda")
    else:
        E, M, K, T = c["E"], c["M"], c["K"], c["capacity"]
        n = _counts(E, c["tokens"], h)
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.long), n.cumsum(0)]).to(torch.int32).cuda()
        s["most"] = (int(n.max()) + 31) // 32 * 32  # host knowledge of the router's plan
        w = (torch.randn(E, M, K, generator=g, device="cuda") * 0.02).bfloat16()
        s["x"] = _activations((T, K), g, torch.bfloat16, 1)
        if c["kind"] == "experts":
            s["w"] = _pack(w, c["fmt"])
            s["scale"] = _input_scale(c, s["x"])
            s["out"] = torch.zeros((T, M), dtype=torch.bfloat16, device="cuda")
        else:
            s["w"] = w
            s["dy"] = (torch.randn(T, M, generator=g, device="cuda") * 1e-3).bfloat16()
            s["scale"] = "amax" if c["fmt"] == "nv" else None
            s["dx"] = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
            s["dw"] = torch.empty((E, M, K), dtype=torch.float32, device="cuda")
    return s


# ----------------------------------------------------------------------------- plain forms
def _scale_of(x, scale):
    """g: given, or from the largest magnitude of all of x."""
    if scale is None:
        return torch.ones(1, device=x.device)
    return scale if torch.is_tensor(scale) else _pow2_scale(x.abs().amax().view(1).float())


def _rounded(x, fmt, g):
    """x (32 bits, [..., depth]; depth a multiple of the block) in 4 bits, read back: code * s, and g aside."""
    x = (x * (1.0 / g)).unflatten(-1, (-1, BLOCK[fmt]))
    a = x.abs().amax(-1, keepdim=True)
    if fmt == "nv":
        s = (a / 6).clamp(max=448.0).to(torch.float8_e4m3fn).float()
    else:
        s = _pow2(((a.view(torch.int32) >> 23) - 2).clamp(min=0))
    q = torch.where(s > 0, x / s, torch.zeros_like(x))
    n = q.abs()
    n = (0.5 * (n > 0.25) + 0.5 * (n >= 0.75) + 0.5 * (n > 1.25) + 0.5 * (n >= 1.75) + 1.0 * (n > 2.5)
         + 1.0 * (n >= 3.5) + 2.0 * (n > 5))
    return (torch.copysign(n, q) * s).flatten(-2)


def _quantized(x, fmt, scale):
    """_rounded with any depth, and the scale g."""
    x = x.float()
    g = _scale_of(x, scale)
    D, B = x.shape[-1], BLOCK[fmt]
    return _rounded(torch.nn.functional.pad(x, (0, -D % B)), fmt, g)[..., :D], g


def _unpacked(w, fmt, R, D):
    """The packed weights' values [E, R, D] without g, and g."""
    values, scales, g = w
    E, B = g.numel(), BLOCK[fmt]
    c = torch.stack([values & 15, values >> 4], -1).view(E, R, -1).long()
    table = torch.tensor([0.0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=values.device)
    t, n = scales.shape[1], scales.shape[2]
    b = scales.view(E, t, n, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(E, t * 128, n * 4)[:, :R]
    s = (b.contiguous().view(torch.float8_e4m3fn).float() if fmt == "nv" else _pow2(b.int()))
    return (table[c] * s.repeat_interleave(B, -1))[..., :D], g


def _activated(y, act):
    if act == "relu":
        return y.clamp(min=0)
    if act == "silu":
        return y / (1 + torch.exp(-y))
    return y * (1 + torch.erf(y * 0.5 ** 0.5)) / 2 if act == "gelu" else y


def _by_expert(x, offsets, most):
    """Tokens [T, C] as [E, most, C], zeros behind each expert's last, and where each one came from."""
    at = offsets[:-1, None].long() + torch.arange(most, device=x.device)
    real = at < offsets[1:, None]
    at = at.clamp(max=x.shape[0] - 1)
    return torch.where(real[..., None], x[at], torch.zeros((), device=x.device, dtype=x.dtype)), at, real


def _back(y, at, real, like):
    """The experts' rows [E, most, C] at their tokens' places; zeros elsewhere."""
    out = torch.zeros(like.shape, device=y.device)
    out[at[real]] = y[real]
    return out


def run(s):
    return _own(s) if own else _plain(s)


def _plain(s):
    c = s["case"]
    fmt = c["fmt"]
    if c["kind"] == "round":
        x = s["x"].float()
        if s["bits"] is not None:
            keep = (s["bits"][..., None] >> torch.arange(32, device=x.device)) & 1
            x = torch.where(keep.flatten(-2)[:, :x.shape[1]] > 0, x, torch.zeros_like(x))
        q, g = _quantized(x if c["axis"] == 1 else x.t(), fmt, s["scale"])
        q = q * g
        return (q if c["axis"] == 1 else q.t()).to(s["x"].dtype)
    if c["kind"] == "linear":
        w, gw = _unpacked(s["w"], fmt, c["M"], c["K"])
        x, gx = _quantized(s["x"] if c["axis"] == 1 else s["x"].t(), fmt, s["scale"])
        y = (w[0] @ x.t()) * (gw * gx)
        if s["bias"] is not None:
            y = y + s["bias"][:, None]
        y = _activated(y, c["act"]).to(s["out"].dtype)
        return y.t().contiguous() if c["axis"] == 1 else y
    if c["kind"] == "grad":
        w, gw = _quantized(s["w"].t(), fmt, s["scale"])
        d, gd = _quantized(s["dy"].t(), fmt, s["scale"])
        dx = (w @ d.t()) * (gw * gd)
        d, gd = _quantized(s["dy"], fmt, s["scale"])
        x, gx = _quantized(s["x"], fmt, s["scale"])
        return dx.bfloat16(), (d @ x.t()) * (gd * gx)
    x, at, real = _by_expert(s["x"], s["offsets"], s["most"])
    if c["kind"] == "experts":
        w, gw = _unpacked(s["w"], fmt, c["M"], c["K"])
        x, gx = _quantized(x, fmt, s["scale"])
        return _back(torch.bmm(x, w.transpose(1, 2)) * (gw * gx)[:, None, None], at, real, s["out"]).bfloat16()
    d, at, real = _by_expert(s["dy"], s["offsets"], s["most"])
    w = s["w"].float().transpose(1, 2)
    gw = _pow2_scale(w.abs().amax((1, 2)))[:, None, None] if fmt == "nv" else torch.ones(c["E"], 1, 1, device=w.device)
    w = _rounded(torch.nn.functional.pad(w, (0, -c["M"] % BLOCK[fmt])), fmt, gw)[..., :c["M"]]
    q, gd = _quantized(d, fmt, s["scale"])
    dx = _back(torch.bmm(q, w.transpose(1, 2)) * (gw * gd), at, real, s["dx"]).bfloat16()
    q, gd = _quantized(d.transpose(1, 2), fmt, s["scale"])
    x, gx = _quantized(x.transpose(1, 2), fmt, s["scale"])
    return dx, torch.bmm(q, x.transpose(1, 2)) * (gd * gx)


# ----------------------------------------------------------------------------- the framework's calls
def _own(s):
    import pruning_hinm_spmm_b200 as H

    c = s["case"]
    fmt = H.HINM_FP4_NV if c["fmt"] == "nv" else H.HINM_FP4_MX
    keep = s.setdefault("own", {})  # the buffers and weights that a program lays out once
    if c["kind"] == "round":
        q = keep["q"] = H.hinm_fp4_quantize(s["x"], fmt, axis=c["axis"], bitmask=s["bits"],
                                            tensor_scale=s["scale"], out=keep.get("q"))
        return H.hinm_fp4_dequantize(q, axis=c["axis"], out=s["out"])
    if c["kind"] in ("linear", "experts") and "w" not in keep:
        keep["w"] = H.Fp4Matrix(format=fmt, batch=c.get("E", 1), rows=c["M"], depth=c["K"], values=s["w"][0],
                                scales=s["w"][1], tensor_scale=s["w"][2] if c["fmt"] == "nv" else None)
    if c["kind"] == "linear":
        x = keep["x"] = H.hinm_fp4_quantize(s["x"], fmt, axis=c["axis"], tensor_scale=s["scale"],
                                            out=keep.get("x"))
        act = {"none": H.HINM_ACT_NONE, "relu": H.HINM_ACT_RELU, "silu": H.HINM_ACT_SILU,
               "gelu": H.HINM_ACT_GELU}[c["act"]]
        return H.hinm_fp4_matmul(keep["w"], x, Y_out=s["out"], transposed=c["axis"] == 1, bias=s["bias"],
                                 activation=act)
    if c["kind"] == "grad":
        def quantized(name, x, axis):
            keep[name] = H.hinm_fp4_quantize(x, fmt, axis=axis, tensor_scale=s["scale"], out=keep.get(name))
            return keep[name]
        H.hinm_fp4_matmul(quantized("w", s["w"], 0), quantized("d", s["dy"], 0), Y_out=s["dx"])
        H.hinm_fp4_matmul(quantized("d2", s["dy"], 1), quantized("x", s["x"], 1), Y_out=s["dw"])
        return s["dx"], s["dw"]

    def tokens(name, x, axis, ragged):
        keep[name] = H.hinm_fp4_quantize(x, fmt, axis=axis, offsets=s["offsets"], ragged=ragged,
                                         tensor_scale=s["scale"], out=keep.get(name))
        return keep[name]
    if c["kind"] == "experts":
        return H.hinm_fp4_grouped_matmul(keep["w"], tokens("x", s["x"], 1, H.HINM_RAGGED_ROWS), Y_out=s["out"],
                                         transposed=True)
    w = keep["w"] = H.hinm_fp4_quantize(s["w"], fmt, axis=0, tensor_scale=s["scale"], out=keep.get("w"))
    H.hinm_fp4_grouped_matmul(w, tokens("d", s["dy"], 1, H.HINM_RAGGED_ROWS), Y_out=s["dx"], transposed=True)
    H.hinm_fp4_grouped_weight_grad(tokens("d2", s["dy"], 0, H.HINM_RAGGED_DEPTH),
                                   tokens("x", s["x"], 0, H.HINM_RAGGED_DEPTH), Y_out=s["dw"])
    return s["dx"], s["dw"]


# ----------------------------------------------------------------------------- what a pass cannot do without
def _size(dtype):
    return {"bf16": 2, "fp16": 2, "fp32": 4}[dtype]


def work(case):
    c = case
    four = 0.5 + 1.0 / BLOCK[c["fmt"]]  # bytes an element
    if c["kind"] == "round":  # read, written in 4 bits, read from there, written as values
        n = c["rows"] * c["depth"]
        return {"bytes": n * (2 * _size(c["dtype"]) + 2 * four + (0.125 if c["mask"] else 0)), "flops": 0}
    if c["kind"] == "linear":
        M, K, N = c["M"], c["K"], c["N"]
        return {"bytes": M * K * four + 2 * K * N + M * N * _size(c["out"]), "flops": 2 * M * K * N}
    if c["kind"] == "grad":
        M, K, N = c["M"], c["K"], c["N"]
        return {"bytes": 2 * (M * K + M * N + K * N) + 2 * K * N + 4 * M * K, "flops": 4 * M * K * N}
    E, M, K, T = c["E"], c["M"], c["K"], c["tokens"]
    if c["kind"] == "experts":
        return {"bytes": min(E, T) * M * K * four + 2 * T * (K + M), "flops": 2 * T * M * K}
    return {"bytes": E * M * K * (2 + 4) + 2 * T * (2 * K + M), "flops": 4 * T * M * K}


# ----------------------------------------------------------------------------- from the definition, in 64 bits
def _x_pow2(amax):
    """Smallest power of two g with amax <= 2688 g."""
    a = float(amax)
    if a == 0:
        return 2.0 ** -126
    k = math.ceil(math.log2(a / TOP))
    while a > TOP * 2.0 ** k:
        k += 1
    while a <= TOP * 2.0 ** (k - 1):
        k -= 1
    return 2.0 ** max(-126, min(126, k))


def _x_nearest(v, grid):
    """The nearest of a grid of ascending values, of two as near the one at the even place; 64 bits."""
    hi = torch.searchsorted(grid, v.contiguous()).clamp(1, grid.numel() - 1)
    lo = hi - 1
    up, down = grid[hi] - v, v - grid[lo]
    at = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return grid[at]


def _x_quantized(x, fmt, scale):
    """x [rows, depth] in 64 bits after the round trip through 4 bits, with its scale g in it."""
    R, D = x.shape
    B = BLOCK[fmt]
    g = 1.0
    if scale is not None:
        g = float(scale) if torch.is_tensor(scale) else _x_pow2(x.abs().max() if x.numel() else 0)
    # the definition divides by g in 32 bits: its reciprocal and the product are rounded to them
    inv = float(torch.tensor(1.0 / g, dtype=torch.float64).float())
    p = torch.zeros(R, -(-D // B) * B, dtype=torch.float64, device=x.device)
    p[:, :D] = (x * inv).float().double()
    p = p.view(R, -1, B)
    a = p.abs().max(-1, keepdim=True).values
    e2m1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    if fmt == "nv":
        e4m3 = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1]
        s = _x_nearest(torch.clamp(a / 6, max=448.0), torch.tensor(e4m3, dtype=torch.float64, device=x.device))
    else:
        m = torch.frexp(a).mantissa  # in [1/2, 1): a / (2 m) is 2 ** floor(log2(a)), exactly
        s = torch.where(a > 0, a / (8 * m), torch.zeros_like(a)).clamp(min=2.0 ** -127)
    q = _x_nearest(torch.where(s > 0, p.abs() / s, torch.zeros_like(p)), e2m1)
    return (torch.sign(p) * q * s).view(R, -1)[:, :D] * g


def _x_weight(w, fmt, e, R, D):
    """Expert e of the packed weights, read byte by byte from the layout's definition."""
    values, scales, g = w
    dev = values.device
    mag = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=dev)
    r, d = torch.arange(R, device=dev)[:, None], torch.arange(D, device=dev)[None]
    nib = (values[e * R:(e + 1) * R].int()[r, d // 2] >> (4 * (d % 2))) & 15
    v = mag[(nib & 7).long()] * (1.0 - 2.0 * (nib >> 3).double())
    b = d // BLOCK[fmt]
    code = scales[e][r // 128, b // 4, 16 * (r % 32) + 4 * (r // 32 % 4) + b % 4].int()
    if fmt == "nv":
        ex, m = (code >> 3) & 15, (code & 7).double()
        s = torch.where(ex > 0, (8 + m) * 2.0 ** (ex.double() - 10), m * 2.0 ** -9)
    else:
        s = 2.0 ** (code.double() - 127)
    return v * s * float(g[e])


def exact(case, seed):
    s, c = prepare(case, seed), case
    fmt = c["fmt"]
    if c["kind"] == "round":
        x = s["x"].double()
        if s["bits"] is not None:
            col = torch.arange(x.shape[1], device=x.device)
            x = x * ((s["bits"].long()[:, col // 32] >> (col % 32)) & 1)
        return _x_quantized(x, fmt, s["scale"]) if c["axis"] == 1 else _x_quantized(x.t(), fmt, s["scale"]).t()
    if c["kind"] == "linear":
        x = s["x"].double()
        y = _x_weight(s["w"], fmt, 0, c["M"], c["K"]) @ _x_quantized(x if c["axis"] == 1 else x.t(), fmt, s["scale"]).t()
        if s["bias"] is not None:
            y += s["bias"].double()[:, None]
        y = {"none": lambda v: v, "relu": lambda v: v.clamp(min=0), "silu": lambda v: v * torch.sigmoid(v),
             "gelu": lambda v: 0.5 * v * torch.erfc(-v / math.sqrt(2.0))}[c["act"]](y)
        return y.t() if c["axis"] == 1 else y
    if c["kind"] == "grad":
        dy, x, w = s["dy"].double(), s["x"].double(), s["w"].double()
        return (_x_quantized(w.t(), fmt, s["scale"]) @ _x_quantized(dy.t(), fmt, s["scale"]).t(),
                _x_quantized(dy, fmt, s["scale"]) @ _x_quantized(x, fmt, s["scale"]).t())
    o = s["offsets"].tolist()
    real = s["x"][:o[-1]].double()
    over = lambda t: torch.tensor([_x_pow2(t.abs().max())]) if s["scale"] == "amax" else s["scale"]  # noqa: E731
    gx = over(real)
    if c["kind"] == "experts":
        y = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            if o[e + 1] > o[e]:
                y[o[e]:o[e + 1]] = _x_quantized(real[o[e]:o[e + 1]], fmt, gx) @ _x_weight(s["w"], fmt, e, c["M"], c["K"]).t()
        return y
    dy = s["dy"][:o[-1]].double()
    gd = over(dy)
    dx = torch.zeros(s["dx"].shape, dtype=torch.float64, device="cuda")
    dw = torch.zeros(s["dw"].shape, dtype=torch.float64, device="cuda")
    for e in range(c["E"]):
        if o[e + 1] > o[e]:
            d, x = dy[o[e]:o[e + 1]], real[o[e]:o[e + 1]]
            dx[o[e]:o[e + 1]] = _x_quantized(d, fmt, gd) @ _x_quantized(s["w"][e].double().t(), fmt, s["scale"]).t()
            dw[e] = _x_quantized(d.t(), fmt, gd) @ _x_quantized(x.t(), fmt, gx).t()
    return dx, dw
