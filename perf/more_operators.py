"""More operators around the step, as they are measured: the norm in front of a
layer with its gradients, the microscaled 4-bit copy of a matrix, and the
product of two such copies.

Four operators:

  norm_forward   y = (x - mean) rstd w + b along each row ("layer"), or
                 y = x rstd w + b with rstd of the mean square ("rms")
  norm_backward  dx = rstd (g - mean(g) - xhat mean(g xhat)) + r with
                 g = dy w, xhat = (x - mean) rstd (without the term mean(g) for
                 "rms"); dw = column sums of dy xhat, db = column sums of dy
  mx4_quantize   a matrix as 4-bit codes with one power-of-two scale for 32
                 neighbours of a row (and, for its transpose, of a column), and
                 the values that they stand for read back from them
  mx4_product    y = act(A B^T + bias) + r of two matrices held so

A block of 32 elements with largest magnitude a has the scale 2^s, s =
max(floor(log2 a) - 2, -127), and each element becomes the nearest of 0, 0.5,
1, 1.5, 2, 3, 4 and 6 times the scale, with its sign; halfway cases take the
one whose code is even, and what is above takes 6.  A block of zeros has s =
-127.  In memory a row is whole blocks of 16 bytes, element 2 i of a block in the
low half of byte i (sign, then three bits of magnitude), zeros behind the row's
end, and its scales are bytes s + 127, rounded up to a multiple of 16 by zeros.

With ``own`` false, ``run`` computes them with elementary torch operations in
32 bits; with ``own`` true, through rank_step_amd.binding.
"""

import math

import torch

own = False

WORKSPACE_BYTES = 64 << 20
EPS = 1e-5


# ---------------------------------------------------------------- the cases

def listed():
    nf, nb, q, p = "norm_forward", "norm_backward", "mx4_quantize", "mx4_product"
    return [
        # one token in front of a projection of the 7B block: the call itself
        {"name": "norm one token", "op": nf, "kind": "rms", "m": 1, "n": 4096, "dtype": "bf16", "w": "bf16",
         "bias": False, "stats": False},
        # a long batch in training, the row statistics kept for the backward pass
        {"name": "norm 8192 tokens", "op": nf, "kind": "layer", "m": 8192, "n": 4096, "dtype": "bf16", "w": "bf16",
         "bias": True, "stats": True},
        # the width of the 128 MiB MLP's layers, fp32: rows that start off every vector boundary
        {"name": "norm odd fp32", "op": nf, "kind": "layer", "m": 1000, "n": 1365, "dtype": "f32", "w": "f32",
         "bias": True, "stats": True},
        # its gradients over the long batch, the residual branch's gradient added on the way
        {"name": "norm grad 8192 tokens", "op": nb, "kind": "layer", "m": 8192, "n": 4096, "dtype": "bf16", "w": "bf16",
         "bias": True, "residual": True, "dw": "bf16", "add": False},
        # the MLP's width again, few rows, added to the fp32 gradients that accumulate over micro-batches
        {"name": "norm grad odd fp32", "op": nb, "kind": "layer", "m": 333, "n": 1365, "dtype": "f32", "w": "f32",
         "bias": True, "residual": False, "dw": "f32", "add": True},
        # a rank's shard of the 7B block's gate projection at N = 8: fp32 master weights to the 4-bit copy and back
        {"name": "mx4 weight shard", "op": q, "rows": 1376, "cols": 4096, "dtype": "f32", "both": False},
        # a layer's gradient over a long batch, for the products that contract over features and over tokens
        {"name": "mx4 8192 tokens both ways", "op": q, "rows": 8192, "cols": 4096, "dtype": "bf16", "both": True},
        # a few rows of an odd width: blocks that end early, and the calls themselves
        {"name": "mx4 odd small", "op": q, "rows": 37, "cols": 251, "dtype": "f32", "both": False},
        # one token through an attention output projection of the 7B block
        {"name": "product one token", "op": p, "m": 1, "n": 4096, "k": 4096, "y": "bf16", "act": "none",
         "bias": False, "residual": True, "z": False},
        # sixteen tokens through its gate projection
        {"name": "product 16 tokens", "op": p, "m": 16, "n": 11008, "k": 4096, "y": "bf16", "act": "silu",
         "bias": False, "residual": False, "z": False},
        # a long batch through the gate projection of the 70B block, the pre-activation kept: the largest product
        {"name": "product 8192 tokens", "op": p, "m": 8192, "n": 28672, "k": 8192, "y": "bf16", "act": "silu",
         "bias": False, "residual": False, "z": True},
        # a weight gradient of the 128 MiB MLP, contracted over 2047 tokens and added to the fp32 gradient in place
        {"name": "product odd weight grad", "op": p, "m": 1024, "n": 1365, "k": 2047, "y": "f32", "act": "none",
         "bias": False, "residual": "in place", "z": False},
    ]


def _spread(rng, lo, hi):
    """Log-uniform in [lo, hi]; half of the larger ones a multiple of 64, the others any number."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v >= 64 and rng.random() < 0.5:
        v -= v % 64
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["norm_forward", "norm_backward", "mx4_quantize", "mx4_product", "mx4_product"])
    if op == "mx4_quantize":
        return {"op": op, "rows": _spread(rng, 1, 8192), "cols": _spread(rng, 32, 11008),
                "dtype": rng.choice(["bf16", "f32"]), "both": rng.random() < 0.5}
    m = _spread(rng, 1, 8192)
    if op == "mx4_product":
        n, k = _spread(rng, 64, 28672), _spread(rng, 64, 11008)
        m = min(m, 8192 * 28672 * 8192 // (n * k))  # no more than the largest listed product
        return {"op": op, "m": m, "n": n, "k": k, "y": rng.choice(["bf16", "bf16", "f32"]),
                "act": rng.choice(["none", "none", "relu", "gelu", "silu"]), "bias": rng.random() < 0.5,
                "residual": rng.choice([False, True, "in place"]), "z": rng.random() < 0.5}
    t = rng.choice(["bf16", "f32"])
    c = {"op": op, "kind": rng.choice(["layer", "rms"]), "m": m, "n": _spread(rng, 64, 11008), "dtype": t,
         "w": rng.choice([t, "bf16"]), "bias": rng.random() < 0.5}
    if op == "norm_forward":
        return c | {"stats": rng.random() < 0.7}
    return c | {"residual": rng.random() < 0.5, "dw": rng.choice(["bf16", "f32"]), "add": rng.random() < 0.5}


_BYTES = {"bf16": 2, "f32": 4}


def _codes(cols):
    """Bytes of a row's codes: whole blocks."""
    return 16 * ((cols + 31) // 32)


def _scales(cols):
    """Bytes of a row's scales, rounded up to 16."""
    return 16 * ((cols + 511) // 512)


def work(case):
    op = case["op"]
    if op == "mx4_quantize":
        r, c = case["rows"], case["cols"]
        copy = r * (_codes(c) + (c + 31) // 32)
        if case["both"]:
            copy += c * (_codes(r) + (r + 31) // 32)
        values = (2 if case["both"] else 1) * r * c * 2
        # the matrix is read, its copies are written, read again, and their values are written
        return {"bytes": r * c * _BYTES[case["dtype"]] + 2 * copy + values, "flops": 4 * r * c * (2 if case["both"] else 1)}
    m, n = case["m"], case["n"]
    if op == "mx4_product":
        k, e = case["k"], _BYTES[case["y"]]
        b = (m + n) * (_codes(k) + (k + 31) // 32) + m * n * e
        b += (2 * n if case["bias"] else 0) + (m * n * e if case["residual"] else 0) + (2 * m * n if case["z"] else 0)
        return {"bytes": b, "flops": 2 * m * n * k}
    e, layer = _BYTES[case["dtype"]], case["kind"] == "layer"
    vectors = n * _BYTES[case["w"]]
    if op == "norm_forward":
        vectors += n * _BYTES[case["w"]] if case["bias"] else 0
        stats = (8 if layer else 4) * m if case["stats"] else 0
        return {"bytes": 2 * m * n * e + vectors + stats, "flops": (8 if layer else 5) * m * n}
    vectors += n * _BYTES[case["dw"]] * (2 if case["bias"] else 1) * (2 if case["add"] else 1)
    matrices = 4 if case["residual"] else 3
    return {"bytes": matrices * m * n * e + vectors + (8 if layer else 4) * m, "flops": (14 if layer else 11) * m * n}


# ---------------------------------------------------------------- inputs

_TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


def _blocks(x):
    """[rows, cols] as [rows, blocks, 32], zeros behind the row's end, in 32 bits."""
    pad = -x.shape[1] % 32
    x = x.float()
    if pad:
        x = torch.cat([x, torch.zeros(x.shape[0], pad, dtype=x.dtype, device=x.device)], dim=1)
    return x.reshape(x.shape[0], -1, 32)


def _plain_codes(x):
    """Codes [rows, blocks, 32] and scale exponents [rows, blocks, 1]."""
    x = _blocks(x)
    mantissa, exponent = torch.frexp(x.abs().amax(dim=2, keepdim=True))
    # frexp's mantissa is in [0.5, 1), or 0
    s = torch.where(mantissa == 0, torch.full_like(exponent, -127), (exponent - 3).clamp(min=-127))
    v = torch.ldexp(x.abs(), -s)
    code = ((v > 0.25).int() + (v >= 0.75).int() + (v > 1.25).int() + (v >= 1.75).int()
            + (v > 2.5).int() + (v >= 3.5).int() + (v > 5.0).int())
    return code + 8 * (x < 0).int(), s


def _plain_decode(code, s):
    """The values of codes [rows, blocks, 32] in 32 bits."""
    m = (code & 7).float()
    # 0, 0.5, 1, 1.5 by halves; 2 and 3 by ones; 4 and 6 by twos
    v = torch.where(m < 4, 0.5 * m, torch.where(m < 6, m - 2.0, 2.0 * m - 8.0))
    v = torch.ldexp(v, s)
    return torch.where(code >= 8, -v, v).reshape(code.shape[0], -1)


def _pack(code, s):
    """The two arrays in memory: bytes of two codes, and scale bytes rounded up to 16 a row."""
    rows, blocks = s.shape[0], s.shape[1]
    c = code.reshape(rows, blocks * 16, 2)
    packed = (c[:, :, 0] | (c[:, :, 1] << 4)).to(torch.uint8)
    scales = torch.zeros(rows, (blocks + 15) // 16 * 16, dtype=torch.uint8, device=s.device)
    scales[:, :blocks] = (s.reshape(rows, blocks) + 127).to(torch.uint8)
    return packed.contiguous(), scales


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op = case["op"]

    def normal(rows, cols, std, dtype="bf16"):
        return (torch.randn(rows, cols, generator=g, device=dev) * std).to(_TORCH[dtype])

    def empty(rows, cols, dtype):
        return torch.empty(rows, cols, dtype=dtype, device=dev)

    s = {"case": case}
    if op == "mx4_quantize":
        r, c = case["rows"], case["cols"]
        s["x"] = normal(r, c, 0.02, case["dtype"])
        for t, rows, cols in (("", r, c), ("_t", c, r))[: 2 if case["both"] else 1]:
            s["codes" + t] = empty(rows, _codes(cols), torch.uint8)
            s["scales" + t] = empty(rows, _scales(cols), torch.uint8)
            s["values" + t] = empty(rows, cols, torch.bfloat16)
        return s
    m, n = case["m"], case["n"]
    s["workspace"] = torch.empty(WORKSPACE_BYTES, dtype=torch.uint8, device=dev)
    if op == "mx4_product":
        k = case["k"]
        s["a"], s["a_scales"] = _pack(*_plain_codes(normal(m, k, 1.0, "f32")))
        s["b"], s["b_scales"] = _pack(*_plain_codes(normal(n, k, 0.02, "f32")))
        s["bias"] = normal(1, n, 0.02).reshape(n) if case["bias"] else None
        s["residual"] = normal(m, n, 1.0, case["y"]) if case["residual"] else None
        s["y"] = s["residual"] if case["residual"] == "in place" else empty(m, n, _TORCH[case["y"]])
        s["z"] = empty(m, n, torch.bfloat16) if case["z"] else None
        return s
    # activations whose features differ in size and lie off zero
    t = case["dtype"]
    x = normal(m, n, 1.0, "f32") * (1.0 + normal(1, n, 0.2, "f32")) + normal(1, n, 0.5, "f32")
    s["x"] = x.to(_TORCH[t])
    s["weight"] = (1.0 + normal(1, n, 0.1, "f32")).to(_TORCH[case["w"]]).reshape(n)
    if op == "norm_forward":
        s["bias"] = normal(1, n, 0.1, case["w"]).reshape(n) if case["bias"] else None
        s["y"] = empty(m, n, _TORCH[t])
        if case["stats"]:
            s["rstd"] = torch.empty(m, device=dev)
            if case["kind"] == "layer":
                s["mean"] = torch.empty(m, device=dev)
        return s
    # the forward pass kept these
    d = s["x"].double()
    if case["kind"] == "layer":
        s["mean"] = d.mean(dim=1).float()
        d = d - d.mean(dim=1, keepdim=True)
    s["rstd"] = (d.square().mean(dim=1) + EPS).rsqrt().float()
    s["dy"] = normal(m, n, 1e-3, t)
    s["residual"] = normal(m, n, 1e-3, t) if case["residual"] else None
    s["dx"] = empty(m, n, _TORCH[t])
    s["dw"] = normal(1, n, 1e-2, case["dw"]).reshape(n)
    s["db"] = normal(1, n, 1e-2, case["dw"]).reshape(n) if case["bias"] else None
    return s


# ---------------------------------------------------------------- the plain form

def _plain_act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _plain_values(codes, scales, cols):
    """The values of a matrix as it lies in memory, in 32 bits."""
    rows, blocks = codes.shape[0], codes.shape[1] // 16
    c = torch.stack([codes & 15, codes >> 4], dim=2).reshape(rows, blocks, 32)
    s = scales[:, :blocks].int().reshape(rows, blocks, 1) - 127
    return _plain_decode(c, s)[:, :cols]


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "mx4_quantize":
        r, c = case["rows"], case["cols"]
        out = {"values": _plain_decode(*_plain_codes(s["x"]))[:, :c].to(torch.bfloat16)}
        if case["both"]:
            out["values_t"] = _plain_decode(*_plain_codes(s["x"].t()))[:, :r].to(torch.bfloat16)
        return out
    if op == "mx4_product":
        k = case["k"]
        z = _plain_values(s["a"], s["a_scales"], k) @ _plain_values(s["b"], s["b_scales"], k).t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _plain_act(z, case["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        if case["residual"] == "in place":
            s["y"].copy_(y)
            out = {"y": s["y"]}
        else:
            out = {"y": y.to(_TORCH[case["y"]])}
        if case["z"]:
            out["z"] = z.to(torch.bfloat16)
        return out
    layer, x, w = case["kind"] == "layer", s["x"].float(), s["weight"].float()
    if op == "norm_forward":
        out = {}
        if layer:
            mean = x.mean(dim=1, keepdim=True)
            x = x - mean
        rstd = 1 / torch.sqrt((x * x).mean(dim=1, keepdim=True) + EPS)
        y = x * rstd * w
        if s["bias"] is not None:
            y = y + s["bias"].float()
        out["y"] = y.to(_TORCH[case["dtype"]])
        if case["stats"]:
            out["rstd"] = rstd.reshape(-1)
            if layer:
                out["mean"] = mean.reshape(-1)
        return out
    rstd = s["rstd"].unsqueeze(1)
    xhat = (x - s["mean"].unsqueeze(1) if layer else x) * rstd
    dy = s["dy"].float()
    g = dy * w
    dx = g - xhat * (g * xhat).mean(dim=1, keepdim=True)
    if layer:
        dx = dx - g.mean(dim=1, keepdim=True)
    dx = dx * rstd
    if s["residual"] is not None:
        dx = dx + s["residual"].float()
    sums = {"dw": (dy * xhat).sum(dim=0)}
    if s["db"] is not None:
        sums["db"] = dy.sum(dim=0)
    out = {"dx": dx.to(_TORCH[case["dtype"]])}
    for name, v in sums.items():
        s[name].copy_(s[name].float() + v if case["add"] else v)
        out[name] = s[name]
    return out


# ---------------------------------------------------------------- the framework's calls

def _own(s):
    from rank_step_amd import binding as B
    case, op = s["case"], s["case"]["op"]
    if op == "mx4_quantize":
        r, c = case["rows"], case["cols"]
        B.fsdp_mx4_quantize(s["x"], r, c, x_dtype=case["dtype"], codes=s["codes"], scales=s["scales"],
                            codes_t=s.get("codes_t"), scales_t=s.get("scales_t"))
        B.fsdp_mx4_dequantize(s["values"], s["codes"], s["scales"], r, c)
        if not case["both"]:
            return {"values": s["values"]}
        B.fsdp_mx4_dequantize(s["values_t"], s["codes_t"], s["scales_t"], c, r)
        return {"values": s["values"], "values_t": s["values_t"]}
    m, n = case["m"], case["n"]
    if op == "mx4_product":
        B.fsdp_mx4_product(s["y"], s["a"], s["a_scales"], s["b"], s["b_scales"], m, n, case["k"], y_dtype=case["y"],
                           bias=s["bias"], residual=s["residual"], act=case["act"], z=s["z"], workspace=s["workspace"])
        return {"y": s["y"], "z": s["z"]} if case["z"] else {"y": s["y"]}
    if op == "norm_forward":
        B.fsdp_norm_forward(s["y"], s["x"], m, n, dtype=case["dtype"], kind=case["kind"], weight=s["weight"],
                            bias=s["bias"], w_dtype=case["w"], eps=EPS, mean=s.get("mean"), rstd=s.get("rstd"))
        return {name: s[name] for name in ("y", "rstd", "mean") if name in s}
    B.fsdp_norm_backward(s["dx"], s["dy"], s["x"], m, n, dtype=case["dtype"], kind=case["kind"], weight=s["weight"],
                         w_dtype=case["w"], mean=s.get("mean"), rstd=s["rstd"], residual=s["residual"], dw=s["dw"],
                         db=s["db"], dw_dtype=case["dw"], accumulate=case["add"], workspace=s["workspace"])
    return {"dx": s["dx"], "dw": s["dw"], "db": s["db"]} if case["bias"] else {"dx": s["dx"], "dw": s["dw"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_quantized(x):
    """The values of the 4-bit copy of x: the exponent from the 64-bit format's
    own bits, the element by its distance to the eight magnitudes."""
    rows, cols = x.shape
    full = torch.zeros(rows, -(-cols // 32) * 32, dtype=torch.float64, device=x.device)
    full[:, :cols] = x
    blocks = full.view(rows, -1, 32)
    top = blocks.abs().amax(-1, keepdim=True)
    exponent = ((top.view(torch.int64) >> 52) & 0x7FF) - 1023  # -1023 where the block is zero
    scale = torch.pow(2.0, (exponent - 2).clamp(min=-127).double())
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    middle = (grid[1:] + grid[:-1]) / 2
    v = blocks.abs() / scale
    low, high = torch.bucketize(v, middle, right=False), torch.bucketize(v, middle, right=True)
    nearest = torch.where(low % 2 == 0, low, high)  # they differ halfway, where the even one counts
    return (torch.copysign(grid[nearest], blocks) * scale).view(rows, -1)[:, :cols]


def _exact_decoded(codes, scales, cols):
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64,
                         device=codes.device)
    v = torch.empty(codes.shape[0], codes.shape[1] * 2, dtype=torch.float64, device=codes.device)
    v[:, 0::2] = table[(codes % 16).long()]
    v[:, 1::2] = table[(codes // 16).long()]
    weight = torch.pow(2.0, scales.double() - 127.0)
    return (v * weight.repeat_interleave(32, dim=1)[:, : v.shape[1]])[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "mx4_quantize":
        x = s["x"].double()
        out = {"values": _exact_quantized(x)}
        if case["both"]:
            out["values_t"] = _exact_quantized(x.T.contiguous())
        return out
    if op == "mx4_product":
        k = case["k"]
        z = torch.mm(_exact_decoded(s["a"], s["a_scales"], k), _exact_decoded(s["b"], s["b_scales"], k).T)
        if case["bias"]:
            z += s["bias"].double()
        if case["act"] == "relu":
            y = z.clamp(min=0)
        elif case["act"] == "gelu":
            y = z * torch.special.ndtr(z)
        elif case["act"] == "silu":
            y = z * torch.sigmoid(z)
        else:
            y = z
        if case["residual"]:
            y = y + s["residual"].double()
        return {"y": y, "z": z} if case["z"] else {"y": y}
    layer, x, w = case["kind"] == "layer", s["x"].double(), s["weight"].double()
    if op == "norm_forward":
        if layer:
            var, mean = torch.var_mean(x, dim=1, correction=0)
        else:
            var, mean = x.square().mean(dim=1), torch.zeros(x.shape[0], dtype=torch.float64, device=x.device)
        rstd = (var + EPS).pow(-0.5)
        y = (x - mean[:, None]) * (rstd[:, None] * w[None, :])
        if case["bias"]:
            y += s["bias"].double()
        out = {"y": y}
        if case["stats"]:
            out["rstd"] = rstd
            if layer:
                out["mean"] = mean
        return out
    # dx through the Jacobian's own terms: d xhat_j / d x_i = rstd (delta_ij - [layer] 1/n - xhat_i xhat_j / n)
    n, r = case["n"], s["rstd"].double()[:, None]
    xhat = (x - s["mean"].double()[:, None]) * r if layer else x * r
    dy = s["dy"].double()
    g = dy * w
    dx = r * g - (r / n) * xhat * torch.linalg.vecdot(g, xhat)[:, None]
    if layer:
        dx -= (r / n) * g.sum(dim=1, keepdim=True)
    if case["residual"]:
        dx += s["residual"].double()
    sums = {"dw": torch.linalg.vecdot(dy, xhat, dim=0)}
    if case["bias"]:
        sums["db"] = torch.einsum("ij->j", dy)
    return {"dx": dx} | {name: s[name].double() + v if case["add"] else v for name, v in sums.items()}
