"""The layer's operators, as they are measured: the products that read the
all-gathered weight copy and write the gradient slices, and dropout.

Five operators:

  linear_forward            z = x W^T + b;  y = D(act(z)) + r
  linear_epilogue_backward  dz = D(dy) act'(z), db = column sums of it
  linear_grad_input         dx = dz W
  linear_grad_weight        dW = dz^T x, stored or added to what is there
  dropout                   y = D(x) + r

x, dz, z are bf16 matrices of m rows (tokens); W is [n, k], bf16 or E4M3 codes
with one scale a tensor (value = code / scale), as the step's two all-gather
copies hold it.  D keeps an element and multiplies it by 65536 / (65536 - T),
or drops it to zero.  Its mask is a function of the element's place: element
(i, j) takes 16 bits of the Philox-4x32-10 block (Salmon et al., "Parallel
random numbers: as easy as 1, 2, 3", 2011) whose counter is the block number
i * ceil(n / 8) + j / 8 (low 64 bits) and the draw's offset (high 64 bits) and
whose key is the seed; word (j % 8) / 2, its low half first.  The element is
kept where those bits are at least T = rint(65536 p).

With ``own`` false, ``run`` computes them with elementary torch operations in
32 bits; with ``own`` true, through rank_step_amd.binding.
"""

import math

import numpy as np
import torch

own = False

WORKSPACE_BYTES = 64 << 20


# ---------------------------------------------------------------- the cases

def listed():
    fwd, epi, gin, gwt, drp = ("linear_forward", "linear_epilogue_backward", "linear_grad_input",
                               "linear_grad_weight", "dropout")
    return [
        # one token through an attention output projection of the 7B block: the weight's bytes and the call itself
        {"name": "forward one token", "op": fwd, "m": 1, "n": 4096, "k": 4096, "w": "bf16", "act": "none",
         "bias": False, "residual": True, "z": False, "p": 0.0, "y": "bf16"},
        # sixteen tokens through the 7B block's gate projection, weights from the fp8 all-gather
        {"name": "forward 16 tokens fp8", "op": fwd, "m": 16, "n": 11008, "k": 4096, "w": "e4m3", "act": "silu",
         "bias": False, "residual": False, "z": False, "p": 0.0, "y": "bf16"},
        # the same projection in training, with the pre-activation kept for the backward pass
        {"name": "forward 4096 tokens", "op": fwd, "m": 4096, "n": 11008, "k": 4096, "w": "bf16", "act": "silu",
         "bias": False, "residual": False, "z": True, "p": 0.0, "y": "bf16"},
        # a layer of the 128 MiB MLP, [1024, 1365]: rows of the weight that end off every vector boundary
        {"name": "forward odd layer", "op": fwd, "m": 1000, "n": 1024, "k": 1365, "w": "bf16", "act": "gelu",
         "bias": True, "residual": True, "z": True, "p": 0.1, "y": "bf16"},
        # behind the up projection in training: activation, dropout and bias gradients in one pass
        {"name": "epilogue grad 4096 tokens", "op": epi, "m": 4096, "n": 11008, "act": "gelu", "p": 0.1, "db": "bf16"},
        # the tiny MLP's hidden layer, where the call is what counts
        {"name": "epilogue grad small", "op": epi, "m": 333, "n": 1024, "act": "relu", "p": 0.0, "db": "f32"},
        # the down projection's input gradient over a long batch: the largest product
        {"name": "input grad 8192 tokens", "op": gin, "m": 8192, "n": 4096, "k": 11008, "w": "bf16"},
        # the odd layer's input gradient from the fp8 copy
        {"name": "input grad odd fp8", "op": gin, "m": 1000, "n": 1024, "k": 1365, "w": "e4m3"},
        # an attention projection's weight gradient, written as the bf16 slice that the reduce takes
        {"name": "weight grad 8192 tokens", "op": gwt, "m": 8192, "n": 4096, "k": 4096, "dw": "bf16", "add": False},
        # the odd layer's, added to the fp32 gradient that accumulates over micro-batches
        {"name": "weight grad odd fp32", "op": gwt, "m": 2047, "n": 1024, "k": 1365, "dw": "f32", "add": True},
        # the residual branch's dropout over a long batch
        {"name": "dropout 8192 tokens", "op": drp, "m": 8192, "n": 4096, "dtype": "bf16", "residual": True, "p": 0.1},
        # a few tokens of the tiny MLP in fp32, odd width
        {"name": "dropout small", "op": drp, "m": 37, "n": 251, "dtype": "f32", "residual": False, "p": 0.5},
    ]


def _spread(rng, lo, hi):
    """Log-uniform in [lo, hi]; half of the larger ones a multiple of 64, the others any number."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v >= 64 and rng.random() < 0.5:
        v -= v % 64
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["linear_forward", "linear_forward", "linear_epilogue_backward", "linear_grad_input",
                     "linear_grad_weight", "dropout"])
    n = _spread(rng, 64, 11008)
    c = {"op": op, "m": _spread(rng, 1, 8192), "n": n}
    if op == "linear_forward":
        c |= {"k": _spread(rng, 64, 11008), "w": rng.choice(["bf16", "bf16", "e4m3"]),
              "act": rng.choice(["none", "relu", "gelu", "silu"]), "bias": rng.random() < 0.5,
              "residual": rng.random() < 0.5, "z": rng.random() < 0.5, "p": rng.choice([0.0, 0.0, 0.1, 0.5]),
              "y": rng.choice(["bf16", "bf16", "f32"])}
    elif op == "linear_epilogue_backward":
        c |= {"act": rng.choice(["none", "relu", "gelu", "silu"]), "p": rng.choice([0.0, 0.1, 0.5]),
              "db": rng.choice(["bf16", "f32"])}
    elif op == "linear_grad_input":
        c |= {"k": _spread(rng, 64, 11008), "w": rng.choice(["bf16", "bf16", "e4m3"])}
    elif op == "linear_grad_weight":
        c |= {"k": _spread(rng, 64, 11008), "dw": rng.choice(["bf16", "f32"]), "add": rng.random() < 0.5}
    elif op == "dropout":
        c |= {"dtype": rng.choice(["bf16", "f32"]), "residual": rng.random() < 0.5, "p": rng.choice([0.1, 0.25, 0.5])}
    # no more than the largest listed product: fewer tokens, the layer's width as drawn
    c["m"] = min(c["m"], 8192 * 4096 * 11008 // (n * c["k"]) if "k" in c else c["m"])
    return c


_BYTES = {"bf16": 2, "f32": 4, "e4m3": 1}


def work(case):
    m, n, op = case["m"], case["n"], case["op"]
    if op == "dropout":
        e = _BYTES[case["dtype"]]
        return {"bytes": m * n * e * (3 if case["residual"] else 2), "flops": 2 * m * n}
    if op == "linear_epilogue_backward":
        read = 4 * m * n if case["act"] != "none" else 2 * m * n
        return {"bytes": read + 2 * m * n + n * _BYTES[case["db"]], "flops": 8 * m * n}
    k = case["k"]
    flops = 2 * m * n * k
    if op == "linear_forward":
        y = _BYTES[case["y"]]
        b = 2 * m * k + n * k * _BYTES[case["w"]] + m * n * y
        b += (2 * n if case["bias"] else 0) + (y * m * n if case["residual"] else 0) + (2 * m * n if case["z"] else 0)
        return {"bytes": b, "flops": flops}
    if op == "linear_grad_input":
        return {"bytes": 2 * m * n + n * k * _BYTES[case["w"]] + 2 * m * k, "flops": flops}
    return {"bytes": 2 * m * n + 2 * m * k + n * k * _BYTES[case["dw"]] * (2 if case["add"] else 1), "flops": flops}


# ---------------------------------------------------------------- inputs

_TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    m, n, op = case["m"], case["n"], case["op"]

    def normal(rows, cols, std, dtype="bf16"):
        return (torch.randn(rows, cols, generator=g, device=dev) * std).to(_TORCH[dtype])

    s = {"case": case}
    if op != "dropout" and op != "linear_epilogue_backward":
        k = case["k"]
        if "w" in case:
            s["w"] = normal(n, k, 0.02, "f32")
            if case["w"] == "e4m3":  # the step's own recipe: 448 over the tensor's largest magnitude
                s["w_scale"] = 448.0 / s["w"].abs().max().clamp(min=1e-12).reshape(1)
                codes = (s["w"] * s["w_scale"]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
                s["w"] = codes.view(torch.uint8)
            else:
                s["w"] = s["w"].to(torch.bfloat16)
    if op == "linear_forward":
        s["x"] = normal(m, case["k"], 1.0)
        s["bias"] = normal(1, n, 0.02).reshape(n) if case["bias"] else None
        s["residual"] = normal(m, n, 1.0, case["y"]) if case["residual"] else None
        s["y"] = torch.empty(m, n, dtype=_TORCH[case["y"]], device=dev)
        s["z"] = torch.empty(m, n, dtype=torch.bfloat16, device=dev) if case["z"] else None
    elif op == "linear_epilogue_backward":
        s["dy"] = normal(m, n, 1e-3)
        s["z"] = normal(m, n, 1.0) if case["act"] != "none" else None
        s["dz"] = torch.empty(m, n, dtype=torch.bfloat16, device=dev)
        s["db"] = torch.empty(n, dtype=_TORCH[case["db"]], device=dev)
    elif op == "linear_grad_input":
        s["dz"] = normal(m, n, 1e-3)
        s["dx"] = torch.empty(m, case["k"], dtype=torch.bfloat16, device=dev)
    elif op == "linear_grad_weight":
        s["dz"] = normal(m, n, 1e-3)
        s["x"] = normal(m, case["k"], 1.0)
        s["dw"] = normal(n, case["k"], 0.1, case["dw"])
    else:
        s["x"] = normal(m, n, 1.0, case["dtype"])
        s["residual"] = normal(m, n, 1.0, case["dtype"]) if case["residual"] else None
        s["y"] = torch.empty(m, n, dtype=_TORCH[case["dtype"]], device=dev)
    if case.get("p", 0.0) > 0.0:
        s["dropout"] = {"p": case["p"], "seed": 0x9E3779B97F4A7C15 ^ seed, "offset": (seed << 20) + 3}
    else:
        s["dropout"] = None
    s["workspace"] = torch.empty(WORKSPACE_BYTES, dtype=torch.uint8, device=dev)
    return s


# ---------------------------------------------------------------- the plain form

_M32 = 0xFFFFFFFF


def _plain_mask(rows, cols, rng, dev):
    """The mask, and what kept elements are multiplied by."""
    per_row = (cols + 7) // 8
    block = torch.arange(rows * per_row, dtype=torch.int64, device=dev)
    c0, c1 = block & _M32, block >> 32
    c2 = torch.full_like(block, rng["offset"] & _M32)
    c3 = torch.full_like(block, (rng["offset"] >> 32) & _M32)
    k0, k1 = rng["seed"] & _M32, (rng["seed"] >> 32) & _M32
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((p1 >> 32) & _M32) ^ c1 ^ k0, p1 & _M32, ((p0 >> 32) & _M32) ^ c3 ^ k1, p0 & _M32
        k0, k1 = (k0 + 0x9E3779B9) & _M32, (k1 + 0xBB67AE85) & _M32
    words = torch.stack([c0, c1, c2, c3], dim=1)
    bits = torch.stack([words & 0xFFFF, words >> 16], dim=2).reshape(rows, per_row * 8)[:, :cols]
    t = round(rng["p"] * 65536)
    return bits >= t, (65536.0 / (65536 - t) if t < 65536 else 0.0)


def _plain_drop(v, rng):
    if rng is None:
        return v
    keep, scale = _plain_mask(v.shape[0], v.shape[1], rng, v.device)
    return torch.where(keep, v * scale, torch.zeros_like(v))


def _plain_act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _plain_act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s))


def _plain_weight(s):
    if s["case"]["w"] == "e4m3":
        return s["w"].view(torch.float8_e4m3fn).float() / s["w_scale"]
    return s["w"].float()


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "linear_forward":
        z = s["x"].float() @ _plain_weight(s).t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _plain_drop(_plain_act(z, case["act"]), s["dropout"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        out = {"y": y.to(_TORCH[case["y"]])}
        if case["z"]:
            out["z"] = z.to(torch.bfloat16)
        return out
    if op == "linear_epilogue_backward":
        d = _plain_drop(s["dy"].float(), s["dropout"])
        if case["act"] != "none":
            d = d * _plain_act_grad(s["z"].float(), case["act"])
        return {"dz": d.to(torch.bfloat16), "db": d.sum(0).to(_TORCH[case["db"]])}
    if op == "linear_grad_input":
        return {"dx": (s["dz"].float() @ _plain_weight(s)).to(torch.bfloat16)}
    if op == "linear_grad_weight":
        d = s["dz"].float().t() @ s["x"].float()
        if case["add"]:
            d = s["dw"].float() + d
        s["dw"].copy_(d)
        return {"dw": s["dw"]}
    y = _plain_drop(s["x"].float(), s["dropout"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.to(_TORCH[case["dtype"]])}


# ---------------------------------------------------------------- the framework's calls

def _own(s):
    from rank_step_amd import binding as B
    case, op = s["case"], s["case"]["op"]
    m, n = case["m"], case["n"]
    if op == "linear_forward":
        B.fsdp_linear_forward(s["y"], s["x"], s["w"], m, n, case["k"], w_dtype=case["w"], w_scale=s.get("w_scale"),
                              y_dtype=case["y"], bias=s["bias"], residual=s["residual"], act=case["act"], z=s["z"],
                              dropout=s["dropout"], workspace=s["workspace"])
        return {"y": s["y"], "z": s["z"]} if case["z"] else {"y": s["y"]}
    if op == "linear_epilogue_backward":
        B.fsdp_linear_epilogue_backward(s["dz"], s["dy"], m, n, z=s["z"], act=case["act"], dropout=s["dropout"],
                                        db=s["db"], db_dtype=case["db"], workspace=s["workspace"])
        return {"dz": s["dz"], "db": s["db"]}
    if op == "linear_grad_input":
        B.fsdp_linear_grad_input(s["dx"], s["dz"], s["w"], m, n, case["k"], w_dtype=case["w"],
                                 w_scale=s.get("w_scale"), workspace=s["workspace"])
        return {"dx": s["dx"]}
    if op == "linear_grad_weight":
        B.fsdp_linear_grad_weight(s["dw"], s["dz"], s["x"], m, n, case["k"], dw_dtype=case["dw"],
                                  accumulate=case["add"], workspace=s["workspace"])
        return {"dw": s["dw"]}
    B.fsdp_dropout(s["y"], s["x"], m, n, case["dtype"], s["dropout"], residual=s["residual"])
    return {"y": s["y"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_factor(rows, cols, rng):
    """The dropout factor of every element (0 or 1 / (1 - T / 65536)), from the
    generator's definition in unsigned 64-bit host arithmetic."""
    u = np.uint64
    lo32, sh = u(0xFFFFFFFF), u(32)
    width = -(-cols // 8)
    index = np.add.outer(np.arange(rows, dtype=u) * u(width), np.arange(width, dtype=u))
    ctr = [index & lo32, index >> sh,
           np.full_like(index, u(rng["offset"] & 0xFFFFFFFF)), np.full_like(index, u((rng["offset"] >> 32) & 0xFFFFFFFF))]
    key = [rng["seed"] & 0xFFFFFFFF, (rng["seed"] >> 32) & 0xFFFFFFFF]
    for r in range(10):
        a, b = ctr[0] * u(0xD2511F53), ctr[2] * u(0xCD9E8D57)
        ka, kb = u((key[0] + r * 0x9E3779B9) % (1 << 32)), u((key[1] + r * 0xBB67AE85) % (1 << 32))
        ctr = [(b >> sh) ^ ctr[1] ^ ka, b & lo32, (a >> sh) ^ ctr[3] ^ kb, a & lo32]
    bits = np.empty((rows, width, 8), dtype=np.int32)
    for w in range(4):
        bits[:, :, 2 * w] = (ctr[w] & u(0xFFFF)).astype(np.int32)
        bits[:, :, 2 * w + 1] = (ctr[w] >> u(16)).astype(np.int32)
    t = int(np.rint(rng["p"] * 65536))
    kept = bits.reshape(rows, width * 8)[:, :cols] >= t
    return torch.from_numpy(kept).to("cuda").double() * (1.0 if t == 0 else 0.0 if t == 65536 else 1.0 / (1.0 - t / 65536.0))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = {name: v.double() for name, v in s.items() if isinstance(v, torch.Tensor) and v.dtype in (torch.bfloat16, torch.float32)
         and name in ("x", "w", "bias", "residual", "dy", "dz", "z", "dw", "w_scale")}
    factor = _exact_factor(case["m"], case["n"], s["dropout"]) if s["dropout"] is not None else 1.0
    if case.get("w") == "e4m3":
        # sign, exponent of bias 7, 3 fraction bits; exponent 0 holds the multiples of 2^-9
        code = s["w"].to(torch.int64)
        e, f = (code >> 3) & 15, (code & 7).double()
        mag = torch.where(e == 0, f * 2.0 ** -9, (8 + f) * torch.pow(torch.tensor(2.0, dtype=torch.float64, device=f.device), (e - 10).double()))
        d["w"] = torch.where(code >= 128, -mag, mag) / d["w_scale"]
    if op == "linear_forward":
        z = torch.mm(d["x"], d["w"].T)
        if case["bias"]:
            z += d["bias"]
        if case["act"] == "relu":
            a = z.clamp(min=0)
        elif case["act"] == "gelu":
            a = z * torch.special.ndtr(z)
        elif case["act"] == "silu":
            a = z * torch.sigmoid(z)
        else:
            a = z
        y = a * factor + (d["residual"] if case["residual"] else 0.0)
        return {"y": y, "z": z} if case["z"] else {"y": y}
    if op == "linear_epilogue_backward":
        if case["act"] == "relu":
            slope = torch.heaviside(d["z"], torch.zeros((), dtype=torch.float64, device="cuda"))
        elif case["act"] == "gelu":
            slope = torch.special.ndtr(d["z"]) + d["z"] * torch.exp(d["z"].square() / -2) / math.sqrt(2 * math.pi)
        elif case["act"] == "silu":
            slope = torch.sigmoid(d["z"]) + d["z"] * torch.sigmoid(d["z"]) * torch.sigmoid(-d["z"])
        else:
            slope = 1.0
        dz = d["dy"] * slope * factor
        return {"dz": dz, "db": dz.sum(dim=0)}
    if op == "linear_grad_input":
        return {"dx": torch.mm(d["dz"], d["w"])}
    if op == "linear_grad_weight":
        dw = torch.mm(d["dz"].T, d["x"])
        return {"dw": d["dw"] + dw if case["add"] else dw}
    return {"y": d["x"] * factor + (d["residual"] if case["residual"] else 0.0)}
