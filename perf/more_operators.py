"""Layer norm and the 4-bit linear layer, as they are measured: their cases, inputs, plain forms and the calls of this package.

Two families of a feed-forward block's operators:

  norm      y = (x - mean) * rstd * weight + bias over every row of x, and its backward pass: dx (with the gradient that
            passes the norm by added to it), the weight's and the bias's gradient
  mx4       microscaled 4-bit floating point (blocks of 32 values along K: 4-bit E2M1 elements, one power of two a
            block): quantising rows or a weight, reading the values back, and the fused linear layer
            out = act(A @ B + bias [+ R]) whose operands are held so, A also quantised on its way in

With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits (quantising is exact in them:
a block's scale is a power of two and the borders between elements are compared with as they stand); with ``own`` true
it calls this package.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # the magnitudes of codes 0..7; bit 3 is the sign


# ------------------------------------------------------------------ cases

def _norm(name, M, H, dtype, step, affine=True, residual=False):
    return {"name": name, "op": "norm", "M": M, "H": H, "dtype": dtype, "step": step, "affine": affine,
            "residual": residual}


def _quant(name, rows, K, dtype, transposed=False):
    return {"name": name, "op": "quant", "rows": rows, "K": K, "dtype": dtype, "transposed": transposed}


def _linear(name, M, N, K, dtype, act, a="raw", residual=False):
    return {"name": name, "op": "linear", "M": M, "N": N, "K": K, "dtype": dtype, "act": act, "a": a,
            "residual": residual}


def listed():
    return [
        # one decode step of a small serving batch: the norm's launch latency
        _norm("norm_decode", 32, 4096, "bf16", "forward"),
        # a long prompt through the norm in front of a wide layer
        _norm("norm_prompt", 8192, 4096, "f16", "forward"),
        # odd sizes in 32 bits, with the gradients: a small model's training step
        _norm("norm_ragged", 4097, 1537, "f32", "train"),
        # a training step of a pre-norm block: forward, then backward with the gradient of the block's residual path
        _norm("norm_train", 16384, 4096, "bf16", "train", residual=True),
        # a weight (K,N) as training leaves it into the 4-bit form that serving keeps, and the values read back
        _quant("quant_weight", 14336, 4096, "bf16", transposed=True),
        # a batch of activations of odd width, and the values read back
        _quant("quant_ragged", 4097, 1537, "f16"),
        # a decoded token through a wide projection: the weight's bytes
        _linear("mx4_token", 1, 14336, 4096, "f16", "gelu_tanh"),
        # a serving batch through the projection back, with the residual
        _linear("mx4_batch", 64, 4096, 14336, "bf16", "none", residual=True),
        # odd sizes throughout
        _linear("mx4_ragged", 4097, 3071, 1537, "bf16", "relu"),
        # a gated projection of wide output, the activations already in 4 bits
        _linear("mx4_gate", 1024, 21568, 4096, "f16", "glu", a="codes"),
        # a prompt through a projection in 32-bit output (logits)
        _linear("mx4_logits", 512, 21568, 1024, "f32", "none"),
        # a long prompt through a large projection
        _linear("mx4_prompt", 8192, 14336, 4096, "bf16", "gelu_tanh"),
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm, odd ones among them."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "norm", "quant", "linear", "linear", "linear"))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    if op == "norm":
        H = _log(rng, 32, 16384)
        M = _log(rng, 1, min(65536, (1 << 26) // H))
        step = rng.choice(("forward", "train"))
        case = _norm("", M, H, dtype, step, affine=rng.random() < 0.8, residual=step == "train" and rng.random() < 0.5)
    elif op == "quant":
        K = _log(rng, 32, 16384)
        case = _quant("", _log(rng, 1, min(32768, (1 << 26) // K)), K, dtype, transposed=rng.random() < 0.5)
    else:
        N, K = _log(rng, 64, 16384), _log(rng, 64, 16384)
        M = _log(rng, 1, max(1, min(8192, int(4e11) // (N * K))))
        case = _linear("", M, N, K, dtype, rng.choice(("none", "relu", "gelu_tanh", "glu")),
                       a=rng.choice(("raw", "raw", "codes")), residual=rng.random() < 0.3)
    del case["name"]
    return case


# ----------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.empty(*shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=g)

    def activations(rows, width):
        """Rows of different sizes and a few columns that are larger than the others, as a residual stream has them."""
        x = normal(rows, width)
        x *= torch.exp(0.3 * normal(width)) * (1 + 9 * (torch.rand(width, generator=g, device="cuda") < 0.01))
        return x.mul_(torch.exp(0.5 * normal(rows, 1))).to(dt)

    dt = DTYPES[case["dtype"]]
    s = {"case": dict(case)}
    if case["op"] == "norm":
        M, H = case["M"], case["H"]
        s["x"] = activations(M, H)
        s["weight"] = (1 + normal(H, std=0.2)).to(dt) if case["affine"] else None
        s["bias"] = normal(H, std=0.2).to(dt) if case["affine"] else None
        if case["step"] == "train":
            s["dout"] = normal(M, H).to(dt)
            s["residual"] = normal(M, H).to(dt) if case["residual"] else None
        return s
    if case["op"] == "quant":
        rows, K = case["rows"], case["K"]
        s["x"] = normal(K, rows, std=K ** -0.5).to(dt) if case["transposed"] else activations(rows, K)
        return s
    M, N, K = case["M"], case["N"], case["K"]
    a = activations(M, K)
    if case["a"] == "raw":
        s["A"] = a
    else:
        s["A_codes"], s["A_scales"] = _quantize(a)
    s["B_codes"], s["B_scales"] = _quantize(normal(N, K, std=K ** -0.5))
    s["bias"] = normal(N, std=0.3).to(dt)
    s["Y"] = normal(M, N).to(dt) if case["act"] == "glu" else None
    s["R"] = normal(M, N).to(dt) if case["residual"] else None
    return s


# ------------------------------------------------------------ plain forms

def _blocks(x):
    """(rows, blocks, 32) in 32 bits, the last block of a row filled up with zeros."""
    x = x.float()
    short = -x.shape[1] % 32
    if short:
        x = torch.cat([x, x.new_zeros(x.shape[0], short)], 1)
    return x.view(x.shape[0], -1, 32)


def _magnitudes(x):
    """Of x (rows, blocks, 32): the exponent of every block's scale, and the codes 0..7 of the magnitudes."""
    exponent = torch.frexp(x.abs().amax(2)).exponent - 1 - 2  # the largest value's, less that of the largest element
    exponent = exponent.clamp(-127, 127)
    a = torch.ldexp(x.abs(), -exponent[..., None])
    # borders between neighbours go to the even code
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return exponent, code


def _quantize(x):
    """(codes (rows, blocks*16), scales (rows, blocks)), bytes: element 2i of a row in the low half of byte i."""
    x = _blocks(x)
    exponent, code = _magnitudes(x)
    code = code + 8 * (x < 0)
    code = code.view(x.shape[0], -1, 2)
    scales = torch.where(x.abs().amax(2) > 0, exponent + 127, torch.zeros_like(exponent))
    return (code[..., 0] + 16 * code[..., 1]).to(torch.uint8).contiguous(), scales.to(torch.uint8).contiguous()


def _values(codes, scales, K):
    """The values of codes and scales, (rows, K) in 32 bits."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = table[torch.stack([codes & 15, codes >> 4], 2).int()].view(codes.shape[0], -1, 32)
    return torch.ldexp(v, scales.int()[..., None] - 127).view(codes.shape[0], -1)[:, :K]


def _rounded(x):
    """The values of a matrix after quantising, without the bytes between."""
    b = _blocks(x)
    exponent, code = _magnitudes(b)
    v = torch.tensor(E2M1, device=x.device)[code.int()]
    v = torch.ldexp(torch.where(b < 0, -v, v), exponent[..., None])
    return v.view(x.shape[0], -1)[:, :x.shape[1]]


def _act(x, y, act):
    if act == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x))
    if act == "gelu_tanh":
        return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))
    return x + x * y if act == "glu" else x


def _plain_norm(s):
    c, x = s["case"], s["x"].float()
    mean = x.mean(1, keepdim=True)
    hat = x - mean
    rstd = 1.0 / torch.sqrt((hat * hat).mean(1, keepdim=True) + EPS)
    hat = hat * rstd
    y = hat if s["weight"] is None else hat * s["weight"].float() + s["bias"].float()
    got = {"y": y.to(s["x"].dtype)}
    if c["step"] == "train":
        d = s["dout"].float()
        g = d if s["weight"] is None else d * s["weight"].float()
        dx = rstd * (g - g.mean(1, keepdim=True) - hat * (g * hat).mean(1, keepdim=True))
        if s["residual"] is not None:
            dx = dx + s["residual"].float()
        got |= {"mean": mean[:, 0], "rstd": rstd[:, 0], "dx": dx.to(s["x"].dtype)}
        if s["weight"] is not None:
            got |= {"dweight": (d * hat).sum(0), "dbias": d.sum(0)}
    return got


def _plain_linear(s):
    c = s["case"]
    a = _rounded(s["A"]) if c["a"] == "raw" else _values(s["A_codes"], s["A_scales"], c["K"])
    x = a @ _values(s["B_codes"], s["B_scales"], c["K"]).t() + s["bias"].float()
    if s["R"] is not None:
        x = x + s["R"].float()
    return _act(x, None if s["Y"] is None else s["Y"].float(), c["act"]).to(DTYPES[c["dtype"]])


def _own_norm(fl, s):
    if s["case"]["step"] == "forward":
        return {"y": fl.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS)}
    y, mean, rstd = fl.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, stats=True)
    dx, dweight, dbias = fl.layer_norm_bwd(s["dout"], s["x"], mean, rstd, s["weight"], R=s["residual"],
                                           dweight=s["weight"] is not None, dbias=s["bias"] is not None)
    return {"y": y, "mean": mean, "rstd": rstd, "dx": dx, "dweight": dweight, "dbias": dbias}


def run(s):
    c = s["case"]
    if own:
        import activation_epilogue_amd as fl
        if c["op"] == "norm":
            return _own_norm(fl, s)
        if c["op"] == "quant":
            return fl.dequantize_mx4(fl.quantize_mx4(s["x"], transposed=c["transposed"]), s["x"].dtype)
        a = s["A"] if c["a"] == "raw" else fl.Mx4(s["A_codes"], s["A_scales"], c["K"])
        return fl.fused_linear_mx4(a, fl.Mx4(s["B_codes"], s["B_scales"], c["K"]), s["bias"], s["Y"], act=c["act"],
                                   R=s["R"], dtype=DTYPES[c["dtype"]])
    if c["op"] == "norm":
        return _plain_norm(s)
    if c["op"] == "quant":
        x = s["x"].t() if c["transposed"] else s["x"]
        return _values(*_quantize(x), c["K"]).to(x.dtype)
    return _plain_linear(s)


# ------------------------------------------------------------------- work

def work(case):
    es = SIZES[case["dtype"]]
    if case["op"] == "norm":
        n, H = case["M"] * case["H"], case["H"]
        affine = 2 * H * es if case["affine"] else 0
        if case["step"] == "forward":
            return {"bytes": 2 * n * es + affine, "flops": 8.0 * n}
        # forward: x, y and the statistics; backward: x, dout, dx (and the residual's), the weight's gradients
        moved = (5 + (1 if case["residual"] else 0)) * n * es + 16 * case["M"]
        return {"bytes": moved + (affine + H * es + 8 * H if case["affine"] else 0), "flops": 24.0 * n}
    if case["op"] == "quant":
        # x, its codes and scales written and read again, and the values
        n, blocks = case["rows"] * case["K"], case["rows"] * ((case["K"] + 31) // 32)
        return {"bytes": 2 * n * es + 2 * 17 * blocks, "flops": 4.0 * n}
    M, N, K = case["M"], case["N"], case["K"]
    blocks = (K + 31) // 32
    a = M * K * es if case["a"] == "raw" else M * blocks * 17
    outs = 1 + (1 if case["act"] == "glu" else 0) + (1 if case["residual"] else 0)
    return {"bytes": a + N * blocks * 17 + N * es + outs * M * N * es, "flops": 2.0 * M * N * K}


# ------------------------------------------------------------ in 64 bits

def _nearest(x):
    """The values of x (rows, K) after quantising, in 64 bits: every element's nearest multiple by its own exponent."""
    x = x.double()
    rows, K = x.shape
    out = torch.empty_like(x)
    for lo in range(0, K, 32):  # one block of every row at a time
        b = x[:, lo:lo + 32]
        top = b.abs().max(1, keepdim=True).values
        scale = torch.exp2(torch.frexp(top).exponent.double() - 3.0).clamp(min=2.0 ** -127)
        v = b / scale
        # E2M1 has one bit behind the point's: steps of a half below 2, of 1 to 4, of 2 above; 6 is the largest
        step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0)).to(v.dtype)
        v = (torch.round(v / step) * step).clamp(-6.0, 6.0)  # round: ties to even multiples, which are the even codes
        out[:, lo:lo + 32] = v * scale
    return out


def _read(codes, scales, K):
    """The values of codes and scales in 64 bits, by the format's bits: sign, two of exponent, one of mantissa."""
    c = torch.empty(codes.shape[0], codes.shape[1] * 2, dtype=torch.int64, device=codes.device)
    c[:, 0::2], c[:, 1::2] = codes.long() & 15, codes.long() >> 4
    e, m = (c >> 1) & 3, (c & 1).double()
    v = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2((e - 1).double()))
    v = torch.where(c >= 8, -v, v)
    return (v * torch.exp2(scales.double() - 127).repeat_interleave(32, 1))[:, :K]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quant":
        x = s["x"]
        return _nearest(x.t().contiguous() if case["transposed"] else x)
    if case["op"] == "linear":
        a = _nearest(s["A"]) if case["a"] == "raw" else _read(s["A_codes"], s["A_scales"], case["K"])
        x = torch.mm(a, _read(s["B_codes"], s["B_scales"], case["K"]).t().contiguous()) + s["bias"].double()
        x = x if s["R"] is None else x + s["R"].double()
        act = case["act"]
        if act == "relu":
            return x.clamp(min=0.0)
        if act == "gelu_tanh":  # 0.5 (1 + tanh u) = 1 / (1 + exp(-2u))
            return x / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))
        return x * (1 + s["Y"].double()) if act == "glu" else x
    x = s["x"].double()
    H = x.shape[1]
    mean = x.sum(1) / H
    var = (x * x).sum(1) / H - mean * mean  # 64 bits have room for the difference
    rstd = (var + EPS) ** -0.5
    hat = (x - mean[:, None]) * rstd[:, None]
    w = torch.ones(H, dtype=torch.float64, device=x.device) if s["weight"] is None else s["weight"].double()
    got = {"y": hat * w + (0.0 if s["bias"] is None else s["bias"].double())}
    if case["step"] == "train":
        d = s["dout"].double()
        # the Jacobian of the norm is rstd (1 - 1/H - hat hat^T / H)
        g = d * w
        dx = rstd[:, None] * (g - (g.sum(1, keepdim=True) + hat * (g * hat).sum(1, keepdim=True)) / H)
        got |= {"mean": mean, "rstd": rstd, "dx": dx if s["residual"] is None else dx + s["residual"].double()}
        if s["weight"] is not None:
            got |= {"dweight": (d * hat).sum(0), "dbias": d.sum(0)}
    return got
