"""The operators that serve a quantized layer, as cases to be timed and compared.

A layer that ``gq_quantize_layer`` has written is a packed bit stream of b-bit codes, a scale and
a zero point per row and group: w = scale * (code - zero).  Three operators run it:

* ``norm``: h = x + residual (stored in the inputs' type), the root-mean-square norm
  v = h / sqrt(mean(h^2) + eps) * gamma, and v in 8 bits, one scale a row:
  scale = max|v| / 127, q = rint(v / scale).  The factor 1 / sqrt(..) cancels in q, so
  q = rint(127 u / max|u|) with u = h gamma.
* ``linear``: y = x W^T from the packed weights, x in bf16 or fp32.
* ``quantized``: y = (q qscale) W^T from the packed weights and 8-bit rows.

``step`` is a norm and a product of its 8-bit rows, as one decoder input runs them.  A case's
``ordered`` means groups along a column order: the codes are packed in that order and column k
multiplies x[:, perm[k]].

With ``own`` false every operator is computed in elementary torch operations; with ``own`` true
by the calls of this repository's library.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def _norm(T, n, dtype, residual, out, eps=1e-6):
    return dict(op="norm", T=T, n=n, dtype=dtype, residual=residual, out=out, eps=eps)


def _linear(op, T, m, n, bits, group, dtype, out, ordered=False):
    return dict(op=op, T=T, m=m, n=n, bits=bits, group=group, dtype=dtype, out=out,
                ordered=ordered)


def listed():
    cases = [
        # the attention input of the 8B-shaped block, one token being decoded
        ("norm one token", _norm(1, 4096, "bf16", True, "q8")),
        # the same for the sweep's 8192 calibration tokens
        ("norm calibration", _norm(8192, 4096, "bf16", True, "q8")),
        # an odd width in fp32, no residual, both forms of the output
        ("norm odd width", _norm(777, 1003, "fp32", False, "both", 1e-5)),
        # the down projection (3-bit, group 128) for one token
        ("linear mlp_down one token", _linear("linear", 1, 4096, 14336, 3, 128, "bf16", "bf16")),
        # a few tokens through a small odd layer in fp32: partial words, a ragged last group
        ("linear odd small", _linear("linear", 5, 1000, 1001, 5, 32, "fp32", "fp32")),
        # a batch of requests through the key projection of the 2-bit sweep
        ("linear k_proj batch", _linear("linear", 48, 1024, 4096, 2, 64, "bf16", "bf16")),
        # q_proj quantized in act-order, an odd prompt in fp32
        ("linear q_proj ordered", _linear("linear", 257, 4096, 4096, 4, 128, "fp32", "fp32", True)),
        # the down projection's calibration tokens, to calibrate what follows the layer
        ("linear mlp_down calibration", _linear("linear", 8192, 4096, 14336, 3, 128, "bf16", "bf16")),
        # q_proj (4-bit, group 128) on the 8-bit row of one token
        ("quantized q_proj one token", _linear("quantized", 1, 4096, 4096, 4, 128, "bf16", "bf16")),
        # q, k and v of the 2-bit sweep side by side, sixteen requests
        ("quantized qkv batch", _linear("quantized", 16, 6144, 4096, 2, 64, "bf16", "bf16")),
        # the up projection's calibration tokens in 8 bits
        ("quantized mlp_up calibration", _linear("quantized", 8192, 14336, 4096, 3, 128, "bf16", "bf16")),
        # norm, 8-bit rows and the stacked q, k, v product of one decoded token
        ("step qkv one token", _linear("step", 1, 6144, 4096, 4, 128, "bf16", "bf16")),
    ]
    return [dict(c, name=name) for name, c in cases]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "linear", "linear", "quantized", "quantized", "step"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "norm":
        n = _log(rng, 64, 14336)
        T = _log(rng, 1, 8192 if n <= 8192 else 4096)
        residual = rng.random() < 0.7
        return _norm(T, n, dtype, residual, rng.choice(["q8", "q8", "y", "both"]),
                     rng.choice([1e-6, 1e-5]))
    m, n = _log(rng, 64, 14336), _log(rng, 64, 14336)
    if rng.random() < 0.5:  # widths as layers have them; the others stay odd
        m, n = -(-m // 128) * 128, -(-n // 128) * 128
    most = 8192 * 4096 * 14336 // (m * n)
    T = _log(rng, 1, min(8192, most) if op != "step" else min(256, most))
    group = rng.choice([0, 16, 32, 64, 128, 128])
    return _linear(op, T, m, n, rng.randint(2, 8), group, dtype, dtype,
                   op != "step" and group > 0 and rng.random() < 0.3)


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _tokens(T, n, g):
    """Activations as a decoder has them: a scale per channel, and a few outlier channels."""
    chan = torch.exp(0.5 * torch.randn(n, generator=g, device="cuda"))
    chan[torch.randperm(n, generator=g, device="cuda")[:4]] *= 20
    return torch.randn(T, n, generator=g, device="cuda") * chan


def _pack(codes, bits):
    """m x n codes as an LSB-first stream of b-bit codes per row, in 32-bit words."""
    m, n = codes.shape
    words = -(-n * bits // 32)
    stream = torch.zeros((m, words * 32), dtype=torch.uint8, device=codes.device)
    for i in range(bits):
        stream[:, i:n * bits:bits] = (codes >> i) & 1
    place = torch.arange(32, device=codes.device, dtype=torch.int32)
    packed = torch.empty((m, words), dtype=torch.int32, device=codes.device)
    for a in range(0, m, 2048):
        part = stream[a:a + 2048].view(-1, words, 32).to(torch.int32) << place
        packed[a:a + 2048] = part.sum(2, dtype=torch.int32)
    return packed


def _layer(m, n, bits, group, g):
    """Codes, scales and zero points of a min-max quantized layer (w = scale (code - zero))."""
    w = 0.02 * torch.randn(m, n, generator=g, device="cuda")
    size = group or n
    G = -(-n // size)
    padded = torch.zeros((m, G * size), device="cuda")
    padded[:, :n] = w
    blocks = padded.view(m, G, size)
    lo, hi = blocks.amin(2).clamp(max=0), blocks.amax(2).clamp(min=0)
    top = (1 << bits) - 1
    scales = (hi - lo) / top
    zeros = torch.round(-lo / scales).clamp(0, top)
    codes = (torch.round(blocks / scales[:, :, None]) + zeros[:, :, None]).clamp(0, top)
    codes = codes.view(m, G * size)[:, :n].to(torch.uint8)
    return _pack(codes, bits), scales.contiguous(), zeros.to(torch.uint8).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, T, n = case["op"], case["T"], case["n"]
    dt, out = TYPES[case["dtype"]], case["out"]
    s = dict(case=case)
    x = _tokens(T, n, g)
    if op in ("norm", "step"):
        s["x"] = x.to(dt)
        s["gamma"] = (1 + 0.2 * torch.randn(n, generator=g, device="cuda")).to(dt)
        s["eps"] = case.get("eps", 1e-6)
        s["residual"] = None
        if case.get("residual", True):
            s["residual"] = (3 * _tokens(T, n, g)).to(dt)
        s["sum"] = torch.empty_like(s["x"]) if s["residual"] is not None else None
        s["y"] = torch.empty_like(s["x"]) if out in ("y", "both") else None
        s["q"] = torch.empty((T, n), dtype=torch.int8, device="cuda") if out != "y" else None
        s["qscale"] = torch.empty(T, dtype=torch.float32, device="cuda") if out != "y" else None
    if op == "norm":
        return s
    m = case["m"]
    s["bits"], s["group"] = case["bits"], case["group"]
    s["codes"], s["scales"], s["zeros"] = _layer(m, n, case["bits"], case["group"], g)
    s["perm"] = None
    if case["ordered"]:
        s["perm"] = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
    s["out"] = torch.empty((T, m), dtype=TYPES[out], device="cuda")
    if op == "linear":
        s["x"] = x.to(dt)
    elif op == "quantized":
        s["qscale"] = x.abs().amax(1) / 127
        s["q"] = torch.round(x / s["qscale"][:, None]).to(torch.int8)
    return s


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def _plain_norm(s):
    h = s["x"]
    r = {}
    if s["residual"] is not None:
        h = (h.float() + s["residual"].float()).to(h.dtype)
        r["sum"] = h
    # 64 bits: the codes are decided at borders between two of them
    h = h.double()
    u = h * s["gamma"].double()
    rstd = torch.rsqrt(h.square().mean(1, keepdim=True) + s["eps"])
    if s["y"] is not None:
        r["y"] = (u * rstd).to(s["x"].dtype)
    if s["q"] is not None:
        top = u.abs().amax(1, keepdim=True)
        r["q"] = torch.where(top > 0, torch.round(127 * u / top), 0.0).to(torch.int8)
        r["qscale"] = (top * rstd / 127).float().view(-1)
    return r


def _plain_weights(s):
    n, bits, group = s["n"], s["bits"], s["group"]
    words = s["codes"].to(torch.int64) & 0xFFFFFFFF
    at = torch.arange(n, device="cuda") * bits
    low = words[:, at // 32] >> (at % 32)
    high = words[:, (at // 32 + 1).clamp(max=words.shape[1] - 1)] << (32 - at % 32)
    codes = ((low | high) & ((1 << bits) - 1)).float()
    of = torch.arange(n, device="cuda") // (group or n)
    return s["scales"][:, of] * (codes - s["zeros"].float()[:, of])


def _plain_linear(s, x):
    if s["perm"] is not None:
        x = x[:, s["perm"].long()]
    return x.float() @ _plain_weights(s).T


def run(state):
    s = state
    case = s["case"]
    op = case["op"]
    if own:
        from post_weight_quantization_22_b200 import gq as G
        if op == "linear":
            return G.gq_linear(s["x"], s["codes"], s["scales"], s["zeros"], s["bits"], s["group"],
                               perm=s["perm"], y=s["out"])
        if op == "quantized":
            return G.gq_linear_quantized(s["q"], s["qscale"], s["codes"], s["scales"], s["zeros"],
                                         s["bits"], s["group"], perm=s["perm"], y=s["out"])
        r = G.gq_rmsnorm_quantize(s["x"], s["gamma"], s["eps"], residual=s["residual"],
                                  sum=s["sum"], y=s["y"], q=s["q"], qscale=s["qscale"])
        if op == "step":
            y = G.gq_linear_quantized(r["q"], r["qscale"], s["codes"], s["scales"], s["zeros"],
                                      s["bits"], s["group"], y=s["out"])
            return {"sum": r["sum"], "out": y}
    else:
        s = dict(s, n=case["n"])
        if op == "linear":
            return _plain_linear(s, s["x"]).to(s["out"].dtype)
        if op == "quantized":
            return (_plain_linear(s, s["q"]) * s["qscale"][:, None]).to(s["out"].dtype)
        r = _plain_norm(s)
        if op == "step":
            y = _plain_linear(s, r["q"]) * r["qscale"][:, None]
            return {"sum": r["sum"], "out": y.to(s["out"].dtype)}
    # the 8-bit rows as the values that they stand for
    got = {k: r[k] for k in ("sum", "y") if r.get(k) is not None}
    if r.get("q") is not None:
        got["rows"] = r["q"] * r["qscale"][:, None]
    return got


def work(case):
    op, T, n = case["op"], case["T"], case["n"]
    size = 2 if case["dtype"] == "bf16" else 4
    if op == "norm":
        rows = 1 + (2 if case["residual"] else 0) + (1 if case["out"] != "q8" else 0)
        q8 = T * (n + 4) if case["out"] != "y" else 0
        return {"bytes": rows * T * n * size + n * size + q8, "flops": 8.0 * T * n}
    m, bits = case["m"], case["bits"]
    G = -(-n // (case["group"] or n))
    b = m * (-(-n * bits // 32)) * 4 + m * G * 5 + (4 * n if case["ordered"] else 0)
    b += T * m * (2 if case["out"] == "bf16" else 4)
    if op == "linear":
        b += T * n * size
    elif op == "quantized":
        b += T * (n + 4)
    else:
        b += 3 * T * n * size + n * size
    return {"bytes": float(b), "flops": 2.0 * T * m * n}


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------

def _exact_norm(s):
    x = s["x"].cpu().double().numpy()
    r = {}
    if s["residual"] is not None:
        # the stored sum: an exact sum in 64 bits, rounded to the inputs' type
        x = x + s["residual"].cpu().double().numpy()
        x = torch.from_numpy(x).to(s["x"].dtype).double().numpy()
        r["sum"] = x
    gamma = s["gamma"].cpu().double().numpy()
    rms = np.sqrt(np.einsum("ij,ij->i", x, x) / x.shape[1] + s["eps"])
    q, scale = None, None
    if s["y"] is not None:
        r["y"] = x / rms[:, None] * gamma
    if s["q"] is not None:
        u = x * gamma
        top = np.abs(u).max(1)
        q = np.rint(127 * u / np.where(top > 0, top, 1)[:, None])
        scale = top / rms / 127
        r["rows"] = q * scale[:, None]
    return r, q, scale


def _exact_rows(s, a, b):
    """Rows a..b of the layer in 64 bits, from the stream's single bits."""
    n, bits = s["case"]["n"], s["bits"]
    words = s["codes"][a:b]
    place = torch.arange(32, device="cuda", dtype=torch.int32)
    stream = ((words[:, :, None] >> place) & 1).to(torch.uint8).reshape(b - a, -1)
    codes = torch.zeros((b - a, n), dtype=torch.float64, device="cuda")
    for i in range(bits):
        codes += stream[:, i:n * bits:bits].double() * 2.0 ** i
    size = s["group"] or n
    for k in range(s["scales"].shape[1]):
        part = codes[:, k * size:(k + 1) * size]
        part -= s["zeros"][a:b, k].double()[:, None]
        part *= s["scales"][a:b, k].double()[:, None]
    return codes


def _exact_linear(s, x):
    if s["perm"] is not None:
        x = torch.index_select(x, 1, s["perm"].to(torch.int64))
    m = s["codes"].shape[0]
    y = torch.empty((x.shape[0], m), dtype=torch.float64, device="cuda")
    for a in range(0, m, 1024):
        b = min(m, a + 1024)
        y[:, a:b] = torch.mm(x, _exact_rows(s, a, b).t())
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        return _exact_linear(s, s["x"].double())
    if op == "quantized":
        return _exact_linear(s, s["q"].double() * s["qscale"].double()[:, None])
    r, q, scale = _exact_norm(s)
    if op == "norm":
        return r
    rows = torch.from_numpy(q * scale[:, None]).cuda()
    return {"sum": r["sum"], "out": _exact_linear(s, rows)}
