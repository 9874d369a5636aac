"""FP8 training and serving operators with float32 scales per 128 elements, timed and compared.

Four operators, which a transformer layer runs one after the other:

* ``norm``      h = x + residual, RMSNorm of h, FP8 codes and scales of the normalized row;
* ``norm_bwd``  its gradient for h (with the residual stream's gradient added) and for the weight;
* ``quant``     FP8 codes with a scale per 1 x 128 tile or 128 x 128 block, along the rows,
                along the columns (transposed codes) or both from one read;
* ``gemm``      D = A B^T of such operands: weights in 128 x 128 blocks (forward and input
                gradient), or both sides in 1 x 128 tiles (weight gradient).

``run`` computes them in plain torch, or (``own``) through the package.
"""

import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_MAX = {"e4m3": 448.0, "e5m2": 57344.0}
_TINY = 2.0 ** -126   # the smallest scale
_EPS = 1e-6


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one token of a decoding sequence, hidden size of the MoE layers: launch latency
        dict(name="norm_token", op="norm", rows=1, cols=2048, type="bf16", residual=True, pow2=False, pad=0),
        # a long prefill whose length is no multiple of anything
        dict(name="norm_prefill", op="norm", rows=16387, cols=4096, type="bf16", residual=True, pow2=False, pad=0),
        # a short training batch without a residual gradient
        dict(name="norm_bwd_short", op="norm_bwd", rows=1999, cols=2048, type="bf16", residual=False),
        # a training batch
        dict(name="norm_bwd_batch", op="norm_bwd", rows=16384, cols=4096, type="bf16", residual=True),
        # activations of a training step, for the forward product and the weight gradient
        dict(name="quant_tokens_both", op="quant", rows=4099, cols=4096, type="bf16", format="e4m3",
             block=False, direction="both", pow2=False, pad=0),
        # 32 experts' w13 weights, for the forward product and the input gradient
        dict(name="quant_experts", op="quant", rows=32 * 1536, cols=2048, type="bf16", format="e4m3",
             block=True, direction="both", pow2=False, pad=0),
        # a few tokens through one expert's w13: launch latency
        dict(name="gemm_expert_16", op="gemm", M=16, N=1536, K=2048, a="e4m3", b="e4m3", block=True, out="bf16"),
        # one decoding sequence through a large layer: the weights' bytes
        dict(name="gemm_token", op="gemm", M=1, N=8192, K=8192, a="e4m3", b="e4m3", block=True, out="bf16"),
        # a decoding batch
        dict(name="gemm_batch_128", op="gemm", M=128, N=8192, K=4096, a="e4m3", b="e4m3", block=True, out="bf16"),
        # input gradient (E5M2 gradients) of a batch of odd length
        dict(name="gemm_dgrad_odd", op="gemm", M=4099, N=2056, K=8192, a="e5m2", b="e4m3", block=True, out="bf16"),
        # weight gradient: the sum runs over an odd number of tokens
        dict(name="gemm_wgrad_odd", op="gemm", M=4096, N=2048, K=8195, a="e4m3", b="e4m3", block=False, out="fp32"),
        # prefill through a large layer
        dict(name="gemm_prefill", op="gemm", M=8192, N=8192, K=8192, a="e4m3", b="e4m3", block=True, out="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi, step):
    """A size between lo and hi over its logarithm: mostly multiples of `step`, at times odd."""
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.3 else max(lo, v // step * step)


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "quant", "gemm", "gemm"])
    kind = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("norm", "norm_bwd"):
        cols = _size(rng, 128, 8192, 128)
        rows = _log(rng, 1, min(16384, (16384 * 4096) // (2 * cols)))
        case = dict(op=op, rows=rows, cols=cols, type=kind, residual=rng.random() < 0.7)
        if op == "norm":
            case.update(pow2=False, pad=rng.choice([0, 0, 0, 64]))
        return case
    if op == "quant":
        cols = _size(rng, 128, 8192, 128)
        rows = _log(rng, 1, min(32768, (32 * 1536 * 1024) // cols))
        return dict(op=op, rows=rows, cols=cols, type=kind, format=rng.choice(["e4m3", "e4m3", "e5m2"]),
                    block=rng.random() < 0.4, direction=rng.choice(["rows", "cols", "both"]),
                    pow2=rng.random() < 0.3, pad=rng.choice([0, 0, 0, 64]))
    block = rng.random() < 0.7
    return dict(op=op, M=_log(rng, 1, 8192), N=_size(rng, 64, 8192, 64), K=_size(rng, 128, 8192, 128),
                a=rng.choice(["e4m3", "e4m3", "e5m2"]), b="e4m3", block=block,
                out="bf16" if block and rng.random() < 0.7 else "fp32")


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(rows, cols, g, pad=0):
    """N(0, 1) rows with a few large channels, as hidden states have them."""
    x = torch.randn(rows, cols + pad, generator=g, device="cuda")
    n = max(1, cols // 256)
    x[:, torch.randint(0, cols, (n,), generator=g, device="cuda")] *= 20.0
    return x


def _fit(n, step):
    return (n + step - 1) // step * step


def _operand(rows, cols, fmt, block, g, scale):
    """Codes [rows, cols] and scales of one side of a product, laid out as the quantizer
    lays them out: codes' rows 16 bytes apart or a multiple, tile scales block-major."""
    x = torch.randn(rows, cols, generator=g, device="cuda") * scale
    if not block and rows > 1:
        x[torch.randint(0, rows, (1 + rows // 256,), generator=g, device="cuda")] *= 10.0
    codes, scales = _plain_rows(x, fmt, block, False)
    held = torch.zeros(rows, _fit(cols, 16), dtype=torch.uint8, device="cuda")
    held[:, :cols] = codes.view(torch.uint8)
    if not block:
        laid = torch.zeros(scales.shape[1], _fit(rows, 4), device="cuda")
        laid[:, :rows] = scales.t()
        scales = laid.t()[:rows]
    return held[:, :cols], scales


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "gemm":
        a = _operand(case["M"], case["K"], case["a"], False, g, 1.0)
        b = _operand(case["N"], case["K"], case["b"], case["block"], g, 0.02 if case["block"] else 1.0)
        return dict(case=case, a=a, b=b)
    t = _TYPES[case["type"]]
    rows, cols = case["rows"], case["cols"]
    if case["op"] == "quant":
        w = case["block"]
        x = torch.randn(rows, cols + case["pad"], generator=g, device="cuda").mul_(0.02) if w else \
            _activations(rows, cols, g, case["pad"])
        return dict(case=case, x=x.to(t)[:, :cols])
    weight = (1 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(t)
    if case["op"] == "norm":
        x = torch.randn(rows, cols + case["pad"], generator=g, device="cuda").to(t)[:, :cols]
        res = _activations(rows, cols, g).to(t) if case["residual"] else None
        return dict(case=case, x=x, residual=res, weight=weight)
    grad = (torch.randn(rows, cols, generator=g, device="cuda") * 0.01).to(t)
    res = (torch.randn(rows, cols, generator=g, device="cuda") * 0.01).to(t) if case["residual"] else None
    return dict(case=case, grad=grad, h=_activations(rows, cols, g).to(t), weight=weight, residual=res)


# ------------------------------------------------------------ plain forms --

def _spread(scales, rows, cols, block):
    """The scale of every element from the scales of tiles (1 x 128) or blocks (128 x 128)."""
    s = scales.repeat_interleave(128, 1)[:, :cols]
    return s.repeat_interleave(128, 0)[:rows] if block else s


def _plain_rows(x, fmt, block, pow2):
    """FP8 values and float32 scales of float32 rows x, tiles along the rows:
    scale = amax / max, or the smallest power of two that holds amax."""
    rows, cols = x.shape
    c, r = _fit(cols, 128), _fit(rows, 128) if block else rows
    a = torch.nn.functional.pad(x.abs(), (0, c - cols, 0, r - rows)).view(r, c // 128, 128).amax(2)
    if block:
        a = a.view(r // 128, 128, c // 128).amax(1)
    if pow2:
        m, e = torch.frexp(a)   # the largest FP8 value is 0.875 times a power of two
        top = int(math.log2(_MAX[fmt] / 0.875))
        s = torch.ldexp(torch.ones_like(a), torch.where(m <= 0.875, e - top, e - top + 1).clamp(min=-126))
        s = torch.where(a > 0, s, torch.full_like(s, _TINY))
    else:
        s = (a / _MAX[fmt]).clamp(min=_TINY)
    return (x / _spread(s, rows, cols, block)).to(_FP8[fmt]), s


def _plain_quant(x, case):
    x = x.float()
    out = ()
    if case["direction"] in ("rows", "both"):
        out += _plain_rows(x, case["format"], case["block"], case["pow2"])
    if case["direction"] in ("cols", "both"):
        out += _plain_rows(x.t().contiguous(), case["format"], case["block"], case["pow2"])
    return out


def _plain_norm(s):
    case, t = s["case"], s["x"].dtype
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + _EPS) * s["weight"].float()
    codes, scales = _plain_rows(y, "e4m3", False, case["pow2"])
    return codes, scales, h.to(t) if s["residual"] is not None else None


def _plain_norm_bwd(s):
    g, h, w = s["grad"].float(), s["h"].float(), s["weight"].float()
    r = torch.rsqrt(h.square().mean(1, keepdim=True) + _EPS)
    xh, gw = h * r, g * w
    gh = r * (gw - xh * (gw * xh).mean(1, keepdim=True))
    if s["residual"] is not None:
        gh = gh + s["residual"].float()
    return gh.to(s["h"].dtype), (g * xh).sum(0)


def _plain_gemm(s):
    case = s["case"]
    sides = []
    for (codes, scales), fmt, block in ((s["a"], case["a"], False), (s["b"], case["b"], case["block"])):
        v = codes.contiguous().view(_FP8[fmt]).float()
        sides.append(v * _spread(scales, v.shape[0], v.shape[1], block))
    return (sides[0] @ sides[1].t()).to(_TYPES[case["out"]])


# -------------------------------------------------------------------- run --

def _own(s):
    import fp8_quantization_mx_b200 as mx
    case = s["case"]
    if case["op"] == "gemm":
        (a, sa), (b, sb) = s["a"], s["b"]
        return mx.gemm128(a, sa, b, sb, a_format=mx.E5M2 if case["a"] == "e5m2" else mx.E4M3,
                          b_format=mx.E4M3, out_dtype=_TYPES[case["out"]])
    if case["op"] == "quant":
        fmt = case["format"]
        out = mx.quantize128(s["x"], mx.E5M2 if fmt == "e5m2" else mx.E4M3, block=case["block"],
                             direction=case["direction"], pow2=case["pow2"])
        return tuple(v.view(_FP8[fmt]) if v.dtype == torch.uint8 else v for v in out)
    if case["op"] == "norm":
        codes, scales, h, _ = mx.rms_norm_quantize(s["x"], s["weight"], s["residual"], eps=_EPS,
                                                   pow2=case["pow2"])
        return codes.view(torch.float8_e4m3fn), scales, h
    return mx.rms_norm_bwd(s["grad"], s["h"], s["weight"], eps=_EPS, grad_residual=s["residual"])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "gemm":
        return _plain_gemm(state)
    if op == "quant":
        return _plain_quant(state["x"], state["case"])
    return _plain_norm(state) if op == "norm" else _plain_norm_bwd(state)


# ------------------------------------------------------------------- work --

def work(case):
    if case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        nk = -(-K // 128)
        scales = 4 * nk * (M + (-(-N // 128) if case["block"] else N))
        return {"bytes": M * K + N * K + scales + M * N * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * M * N * K}
    rows, cols = case["rows"], case["cols"]
    n, size = rows * cols, 4 if case["type"] == "fp32" else 2
    if case["op"] == "norm":
        return {"bytes": n * (size * (3 if case["residual"] else 1) + 1) + 4 * rows * -(-cols // 128) + cols * size,
                "flops": 8 * n}
    if case["op"] == "norm_bwd":
        return {"bytes": n * size * (4 if case["residual"] else 3) + cols * (size + 4), "flops": 14 * n}
    ways = 2 if case["direction"] == "both" else 1
    r, c = -(-rows // 128), -(-cols // 128)
    along = {"rows": rows * c, "cols": cols * r, "both": rows * c + cols * r}[case["direction"]]
    scales = r * c * ways if case["block"] else along
    return {"bytes": n * (size + ways) + 4 * scales, "flops": 3 * n * ways}


# ------------------------------------------------------------------ exact --

def _exact_fp8(v, fmt):
    """Nearest FP8 value of float64 v (ties to the even code), by its exponent."""
    bits, low = (3, -6) if fmt == "e4m3" else (2, -14)
    _, e = torch.frexp(v)
    ulp = torch.ldexp(torch.ones_like(v), torch.clamp(e - 1, min=low) - bits)
    return torch.round(v / ulp).mul_(ulp).clamp_(-_MAX[fmt], _MAX[fmt])


def _exact_quant(x, fmt, block, pow2):
    rows, cols = x.shape
    parts = []
    for c in x.split(128, 1):   # the last tile may be narrower
        a = c.abs().amax(1)
        if block:
            a = torch.stack([b.amax() for b in a.split(128)])
        parts.append(a)
    a = torch.stack(parts, 1)
    s = a / _MAX[fmt]
    if pow2:   # the smallest power of two that is not below amax / max, both exact
        e = torch.frexp(s)[1]
        half = torch.ldexp(torch.ones_like(s), e - 1)
        s = torch.where(s <= half, half, 2 * half)
    s = torch.where(a > 0, s, torch.zeros_like(s)).clamp(min=_TINY)
    at = torch.arange(cols, device=x.device) // 128
    full = s[torch.arange(rows, device=x.device) // 128][:, at] if block else s[:, at]
    return _exact_fp8(x / full, fmt), s


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gemm":
        total = None
        (a, sa), (b, sb) = s["a"], s["b"]
        for i, k in enumerate(range(0, case["K"], 1024)):
            p = a[:, k:k + 1024].contiguous().view(_FP8[case["a"]]).double()
            q = b[:, k:k + 1024].contiguous().view(_FP8[case["b"]]).double()
            at = torch.arange(k, k + p.shape[1], device=p.device) // 128
            p *= sa.double()[:, at]
            q *= (sb.double()[torch.arange(case["N"], device=q.device) // 128] if case["block"] else sb.double())[:, at]
            total = p @ q.t() if total is None else total.addmm_(p, q.t())
        return total
    if case["op"] == "quant":
        out = ()
        for way, x in (("rows", s["x"]), ("cols", s["x"].t())):
            if case["direction"] in (way, "both"):
                out += _exact_quant(x.double(), case["format"], case["block"], case["pow2"])
        return out
    w = s["weight"].double()
    if case["op"] == "norm":
        h = s["x"].double() + (0 if s["residual"] is None else s["residual"].double())
        y = h / torch.sqrt((h * h).sum(1, keepdim=True) / case["cols"] + _EPS) * w
        return _exact_quant(y, "e4m3", False, case["pow2"]) + (h if s["residual"] is not None else None,)
    g, h = s["grad"].double(), s["h"].double()
    d = torch.sqrt((h * h).sum(1, keepdim=True) / case["cols"] + _EPS)
    n = h / d
    gh = g * w / d - n * ((g * w * n).sum(1, keepdim=True) / case["cols"]) / d
    return gh + (0 if s["residual"] is None else s["residual"].double()), torch.einsum("rc,rc->c", g, n)
