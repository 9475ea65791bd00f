"""The dense path in 8-bit floating point: what its operators are given, what they compute, and how much work that is.

Four operators, used one after the other around attention and the feed-forward block, from single tokens to whole prompts:

* norm: the residual's addition and a root-mean-square norm, its result in 8 bits with a scale for each 128 columns;
* quant: bf16 values into that format (an attention's output; weights once, with a scale for each block of 128 by 128);
* gemm: a matrix product of two such operands (the projections around attention, and back from the feed-forward block);
* gated: both projections of a gated feed-forward block, silu(gate) * up, the result in 8 bits again.

A code is an e4m3 number, a scale a power of two held as its exponent (e8m0): the smallest one that leaves no code of
its block beyond 448. `run` computes a case in its plain form (elementary torch operations in 32 bits), or with the
package's kernels where `own` is true. `exact` computes it from the definitions in 64 bits.
"""

import math

import torch

own = False

BLOCK = 128  # columns that share one scale; of weights, rows too
TOP = 448.0  # the largest e4m3 number


# ---------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # before a layer in one decode step of 64 sequences: the router behind it reads the bf16 copy
        dict(name="norm_step", op="norm", rows=64, cols=4096, f32=False, copy=True),
        # the same of a long prompt, in front of dense projections alone
        dict(name="norm_prompt", op="norm", rows=8191, cols=4096, f32=False, copy=False),
        # rows of an odd width, whose last scale stands for 16 columns; the addend is the unrounded sum of a layer's experts
        dict(name="norm_ragged", op="norm", rows=2049, cols=5008, f32=True, copy=True),
        # a prompt's attention output, cut out of wider rows, in front of the output projection
        dict(name="quant_prompt", op="quant", rows=4097, cols=8192, extra=1024, block=1),
        # a projection's weights, once
        dict(name="quant_weight", op="quant", rows=12288, cols=4096, extra=0, block=128),
        # the stacked query, key and value projections of one new token, where latency counts
        dict(name="gemm_token", op="gemm", rows=1, n=12288, k=4096, f32=False),
        # the output projection in one decode step of 64 sequences, unrounded
        dict(name="gemm_step", op="gemm", rows=64, n=4096, k=4096, f32=True),
        # the output projection of a prompt's chunk of odd length behind wide heads
        dict(name="gemm_chunk", op="gemm", rows=777, n=4096, k=8192, f32=False),
        # the stacked projections of a long prompt
        dict(name="gemm_prompt", op="gemm", rows=8191, n=12288, k=4096, f32=False),
        # five drafted tokens through a dense feed-forward block's first half
        dict(name="gated_draft", op="gated", rows=5, n=12288, k=4096, e4m3=True),
        # a shared expert in one decode step of 64 sequences
        dict(name="gated_step", op="gated", rows=64, n=1024, k=4096, e4m3=True),
        # a prompt through a dense feed-forward block's first half
        dict(name="gated_prompt", op="gated", rows=4095, n=12288, k=4096, e4m3=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["norm", "quant", "gemm", "gemm", "gated", "gated"])
    cols = 16 * _log(rng, 4, 1024)
    if op in ("norm", "quant"):
        rows = _log(rng, 1, min(8192, 30_000_000 // cols))
        if op == "norm":
            return dict(op="norm", rows=rows, cols=cols, f32=rng.random() < 0.3, copy=rng.random() < 0.5)
        return dict(op="quant", rows=rows, cols=cols, extra=rng.choice([0, 0, 8, 1024]), block=rng.choice([1, 1, 128]))
    rows = _log(rng, 1, 8192)
    most = min(100_000_000, 400_000_000_000 // rows) // (cols * (2 if op == "gated" else 1))
    if op == "gemm":
        return dict(op="gemm", rows=rows, n=_log(rng, 16, min(16384, most)), k=cols, f32=rng.random() < 0.4)
    return dict(op="gated", rows=rows, n=16 * _log(rng, 2, min(16384, most) // 16), k=cols, e4m3=rng.random() < 0.7)


def _blocks(cols):
    return -(-cols // BLOCK)


def work(c):
    if c["op"] == "norm":
        n = c["rows"] * c["cols"]
        return {"bytes": n * (4 + 4 + (4 if c["f32"] else 2) + 1 + (2 if c["copy"] else 0)) + 2 * c["cols"] + c["rows"] * _blocks(c["cols"]), "flops": 6 * n}
    if c["op"] == "quant":
        n = c["rows"] * c["cols"]
        return {"bytes": 3 * n + -(-c["rows"] // c["block"]) * _blocks(c["cols"]), "flops": 3 * n}
    m, n, k = c["rows"], c["n"], c["k"]
    x = m * (k + _blocks(k))
    w = n * k + _blocks(n) * _blocks(k)
    if c["op"] == "gemm":
        return {"bytes": x + w + m * n * (4 if c["f32"] else 2), "flops": 2 * m * n * k}
    return {"bytes": x + 2 * w + (m * (n + _blocks(n)) if c["e4m3"] else 2 * m * n), "flops": 4 * m * n * k + 5 * m * n}


# --------------------------------------------------------------------------------------------------------- inputs
def _quantise(x, block=1):
    """x [rows][cols] (fp32) as e4m3 codes and a power of two for each 128 columns of a row, or of `block` rows."""
    rows, cols = x.shape
    g = torch.nn.functional.pad(x, (0, -cols % BLOCK, 0, -rows % block)).view(-1, block, _blocks(cols), BLOCK)
    part, power = torch.frexp(g.abs().amax((1, 3), keepdim=True))
    e = torch.where(part == 0, -127, power - 9 + (part > 0.875).int()).clamp(min=-127)
    q = torch.ldexp(g, -e).view(-1, _blocks(cols) * BLOCK)[:rows, :cols].to(torch.float8_e4m3fn)
    return q.contiguous(), (e + 127).to(torch.uint8).view(-1, _blocks(cols)).view(torch.float8_e8m0fnu)


def _scales(rows, cols, dev):
    """Room for the scales of `rows` rows of `cols` columns: rows a multiple of four bytes apart."""
    n = _blocks(cols)
    return torch.zeros(rows, (n + 3) // 4 * 4, dtype=torch.uint8, device=dev).view(torch.float8_e8m0fnu)[:, :n]


def _held(x, block=1):
    """x quantised, as a program holds it."""
    q, e = _quantise(x, block)
    scale = _scales(e.shape[0], x.shape[1], x.device)
    scale.view(torch.uint8).copy_(e.view(torch.uint8))
    return q, scale


def _codes(rows, cols, dev):
    return torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device=dev)


def prepare(c, seed):
    dev = torch.device("cuda")
    rng = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=rng, device=dev)

    s = dict(c=c)
    if c["op"] == "norm":
        d = c["cols"]
        size = torch.exp(0.5 * normal(d))  # a residual's columns differ in size
        s["h"] = 3 * normal(c["rows"], d) * size
        s["delta"] = normal(c["rows"], d) * size
        if not c["f32"]:
            s["delta"] = s["delta"].bfloat16()
        s["rho"] = (1 + 0.1 * normal(d)).bfloat16()
        s["q"], s["scale"] = _codes(c["rows"], d, dev), _scales(c["rows"], d, dev)
        s["a"] = torch.empty(c["rows"], d, dtype=torch.bfloat16, device=dev) if c["copy"] else None
    elif c["op"] == "quant":
        wide = normal(c["rows"], c["cols"] + c["extra"]) * (0.02 if c["block"] > 1 else torch.exp(0.5 * normal(1, c["cols"] + c["extra"])))
        s["x"] = wide.bfloat16()[:, :c["cols"]]
        s["q"], s["scale"] = _codes(c["rows"], c["cols"], dev), _scales(-(-c["rows"] // c["block"]), c["cols"], dev)
    else:
        m, n, k = c["rows"], c["n"], c["k"]
        column = torch.exp(0.5 * normal(k))
        column[torch.randint(0, k, (max(1, k // 512),), generator=rng, device=dev)] *= 20  # a few columns stand far out
        s["x_q"], s["x_scale"] = _held(normal(m, k) * column)
        for w in ("w",) if c["op"] == "gemm" else ("gate", "up"):
            s[w + "_q"], s[w + "_scale"] = _held(normal(n, k) / math.sqrt(k), BLOCK)
        if c["op"] == "gemm":
            s["y"] = torch.empty(m, (n + 7) // 8 * 8, dtype=torch.float32 if c["f32"] else torch.bfloat16, device=dev)[:, :n]
        elif c["e4m3"]:
            s["q"], s["scale"] = _codes(m, n, dev), _scales(m, n, dev)
        else:
            s["y"] = torch.empty(m, n, dtype=torch.bfloat16, device=dev)
    if own:
        _handles(s)
    return s


def _handles(s):
    """The matrices' handles and the workspace that a serving program keeps from call to call."""
    from bit_group_quantized_gb300 import lib

    if "q" in s:
        s["out"] = lib.F8Matrix(s["q"], s["scale"], s["c"].get("block", 1))
    if "x_q" in s:
        s["x"] = lib.F8Matrix(s["x_q"], s["x_scale"])
        s |= {w: lib.F8Matrix(s[w + "_q"], s[w + "_scale"], BLOCK) for w in ("w", "gate", "up") if w + "_q" in s}
        s["ws"] = lib.workspace(lib.f8_gemm_workspace_bytes(s.get("w", s.get("up")), s["x"]), s["x_q"].device)


# ------------------------------------------------------------------------------------------------------------ run
def run(s):
    return {"norm": _norm, "quant": _quant, "gemm": _gemm, "gated": _gated}[s["c"]["op"]](s)


def _norm(s):
    if own:
        from bit_group_quantized_gb300 import lib

        lib.bgq_rmsnorm_f8(s["h"], s["rho"], 1e-6, delta=s["delta"], out=s["out"], a=s["a"])
        return s["q"], s["scale"], s["h"], s["a"]
    h = s["h"].add_(s["delta"].float())
    a = h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6) * s["rho"].float()
    q, scale = _quantise(a)
    return q, scale, h, a.bfloat16() if s["c"]["copy"] else None


def _quant(s):
    if own:
        from bit_group_quantized_gb300 import lib

        lib.bgq_f8_quantise(s["x"], out=s["out"])
        return s["q"], s["scale"]
    return _quantise(s["x"].float(), s["c"]["block"])


def _values(q, scale, block=1):
    """The values, in float32, that codes [rows][cols] and their scales stand for."""
    wide = scale.float().repeat_interleave(BLOCK, 1)[:, :q.shape[1]]
    return q.float() * (wide if block == 1 else wide.repeat_interleave(block, 0)[:q.shape[0]])


def _product(s, w):
    return torch.matmul(_values(s["x_q"], s["x_scale"]), _values(s[w + "_q"], s[w + "_scale"], BLOCK).T)


def _gemm(s):
    if own:
        from bit_group_quantized_gb300 import lib

        lib.bgq_f8_gemm(s["w"], s["x"], ws=s["ws"], **{"out_f32" if s["c"]["f32"] else "out": s["y"]})
        return s["y"]
    y = _product(s, "w")
    return y if s["c"]["f32"] else y.bfloat16()


def _gated(s):
    if own:
        from bit_group_quantized_gb300 import lib

        if s["c"]["e4m3"]:
            lib.bgq_f8_swiglu(s["gate"], s["up"], s["x"], h=s["out"], ws=s["ws"])
            return s["q"], s["scale"]
        lib.bgq_f8_swiglu(s["gate"], s["up"], s["x"], out=s["y"], ws=s["ws"])
        return s["y"]
    g = _product(s, "gate")
    h = g / (1 + torch.exp(-g)) * _product(s, "up")
    return _quantise(h) if s["c"]["e4m3"] else h.bfloat16()


# ---------------------------------------------------------------------------------------------------------- exact
def exact(c, seed):
    s = prepare(c, seed)
    return {"norm": _exact_norm, "quant": _exact_quant, "gemm": _exact_gemm, "gated": _exact_gated}[c["op"]](s)


def _exact_codes(x, block):
    """What the codes of x round, and the scales, both as 64-bit numbers."""
    rows, cols = x.shape
    scale = torch.zeros(-(-rows // block), _blocks(cols), dtype=torch.float64, device=x.device)
    for j in range(_blocks(cols)):
        top = x[:, j * BLOCK:(j + 1) * BLOCK].abs().amax(1)
        if block > 1:
            top = torch.stack([t.max() for t in top.split(block)])
        e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -140) / TOP))
        e = torch.where(TOP * torch.exp2(e - 1) >= top, e - 1, torch.where(TOP * torch.exp2(e) < top, e + 1, e))
        scale[:, j] = torch.exp2(e.clamp(min=-127))
    row, column = torch.arange(rows, device=x.device) // block, torch.arange(cols, device=x.device) // BLOCK
    return x / scale[row][:, column], scale


def _exact_norm(s):
    h = s["h"].double() + s["delta"].double()
    a = h * torch.rsqrt(h.square().sum(1) / h.shape[1] + 1e-6)[:, None] * s["rho"].double()
    return (*_exact_codes(a, 1), h, a if s["c"]["copy"] else None)


def _exact_quant(s):
    return _exact_codes(s["x"].double(), s["c"]["block"])


def _exact_values(q, scale, block):
    """Codes and scales by their bits: sign, four bits of exponent, three of fraction."""
    code = torch.arange(256, dtype=torch.float64)
    sign, power, part = torch.where(code < 128, 1.0, -1.0), (code % 128) // 8, code % 8
    value = sign * torch.where(power == 0, part / 8 * 2.0 ** -6, (1 + part / 8) * 2.0 ** (power - 7))
    row, column = torch.arange(q.shape[0], device=q.device) // block, torch.arange(q.shape[1], device=q.device) // BLOCK
    x = value.to(q.device)[q.view(torch.uint8).int()]
    return x * torch.exp2(scale.view(torch.uint8).double() - 127)[row][:, column]


def _exact_product(s, w):
    return _exact_values(s["x_q"], s["x_scale"], 1) @ _exact_values(s[w + "_q"], s[w + "_scale"], BLOCK).T


def _exact_gemm(s):
    return _exact_product(s, "w")


def _exact_gated(s):
    h = torch.nn.functional.silu(_exact_product(s, "gate")) * _exact_product(s, "up")
    return _exact_codes(h, 1) if s["c"]["e4m3"] else h
