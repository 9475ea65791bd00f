"""The attention operators around a 4-bit key/value cache: what they are given, what they compute, and how much work that is.

Three operators, used one after the other between a decoder layer's projections:

* rope: rotary positions with several axes (time, height, width) on the heads of a fused projection;
* cache: new keys and values quantised to 4 bits (a bf16 scale and bias for each 64 columns) as they are written into
  a paged cache, and read back from it as bf16 values;
* attn: attention of grouped query heads over that cache, from one new token a sequence to whole prompts.

`run` computes a case in its plain form (elementary torch operations in 32 bits, 64 for the rotary angles and for the
choice of a code), or with the package's kernels where `own` is true. `exact` computes it from the definitions in 64 bits.
"""

import math

import torch

own = False

GROUP = 64  # columns that share one scale and one bias


# ---------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 64 sequences: the query and key heads of a fused projection, at far positions
        dict(name="rope_step", op="rope", tokens=64, heads=40, extra=8, d=128, rot=128, axes=3, far=1000000, pairs=False, inverse=False),
        # a long prompt with images in it, one axis per time, height and width
        dict(name="rope_prompt", op="rope", tokens=8191, heads=40, extra=8, d=128, rot=128, axes=3, far=40000, pairs=False, inverse=False),
        # a vision tower's two axes on neighbouring columns, the part behind column 64 left as it is; the gradient's direction
        dict(name="rope_image_grad", op="rope", tokens=2304, heads=16, extra=16, d=96, rot=64, axes=2, far=128, pairs=True, inverse=True),
        # one decode step of 64 sequences writes 64 tokens, which are read back
        dict(name="cache_step", op="cache", batch=64, lo=33, hi=16384, q_lo=1, q_hi=1, hkv=8, d=128, page=64, write=True),
        # three prompts of odd lengths written whole, and read back
        dict(name="cache_prompt", op="cache", batch=3, lo=3001, hi=9001, q_lo=3001, q_hi=9001, hkv=8, d=128, page=64, write=True),
        # long sequences read back whole (to move them, or for a kernel that wants bf16)
        dict(name="cache_read", op="cache", batch=5, lo=5000, hi=32000, q_lo=5000, q_hi=32000, hkv=2, d=256, page=16, write=False),
        # the first answers of a chat: one sequence, a short past, where latency counts
        dict(name="attn_short", op="attn", batch=1, lo=513, hi=513, q_lo=1, q_hi=1, hq=32, hkv=8, d=128, page=64, causal=True, window=0, lse=True),
        # one sequence with a long past in one run of memory
        dict(name="attn_long", op="attn", batch=1, lo=131071, hi=131071, q_lo=1, q_hi=1, hq=32, hkv=8, d=128, page=0, causal=True, window=0, lse=True),
        # a served batch of ragged lengths, one new token each
        dict(name="attn_batch", op="attn", batch=64, lo=512, hi=16384, q_lo=1, q_hi=1, hq=32, hkv=8, d=128, page=64, causal=True, window=0, lse=False),
        # drafted tokens verified: five rows a sequence, few wide key heads
        dict(name="attn_verify", op="attn", batch=24, lo=700, hi=9000, q_lo=5, q_hi=5, hq=16, hkv=2, d=256, page=16, causal=True, window=0, lse=True),
        # a prompt from its first token
        dict(name="attn_prompt", op="attn", batch=1, lo=4096, hi=4096, q_lo=4096, q_hi=4096, hq=32, hkv=8, d=128, page=64, causal=True, window=0, lse=False),
        # chunks of three prompts behind longer pasts
        dict(name="attn_chunk", op="attn", batch=3, lo=5000, hi=16000, q_lo=700, q_hi=1100, hq=32, hkv=4, d=128, page=64, causal=True, window=0, lse=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "cache", "attn", "attn"])
    if op == "rope":
        d = rng.choice([64, 96, 128, 256])
        rot = rng.choice([d, d, d // 2])
        return dict(op="rope", tokens=_log(rng, 1, 5000), heads=rng.randint(1, 40), extra=rng.randint(0, 8), d=d, rot=rot,
                    axes=rng.choice([1, 2, 3]), far=_log(rng, 100, 1000000), pairs=rng.random() < 0.4, inverse=rng.random() < 0.3)
    d = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    page = rng.choice([0, 16, 32, 64, 128])
    if op == "cache":
        most = max(2, 16000 * 8 * 128 // (hkv * d))
        batch = _log(rng, 1, 64)
        hi = _log(rng, 1, max(2, min(32000, most // batch)))
        write = rng.random() < 0.6
        q = rng.choice([1, hi])
        return dict(op="cache", batch=batch, lo=max(q, hi // 3) if q == 1 else max(1, hi // 3), hi=hi, q_lo=1 if q == 1 else max(1, hi // 3),
                    q_hi=q, hkv=hkv, d=d, page=page, write=write)
    hq = hkv * rng.choice([1, 2, 3, 4, 8])
    kind = rng.choice(["step", "verify", "prompt"])
    if kind == "prompt":
        batch = rng.randint(1, 3)
        q_hi = _log(rng, 20, 1500)
        hi = max(q_hi, _log(rng, 20, min(8000, 300_000_000_000 // (4 * batch * q_hi * hq * d))))
        q_lo = max(1, q_hi // 2)
        lo = max(q_hi, hi // 2)
    else:
        batch = _log(rng, 1, 64)
        q_lo = q_hi = 1 if kind == "step" else rng.randint(2, 8)
        hi = max(q_hi, _log(rng, 1, 500000 // batch if batch > 4 else 60000))
        hi = min(hi, 60000)
        lo = max(q_hi, hi // 8)
    return dict(op="attn", batch=batch, lo=lo, hi=hi, q_lo=q_lo, q_hi=q_hi, hq=hq, hkv=hkv, d=d, page=page,
                causal=rng.random() < 0.85, window=rng.choice([0, 0, 0, _log(rng, 16, 4096)]), lse=kind != "prompt")


def _spread(lo, hi, n, turn):
    """n lengths between lo and hi, spread evenly over the logarithm, in mixed order: the same for every seed."""
    if n == 1 or lo == hi:
        return [hi] * n
    return [int(round(lo * (hi / lo) ** ((turn + b * 0.6180339887) % 1.0))) for b in range(n)]


def _lengths(c):
    """Tokens in the cache (the new ones among them) and new tokens, for each sequence."""
    kv = _spread(c["lo"], c["hi"], c["batch"], 0.5)
    if c["q_lo"] == c["lo"] and c["q_hi"] == c["hi"]:
        return kv, list(kv)
    return kv, [min(a, b) for a, b in zip(_spread(c["q_lo"], c["q_hi"], c["batch"], 0.25), kv)]


def _sections(c):
    """Rotary pairs of each axis."""
    half, n = c["rot"] // 2, c["axes"]
    rest = [half // n] * n
    rest[0] += half - sum(rest)
    return rest


def work(c):
    if c["op"] == "rope":
        values = c["tokens"] * c["heads"] * c["d"]
        return {"bytes": 4 * values + 4 * c["axes"] * c["tokens"], "flops": 3 * values}
    kv, new = _lengths(c)
    row = c["hkv"] * (c["d"] // 2 + c["d"] // GROUP * 4)  # bytes of one token's keys, or values, in the cache
    if c["op"] == "cache":
        bf16 = sum(new) * c["hkv"] * c["d"] * 2 * 2
        held = sum(new) * row * 2
        return {"bytes": (2 * bf16 if c["write"] else bf16) + held, "flops": 2 * sum(new) * c["hkv"] * c["d"] * (4 if c["write"] else 1)}
    pairs = seen = 0
    for n, m in zip(kv, new):
        first = n
        for j in range(m):
            last = n - m + j + 1 if c["causal"] else n
            begin = max(0, n - m + j + 1 - c["window"]) if c["window"] else 0
            pairs += max(0, last - begin)
            first = min(first, begin)
        seen += n - first
    return {"bytes": 2 * seen * row + 4 * sum(new) * c["hq"] * c["d"] + (4 * sum(new) * c["hq"] if c["lse"] else 0), "flops": 4 * pairs * c["hq"] * c["d"]}


# --------------------------------------------------------------------------------------------------------- inputs
def _quantise(x):
    """Codes [.., d] (as numbers) and (scale, bias) bf16 [.., d/64, 2] of x [.., d]: scale = bf16((max-min)/15),
    bias = bf16(min), code = the nearest whole number to (x-bias)/scale, halves up, within 0..15."""
    g = x.float().unflatten(-1, (-1, GROUP))
    low, high = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    scale, bias = ((high - low) / 15).bfloat16(), low.bfloat16()
    code = torch.floor((g.double() - bias.double()) / scale.double() + 0.5).clamp(0, 15)
    code = torch.where(scale == 0, torch.zeros_like(code), code)
    return code.flatten(-2), torch.cat([scale, bias], -1)


def _pack(code):
    """Codes [.., d] into int32 words [.., d/8], eight to a word, the first in the lowest bits."""
    w = code.to(torch.int64).unflatten(-1, (-1, 8))
    w = (w << torch.arange(0, 32, 4, device=w.device)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def _unpack(q):
    """int32 words [.., d/8] as codes [.., d] in float32."""
    return ((q.unsqueeze(-1) >> torch.arange(0, 32, 4, device=q.device, dtype=torch.int32)) & 15).flatten(-2).float()


def _filled(rng, pages, heads, size, d, dev, spread):
    """Packed codes and scale/bias rows of a cache full of normal values whose columns differ in size as a key's do."""
    q = torch.empty(pages, heads, size, d // 8, dtype=torch.int32, device=dev)
    sb = torch.empty(pages, heads, size, d // GROUP, 2, dtype=torch.bfloat16, device=dev)
    col = torch.exp(spread * torch.randn(heads, 1, d, generator=rng, device=dev))
    step = max(1, (1 << 25) // (heads * size * d))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        code, s = _quantise((torch.randn(n, heads, size, d, generator=rng, device=dev) * col).bfloat16())
        q[p:p + n], sb[p:p + n] = _pack(code), s
    return q, sb


def prepare(c, seed):
    dev = torch.device("cuda")
    rng = torch.Generator(device=dev).manual_seed(seed)
    s = dict(c=c)
    if c["op"] == "rope":
        wide = torch.randn(c["tokens"], c["heads"] + c["extra"], c["d"], generator=rng, device=dev).bfloat16()
        s["x"] = wide[:, :c["heads"]]  # the heads to turn stand in front of others in each token's row
        s["pos"] = torch.randint(0, c["far"], (c["axes"], c["tokens"]), generator=rng, device=dev, dtype=torch.int32)
        s["y"] = torch.empty(c["tokens"], c["heads"], c["d"], dtype=torch.bfloat16, device=dev)
    else:
        kv, new = _lengths(c)
        size = c["page"] or (max(kv) + 15) // 16 * 16
        need = [(n + size - 1) // size for n in kv]
        pool = sum(need) + (3 if c["page"] else 0)
        s["k_q"], s["k_sb"] = _filled(rng, pool, c["hkv"], size, c["d"], dev, 0.4)
        s["v_q"], s["v_sb"] = _filled(rng, pool, c["hkv"], size, c["d"], dev, 0.1)
        s["pages"] = None
        if c["page"]:  # the pages of a sequence lie anywhere in the pool
            at = torch.randperm(pool, generator=rng, device=dev)[:sum(need)].to(torch.int32)
            held = torch.arange(max(need), device=dev) < torch.tensor(need, device=dev).unsqueeze(1)
            s["pages"] = torch.full((c["batch"], max(need)), -1, dtype=torch.int32, device=dev).masked_scatter_(held, at)
        s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=dev)
        s["q_start"] = torch.tensor([sum(new[:b]) for b in range(c["batch"] + 1)], dtype=torch.int32, device=dev)
        s["rows"], s["max_q"], s["max_kv"] = sum(new), max(new), max(kv)
        if c["op"] == "cache":
            s["k"], s["v"] = (torch.randn(s["rows"], c["hkv"], c["d"], generator=rng, device=dev).bfloat16() for _ in range(2))
            s["k_out"], s["v_out"] = torch.empty_like(s["k"]), torch.empty_like(s["v"])
        else:
            s["q"] = (1.5 * torch.randn(s["rows"], c["hq"], c["d"], generator=rng, device=dev)).bfloat16()
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(s["rows"], c["hq"], dtype=torch.float32, device=dev) if c["lse"] else None
    if own:
        _handles(s)
    return s


def _handles(s):
    """The argument structs and the workspace that a serving program keeps from call to call."""
    from bit_group_quantized_gb300 import lib

    c = s["c"]
    if c["op"] == "rope":
        s["plan"] = lib.RopePlan(c["d"], c["rot"], 10000.0, _sections(c), pairs=c["pairs"])
        return
    s["cache"] = lib.KV4Cache(s["k_q"], s["k_sb"], s["v_q"], s["v_sb"])
    s["seqs"] = lib.KV4Seqs(s["kv_len"], rows=s["rows"], pages=s["pages"], q_start=s["q_start"], max_q=s["max_q"])
    if c["op"] == "attn":
        s["ws"] = lib.workspace(lib.kv4_attention_workspace_bytes(s["cache"], s["seqs"], c["hq"]), s["q"].device)


# ------------------------------------------------------------------------------------------------------------ run
def run(s):
    return {"rope": _rope, "cache": _cache, "attn": _attn}[s["c"]["op"]](s)


def _rope(s):
    c = s["c"]
    if own:
        from bit_group_quantized_gb300 import lib

        return lib.bgq_rope(s["plan"], s["x"], s["pos"], y=s["y"], inverse=c["inverse"])
    half = c["rot"] // 2
    axis = torch.repeat_interleave(torch.arange(c["axes"], device=s["x"].device), torch.tensor(_sections(c), device=s["x"].device))
    turn = 10000.0 ** (-torch.arange(half, device=s["x"].device, dtype=torch.float64) / half)
    angle = s["pos"].double()[axis].T * turn  # [tokens][half]
    cos, sin = torch.cos(angle).float().unsqueeze(1), torch.sin(angle).float().unsqueeze(1)
    if c["inverse"]:
        sin = -sin
    x = s["x"].float()
    a, b = (x[..., 0:c["rot"]:2], x[..., 1:c["rot"]:2]) if c["pairs"] else (x[..., :half], x[..., half:c["rot"]])
    a, b = a * cos - b * sin, a * sin + b * cos
    front = torch.stack([a, b], -1).flatten(-2) if c["pairs"] else torch.cat([a, b], -1)
    return torch.cat([front, x[..., c["rot"]:]], -1).bfloat16()


def _places(s, longest):
    """Page and place within the page of tokens 0..longest-1 of every sequence (page 0 where there is none), [batch][longest]."""
    t = torch.arange(longest, device=s["kv_len"].device)
    size = s["k_q"].shape[2]
    if s["pages"] is None:
        page = torch.arange(len(s["kv_len"]), device=t.device).unsqueeze(1).expand(-1, longest)
    else:
        page = s["pages"][:, torch.clamp(t // size, max=s["pages"].shape[1] - 1)].long().clamp(min=0)
    return page, (t % size).unsqueeze(0).expand(len(s["kv_len"]), -1)


def _row_places(s):
    """Page and place within the page of the token of every row."""
    row = torch.arange(s["rows"], device=s["kv_len"].device)
    b = torch.searchsorted(s["q_start"][1:].long(), row, right=True)
    t = s["kv_len"].long()[b] - s["q_start"].long()[b + 1] + row
    size = s["k_q"].shape[2]
    page = b if s["pages"] is None else s["pages"].long()[b, t // size]
    return page, t % size


def _values(q, sb, page, place):
    """The values, in float32, of the tokens at these pages and places: [.., heads, d]."""
    code, pair = _unpack(q[page, :, place]), sb[page, :, place].float()
    return (code.unflatten(-1, (-1, GROUP)) * pair[..., 0:1] + pair[..., 1:2]).flatten(-2)


def _cache(s):
    if own:
        from bit_group_quantized_gb300 import lib

        if s["c"]["write"]:
            lib.bgq_kv4_append(s["cache"], s["seqs"], s["k"], s["v"])
        return lib.bgq_kv4_read(s["cache"], s["seqs"], k=s["k_out"], v=s["v_out"])
    page, place = _row_places(s)
    if s["c"]["write"]:
        for x, q, sb in ((s["k"], s["k_q"], s["k_sb"]), (s["v"], s["v_q"], s["v_sb"])):
            code, pair = _quantise(x)
            q[page, :, place], sb[page, :, place] = _pack(code), pair
    return tuple(_values(q, sb, page, place).bfloat16() for q, sb in ((s["k_q"], s["k_sb"]), (s["v_q"], s["v_sb"])))


def _attn(s):
    c = s["c"]
    if own:
        from bit_group_quantized_gb300 import lib

        lib.bgq_kv4_attention(s["cache"], s["seqs"], s["q"], causal=c["causal"], window=c["window"], out=s["out"], lse=s["lse"], ws=s["ws"])
        return (s["out"], s["lse"]) if c["lse"] else s["out"]
    dev, n, m = s["q"].device, s["max_kv"], s["max_q"]
    batch, hkv, group, d = c["batch"], c["hkv"], c["hq"] // c["hkv"], c["d"]
    page, place = _places(s, n)
    start, kv_len = s["q_start"].long(), s["kv_len"].long()
    new = start[1:] - start[:-1]
    # the rows as a padded batch [batch][hkv][m*group][d]
    j = torch.arange(m, device=dev)
    row = torch.clamp(start[:-1].unsqueeze(1) + j, max=s["rows"] - 1)
    q = s["q"].float()[row].unflatten(2, (hkv, group)).permute(0, 2, 1, 3, 4).reshape(batch, hkv, m * group, d)
    at = (kv_len - new).unsqueeze(1) + j  # a row's own position
    t = torch.arange(n, device=dev)
    seen = t < kv_len.view(-1, 1, 1)
    if c["causal"]:
        seen = seen & (t <= at.unsqueeze(2))
    if c["window"]:
        seen = seen & (t > at.unsqueeze(2) - c["window"])
    seen = (seen & (j < new.unsqueeze(1)).unsqueeze(2)).repeat_interleave(group, 1).unsqueeze(1)  # [batch][1][m*group][n]
    k = _values(s["k_q"], s["k_sb"], page, place).transpose(1, 2)
    p = torch.matmul(q, k.transpose(2, 3)).mul_(1 / math.sqrt(d)).masked_fill_(~seen, -math.inf)
    del k
    top = p.amax(-1, keepdim=True)
    safe = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = p.sub_(safe).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, _values(s["v_q"], s["v_sb"], page, place).transpose(1, 2))
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (safe + torch.log(total)).squeeze(-1)
    # back to rows
    b = torch.searchsorted(start[1:], torch.arange(s["rows"], device=dev), right=True)
    i = torch.arange(s["rows"], device=dev) - start[b]
    out = o.view(batch, hkv, m, group, d).permute(0, 2, 1, 3, 4)[b, i].reshape(s["rows"], c["hq"], d).bfloat16()
    if not c["lse"]:
        return out
    return out, lse.view(batch, hkv, m, group).permute(0, 2, 1, 3)[b, i].reshape(s["rows"], c["hq"])


# ---------------------------------------------------------------------------------------------------------- exact
def exact(c, seed):
    s = prepare(c, seed)
    return {"rope": _exact_rope, "cache": _exact_cache, "attn": _exact_attn}[c["op"]](s)


def _exact_rope(s):
    c = s["c"]
    x, y, first = s["x"].double(), s["x"].double().clone(), 0
    for axis, count in enumerate(_sections(c)):
        for i in range(first, first + count):
            angle = s["pos"][axis].double() * math.pow(10000.0, -2.0 * i / c["rot"])
            z = torch.polar(torch.ones_like(angle), -angle if c["inverse"] else angle).unsqueeze(1)
            lo, hi = (2 * i, 2 * i + 1) if c["pairs"] else (i, i + c["rot"] // 2)
            turned = torch.complex(x[..., lo], x[..., hi]) * z
            y[..., lo], y[..., hi] = turned.real, turned.imag
        first += count
    return y


def _exact_token(q, sb):
    """The values that packed rows [.., d/8] with pairs [.., d/64, 2] stand for, in 64 bits."""
    word = q.long() & 0xFFFFFFFF
    code = torch.stack([(word // 16 ** i) % 16 for i in range(8)], -1).flatten(-2).double()
    return code * sb[..., 0].double().repeat_interleave(GROUP, -1) + sb[..., 1].double().repeat_interleave(GROUP, -1)


def _exact_cache(s):
    outs = []
    for name in ("k", "v"):
        if s["c"]["write"]:
            g = s[name].double().unflatten(-1, (-1, GROUP))
            bias = g.min(-1, keepdim=True).values
            scale = ((g.max(-1, keepdim=True).values - bias) / 15).bfloat16().double()
            steps = (g - bias) / torch.where(scale > 0, scale, torch.ones_like(scale))
            code = torch.where(scale > 0, torch.ceil(steps - 0.5) + (torch.ceil(steps - 0.5) == steps - 0.5), torch.zeros_like(g))
            outs.append((code.clamp(0, 15) * scale + bias).flatten(-2))
            continue
        page, place = _row_places(s)
        outs.append(_exact_token(s[name + "_q"][page, :, place], s[name + "_sb"][page, :, place]))
    return tuple(outs)


def _exact_attn(s):
    c = s["c"]
    kv, new = _lengths(c)
    size, group, first, outs, lses = s["k_q"].shape[2], c["hq"] // c["hkv"], 0, [], []
    for b, (n, m) in enumerate(zip(kv, new)):
        t = torch.arange(n, device=s["q"].device)
        page = torch.full_like(t, b) if s["pages"] is None else s["pages"][b].long()[t // size]
        at = torch.arange(n - m, n, device=t.device).unsqueeze(1)
        hidden = (t > at) if c["causal"] else torch.zeros(m, n, dtype=torch.bool, device=t.device)
        if c["window"]:
            hidden = hidden | (t <= at - c["window"])
        heads, logs = [], []
        for h in range(c["hkv"]):
            k = _exact_token(s["k_q"][page, h, t % size], s["k_sb"][page, h, t % size])
            v = _exact_token(s["v_q"][page, h, t % size], s["v_sb"][page, h, t % size])
            for g in range(group):
                x = s["q"][first:first + m, h * group + g].double() @ k.T / math.sqrt(c["d"])
                x = torch.where(hidden, torch.full_like(x, -math.inf), x)
                log = torch.logsumexp(x, -1, keepdim=True)
                heads.append(torch.exp(x - torch.where(log == -math.inf, torch.zeros_like(log), log)) @ v)
                logs.append(log[:, 0])
        outs.append(torch.stack(heads, 1))
        lses.append(torch.stack(logs, 1))
        first += m
    out = torch.cat(outs)
    return (out, torch.cat(lses)) if c["lse"] else out
