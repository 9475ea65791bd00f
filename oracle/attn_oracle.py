"""fp64 CPU oracle for the attention operators: rotary positions, the 4-bit cache, attention over it.

TEST INFRASTRUCTURE ONLY, like ``bgq_oracle``: the plain definitions in float64 with numpy, sharing no code with the
library. Cache arrays are the packed words and bf16 bit patterns as stored.
"""

from __future__ import annotations

import numpy as np

from oracle.bgq_oracle import bf16_to_f64, f64_to_bf16_bits

GROUP = 64


def rope_axes(half: int, sections, cycle: bool = False) -> list[int]:
    """Axis of every pair."""
    if cycle:
        return [i % len(sections) if i // len(sections) < sections[i % len(sections)] else 0 for i in range(half)]
    return [a for a, n in enumerate(sections) for _ in range(n)]


def rope(x, pos, rot: int, theta: float, sections, pairs=False, cycle=False, restart=False, inverse=False) -> np.ndarray:
    """x [tokens][heads][d], pos int [n_axes][tokens]."""
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    half = rot // 2
    axis = rope_axes(half, sections, cycle)
    start = np.cumsum([0] + list(sections))
    for i in range(half):
        sec = rope_axes(half, sections)[i]  # frequencies restart with the sections, which CYCLE does not have
        f = theta ** (-(i - start[sec]) / sections[sec]) if restart else theta ** (-2.0 * i / rot)
        # reduced modulo a turn in extended precision: positions reach 2^31
        t = np.asarray(pos[axis[i]]).astype(np.longdouble) * np.longdouble(f)
        t = np.float64(np.remainder(t, 2 * np.longdouble("3.14159265358979323846264338327950288")))[:, None]
        if inverse:
            t = -t
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + half)
        y[..., a] = x[..., a] * np.cos(t) - x[..., b] * np.sin(t)
        y[..., b] = x[..., a] * np.sin(t) + x[..., b] * np.cos(t)
    return y


def kv4_quantise(x):
    """x [.., d] (finite, exact bf16 values) -> codes int [.., d], scale and bias (bf16 values) [.., d/64], and how far
    (x - bias)/scale is from the nearest half (the codes next to one may go either way in fp32)."""
    g = np.asarray(x, dtype=np.float64).reshape(*x.shape[:-1], -1, GROUP)
    low, high = g.min(-1), g.max(-1)
    scale = bf16_to_f64(f64_to_bf16_bits((high - low) / 15.0))
    scale = np.where(scale < 2.0 ** -126, 0.0, scale)
    steps = (g - low[..., None]) / np.where(scale > 0, scale, 1.0)[..., None]
    code = np.where(scale[..., None] > 0, np.clip(np.floor(steps + 0.5), 0, 15), 0).astype(np.int64)
    edge = np.abs(steps - np.floor(steps) - 0.5)
    return code.reshape(x.shape), scale, low, np.where(edge == 0, 1.0, edge).reshape(x.shape)


def kv4_pack(code) -> np.ndarray:
    w = np.asarray(code, dtype=np.uint32).reshape(*code.shape[:-1], -1, 8)
    return np.bitwise_or.reduce(w << (4 * np.arange(8, dtype=np.uint32)), axis=-1)


def kv4_unpack(q) -> np.ndarray:
    q = np.asarray(q).view(np.uint32)
    return ((q[..., None] >> (4 * np.arange(8, dtype=np.uint32))) & 15).reshape(*q.shape[:-1], q.shape[-1] * 8).astype(np.float64)


def kv4_values(q, sb_bits) -> np.ndarray:
    """Packed rows [.., d/8] with pairs [.., d/64, 2] -> values [.., d]."""
    s = bf16_to_f64(sb_bits)
    return kv4_unpack(q) * np.repeat(s[..., 0], GROUP, -1) + np.repeat(s[..., 1], GROUP, -1)


def slot(t: int, b: int, pages, page_size: int, n_pages: int):
    """(page, place) of token t of sequence b, None if absent."""
    p, at = t // page_size, t % page_size
    if t < 0 or p >= (1 if pages is None else pages.shape[1]):
        return None
    page = b if pages is None else int(pages[b, p])
    return (page, at) if 0 <= page < n_pages else None


def kv4_attention(cache, kv_len, q_start, rows, pages, q, scale, causal=True, window=0):
    """cache: (k_q, k_sb bits, v_q, v_sb bits) as [n_pages][heads][page_size][..]; q [rows][q_heads][d] float64.
    Returns out and lse (NaN in rows of no sequence), and for error bounds sum p (|v| + 8 s), s the scale of v's group,
    and max_t scale * sum |q k|."""
    k_q, k_sb, v_q, v_sb = cache
    n_pages, hkv, size = k_q.shape[:3]
    hq, d = q.shape[1:]
    out, size_v = np.full((rows, hq, d), np.nan), np.zeros((rows, hq, d))
    lse, size_s = np.full((rows, hq), np.nan), np.zeros((rows, hq))
    for b, n in enumerate(int(v) for v in kv_len):
        first, m = int(q_start[b]), int(q_start[b + 1] - q_start[b])
        n = max(n, 0)
        at = [(t, slot(t, b, pages, size, n_pages)) for t in range(n)]
        tok = np.array([t for t, s in at if s is not None], dtype=np.int64)
        page = np.array([s[0] for _, s in at if s is not None], dtype=np.int64)
        place = np.array([s[1] for _, s in at if s is not None], dtype=np.int64)
        pos = n - m + np.arange(m)
        seen = np.ones((m, len(tok)), dtype=bool)
        if causal:
            seen &= tok[None] <= pos[:, None]
        if window > 0:
            seen &= tok[None] > pos[:, None] - window
        for h in range(hkv):
            vs = np.repeat(np.abs(bf16_to_f64(v_sb[page, h, place])[..., 0]), GROUP, -1)
            K, V = kv4_values(k_q[page, h, place], k_sb[page, h, place]), kv4_values(v_q[page, h, place], v_sb[page, h, place])
            for g in range(h * hq // hkv, (h + 1) * hq // hkv):
                for j in range(m):  # row by row: what a row may not see never enters its sums
                    see = seen[j]
                    if not see.any():
                        out[first + j, g], lse[first + j, g] = 0.0, -np.inf
                        continue
                    qj = q[first + j, g]
                    s = K[see] @ qj * scale
                    top = s.max()
                    e = np.exp(s - top)
                    lse[first + j, g] = top + np.log(e.sum())
                    out[first + j, g] = (e / e.sum()) @ V[see]
                    size_v[first + j, g] = (e / e.sum()) @ (np.abs(V[see]) + 8 * vs[see])
                    size_s[first + j, g] = (np.abs(K[see]) @ np.abs(qj)).max() * abs(scale)
    return out, lse, size_v, size_s
