"""The operators around the top-k from their definitions, in numpy and 64 bits, for the tests."""
import math

import numpy as np


# ------------------------------------------------------------------ gate ---------

def scores(x, scoring):
    x = np.asarray(x, dtype=np.float64)
    if scoring == "sigmoid":
        return 1.0 / (1.0 + np.exp(-x))
    top = x.max(-1, keepdims=True, initial=-np.inf)
    e = np.exp(x - np.where(np.isinf(top), 0.0, top))
    total = e.sum(-1, keepdims=True)
    return e / np.where(total > 0, total, 1.0)


def route_weights(x, chosen, scoring, renormalise, scale):
    w = np.take_along_axis(scores(x, scoring), chosen, -1)
    if renormalise:
        total = w.sum(-1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    return scale * w


def route(x, k, scoring, bias=None, groups=1, topk_groups=1, group_score="max"):
    """(experts, margin): each row's choice, and how near it came to another one (the least
    gap between choice values, or group scores, that a rounding could swap)."""
    x = np.asarray(x, dtype=np.float64)
    s = scores(x, scoring)
    c = x if bias is None else s + np.asarray(bias, dtype=np.float64)
    rows, E = x.shape
    size = E // groups
    experts, margin = np.zeros((rows, k), dtype=np.int64), np.full(rows, np.inf)
    for r in range(rows):
        open_ = np.ones(E, dtype=bool)
        if groups > 1:
            by = (c if group_score == "max" or bias is not None else s)[r].reshape(groups, size)
            top = np.sort(by, -1)[:, ::-1]
            gs = top[:, 0] if group_score == "max" or size == 1 else top[:, 0] + top[:, 1]
            order = np.argsort(-gs, kind="stable")
            if topk_groups < groups:
                margin[r] = gs[order[topk_groups - 1]] - gs[order[topk_groups]]
            open_ = np.isin(np.arange(E) // size, order[:topk_groups])
        at = np.flatnonzero(open_)
        at = at[np.argsort(-c[r][at], kind="stable")]
        experts[r] = at[:k]
        gaps = -np.diff(c[r][at[:k + 1]])
        if gaps.size:
            margin[r] = min(margin[r], gaps.min())
    return experts, margin


def route_gradient(g, x, chosen, scoring, renormalise, scale):
    """sum_j g_j dw_j / dx_e with the choice held: the chain through w = scale s / D."""
    s = scores(x, scoring)
    sc = np.take_along_axis(s, chosen, -1)
    g = np.asarray(g, dtype=np.float64)
    if renormalise:
        D = sc.sum(-1, keepdims=True)
        d = np.where(D > 0, scale * (g / np.where(D > 0, D, 1) - (g * sc).sum(-1, keepdims=True) / np.where(D > 0, D, 1) ** 2), 0)
    else:
        d = scale * g
    full = np.zeros_like(s)
    np.put_along_axis(full, chosen, d, -1)
    if scoring == "sigmoid":
        return full * s * (1 - s)
    return s * (full - (full * s).sum(-1, keepdims=True))


# ------------------------------------------------------------------ verification --

def verify(x, drafts, uniforms, noise, q=None, lens=None, temperature=1.0):
    """(tokens, accepted, probs, margin): margin is the least relative gap of any comparison the
    answer hangs on (u q against p, the race's best against its second)."""
    B, rows, V = x.shape
    S = rows - 1
    t_of = np.broadcast_to(np.asarray(temperature, dtype=np.float64), (B,))
    tokens, probs = np.full((B, rows), -1, dtype=np.int64), np.zeros((B, rows))
    accepted, margin = np.zeros(B, dtype=np.int64), np.full(B, np.inf)
    for b in range(B):
        limit = S if lens is None else min(max(int(lens[b]), 0), S)
        for i in range(rows):
            row = x[b, i].astype(np.float64)
            p = np.zeros(V)
            if np.isneginf(row).all():
                pass
            elif t_of[b] > 0:
                p = scores(row[None] / t_of[b], "softmax")[0]
            else:
                p[int(row.argmax())] = 1.0
            r = p
            if i < limit:
                t = int(drafts[b, i])
                qi = np.zeros(V)
                if q is not None:
                    qi = q[b, i].astype(np.float64)
                elif 0 <= t < V:
                    qi[t] = 1.0
                if 0 <= t < V:
                    uq = float(uniforms[b, i]) * qi[t]
                    margin[b] = min(margin[b], abs(uq - p[t]) / max(uq, p[t], 1e-300))
                    if uq < p[t]:
                        tokens[b, i], probs[b, i] = t, p[t]
                        accepted[b] += 1
                        continue
                r = np.maximum(p - qi, 0)
                r = r if r.max() > 0 else p
            race = r / noise[b].astype(np.float64)
            if race.max() > 0:
                v = int(race.argmax())
                tokens[b, i], probs[b, i] = v, p[v]
                rest = np.delete(race, v)
                if rest.size:
                    margin[b] = min(margin[b], 1 - rest.max() / race[v])
            break
    return tokens, accepted, probs, margin


# ------------------------------------------------------------------ 4-bit cache ---

def bf16(x):
    """fp32 values rounded to bf16 (nearest, ties to even)."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    u = (u + np.uint64(0x7FFF) + ((u >> np.uint64(16)) & np.uint64(1))) & np.uint64(0xFFFF0000)
    return u.astype(np.uint32).view(np.float32)


def quantise(x):
    """Codes, s and m of each row, in the fp32 steps the format is defined by."""
    x = np.asarray(x, dtype=np.float32)
    m = bf16(x.min(-1))
    s = bf16((x.max(-1) - m) * np.float32(1.0 / 15.0))
    tiny = s < np.float32(2.0 ** -126)
    inv = np.where(tiny, np.float32(0), np.float32(1) / np.where(tiny, np.float32(1), s)).astype(np.float32)
    codes = np.clip(np.rint((x - m[..., None]) * inv[..., None]), 0, 15).astype(np.uint8)
    return codes, s, m


def value(codes, s, m):
    return codes.astype(np.float64) * s.astype(np.float64)[..., None] + m.astype(np.float64)[..., None]


def pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def unpack(packed):
    return np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], 2 * packed.shape[-1])


def attention(q, kv, lens, indices=None, scale=None):
    """out and lse in 64 bits.  kv(b, h, positions) gives the key and value rows (64 bits) of
    those positions, and which of them have a page."""
    B, Q, hq, D = q.shape
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    heads = kv.heads
    out, lse = np.zeros((B, Q, hq, D)), np.full((B, Q, hq), -np.inf)
    for b in range(B):
        for i in range(Q):
            end = int(min(max(int(lens[b]), 0), kv.width)) - (Q - 1 - i)
            pos = np.arange(max(end, 0)) if indices is None else indices[b, i].astype(np.int64)
            pos = pos[(pos >= 0) & (pos < end)]
            for h in range(heads):
                k, v, there = kv(b, h, pos)
                k, v = k[there], v[there]
                if not len(k):
                    continue
                for j in range(h * (hq // heads), (h + 1) * (hq // heads)):
                    s = k @ q[b, i, j].astype(np.float64) * scale
                    top = s.max()
                    p = np.exp(s - top)
                    lse[b, i, j] = top + math.log(p.sum())
                    out[b, i, j] = p @ v / p.sum()
    return out, lse
