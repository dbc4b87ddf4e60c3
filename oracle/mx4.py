"""Microscaled 4-bit floating point (the E2M1 / E8M0 block format of the OCP Microscaling
Formats specification 1.0, blocks of 32), its products, the selection of experts and
their FFN, in fp64 from the definitions."""
import numpy as np

GRID = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])          # code & 7; bit 3 is the sign


def mx4_quantize(x):
    """x [..., K] (fp32 or bf16 values) -> codes uint8 [..., K / 2], scale bytes uint8 [..., K / 32]."""
    x = np.asarray(x, dtype=np.float64)
    g = x.reshape(x.shape[:-1] + (-1, 32))
    bad = ~np.isfinite(g).all(-1)
    g = np.where(bad[..., None], 0, g)
    a = np.abs(g).max(-1)
    _, e = np.frexp(a)                                # a = m 2^e, m in [0.5, 1): floor(log2 a) = e - 1
    e = np.where(a > 0, np.maximum(e - 3, -127), -127)
    r = np.abs(np.ldexp(g, -e[..., None].astype(np.int32)))
    # distance to every grid value; of two equally near ones the even code
    d = np.abs(r[..., None] - GRID)
    near = d == d.min(-1, keepdims=True)
    q = np.argmax(near * (1 + (np.arange(8) % 2 == 0)), -1)
    q = np.where(r >= 6, 7, q) + 8 * np.signbit(g)
    q = np.where(bad[..., None], 0, q).reshape(x.shape).astype(np.uint8)
    return q[..., 0::2] | (q[..., 1::2] << 4), np.where(bad, 255, e + 127).astype(np.uint8)


def mx4_values(codes, scale):
    """fp64 values [..., K] of codes and scale bytes."""
    n = np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[:-1] + (-1,))
    v = np.where(n & 8, -GRID[n & 7], GRID[n & 7])
    s = np.where(scale == 255, np.nan, np.ldexp(1.0, scale.astype(np.int32) - 127))
    return v * np.repeat(s, 32, -1)


def moe_select(logits, top_k, score="softmax", bias=None, groups=1, top_groups=1, group_best=1, renormalize=False,
               scale=1.0):
    """(ids int32, weights fp64) [M][top_k], token by token."""
    ids, weights = [], []
    for l in np.asarray(logits, dtype=np.float64):
        E = len(l)
        nan = np.isnan(l).any()
        masked = np.isnan(l) | (l == -np.inf)
        live = np.where(masked, -np.inf, l)
        with np.errstate(invalid="ignore", over="ignore"):
            if score == "sigmoid":
                s = np.where(masked, 0, 1 / (1 + np.exp(-live)))
            elif masked.all():
                s = np.zeros(E)
            else:
                s = np.exp(live - live.max())
                s = s / s.sum()
        c = np.where(masked, -np.inf, s if bias is None else s + np.asarray(bias, dtype=np.float64))
        value = [sum(sorted(c[g * (E // groups):(g + 1) * (E // groups)], reverse=True)[:group_best])
                 for g in range(groups)]
        kept = sorted(range(groups), key=lambda g: (-value[g], g))[:top_groups]
        rank = c if bias is not None else np.where(masked, -np.inf, l)
        order = sorted((e for e in range(E) if e // (E // groups) in kept), key=lambda e: (-rank[e], e))[:top_k]
        w = s[order]
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else np.zeros(top_k)
        ids.append(order)
        weights.append(np.full(top_k, np.nan) if nan else w * scale)
    return np.array(ids, dtype=np.int32).reshape(-1, top_k), np.array(weights).reshape(-1, top_k)


def gated(g, u, act):
    if act == "silu":
        with np.errstate(over="ignore"):
            return g / (1 + np.exp(-g)) * u
    return 0.5 * g * (1 + np.tanh(np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3))) * u


def mx4_moe(gate, up, down, x, ids, weights, act):
    """(y, bound) fp64 [M][D] for fp64 weight stacks, and what y may be off by: sums of K products in fp32 (each of
    at most K additions off by 2^-23 of the sum of magnitudes), h rounded to 16 bits (2^-16) after an
    activation whose slope is under 1.13, off by 2^-18 of itself and 2^-22 |g| (1 + tanh cancels
    for negative g), and y rounded to bf16."""
    M, D = x.shape
    y, b = np.zeros((M, D)), np.zeros((M, D))
    for m in range(M):
        for e, w in zip(ids[m], weights[m]):
            if not 0 <= e < len(gate):
                continue
            F = len(gate[e])
            g, u = gate[e] @ x[m], up[e] @ x[m]
            tg, tu = (D * 2.0 ** -23 * (np.abs(v[e]) @ np.abs(x[m])) for v in (gate, up))
            h = gated(g, u, act)
            a = np.abs(gated(g, np.ones(F), act))
            dh = 1.13 * tg * (np.abs(u) + tu) + a * tu + 2.0 ** -18 * np.abs(h) + 2.0 ** -22 * np.abs(g * u)
            dh = dh + 2.0 ** -16 * (np.abs(h) + dh)
            y[m] += w * (down[e] @ h)
            s = np.abs(down[e])
            b[m] += abs(w) * (s @ dh + (F + len(ids[m]) + 2) * 2.0 ** -23 * (s @ (np.abs(h) + dh)))
    return y, b + 2.0 ** -8 * (np.abs(y) + b)
