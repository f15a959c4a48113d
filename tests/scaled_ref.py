"""Plain 64-bit forms (numpy) of the scored router and of the float8 block-scaled operators, with
bounds on what fp32 arithmetic may differ from them by."""
from __future__ import annotations

import numpy as np

BLOCK = 128


def blocks(n: int) -> int:
    return -(-n // BLOCK)


def _decode_table() -> np.ndarray:
    """The value of each of the 256 e4m3 codes."""
    c = np.arange(256)
    ex, man = (c >> 3) & 15, c & 7
    v = np.where(ex == 0, man * 2.0 ** -9, (8 + man) * 2.0 ** (ex - 10.0))
    v[(c & 127) == 127] = np.nan
    return np.where(c >= 128, -v, v)


E4M3 = _decode_table()
_POS = E4M3[:127]
_MID = (_POS[1:] + _POS[:-1]) / 2


def encode(v: np.ndarray) -> np.ndarray:
    """Codes of the nearest e4m3 values (|v| clamped to 448), halfway cases to the even code."""
    m = np.abs(v)
    lo, hi = np.searchsorted(_MID, m, "left"), np.searchsorted(_MID, m, "right")
    code = np.where((lo != hi) & (lo % 2 == 1), hi, lo)
    return (code + 128 * np.signbit(v)).astype(np.uint8)


def quantize(x: np.ndarray):
    """x [T][K] -> (codes [T][K], scales [blocks][T] fp32): the operator's definition."""
    T, K = x.shape
    x = x.astype(np.float64)
    q = np.zeros((T, K), np.uint8)
    s = np.zeros((blocks(K), T), np.float32)
    for b in range(blocks(K)):
        part = x[:, b * BLOCK:(b + 1) * BLOCK]
        fin = np.isfinite(part).all(1)
        amax = np.where(fin, np.abs(np.where(np.isfinite(part), part, 0)).max(1), 0)
        sc = (amax.astype(np.float32) / np.float32(448)).astype(np.float32)
        s[b] = sc
        ok = sc > 0
        r = np.zeros_like(part)
        r[ok] = part[ok] / sc[ok].astype(np.float64)[:, None]
        q[:, b * BLOCK:(b + 1) * BLOCK] = np.where(ok[:, None], encode(r), 0)
    return q, s


def wide_act(q, s):
    """Codes [T][K] and scales [blocks][T] as float64 values."""
    return E4M3[q] * np.repeat(s.T.astype(np.float64), BLOCK, 1)[:, :q.shape[1]]


def wide_weight(q, s):
    """Codes [N][K] and scales [blocks][blocks] as float64 values."""
    n, k = q.shape
    return E4M3[q] * np.repeat(np.repeat(s.astype(np.float64), BLOCK, 0)[:n], BLOCK, 1)[:, :k]


# fp32 error of a block-scaled product relative to the sum of the magnitudes of its terms: a block
# is four accumulator steps of 32 products, each step rounding or truncating to 24 bits (2^-23,
# taken twice since the products are aligned before they are summed); its two scale roundings
# and its addition are 3 * 2^-24, and the running total rounds once per block.
def product_error(nb: int) -> float:
    return 8 * 2.0 ** -23 + (nb + 3) * 2.0 ** -24


def matmul(a, b):
    """(out, sum of magnitudes) of widened activations [M][K] and weights [N][K]."""
    return a @ b.T, np.abs(a) @ np.abs(b).T


def experts(x, ids, w, gate, W):
    """The experts' layer in 64 bits: x [T][H] (values as the operator reads them), ids, w [T][k],
    gate [T] or None, W: dict of (codes, scales) of gate, up, down, with `shared`.

    Returns (out, tol, half): tol bounds what fp32 arithmetic may change, half what holding every
    y in fp16 times a power of two per 128 columns adds (batches of more than 4 tokens with a
    16-bit output): 2^-11 of |y|, and half of fp16's smallest step times the power, which is
    less than four times what the largest possible sum asks for.  In tol, g and u carry
    product_error; h = silu(g) u inherits them (|silu'| <= 1.1) with a few fp32 roundings; a
    value of h whose quotient lies that close to a rounding boundary may take the neighbouring
    e4m3 value; y and the weighted sum round in fp32."""
    T, H = x.shape
    E = W["gate"][0].shape[0] - int(W["shared"])
    xq = wide_act(*quantize(x))
    out, tol, half = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))
    jobs = [(e, [(t, w[t, j]) for t in range(T) for j in range(ids.shape[1]) if ids[t, j] == e])
            for e in range(E)]
    if W["shared"]:
        jobs.append((E, [(t, 1.0 if gate is None else gate[t]) for t in range(T)]))
    for e, rows in jobs:
        if not rows:
            continue
        t = np.array([r[0] for r in rows])
        c = np.array([r[1] for r in rows], np.float64)[:, None]
        m = {n: wide_weight(W[n][0][e], W[n][1][e]) for n in ("gate", "up", "down")}
        F = m["gate"].shape[0]
        g, ga = matmul(xq[t], m["gate"])
        u, ua = matmul(xq[t], m["up"])
        eps = product_error(blocks(H))
        sig = 1 / (1 + np.exp(-g))
        h = g * sig * u
        dh = 1.1 * np.abs(u) * ga * eps + np.abs(g * sig) * ua * eps + 8 * 2.0 ** -24 * np.abs(h)
        hq, hs = quantize(h)
        hv = wide_act(hq, hs)
        s = np.repeat(hs.T.astype(np.float64), BLOCK, 1)[:, :F]
        ds = np.repeat(np.stack([dh[:, b * BLOCK:(b + 1) * BLOCK].max(1) / 448
                                 for b in range(blocks(F))], 1), BLOCK, 1)[:, :F]
        s1 = np.where(s > 0, s, 1)
        r = np.abs(h) / s1
        dr = dh / s1 + r * ds / s1 + r * 2.0 ** -22
        low, high = E4M3[encode(np.maximum(r - dr, 0))], E4M3[encode(np.minimum(r + dr, 448))]
        dv = np.maximum(high - E4M3[encode(r)], E4M3[encode(r)] - low) * s + np.abs(hv) * (
            ds / s1 + 2.0 ** -23)
        y, ya = matmul(hv, m["down"])
        ty = dv @ np.abs(m["down"]).T + ya * product_error(blocks(F))
        np.add.at(out, t, c * y)
        top = (hs.T.astype(np.float64)[:, None, :] * W["down"][1][e].astype(np.float64)).max(2)
        power = 4 * np.repeat(top, BLOCK, 1)[:, :H] * blocks(F) * 128 * 448.0 ** 2 / 65504
        np.add.at(half, t, np.abs(c) * (np.abs(y) * 2.0 ** -11 + 2.0 ** -25 * power))
        np.add.at(tol, t, np.abs(c) * (ty + np.abs(y) * (ids.shape[1] + 3) * 2.0 ** -24))
    return out, tol, half


def random_weights(rng, n, rows, cols):
    """Codes [n][rows][cols] (no NaN) and scales [n][blocks][blocks]."""
    q = encode(np.clip(rng.standard_normal((n, rows, cols)) * 130, -448, 448))
    s = np.exp(0.5 * rng.standard_normal((n, blocks(rows), blocks(cols)))) / (130 * cols ** 0.5)
    return q, s.astype(np.float32)


def route(l, k, score, n_group, topk_group, group_top, renorm, scale, bias):
    """(ids, w) of logits [T][E] by the rule in 64 bits."""
    T, E = l.shape
    l = l.astype(np.float64)
    if score == "softmax":
        z = np.exp(l - l.max(1, keepdims=True))
        s = z / z.sum(1, keepdims=True)
    else:
        s = 1 / (1 + np.exp(-np.maximum(l, -700)))
        s = np.where(l < -700, 0.0, s)
    v = s if bias is None else s + bias.astype(np.float64)
    by = (l if bias is None else v).copy()
    if n_group > 1:
        per = E // n_group
        part = v.reshape(T, n_group, per) if group_top == 2 else by.reshape(T, n_group, per)
        total = np.sort(part, 2)[:, :, per - group_top:].sum(2)
        keep = np.argsort(-total, 1, kind="stable")[:, :topk_group]
        on = np.zeros((T, n_group), bool)
        np.put_along_axis(on, keep, True, 1)
        by[~np.repeat(on, per, 1)] = -np.inf
    ids = np.argsort(-by, 1, kind="stable")[:, :k]
    w = np.take_along_axis(s, ids, 1)
    if renorm:
        tot = w.sum(1, keepdims=True)
        w = np.where(tot > 0, w / np.where(tot > 0, tot, 1), 0)
    return ids.astype(np.int32), w * scale


def group(ids, E):
    """(counts, offsets, perm, inv_perm) of ids [T][k], stable in token order."""
    flat = ids.ravel()
    perm = np.argsort(flat, kind="stable").astype(np.int32)
    inv = np.empty_like(perm)
    inv[perm] = np.arange(flat.size)
    counts = np.bincount(flat, minlength=E).astype(np.int32)
    return counts, np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), perm, inv
