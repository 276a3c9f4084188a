"""Plain 64-bit statements of the serving operators for their tests: numpy,
one element, row or page at a time, written from the definitions."""
from __future__ import annotations

import math

import numpy as np
import torch

INF = 2 ** 31 - 1


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().to("cpu").double().numpy()


def rotate(x, pos, theta, rot, layout, scale=None, scale_all=1.0, amp=1.0, inverse=False):
    """x [..., H, d] float64, pos [...]: (y, bound): the rotation and, per
    element, amp (|x0| + |x1|) of its pair (0 where the dim passes through)."""
    n = rot // 2
    y, mag = x.copy(), np.zeros_like(x)
    for c in range(n):
        f = theta ** (-2.0 * c / rot) * (1.0 if scale is None else scale[c]) * scale_all
        ang = pos.astype(np.float64) * f * (-1.0 if inverse else 1.0)
        co, si = np.cos(ang)[..., None], np.sin(ang)[..., None]
        split, pair = (c, n + c), (2 * c, 2 * c + 1)
        src = pair if layout == 0 or (layout == 2 and inverse) else split
        dst = pair if layout == 0 or (layout == 2 and not inverse) else split
        a, b = x[..., src[0]], x[..., src[1]]
        y[..., dst[0]], y[..., dst[1]] = amp * (a * co - b * si), amp * (a * si + b * co)
        mag[..., dst[0]] = mag[..., dst[1]] = abs(amp) * (np.abs(a) + np.abs(b))
    return y, mag


def assert_rotation(got: torch.Tensor, ref, mag, tag=""):
    """The angle, reduced in fp64, is rounded to fp32 (|r| <= pi: 2^-23 abs);
    sincosf is within 2^-22 of it; amplitude times cos or sin rounds twice and
    the two products and their sum three times (2^-24 relative each): together
    below 2^-20 (|x0| + |x1|) amp. Then one rounding to bf16, 2^-8 relative."""
    g = f64(got).reshape(ref.shape)
    d = 2.0 ** -20 * mag
    tol = 2.0 ** -8 * (np.abs(ref) + d) + d
    assert np.isfinite(g).all(), tag
    bad = np.abs(g - ref) > tol
    assert not bad.any(), f"{tag}: {bad.sum()} off, first at {np.argwhere(bad)[0].tolist()}"


def chains(parents, n):
    """Per node: itself and its ancestors."""
    out = []
    for t in range(n):
        out.append([t] + (out[parents[t]] if parents[t] >= 0 else []))
    return out


def tree(q, keys, vals, lens, nodes, parents, cut, scale=None):
    """q [B,T,Hq,d] float64; keys, vals: per sequence [Hkv, len + nodes, d].
    Returns O, LSE, and two arrays that a tolerance needs: A [B,T,Hq,d] =
    softmax-weighted |v|, and E [B,Hq,T] = the largest sum |q||k| scale of the row."""
    B, T, Hq, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    O, A = np.zeros_like(q), np.zeros_like(q)
    lse, E = np.full((B, Hq, T), -np.inf), np.zeros((B, Hq, T))
    for b in range(B):
        ch = chains(parents[b], nodes[b])
        L = lens[b]
        for t in range(nodes[b]):
            at = L + len(ch[t]) - 1
            slot = np.array(list(range(L)) + [L + u for u in ch[t]])
            where = np.array(list(range(L)) + [L + len(ch[u]) - 1 for u in ch[t]])
            dist = at - where
            for h in range(Hq):
                hk = h // (Hq // keys[b].shape[0])
                k, v = keys[b][hk][slot], vals[b][hk][slot]
                s = np.zeros(len(slot))
                for g in range(d // 16):
                    w = INF if cut is None else cut[g]
                    part = k[:, 16 * g:16 * g + 16] @ q[b, t, h, 16 * g:16 * g + 16]
                    s += np.where(dist <= w, part, 0.0)
                s *= scale
                E[b, h, t] = scale * (np.abs(np.nan_to_num(k)) @ np.abs(q[b, t, h])).max()
                m = s.max()
                p = np.exp(s - m)
                O[b, t, h] = p @ v / p.sum()
                A[b, t, h] = p @ np.abs(v) / p.sum()
                lse[b, h, t] = m + math.log(p.sum())
    return O, lse, A, E


def assert_tree(o, lse, ref, tag=""):
    """Tolerance. The products of bf16 values are exact in fp32; each logit
    sums d <= 128 of them in fp32, off by at most (d + 8) 2^-24 sum|q||k| scale
    =: s (the scale's own rounding and the exponent's included), E holds the
    row's largest. The softmax weights are then off by a factor e^(2s), the
    exponential itself by 2^-20, and P rounds to bf16 (2^-8): O moves by at
    most (2^-8 + 2 s' + 2^-19) A, A = sum p|v| / sum p, plus its own rounding
    2^-8 |O|. The LSE moves by s + 2^-19, and rounds (2^-23 |lse|)."""
    O, L, A, E = ref
    g, gl = f64(o), f64(lse)
    s = (128 + 8) * 2.0 ** -24 * E + 2.0 ** -22 * np.abs(np.where(np.isfinite(L), L, 0.0))
    sb = np.transpose(s, (0, 2, 1))[..., None]
    w = 2.0 ** -8 + 2.1 * sb + 2.0 ** -19
    tol = w * A + 2.0 ** -8 * (np.abs(O) + w * A)
    assert np.isfinite(g).all(), f"{tag}: non-finite O"
    bad = np.abs(g - O) > tol
    assert not bad.any(), f"{tag}: O {bad.sum()} off, first at {np.argwhere(bad)[0].tolist()}, worst " \
                          f"{(np.abs(g - O) - tol).max():.3e}"
    none = np.isneginf(L)
    assert np.array_equal(none, np.isneginf(gl)), f"{tag}: empty rows"
    with np.errstate(invalid="ignore"):
        badl = np.abs(gl - L) > s + 2.0 ** -19 + 2.0 ** -22 * np.abs(L)
    assert not (badl & ~none).any(), f"{tag}: LSE off at {np.argwhere(badl & ~none)[0].tolist()}"


def pages_update(refs, table, lens, parent, keep, new, P):
    """The transaction on lists; returns (refs, table, lens, copies, info)."""
    B, MP = len(table), len(table[0])
    pool = len(refs)
    up = lambda x: -(-x // P)  # noqa: E731
    same = lambda code, taken=0, free=0: (list(refs), [list(r) for r in table], list(lens), [[-1, -1, 0]] * B,  # noqa: E731
                                          [code, taken, free, 0])
    if any(r < 0 for r in refs):
        return same(2)
    for b in range(B):
        if not (0 <= lens[b] <= MP * P and 0 <= keep[b] <= new[b] <= MP * P):
            return same(2)
        if keep[b] > 0 and not (0 <= parent[b] < B and keep[b] <= lens[parent[b]]):
            return same(2)
        if any(not 0 <= p < pool for p in table[b][:up(lens[b])]):
            return same(2)
    r = list(refs)
    for b in range(B):
        for p in table[b][:up(lens[b])]:
            r[p] -= 1
    if any(x < 0 for x in r):  # a page with more holders among the rows than its count says
        return same(2)
    rows = [list(table[parent[b]][:up(keep[b])]) if keep[b] else [] for b in range(B)]
    for row in rows:
        for p in row:
            r[p] += 1
    writers = {}
    for b in range(B):
        if new[b] > keep[b] and keep[b] % P:
            writers.setdefault(rows[b][-1], []).append(b)
    copying = set()
    for p, who in writers.items():
        if r[p] > 1:
            copying.update(who[1:] if len(who) == r[p] else who)
    need = sum(up(new[b]) - up(keep[b]) + (b in copying) for b in range(B))
    free = [p for p in range(pool) if r[p] == 0]
    if need > len(free):
        return same(1, need, len(free))
    at, copies = 0, []
    for b in range(B):
        if b in copying:
            src = rows[b].pop()
            r[src] -= 1
            copies.append([src, free[at], keep[b] % P])
        else:
            copies.append([-1, -1, 0])
        while len(rows[b]) < up(new[b]):
            rows[b].append(free[at])
            r[free[at]] = 1
            at += 1
    return r, [row + [-1] * (MP - len(row)) for row in rows], list(new), copies, [0, need, len(free), len(copying)]
