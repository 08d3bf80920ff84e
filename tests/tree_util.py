"""A speculative step from drafted trees in numpy and 64 bits, from its definitions
(include/photon_paged.h): which nodes see which, attention of a tree over a paged
cache, verification, and where accepted rows move to."""
from __future__ import annotations

import numpy as np

import int4_util as I


def random_parents(rng, n, kind="tree"):
    """parents of one tree: a chain, a random tree below node 0, or several roots."""
    if kind == "chain":
        return np.arange(-1, n - 1, dtype=np.int32)
    low = -1 if kind == "forest" else 0
    return np.array([-1] + [rng.integers(low, i) for i in range(1, n)], dtype=np.int32)[:n]


def sees(parents):
    """[i][j]: node j is node i or an ancestor of it."""
    n = len(parents)
    m = np.eye(n, dtype=bool)
    for i, up in enumerate(parents):
        if up >= 0:
            m[i] |= m[up]
    return m


def depths(parents):
    return sees(parents).sum(1) - 1


def cached_rows(pool, table, length, dtype):
    """Rows 0 .. length - 1 of a context in 64 bits, [length][hkv][d]."""
    j = np.arange(length)
    return I.to_f64(pool[table[j // 16], :, j % 16], dtype)


def tree_attention(q, k, v, parents, scale, eps, there=None):
    """One sequence: q [n][hq][d], k and v [ctx][hkv][d] in 64 bits -> (out, bound).

    Bound, for finite inputs: with A = log2(e) |scale| sum |q| max |k|, a score is off by
    at most 2^-22 A (fp32 accumulation of head_dim products, the tensor cores keep at least
    22 bits), which the weights' quotient turns into 2 ln 2 2^-22 A of the largest |v|; each
    weight is rounded to the storage type, half a step, eps / 2 of itself, and the
    exponentials, the partials' join and the sums add 2^-18; then one rounding of the
    output, eps / 2 of it (subnormals of fp16: 2^-25)."""
    n, hq, d = q.shape
    ctx, hkv = k.shape[:2]
    see = np.ones((n, ctx), dtype=bool)
    see[:, ctx - n:] = sees(parents)
    if there is not None:
        see &= there
        k, v = np.where(there[:, None, None], k, 0), np.where(there[:, None, None], v, 0)
    out, bound = np.zeros((n, hq, d)), np.zeros((n, hq, 1))
    for h in range(hq):
        kk, vv = k[:, h // (hq // hkv)], v[:, h // (hq // hkv)]
        x = np.where(see, scale * (q[:, h] @ kk.T), -np.inf)
        top = x.max(-1, keepdims=True)
        p = np.exp(x - np.where(np.isfinite(top), top, 0))
        s = p.sum(-1, keepdims=True)
        out[:, h] = (p @ vv) / np.where(s > 0, s, 1)
        mag = 1.4427 * abs(scale) * np.abs(q[:, h]).sum(-1) * np.abs(kk).max()
        bound[:, h, 0] = (2 * np.log(2) * 2.0 ** -22 * mag + eps / 2 + 2.0 ** -18) * np.abs(vv).max()
    return out, bound + eps / 2 * (np.abs(out) + bound) + 2.0 ** -25


def probabilities(x):
    """Entries as photon_verify_tree takes them."""
    return np.clip(np.nan_to_num(np.asarray(x, dtype=np.float64), nan=0.0, posinf=1.0), 0, 1)


def verify(p, q, tokens, parents, accept, sample):
    """One sequence: p, q (None: chosen children) [n][vocab], -> (path, next token)."""
    p = probabilities(p)
    q = None if q is None else probabilities(q)
    accept = np.asarray(accept, dtype=np.float64)
    n, vocab = p.shape
    node, path = 0, [0]
    while True:
        r, z, down = p[node].copy(), 1.0, None
        for i in range(node + 1, n):
            x = int(tokens[i])
            if parents[i] != node or not 0 <= x < vocab:
                continue
            share = 1.0 if q is None else q[node, x]
            if r[x] > accept[i] * z * share:
                down = i
                break
            if q is None:
                z, r[x] = max(0.0, z - r[x]), 0.0
            else:
                r = np.maximum(r / (z if z > 0 else 1.0) - q[node], 0)
                z = r.sum()
        if down is None:
            break
        node = down
        path.append(node)
    if not r.sum() > 0:
        r = p[node]
    sums = np.cumsum(r)
    if not sums[-1] > 0:
        return path, -1
    above = np.flatnonzero((sums > np.float64(sample) * sums[-1]) & (r > 0))
    return path, int(above[0]) if len(above) else int(np.flatnonzero(r)[-1])


def compacted(pool, table, ctx, n, path):
    """The pool with a path's rows moved, and what was there otherwise."""
    new = pool.copy()
    for j, node in enumerate(path):
        to, of = ctx - n + j, ctx - n + node
        new[table[to // 16], :, to % 16] = pool[table[of // 16], :, of % 16]
    return new
