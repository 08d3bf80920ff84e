"""The 4-bit KV cache in numpy and 64 bits, from its definition: a row holds lo
(its smallest element), step = (largest - smallest) / 15 rounded once to the
storage type, and per element n = clamp(round_half_even((x - lo) / step), 0,
15); element x stands for lo + n * step.  Storage types travel as numpy
float16, or as uint16 bits for bf16."""
from __future__ import annotations

import numpy as np

import workloads as W

EPS = {W.DTYPE_F16: 2.0 ** -10, W.DTYPE_BF16: 2.0 ** -7, W.DTYPE_F32: 2.0 ** -23}


def to_f64(a: np.ndarray, dtype: int) -> np.ndarray:
    if dtype == W.DTYPE_BF16:
        return (a.astype(np.uint32) << np.uint32(16)).view(np.float32).astype(np.float64)
    return a.astype(np.float64)


def narrow(x: np.ndarray, dtype: int) -> np.ndarray:
    """float64 -> storage type with one rounding to nearest even."""
    x = np.asarray(x, dtype=np.float64)
    if dtype == W.DTYPE_F16:
        return x.astype(np.float16)
    if dtype == W.DTYPE_F32:
        return x.astype(np.float32)
    # to 32 bits towards zero with what was cut off kept in the last bit, then to bf16
    f = x.astype(np.float32)
    bits = f.view(np.uint32).copy()
    off = f.astype(np.float64) != x
    over = off & (np.abs(f.astype(np.float64)) > np.abs(x))
    bits[over] -= np.uint32(1)
    bits[off] |= np.uint32(1)
    rounded = (bits + np.uint32(0x7FFF) + ((bits >> np.uint32(16)) & np.uint32(1))) >> np.uint32(16)
    nan = np.isnan(x)
    rounded[nan] = 0x7FC0
    return rounded.astype(np.uint16)


def record_bytes(d: int) -> int:
    return 8 * d + 64


def quantise(x: np.ndarray, dtype: int):
    """Rows [..., d] of the storage type -> (codes uint8 [..., d], step, lo in the storage type)."""
    v = to_f64(x, dtype)
    bad = ~np.isfinite(v).all(-1)
    v = np.where(bad[..., None], 0.0, v)
    lo = v.min(-1)
    step = narrow((v.max(-1) - lo) / 15.0, dtype)
    s = to_f64(step, dtype)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(s[..., None] > 0, (v - lo[..., None]) / s[..., None], 0.0)
    codes = np.clip(np.rint(q), 0, 15).astype(np.uint8)
    lo = narrow(lo, dtype)
    nan = narrow(np.array([np.nan]), dtype)[0]
    step = np.where(bad, nan, step)
    lo = np.where(bad, nan, lo)
    codes[bad] = 0
    return codes, step.astype(narrow(np.zeros(1), dtype).dtype), lo.astype(step.dtype)


def values(codes, step, lo, dtype):
    return to_f64(lo, dtype)[..., None] + codes.astype(np.float64) * to_f64(step, dtype)[..., None]


def store_row(pool: np.ndarray, keys: bool, d: int, block: int, head: int, row: int, codes, step,
              lo) -> None:
    """Put one row into a pool (uint8 [NB][Hkv][record])."""
    rec = pool[block, head]
    packed = (codes[0::2] | (codes[1::2] << 4)).astype(np.uint8)
    if keys:
        rec[row * (d // 2):(row + 1) * (d // 2)] = packed
    else:
        for c in range(d // 4):
            at = (row // 2) * d + 4 * c + 2 * (row % 2)
            rec[at:at + 2] = packed[2 * c:2 * c + 2]
    pair = np.array([step, lo]).view(np.uint8)
    rec[8 * d + 4 * row:8 * d + 4 * row + 4] = pair


def load_rows(pool: np.ndarray, keys: bool, d: int, table, ctx: int, dtype: int) -> np.ndarray:
    """Values [Hkv][ctx][d] of one context, in 64 bits."""
    hkv = pool.shape[1]
    out = np.zeros((hkv, ctx, d))
    storage = np.float16 if dtype == W.DTYPE_F16 else np.uint16
    for blk in range((ctx + 15) // 16):
        rec = pool[int(table[blk])]                                   # [Hkv][record]
        n = min(16, ctx - 16 * blk)
        if keys:
            packed = rec[:, :8 * d].reshape(hkv, 16, d // 2)
        else:
            packed = rec[:, :8 * d].reshape(hkv, 8, d // 4, 2, 2).transpose(0, 1, 3, 2, 4)
            packed = packed.reshape(hkv, 16, d // 2)
        codes = np.stack([packed & 15, packed >> 4], -1).reshape(hkv, 16, d)
        pairs = np.ascontiguousarray(rec[:, 8 * d:]).view(storage).reshape(hkv, 16, 2)
        out[:, 16 * blk:16 * blk + n] = values(codes, pairs[..., 0], pairs[..., 1], dtype)[:, :n]
    return out


def build_pools(seed: int, *, contexts, hkv: int, d: int, dtype: int, spare: int = 3,
                mbs: int = 0, scale_of=None, num_blocks: int = 0):
    """Pools of normal rows for these contexts, in permuted blocks; every other
    byte, rows behind a context's end among them, is 0xFF (its pairs are NaN).
    scale_of(row index of the sequence) scales a row.  Returns (k_pool, v_pool,
    block_tables, context_lens)."""
    rng = np.random.Generator(np.random.PCG64(seed))
    used = [(c + 15) // 16 for c in contexts]
    nb = num_blocks or sum(used) + spare
    mbs = mbs or max(1, max(used))
    perm = rng.permutation(nb).astype(np.int32)
    pools = [np.full((nb, hkv, record_bytes(d)), 0xFF, dtype=np.uint8) for _ in range(2)]
    tables = np.full((len(contexts), mbs), -1, dtype=np.int32)
    at = 0
    for b, ctx in enumerate(contexts):
        tables[b, :used[b]] = perm[at:at + used[b]]
        at += used[b]
        if not ctx:
            continue
        for which, pool in enumerate(pools):
            rows = rng.standard_normal((ctx, hkv, d))
            if scale_of is not None:
                rows *= np.array([scale_of(j) for j in range(ctx)])[:, None, None]
            codes, step, lo = quantise(narrow(rows, dtype), dtype)
            packed = (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)
            pair = np.stack([step, lo], -1).view(np.uint8).reshape(ctx, hkv, 4)
            j = np.arange(ctx)
            blk, off = tables[b][j // 16], j % 16
            for r in range(16):
                sel = off == r
                if which == 0:
                    idx = r * (d // 2) + np.arange(d // 2)
                else:
                    idx = (r // 2) * d + 2 * (r % 2) + np.arange(d // 4)[:, None] * 4 + np.arange(2)
                pool[blk[sel][:, None, None], np.arange(hkv)[None, :, None],
                     idx.reshape(-1)[None, None, :]] = packed[sel]
                pool[blk[sel], :, 8 * d + 4 * r:8 * d + 4 * r + 4] = pair[sel]
    return pools[0], pools[1], tables, np.asarray(contexts, dtype=np.int32)


def decode(q, k_pool, v_pool, tables, contexts, scale, dtype):
    """softmax(scale q K) V over each context in 64 bits; returns (out, bound)
    where bound is how far a result of the documented arithmetic may be off:
      * scores in fp32: each of the head_dim products and sums may lose 2^-22 of
        the sum of magnitudes A (the tensor cores' fp32 accumulation keeps at
        least 22 bits), the softmax weight then loses ln 2 x that in the log2
        domain, 2 x for numerator and denominator, of values up to max |V|;
      * weights as fp16 plus residual: 2^-22, exponentials 2^-22, sums 2^-22
        a step: 2^-18 of max |V| covers 16 of them;
      * one rounding of the output: half a step, eps / 2 of |out|, and half the
        smallest subnormal."""
    qf = to_f64(q, dtype)
    B, hq, d = qf.shape
    hkv = k_pool.shape[1]
    G = hq // hkv
    out = np.zeros((B, hq, d))
    bound = np.zeros((B, hq, d))
    for b in range(B):
        ctx = int(contexts[b])
        if ctx == 0:
            continue
        k = load_rows(k_pool, True, d, tables[b], ctx, dtype)
        v = load_rows(v_pool, False, d, tables[b], ctx, dtype)
        for h in range(hq):
            s = scale * (k[h // G] @ qf[b, h])
            p = np.exp(s - s.max())
            out[b, h] = (p / p.sum()) @ v[h // G]
            # |lo| + n step <= |lo| + (hi - lo), at most three times the row's magnitude
            mags = 3 * np.abs(k[h // G]).max(-1) * np.abs(qf[b, h]).sum() * abs(scale) * 1.4427
            loss = 2 * np.log(2) * mags.max() * 2.0 ** -22 + 2.0 ** -18
            bound[b, h] = loss * 3 * np.abs(v[h // G]).max()
    bound += EPS[dtype] / 2 * (np.abs(out) + bound) + (2.0 ** -25 if dtype == W.DTYPE_F16 else 0.0)
    return out, bound
