"""The 4-bit KV cache on the GPU against the definition in 64 bits: codes and
pairs bit for bit, read-back values to one rounding, attention within the
bound of its documented arithmetic (int4_util.decode)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import int4_util as I
import paged_kv_attention_photon_gb300 as P
import workloads as W
from gpu_util import dev, host, to_float64

pytestmark = pytest.mark.gpu
TYPES = [W.DTYPE_F16, W.DTYPE_BF16]


def shape_for(*, seqs, hq, hkv, d, nb, mbs, dtype):
    return P.PagedShape.make(num_seqs=seqs, num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                             num_blocks=nb, max_blocks_per_seq=mbs, dtype=dtype)


def ok_status():
    st, bits = P.photon_get_last_device_error()
    assert st == 0, bits


def run_write(k, v, slots, nb, dtype, k_stride=0, v_stride=0, kd=None, vd=None):
    T, hkv, d = k.shape
    pools = [torch.full((nb, hkv, I.record_bytes(d)), 0xFF, dtype=torch.uint8, device="cuda")
             for _ in range(2)]
    shape = shape_for(seqs=1, hq=hkv, hkv=hkv, d=d, nb=nb, mbs=1, dtype=dtype)
    P.photon_cache_write_int4(dev(k) if kd is None else kd, k_stride,
                              dev(v) if vd is None else vd, v_stride, dev(slots), T, *pools, shape)
    return [p.cpu().numpy() for p in pools]


def want_pools(k, v, slots, nb, dtype):
    T, hkv, d = k.shape
    want = [np.full((nb, hkv, I.record_bytes(d)), 0xFF, dtype=np.uint8) for _ in range(2)]
    for which, (x, pool) in enumerate(zip((k, v), want)):
        codes, step, lo = I.quantise(x, dtype)
        for t in range(T):
            if 0 <= slots[t] < nb * 16:
                for h in range(hkv):
                    I.store_row(pool, which == 0, d, slots[t] // 16, h, slots[t] % 16, codes[t, h],
                                step[t, h], lo[t, h])
    return want


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,hkv", [(1, 1), (3, 2), (37, 8), (130, 3)])
def test_write_bit_exact(dtype, d, T, hkv):
    rng = np.random.default_rng(T * d + hkv)
    nb = T // 16 + 3
    slots = rng.permutation(nb * 16)[:T].astype(np.int64)
    k = I.narrow(rng.standard_normal((T, hkv, d)) * np.exp(rng.uniform(-6, 6, (T, hkv, 1))), dtype)
    v = I.narrow(rng.standard_normal((T, hkv, d)) + 3, dtype)
    if T > 2:
        slots[1] = -1
    got = run_write(k, v, slots, nb, dtype)
    ok_status()
    for a, b in zip(got, want_pools(k, v, slots, nb, dtype)):
        assert np.array_equal(a, b)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
def test_write_hard_rows(dtype, d):
    """Constant, tiny, huge and one-outlier rows, rows on a grid that puts many elements
    exactly between two codes, and rows of few distinct values."""
    rng = np.random.default_rng(5)
    top = 65504.0 if dtype == W.DTYPE_F16 else 3.3e38
    low = 2.0 ** -24 if dtype == W.DTYPE_F16 else 2.0 ** -130
    rows = [np.zeros(d), np.full(d, 1.5), np.full(d, -0.0), np.full(d, top), np.full(d, -top),
            rng.choice([-top, top], d), rng.uniform(-1, 1, d) * top,
            rng.integers(0, 9, d) * low, rng.integers(-40, 40, d) * low,
            np.concatenate([rng.standard_normal(d - 1), [500.0]]),
            np.concatenate([np.full(d - 1, -7.0), [-6.5]])]
    for unit in (1.0, 0.25, 2.0 ** -9, 3.0):
        # steps of exactly 2 units: odd multiples of the unit lie on a border
        rows.append(np.concatenate([rng.integers(0, 31, d - 2), [0, 30]]) * unit)
        rows.append(np.concatenate([rng.integers(-15, 16, d - 2), [-15, 15]]) * unit)
    for s in range(64):   # many steps near the border of two storage values
        rows.append(np.round(rng.standard_normal(d) * 64) / 64 * (1 + s))
    x = I.narrow(np.stack(rows)[:, None, :], dtype)
    T = x.shape[0]
    nb = T // 16 + 1
    slots = np.arange(T, dtype=np.int64)[::-1].copy()
    got = run_write(x, x[::-1].copy(), slots, nb, dtype)
    ok_status()
    want = want_pools(x, x[::-1].copy(), slots, nb, dtype)
    for a, b in zip(got, want):
        # a row's smallest element may be either zero
        for pool in (a, b):
            pairs = pool[:, :, 8 * d:].reshape(nb, 1, 16, 4)
            pairs[..., 3][(pairs[..., 2] == 0) & (pairs[..., 3] == 0x80)] = 0
        assert np.array_equal(a, b)


@pytest.mark.parametrize("dtype", TYPES)
def test_write_rows_that_are_not_finite(dtype):
    d, hkv = 128, 2
    rng = np.random.default_rng(8)
    x = rng.standard_normal((6, hkv, d))
    x[1, 0, 5] = np.nan
    x[2, 1, 127] = np.inf
    x[3, 0, 0] = -np.inf
    k = I.narrow(x, dtype)
    slots = np.arange(6, dtype=np.int64)
    got = run_write(k, k, slots, 1, dtype)
    ok_status()
    storage = np.float16 if dtype == W.DTYPE_F16 else np.uint16
    for pool in got:
        pairs = I.to_f64(np.ascontiguousarray(pool[:, :, 8 * d:]).view(storage), dtype)
        pairs = pairs.reshape(hkv, 16, 2)
        bad = np.zeros((hkv, 16), bool)
        bad[0, 1] = bad[1, 2] = bad[0, 3] = True
        bad[:, 6:] = True     # never written
        assert np.array_equal(np.isnan(pairs).any(-1), bad)
        assert np.array_equal(np.isnan(pairs).all(-1), bad)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
def test_write_strides_and_bad_slots(dtype, d):
    """A slice of a fused projection; slots outside the pool flag bit 2 and skip their row."""
    rng = np.random.default_rng(11)
    T, hkv, nb = 19, 4, 3
    fused = I.narrow(rng.standard_normal((T, 3 * hkv, d)), dtype)
    slots = rng.permutation(nb * 16)[:T].astype(np.int64)
    slots[4], slots[7], slots[18] = nb * 16, -5, 1 << 40
    on = dev(fused)
    got = run_write(fused[:, :hkv], fused[:, 2 * hkv:], slots, nb, dtype, 3 * hkv * d, 3 * hkv * d,
                    on, on[:, 2 * hkv:])
    st, bits = P.photon_get_last_device_error()
    assert (st, bits) == (6, 2)
    k, v = np.ascontiguousarray(fused[:, :hkv]), np.ascontiguousarray(fused[:, 2 * hkv:])
    for a, b in zip(got, want_pools(k, v, slots, nb, dtype)):
        assert np.array_equal(a, b)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
def test_gather(dtype, d):
    contexts = [0, 1, 15, 16, 17, 50]
    hkv = 3
    kp, vp, bt, cl = I.build_pools(21, contexts=contexts, hkv=hkv, d=d, dtype=dtype, mbs=6)
    shape = shape_for(seqs=6, hq=hkv, hkv=hkv, d=d, nb=kp.shape[0], mbs=6, dtype=dtype)
    like = np.zeros((6, hkv, 96, d), dtype=np.float16 if dtype == W.DTYPE_F16 else np.uint16)
    out = [torch.full(like.shape, -1, dtype=torch.int16, device="cuda") for _ in range(2)]
    P.photon_paged_gather_int4(dev(kp), dev(vp), dev(bt), dev(cl), *out, shape)
    ok_status()
    for which, (pool, t) in enumerate(zip((kp, vp), out)):
        got = I.to_f64(host(t, like), dtype)
        for b, ctx in enumerate(contexts):
            want = I.load_rows(pool, which == 0, d, bt[b], ctx, dtype)
            # fp32 first (2^-24), then half a step of the storage type
            tol = np.abs(want) * (I.EPS[dtype] / 2 + 2.0 ** -23) + 2.0 ** -25
            assert (np.abs(got[b, :, :ctx] - want) <= tol).all()
            assert not got[b, :, ctx:].any()
    # a block outside the pool and a length outside the table: zeros and the error bits
    bt2, cl2 = bt.copy(), cl.copy()
    bt2[5, 1] = kp.shape[0]
    cl2[4] = 97
    P.photon_paged_gather_int4(dev(kp), dev(vp), dev(bt2), dev(cl2), *out, shape)
    st, bits = P.photon_get_last_device_error()
    assert (st, bits) == (6, 1 | 4)
    got = I.to_f64(host(out[0], like), dtype)
    assert not got[5, :, 16:32].any() and got[5, :, 32:50].any() and not got[4].any()


@pytest.mark.parametrize("dtype,tiny", [(W.DTYPE_F16, 2.0 ** -24), (W.DTYPE_BF16, 2.0 ** -30)])
def test_gather_rounds_once(dtype, tiny):
    """Values halfway between two of the storage type's but for a lo far below them."""
    rng = np.random.default_rng(31)
    d, n = 64, 256
    x = rng.uniform(tiny, 4.0, (n, 1, d))
    x[:, 0, 0] = np.where(np.arange(n) % 2, tiny, -tiny)
    x[:, 0, 1] = rng.uniform(0.5, 4.0, n)
    x = I.narrow(np.clip(x, x[:, :, :1], x[:, :, 1:2]), dtype)
    codes, step, lo = I.quantise(x, dtype)
    pool = np.zeros((n // 16, 1, I.record_bytes(d)), dtype=np.uint8)
    for which in (True, False):
        for t in range(n):
            I.store_row(pool, which, d, t // 16, 0, t % 16, codes[t, 0], step[t, 0], lo[t, 0])
        shape = shape_for(seqs=1, hq=1, hkv=1, d=d, nb=n // 16, mbs=n // 16, dtype=dtype)
        table = dev(np.arange(n // 16, dtype=np.int32)[None])
        out = [torch.zeros((1, 1, n, d), dtype=torch.int16, device="cuda") for _ in range(2)]
        P.photon_paged_gather_int4(dev(pool), dev(pool), table, dev(np.array([n], np.int32)), *out,
                                   shape)
        ok_status()
        exact = I.values(codes, step, lo, dtype)[:, 0]
        first = exact.astype(np.float32).astype(np.float64)
        assert (I.narrow(first, dtype) != I.narrow(exact, dtype)).any()   # rounding twice shows
        assert np.array_equal(host(out[0 if which else 1], x).reshape(n, d), I.narrow(exact, dtype))


class Decode:
    """One decode call's device buffers; the output starts as -1 bits, the workspace as NaNs."""

    def __init__(self, seed, contexts, hq, hkv, d, dtype, **pool):
        self.kp, self.vp, self.bt, self.cl = I.build_pools(seed, contexts=contexts, hkv=hkv, d=d,
                                                           dtype=dtype, **pool)
        rng = np.random.default_rng(seed + 1)
        self.q = I.narrow(rng.standard_normal((len(contexts), hq, d)), dtype)
        self.dtype, self.scale = dtype, d ** -0.5
        self.shape = shape_for(seqs=len(contexts), hq=hq, hkv=hkv, d=d, nb=self.kp.shape[0],
                               mbs=self.bt.shape[1], dtype=dtype)
        self.ws_bytes = P.photon_paged_decode_int4_workspace_size(self.shape)
        self.ws = torch.full((max(16, self.ws_bytes),), 0xFF, dtype=torch.uint8, device="cuda")
        self.out = torch.full(self.q.shape, -1, dtype=torch.int16, device="cuda")
        self.up()

    def up(self):
        self.dev = [dev(x) for x in (self.q, self.kp, self.vp, self.bt, self.cl)]

    def run(self, stream=None):
        P.photon_paged_decode_int4(*self.dev, self.scale, self.out, self.ws, self.ws_bytes,
                                   self.shape, stream)

    def got(self):
        return I.to_f64(host(self.out, self.q), self.dtype)

    def check(self):
        want, bound = I.decode(self.q, self.kp, self.vp, self.bt, self.cl, self.scale, self.dtype)
        got = self.got()
        assert np.isfinite(got).all()
        worst = (np.abs(got - want) - bound).max()
        assert worst <= 0, f"off by {np.abs(got - want).max()}, {worst} over the bound"


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (4, 1), (8, 1), (12, 3)])
def test_decode(dtype, d, hq, hkv):
    c = Decode(31 + hq, [0, 1, 15, 16, 17, 63, 64, 65, 300, 1, 0, 129], hq, hkv, d, dtype)
    for _ in range(2):   # the workspace's last contents do not matter
        c.run()
        ok_status()
        c.check()


@pytest.mark.parametrize("hq,hkv,d", [(2, 1, 64), (8, 1, 128)])
def test_decode_one_long_context(hq, hkv, d):
    c = Decode(41, [20011], hq, hkv, d, W.DTYPE_F16)
    c.run()
    ok_status()
    c.check()


@pytest.mark.parametrize("hq,hkv,d", [(16, 8, 128), (16, 16, 64), (64, 8, 64), (12, 6, 64),
                                      (12, 12, 128)])
def test_decode_many_heads(hq, hkv, d):
    """8, 4 and 2 KV heads of a block read together."""
    c = Decode(37, [0, 33, 700, 16, 1], hq, hkv, d, W.DTYPE_F16)
    c.run()
    ok_status()
    c.check()


def test_decode_large_batch():
    """More sequences than threads of a CTA, empty ones in a row, more units than warps."""
    rng = np.random.default_rng(2)
    contexts = [int(x) for x in rng.integers(0, 40, 700)]
    contexts[100:240] = [0] * 140
    contexts[5], contexts[699], contexts[0] = 3000, 0, 0
    c = Decode(43, contexts, 8, 4, 64, W.DTYPE_BF16)
    c.run()
    ok_status()
    c.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("direction", [1, -1])
def test_decode_rows_of_very_different_size(dtype, direction):
    """K and V rows that grow, or shrink, by 2^13 along the context: the running maximum
    and the V steps' scale move."""
    n = 400
    c = Decode(47, [n], 4, 2, 128, dtype, scale_of=lambda j: 2.0 ** (direction * (j * 13 / n)
                                                                     - (13 if direction > 0 else 0)))
    c.scale = 1.0
    c.run()
    ok_status()
    c.check()


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_decode_scales(scale):
    c = Decode(53, [77, 5, 200], 8, 2, 64, W.DTYPE_F16)
    c.scale = scale
    c.run()
    ok_status()
    c.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("size", [2.0 ** -14, 2.0 ** 10])
def test_decode_small_and_large_queries(dtype, size):
    c = Decode(59, [40, 17], 4, 2, 128, dtype)
    c.q = I.narrow(I.to_f64(c.q, dtype) * size, dtype)
    c.scale /= size
    c.up()
    c.run()
    ok_status()
    c.check()


def test_decode_nan_row_stays_with_its_sequence():
    """A cached row that reads back as NaN, or a NaN query, reaches its own heads only."""
    c = Decode(61, [30, 30, 30], 8, 2, 64, W.DTYPE_F16)
    blk = int(c.bt[1, 0])
    c.kp[blk, 0, 8 * 64 + 12:8 * 64 + 16] = 0xFF      # row 3 of KV head 0 of sequence 1
    c.q[2, 5, 1] = np.nan
    c.up()
    c.run()
    ok_status()
    bad = np.isnan(c.got()).any(-1)
    want = np.zeros((3, 8), bool)
    want[1, :4] = True
    want[2, 5] = True
    assert np.array_equal(bad, want)


def test_decode_bad_tables_and_lengths():
    c = Decode(67, [40, 100, 33], 4, 2, 128, W.DTYPE_F16)
    want, bound = I.decode(c.q, c.kp, c.vp, c.bt, c.cl, c.scale, c.dtype)
    c.cl[0] = c.bt.shape[1] * 16 + 1
    c.cl[2] = -1
    c.up()
    c.run()
    assert P.photon_get_last_device_error() == (6, 4)
    got = c.got()
    assert not got[0].any() and not got[2].any()
    assert (np.abs(got[1] - want[1]) <= bound[1]).all()
    # a block id outside the pool: its keys are absent
    c.cl[:] = [16, 100, 48]
    c.bt[1, 3] = c.kp.shape[0]
    c.bt[0, 0] = -7                # the whole context
    c.up()
    c.run()
    assert P.photon_get_last_device_error() == (6, 1)
    got = c.got()
    assert not got[0].any()
    kept = np.r_[0:48, 64:100]
    k = np.concatenate([I.load_rows(c.kp, True, 128, c.bt[1], 48, c.dtype),
                        I.load_rows(c.kp, True, 128, c.bt[1, 4:], 36, c.dtype)], 1)
    v = np.concatenate([I.load_rows(c.vp, False, 128, c.bt[1], 48, c.dtype),
                        I.load_rows(c.vp, False, 128, c.bt[1, 4:], 36, c.dtype)], 1)
    assert k.shape[1] == kept.size
    for h in range(4):
        s = c.scale * (k[h // 2] @ I.to_f64(c.q, c.dtype)[1, h])
        p = np.exp(s - s.max())
        assert (np.abs(got[1, h] - (p / p.sum()) @ v[h // 2]) <= bound[1, h] + 1e-3).all()


def test_decode_captured_and_on_another_stream():
    """Two calls with workspaces of their own in one graph, replayed with other lengths and
    queries; a call on a side stream."""
    a = Decode(71, [300, 17, 64], 8, 4, 64, W.DTYPE_F16, mbs=20)
    b = Decode(73, [5, 900], 8, 1, 128, W.DTYPE_BF16)
    a.run(), b.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run(), b.run()
    a.cl[:] = [255, 1, 0]
    a.q = a.q[::-1].copy()
    a.dev[0].copy_(dev(a.q))
    a.dev[4].copy_(dev(a.cl))
    for _ in range(2):
        graph.replay()
    ok_status()
    a.check()
    b.check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a.cl[:] = [300, 17, 64]
    with torch.cuda.stream(side):
        a.dev[4].copy_(dev(a.cl))
        a.run()
    side.synchronize()
    a.check()


def test_pool_offsets_past_32_bits():
    """Pools of more than 4 GiB whose used blocks are at the far end."""
    d, hkv, nb = 128, 8, 500_000
    small = Decode(79, [40, 100], 16, hkv, d, W.DTYPE_F16)
    n = small.kp.shape[0]
    shape = shape_for(seqs=2, hq=16, hkv=hkv, d=d, nb=nb, mbs=small.bt.shape[1], dtype=W.DTYPE_F16)
    assert P.photon_cache_int4_bytes(shape) > 1 << 32
    pools = []
    for x in (small.kp, small.vp):
        t = torch.empty((nb, hkv, I.record_bytes(d)), dtype=torch.uint8, device="cuda")
        t[nb - n:] = dev(x)
        pools.append(t)
    bt = np.where(small.bt >= 0, small.bt + nb - n, -1).astype(np.int32)
    P.photon_paged_decode_int4(small.dev[0], *pools, dev(bt), small.dev[4], small.scale, small.out,
                               small.ws, small.ws_bytes, shape)
    ok_status()
    small.check()
    # and a write there
    rng = np.random.default_rng(3)
    k = I.narrow(rng.standard_normal((2, hkv, d)), W.DTYPE_F16)
    slots = np.array([nb * 16 - 1, (nb - n) * 16 + 3], dtype=np.int64)
    P.photon_cache_write_int4(dev(k), 0, dev(k), 0, dev(slots), 2, *pools, shape)
    ok_status()
    want = want_pools(k, k, slots - (nb - n) * 16, n, W.DTYPE_F16)
    for pool, w in zip(pools, want):
        got = pool[nb - n:].cpu().numpy()
        for s, t in ((n * 16 - 1, 0), (3, 1)):
            pair = slice(8 * d + 4 * (s % 16), 8 * d + 4 * (s % 16) + 4)
            assert np.array_equal(got[s // 16, :, pair], w[s // 16, :, pair])


def test_write_then_decode():
    """A step at a time: the new rows go in, the attention sees them."""
    dtype, hq, hkv, d = W.DTYPE_BF16, 8, 4, 64
    c = Decode(83, [33, 16, 1], hq, hkv, d, dtype, mbs=4)
    rng = np.random.default_rng(4)
    fresh = [b for b in range(c.kp.shape[0]) if b not in c.bt]
    for step in range(3):
        slots = np.zeros(3, dtype=np.int64)
        for b in range(3):
            pos = int(c.cl[b])
            if pos % 16 == 0:
                c.bt[b, pos // 16] = fresh.pop()
            slots[b] = int(c.bt[b, pos // 16]) * 16 + pos % 16
            c.cl[b] += 1
        k = I.narrow(rng.standard_normal((3, hkv, d)), dtype)
        v = I.narrow(rng.standard_normal((3, hkv, d)), dtype)
        P.photon_cache_write_int4(dev(k), 0, dev(v), 0, dev(slots), 3, c.dev[1], c.dev[2], c.shape)
        for which, (x, pool) in enumerate(((k, c.kp), (v, c.vp))):
            codes, st, lo = I.quantise(x, dtype)
            for b in range(3):
                for h in range(hkv):
                    I.store_row(pool, which == 0, d, slots[b] // 16, h, slots[b] % 16, codes[b, h],
                                st[b, h], lo[b, h])
        c.dev[3], c.dev[4] = dev(c.bt), dev(c.cl)
        c.run()
        ok_status()
        assert np.array_equal(c.dev[1].cpu().numpy(), c.kp)
        assert np.array_equal(c.dev[2].cpu().numpy(), c.vp)
        c.check()


def test_decode_of_empty_contexts_only():
    c = Decode(89, [0, 0, 0], 4, 2, 64, W.DTYPE_F16)
    c.run()
    ok_status()
    assert not c.got().any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale", [0.0, 1e-20, -1e-20, 0.125])
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (8, 1, 128)])
def test_decode_zero_and_tiny_queries(dtype, scale, hq, hkv, d):
    """Rows of q that are zero, or (bf16) far below 1: every weight is 1 or nearly so, and keys
    that are not there weigh nothing, whatever part of the last 32 they are."""
    c = Decode(97, [5, 16, 33, 64, 70, 200], hq, hkv, d, dtype)
    c.scale = scale
    q = I.to_f64(c.q, dtype)
    q[:, 1::2] = 0.0
    q[1:4, ::2] *= 2.0 ** -60
    c.q = I.narrow(q, dtype)
    c.up()
    c.run()
    ok_status()
    c.check()
    c.bt[5, 3] = c.kp.shape[0]     # and a block that is not in the pool
    c.up()
    c.run()
    assert P.photon_get_last_device_error() == (6, 1)
    assert np.isfinite(c.got()).all()


@pytest.mark.parametrize("size", [2.0 ** 112, 2.0 ** 118, 2.0 ** 121])
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (8, 1, 128)])
def test_decode_queries_near_the_types_largest(size, hq, hkv, d):
    """bf16 rows whose scale brings the scores back to ordinary ones."""
    c = Decode(101, [40, 17, 129], hq, hkv, d, W.DTYPE_BF16)
    c.q = I.narrow(np.abs(I.to_f64(c.q, c.dtype)) * size, c.dtype)
    c.scale /= size
    c.up()
    c.run()
    ok_status()
    c.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("keys", [1568, 13900])
@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 64), (4, 1, 128), (8, 1, 64), (8, 1, 128)])
def test_decode_many_keys_of_little_weight(dtype, keys, hq, hkv, d):
    """A first key holds nearly all of the weight and has a small V; each key behind it weighs
    e^-17 to e^-19 and has an ordinary V.  The sequences share one table, and are so many that
    a run of the split has as many keys as a context.

    Bound: every sum of keys / 16 products of 16 keys in fp32 may lose 2^-22 of the magnitudes
    M = sum p (|lo| + 15 step) a product; then the output's rounding."""
    rng = np.random.default_rng(keys + hq)
    scale = 8.0 / d
    # constant K rows, so scores are exact: 17 (1 + s / 64) for the first key, 0 for the others
    k = np.zeros((keys, 1, d))
    k[0] = 2.125
    v = rng.standard_normal((keys, 1, d))
    v[0] *= 0.003
    rows = [I.quantise(I.narrow(x, dtype), dtype) for x in (k, v)]
    blocks = (keys + 15) // 16
    pools = [np.full((blocks, 1, I.record_bytes(d)), 0xFF, dtype=np.uint8) for _ in range(2)]
    for which, (codes, step, lo) in enumerate(rows):
        for j in range(keys):
            I.store_row(pools[which], which == 0, d, j // 16, 0, j % 16, codes[j, 0], step[j, 0],
                        lo[j, 0])
    seqs = 2600
    q = np.ones((hq, d)) * (1 + np.arange(hq) / 64)[:, None]
    on_q = dev(np.broadcast_to(I.narrow(q, dtype), (seqs, hq, d)))
    table = dev(np.broadcast_to(np.arange(blocks, dtype=np.int32), (seqs, blocks)))
    shape = shape_for(seqs=seqs, hq=hq, hkv=1, d=d, nb=blocks, mbs=blocks, dtype=dtype)
    n = P.photon_paged_decode_int4_workspace_size(shape)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    out = torch.full((seqs, hq, d), -1, dtype=torch.int16, device="cuda")
    P.photon_paged_decode_int4(on_q, dev(pools[0]), dev(pools[1]), table,
                               dev(np.full(seqs, keys, np.int32)), scale, out, ws, n, shape)
    ok_status()
    got = I.to_f64(host(out, np.zeros((seqs, hq, d), np.float16 if dtype == W.DTYPE_F16 else np.uint16)),
                   dtype)
    codes, step, lo = (x[:, 0] for x in rows[1])
    value, size = I.values(codes, step, lo, dtype), np.abs(I.to_f64(lo, dtype)) + 15 * I.to_f64(step, dtype)
    for s in range(hq):
        p = np.exp(scale * (I.to_f64(I.narrow(k, dtype), dtype)[:, 0] @ q[s] - 2.125 * q[s].sum()))
        want = (p @ value) / p.sum()
        tol = keys / 16 * 2.0 ** -22 * (p @ size)
        tol += I.EPS[dtype] / 2 * (np.abs(want) + tol) + (2.0 ** -25 if dtype == W.DTYPE_F16 else 0.0)
        assert (np.abs(got[:, s] - want) <= tol).all(), (np.abs(got[:, s] - want) / tol).max()


def borders(rng, d):
    """Rows with steps of exactly 2, odd multiples of 1 lying between two codes, and others."""
    rows = [np.concatenate([rng.integers(0, 31, d - 2), [0, 30]]) for _ in range(20)]
    rows += [np.concatenate([rng.integers(-15, 16, d - 2), [-15, 15]]) for _ in range(20)]
    return np.stack(rows + [rng.standard_normal(d) * 8 for _ in range(200)])


@pytest.mark.parametrize("dtype,size", [(W.DTYPE_F16, 2.0 ** -12), (W.DTYPE_F16, 2.0 ** -20)] +
                         [(W.DTYPE_BF16, 2.0 ** -e) for e in (12, 16, 40, 80, 98, 104, 120)])
@pytest.mark.parametrize("d", [64, 128])
def test_write_small_ranges(dtype, size, d):
    """Steps far below 1, down to where they have few bits (fp16) or fp32 ends (bf16)."""
    x = I.narrow(borders(np.random.default_rng(int(-np.log2(size))), d)[:, None] * size, dtype)
    T = x.shape[0]
    slots = np.arange(T, dtype=np.int64)
    got = run_write(x, x, slots, T // 16, dtype)
    ok_status()
    for a, b in zip(got, want_pools(x, x, slots, T // 16, dtype)):
        assert np.array_equal(a, b)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("unit", [1.0, 2.0 ** 5, 2.0 ** -3])
def test_write_elements_that_decide_a_border_by_their_last_bits(dtype, d, unit):
    """lo is a half-integer number of steps, so an element near 0 is next to a border: zero lies
    on it (even code), the smallest ones above and below it by less than fp32 keeps of x - lo."""
    tiny = 2.0 ** -24 if dtype == W.DTYPE_F16 else 2.0 ** -30 * unit
    rows, where = [], []
    for below in range(15):          # lo = -(below + 1/2) steps, hi = 15 steps more
        lo = -(below + 0.5)
        x = np.linspace(0.25, 0.45, d) * (1 if below < 14 else -1)
        x[0], x[1] = lo, lo + 15
        small = [tiny, -tiny, 2 * tiny, -2 * tiny, 0.0]
        x[2:7] = np.array(small) / unit
        x[d - 5:] = np.array(small[::-1]) / unit
        rows.append(x * unit)
        up, even = below + 1, below + 1 if below % 2 else below
        where.append([up, below, up, below, even])
    x = I.narrow(np.stack(rows)[:, None], dtype)
    codes, step, lo = I.quantise(x, dtype)
    assert (I.to_f64(step, dtype) == unit).all()
    # the oracle's own quotient is in 64 bits, which hold lo + 2^-30; checked against the definition
    assert np.array_equal(codes[:, 0, 2:7], np.array(where))
    slots = np.arange(15, dtype=np.int64)
    got = run_write(x, x, slots, 1, dtype)
    ok_status()
    for a, b in zip(got, want_pools(x, x, slots, 1, dtype)):
        assert np.array_equal(a, b)


def packed_pools(k, v, slots, nb, dtype):
    """want_pools, by arrays."""
    T, hkv, d = k.shape
    want = []
    kept = (slots >= 0) & (slots < nb * 16)
    blk, row = slots[kept] // 16, slots[kept] % 16
    for which, x in enumerate((k, v)):
        pool = np.full((nb, hkv, I.record_bytes(d)), 0xFF, dtype=np.uint8)
        codes, step, lo = (y[kept] for y in I.quantise(x, dtype))
        packed = (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)
        at = np.arange(d // 2)
        if which == 0:
            byte = row[:, None] * (d // 2) + at
        else:
            byte = row[:, None] // 2 * d + at // 2 * 4 + row[:, None] % 2 * 2 + at % 2
        heads = np.arange(hkv)[None, :, None]
        pool[blk[:, None, None], heads, byte[:, None]] = packed
        pair = np.stack([step, lo], -1).view(np.uint8).reshape(len(blk), hkv, 4)
        pool[blk[:, None, None], heads, 8 * d + 4 * row[:, None, None] + np.arange(4)] = pair
        want.append(pool)
    return want


def test_packed_pools_are_the_oracles():
    rng = np.random.default_rng(1)
    for dtype in TYPES:
        x = I.narrow(rng.standard_normal((30, 3, 64)), dtype)
        slots = rng.permutation(48)[:30].astype(np.int64)
        slots[[2, 5]] = -1, 48
        for a, b in zip(packed_pools(x, x[::-1], slots, 3, dtype), want_pools(x, x[::-1], slots, 3, dtype)):
            assert np.array_equal(a, b)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv", [1, 3, 5, 7, 8, 12])
def test_write_several_rounds(dtype, d, hkv):
    """More rows than two rounds of the grid (3 / 2 CTAs per SM of 8 warps, 512 / d rows each a
    round), with head counts that do not divide a round: a warp's next token and head are carried on."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    round_rows = sms * 3 // 2 * 8 * (512 // d)
    T = (2 * round_rows + round_rows // 2) // hkv + 1
    rng = np.random.default_rng(T + d)
    nb = T // 16 + 2
    slots = rng.permutation(nb * 16)[:T].astype(np.int64)
    slots[::97] = -1
    slots[T - 2] = nb * 16          # a bad slot in the last round
    fused = I.narrow(rng.standard_normal((T, 2 * hkv, d)) * np.exp(rng.uniform(-3, 3, (T, 1, 1))), dtype)
    on, stride = dev(fused), 2 * hkv * d
    got = run_write(fused[:, :hkv], fused[:, hkv:], slots, nb, dtype, stride, stride, on, on[:, hkv:])
    assert P.photon_get_last_device_error() == (6, 2)
    for a, b in zip(got, packed_pools(fused[:, :hkv], fused[:, hkv:], slots, nb, dtype)):
        assert np.array_equal(a, b)


@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 64), (16, 2, 128)])
def test_decode_two_streams_at_once_and_repeated(hq, hkv, d):
    """Two calls in flight with workspaces of their own, again and again: the same bits."""
    rng = np.random.default_rng(6)
    cases = [Decode(103, [int(x) for x in rng.integers(0, 900, 40)], hq, hkv, d, W.DTYPE_F16),
             Decode(107, [2000, 3, 700], 8, 4, 64, W.DTYPE_BF16)]
    streams = [torch.cuda.Stream() for _ in cases]
    first = []
    for c in cases:
        c.run()
        ok_status()
        c.check()
        first.append(c.out.clone())
    for _ in range(5):
        for c in cases:
            c.out.fill_(-1)
        torch.cuda.synchronize()
        for _ in range(4):
            for c, s in zip(cases, streams):
                c.run(s)
        torch.cuda.synchronize()
        for c, f in zip(cases, first):
            assert torch.equal(c.out, f)
    ok_status()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("hq,hkv,d", [(2, 1, 64), (4, 1, 128), (8, 1, 64), (8, 1, 128)])
@pytest.mark.parametrize("size", [1e3, 2e5, 7e6, 3e7, 1e8, 1e9, 1e10])
def test_decode_scores_far_from_zero(dtype, hq, hkv, d, size):
    """Scores of that size (log2 domain), so far apart that only the keys of the largest one weigh
    anything; those are equal, and the output is the mean of their V.  Constant K rows, so equal
    rows have equal scores whatever the products lose."""
    rng = np.random.default_rng(int(size) % 1000 + d)
    contexts = [300, 77, 1, 520]
    kp, vp, bt, cl = I.build_pools(113, contexts=contexts, hkv=1, d=d, dtype=dtype)
    ladder = np.array([0.25, 0.5, 0.625, 0.75, 0.875, 1.0]) * 1.37
    picks = []
    for b, n in enumerate(contexts):
        # rising in steps, so that the maximum moves several times, the largest a few times over
        pick = np.sort(rng.integers(0, len(ladder), n))
        pick[rng.integers(0, n, n // 3)] = 0
        picks.append(pick)
        codes, step, lo = I.quantise(I.narrow(np.broadcast_to(ladder[pick][:, None], (n, d)), dtype), dtype)
        for j in range(n):
            I.store_row(kp, True, d, bt[b, j // 16], 0, j % 16, codes[j], step[j], lo[j])
    q = I.narrow(np.full((len(contexts), hq, d), 3.0) + np.arange(hq)[None, :, None] / 4, dtype)
    scale = size / (1.4427 * 1.37 * 3.0 * d)
    shape = shape_for(seqs=len(contexts), hq=hq, hkv=1, d=d, nb=kp.shape[0], mbs=bt.shape[1], dtype=dtype)
    n = P.photon_paged_decode_int4_workspace_size(shape)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for sign in (1, -1):     # a negative scale turns the ladder round
        out = torch.full(q.shape, -1, dtype=torch.int16, device="cuda")
        P.photon_paged_decode_int4(dev(q), dev(kp), dev(vp), dev(bt), dev(cl), sign * scale, out, ws, n,
                                   shape)
        ok_status()
        got = I.to_f64(host(out, q), dtype)
        for b, ctx in enumerate(contexts):
            v = I.load_rows(vp, False, d, bt[b], ctx, dtype)[0]
            top = picks[b] == (picks[b].max() if sign > 0 else picks[b].min())
            want = v[top].mean(0)
            # sums of up to ctx weights of 1: 2^-22 each; the other keys weigh 2^-100 and less
            tol = ctx * 2.0 ** -22 * np.abs(v).max()
            tol = tol + I.EPS[dtype] / 2 * (np.abs(want) + tol) + 2.0 ** -25
            assert (np.abs(got[b] - want) <= tol).all(), (sign, b, np.abs(got[b] - want).max())
