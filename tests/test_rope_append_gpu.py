"""photon_rope_cache_append against its formula in 64 bits.  Bound: two products and a sum in
fp32, each off by 2^-24 of what it gives, so 3 x 2^-24 of |x[a]| + |x[b]|, then one rounding,
eps / 2 of the result (fp16 and bf16 subnormals: half of the smallest step).  What is copied is
compared bit for bit, the pools' other rows too."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import int4_util as I
import paged_kv_attention_photon_gb300 as P
import workloads as W
from gpu_util import dev, host, rope_table

pytestmark = pytest.mark.gpu
TYPES = [W.DTYPE_F32, W.DTYPE_F16, W.DTYPE_BF16]
TINY = {W.DTYPE_F32: 2.0 ** -149, W.DTYPE_F16: 2.0 ** -25, W.DTYPE_BF16: 2.0 ** -134}


def bits(a):
    return np.ascontiguousarray(a).view(np.uint8)


class Case:
    def __init__(self, *, T, hq, hkv, d, dtype, rotary, pairs, seed=0, extra=0, max_pos=300, NB=None):
        rng = np.random.default_rng(seed)
        self.T, self.hq, self.hkv, self.d, self.dtype = T, hq, hkv, d, dtype
        self.rotary, self.pairs, self.max_pos = rotary, pairs, max_pos
        self.NB = NB or (T + 15) // 16 + 3
        self.fused = I.narrow(rng.standard_normal((T, hq + 2 * hkv + extra, d)), dtype)
        self.pos = rng.integers(0, max_pos, T).astype(np.int32)
        self.slots = rng.permutation(self.NB * 16)[:T].astype(np.int64)
        self.pools = [I.narrow(rng.standard_normal((self.NB, hkv, 16, d)), dtype) for _ in range(2)]
        self.table = rope_table(1e4, max_pos, rotary)
        self.shape = P.PagedShape.make(num_seqs=0, num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                                       num_blocks=self.NB, max_blocks_per_seq=1, dtype=dtype)
        self.before = I.narrow(np.full((T, hq, d), -1.0), dtype)

    def run(self, in_place=False, keys_only=False, stream=None):
        """q_out (or q in place) and the pools after the call, in the storage type."""
        on = dev(self.fused)
        pools = [dev(p) for p in self.pools]
        stride, hq, hkv = self.fused.shape[1] * self.d, self.hq, self.hkv
        k, v = on[:, hq:], on[:, hq + hkv:]
        qo, so = (on, stride) if in_place else (dev(self.before), 0)
        q = None if keys_only else on
        P.photon_rope_cache_append(q, 0 if keys_only else stride, k, stride, v, stride, dev(self.pos),
                                   self.table, self.max_pos, self.rotary, self.pairs,
                                   dev(self.slots), self.T, None if keys_only else qo, so, *pools,
                                   self.shape, stream)
        pools = [host(p, h) for p, h in zip(pools, self.pools)]
        if in_place:
            back = host(on, self.fused)
            assert np.array_equal(bits(back[:, hq:]), bits(self.fused[:, hq:]))
            return back[:, :hq], *pools
        return host(qo, self.before), *pools

    def turned(self, x):
        """(z, fp32 bound) of rows x [T][h][d] in 64 bits."""
        half = self.rotary // 2
        i = np.arange(half)
        a, b = (2 * i, 2 * i + 1) if self.pairs else (i, i + half)
        ok = (self.pos >= 0) & (self.pos < self.max_pos)
        t = self.table.cpu().numpy().astype(np.float64)[np.where(ok, self.pos, 0)][:, None]
        cos = np.where(ok[:, None, None], t[..., 0], 1.0)
        sin = np.where(ok[:, None, None], t[..., 1], 0.0)
        z, m = x.copy(), np.zeros_like(x)
        z[..., a], z[..., b] = x[..., a] * cos - x[..., b] * sin, x[..., b] * cos + x[..., a] * sin
        m[..., a] = m[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * ok[:, None, None]
        return z, m * 3 * 2.0 ** -24

    def check(self, got, keys_only=False):
        q, kc, vc = got
        hq, hkv = self.hq, self.hkv
        x = I.to_f64(self.fused, self.dtype)
        z, m = self.turned(x)
        bound = m + I.EPS[self.dtype] / 2 * (np.abs(z) + m) * (m > 0) + TINY[self.dtype] * (m > 0)
        there = self.pos >= 0
        off = np.abs(I.to_f64(q, self.dtype) - z[:, :hq])
        if not keys_only:
            assert (off <= bound[:, :hq])[there].all(), off[there].max()
        left = q if keys_only else q[~there]
        assert np.array_equal(bits(left), bits(self.before if keys_only else self.before[~there]))
        want_k, want_v = I.to_f64(self.pools[0], self.dtype), self.pools[1].copy()
        bound_k = np.zeros_like(want_k)
        for t in range(self.T):
            s = self.slots[t]
            if there[t] and 0 <= s < self.NB * 16:
                want_k[s // 16, :, s % 16] = z[t, hq:hq + hkv]
                bound_k[s // 16, :, s % 16] = bound[t, hq:hq + hkv]
                want_v[s // 16, :, s % 16] = self.fused[t, hq + hkv:hq + 2 * hkv]
        assert np.array_equal(bits(vc), bits(want_v))
        assert (np.abs(I.to_f64(kc, self.dtype) - want_k) <= bound_k).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pairs", [0, 1])
@pytest.mark.parametrize("T,hq,hkv,d,rotary", [
    (1, 1, 1, 64, 64), (5, 4, 2, 128, 128), (33, 16, 8, 128, 64), (17, 8, 1, 64, 16),
    (70, 32, 8, 64, 32), (9, 40, 5, 128, 112), (3, 24, 3, 128, 48)])
def test_layouts_and_parts(dtype, pairs, T, hq, hkv, d, rotary):
    c = Case(T=T, hq=hq, hkv=hkv, d=d, dtype=dtype, rotary=rotary, pairs=pairs, seed=T)
    c.check(c.run())
    assert P.photon_get_last_device_error()[0] == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pairs", [0, 1])
def test_in_place_strides_and_keys_alone(dtype, pairs):
    c = Case(T=19, hq=8, hkv=4, d=128, dtype=dtype, rotary=96, pairs=pairs, extra=3, seed=2)
    out = c.run()
    c.check(out)
    for a, b in zip(out, c.run(in_place=True)):
        assert np.array_equal(bits(a), bits(b))
    alone = c.run(keys_only=True)
    c.check(alone, keys_only=True)
    for a, b in zip(out[1:], alone[1:]):
        assert np.array_equal(bits(a), bits(b))


def test_padding_and_what_lies_outside():
    c = Case(T=12, hq=4, hkv=2, d=64, dtype=W.DTYPE_F16, rotary=64, pairs=0, seed=4)
    c.pos[[3, 11]] = [-1, -7]       # padding, with and without a slot
    c.slots[[3, 5]] = [-1, -9]      # a token that is not stored
    c.fused[11] = np.nan            # padding is not looked at
    c.check(c.run())
    assert P.photon_get_last_device_error()[0] == 0
    c.slots[7] = c.NB * 16
    c.check(c.run())
    assert P.photon_get_last_device_error() == (6, 2)
    c.pos[8] = c.max_pos
    c.fused[8, :, 5] = np.inf       # unturned is not turned by no angle
    c.slots[7] = 1 << 40
    q, kc, vc = c.run()
    assert P.photon_get_last_device_error() == (6, 18)
    assert np.array_equal(bits(q[8]), bits(c.fused[8, :4]))
    s = c.slots[8]
    assert np.array_equal(bits(kc[s // 16, :, s % 16]), bits(c.fused[8, 4:6]))


def test_an_infinity_keeps_to_its_pair():
    c = Case(T=3, hq=2, hkv=1, d=64, dtype=W.DTYPE_F32, rotary=32, pairs=1, seed=6)
    c.pos[:] = [1, 2, 3]
    c.fused[1, 0, 4] = np.inf
    c.fused[2, 1, 40] = np.nan
    q = c.run()[0]
    bad = ~np.isfinite(q)
    want = np.zeros_like(bad)
    want[1, 0, 4:6] = want[2, 1, 40] = True
    assert np.array_equal(bad, want)


def test_offsets_past_32_bits():
    """Rows 4 MB apart and a pool of more than 4 GiB, whose last slots are written."""
    c = Case(T=1100, hq=4, hkv=2, d=64, dtype=W.DTYPE_F16, rotary=64, pairs=0, seed=9, NB=80)
    stride, width, NB = 1 << 21, 8 * 64, 1200000
    big = torch.empty((c.T, stride), dtype=torch.float16, device="cuda")
    big[:, :width] = dev(c.fused).reshape(c.T, width)
    kc = torch.zeros((NB, 2, 16, 64), dtype=torch.float16, device="cuda")   # 4.9 GB
    vc = torch.zeros_like(kc)
    far = (NB - 80) * 16
    qo = dev(c.before)
    c.shape.num_blocks = NB
    P.photon_rope_cache_append(big, stride, big[:, 256:], stride, big[:, 384:], stride, dev(c.pos),
                               c.table, c.max_pos, 64, 0, dev(c.slots + far), c.T, qo, 0, kc, vc,
                               c.shape)
    assert not kc[:NB - 80].any() and not vc[:NB - 80].any()
    c.pools = [np.zeros_like(p) for p in c.pools]
    c.check([host(qo, c.before), host(kc[-80:], c.pools[0]), host(vc[-80:], c.pools[1])])


def test_captured_and_on_another_stream():
    c = Case(T=9, hq=4, hkv=2, d=64, dtype=W.DTYPE_F16, rotary=64, pairs=0, seed=8)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = c.run()
    c.check(got)
    on, stride = dev(c.fused), 8 * 64
    qo, pools = dev(c.before), [dev(p) for p in c.pools]
    pos, slots = dev(c.pos), dev(c.slots)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.photon_rope_cache_append(on, stride, on[:, 4:], stride, on[:, 6:], stride, pos, c.table,
                                   c.max_pos, 64, 0, slots, 9, qo, 0, *pools, c.shape)
    c.pos = (c.pos + 77) % c.max_pos
    c.slots = np.roll(c.slots, 2)
    pos.copy_(dev(c.pos))
    slots.copy_(dev(c.slots))
    graph.replay()
    torch.cuda.synchronize()
    c.check([host(qo, c.before), *[host(p, h) for p, h in zip(pools, c.pools)]])
