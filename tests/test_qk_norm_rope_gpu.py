"""photon_qk_norm_rope against its formula in 64 bits.  Bounds: the output's
rounding (eps / 2 of |z|), and fp32 arithmetic before it: the sum of squares
(head_dim + 5 additions of positive terms, 2^-24 each, halved by the root), the
root, reciprocal and products of the norm, and two products and a sum of the
rotation: (133 / 2 + 8) x 2^-24 < 2^-17 of |y[k]| + |y[k + r/2]|."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import int4_util as I
import paged_kv_attention_photon_gb300 as P
import workloads as W
from gpu_util import dev, host, rope_table

pytestmark = pytest.mark.gpu
BASE = 1e4


def axis_of(sections, dealt):
    half, n = sum(sections), len(sections)
    axis = np.zeros(half, dtype=int)
    if dealt:
        for a in range(1, n):
            for i in range(sections[a]):
                axis[a + n * i] = a
    else:
        axis = np.repeat(np.arange(n), sections)
    return axis


def formula(x, weight, eps, pos, table, sections, dealt, max_pos):
    """x [T][H][d] and weight in 64 bits -> (z, bound without the output's rounding)."""
    half = sum(sections)
    y = x if weight is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    axis = axis_of(sections, dealt)
    ok = ((pos >= 0) & (pos < max_pos)).all(0)
    turn = table[np.where(ok, pos, 0)[axis].T, np.arange(half)]        # [T][half][2]
    cos, sin = turn[:, None, :, 0], turn[:, None, :, 1]
    z = y.copy()
    a, b = y[..., :half], y[..., half:2 * half]
    z[..., :half] = a * cos - b * sin
    z[..., half:2 * half] = b * cos + a * sin
    z = np.where(ok[:, None, None], z, y)
    mag = np.abs(y).copy()
    mag[..., :half] += np.abs(b)
    mag[..., half:2 * half] += np.abs(a)
    return z, mag * 2.0 ** -17


class Case:
    def __init__(self, *, T, hq, hkv, d, dtype, sections, dealt=False, seed=0, extra=0,
                 max_pos=512, size=1.0, norm=True, eps=1e-6):
        rng = np.random.default_rng(seed)
        self.__dict__.update(T=T, hq=hq, hkv=hkv, d=d, dtype=dtype, sections=sections, dealt=dealt,
                             max_pos=max_pos, eps=eps)
        self.fused = I.narrow(rng.standard_normal((T, hq + hkv + extra, d)) * size, dtype)
        self.w = [I.narrow(1 + 0.2 * rng.standard_normal(d), dtype) if norm else None
                  for _ in range(2)]
        self.pos = rng.integers(0, max_pos, (len(sections), T)).astype(np.int32)
        self.table = rope_table(BASE, max_pos, 2 * sum(sections))
        self.shape = P.PagedShape.make(num_seqs=0, num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                                       num_blocks=0, max_blocks_per_seq=1, dtype=dtype)

    def run(self, in_place=False, stream=None):
        on = dev(self.fused)
        stride = self.fused.shape[1] * self.d
        q, k = on, on[:, self.hq:]
        if in_place:
            qo, ko, so = q, k, stride
        else:
            qo = torch.full((self.T, self.hq, self.d), -1, dtype=on.dtype, device="cuda")
            ko = torch.full((self.T, self.hkv, self.d), -1, dtype=on.dtype, device="cuda")
            so = 0
        w = [None if x is None else dev(x) for x in self.w]
        P.photon_qk_norm_rope(q, stride, k, stride, *w, self.eps, dev(self.pos), self.table,
                              self.max_pos, P.RopeAxes.make(self.sections, self.dealt), self.T, qo,
                              so, ko, so, self.shape, stream)
        if in_place:
            back = host(on, self.fused)
            assert np.array_equal(back[:, self.hq + self.hkv:].view(np.uint8),
                                  self.fused[:, self.hq + self.hkv:].view(np.uint8))
            return [I.to_f64(x, self.dtype) for x in (back[:, :self.hq],
                                                      back[:, self.hq:self.hq + self.hkv])]
        return [I.to_f64(host(t, self.fused[:, :n]), self.dtype)
                for t, n in ((qo, self.hq), (ko, self.hkv))]

    def want(self):
        x = I.to_f64(self.fused, self.dtype)
        table = self.table.cpu().numpy().astype(np.float64)
        w = [None if v is None else I.to_f64(v, self.dtype) for v in self.w]
        return [formula(y, v, self.eps, self.pos, table, self.sections, self.dealt, self.max_pos)
                for y, v in ((x[:, :self.hq], w[0]), (x[:, self.hq:self.hq + self.hkv], w[1]))]

    def check(self, got, rows=slice(None)):
        for g, (z, b) in zip(got, self.want()):
            bound = b + I.EPS[self.dtype] / 2 * (np.abs(z) + b) + \
                (2.0 ** -25 if self.dtype == W.DTYPE_F16 else 2.0 ** -134)
            assert np.isfinite(g[rows]).all()
            assert (np.abs(g - z) <= bound)[rows].all(), np.abs(g - z)[rows].max()


@pytest.mark.parametrize("dtype", [W.DTYPE_F32, W.DTYPE_F16, W.DTYPE_BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,hq,hkv", [(1, 1, 1), (5, 4, 2), (33, 16, 4), (7, 40, 5), (130, 8, 1)])
def test_one_axis(dtype, d, T, hq, hkv):
    c = Case(T=T, hq=hq, hkv=hkv, d=d, dtype=dtype, sections=[d // 2], seed=T)
    c.check(c.run())
    assert P.photon_get_last_device_error()[0] == 0


@pytest.mark.parametrize("dtype", [W.DTYPE_F32, W.DTYPE_BF16])
@pytest.mark.parametrize("d,sections,dealt", [
    (128, [24, 20, 20], False), (128, [24, 20, 20], True), (64, [16, 16], False),
    (64, [12, 10, 10], True), (128, [0, 32, 32], False), (128, [10, 10, 10, 10], True),
    (64, [5, 1, 1, 1], False), (128, [48], False), (128, [8], False), (64, [8, 8], True)])
def test_several_axes_and_partial_rotation(dtype, d, sections, dealt):
    c = Case(T=21, hq=4, hkv=2, d=d, dtype=dtype, sections=sections, dealt=dealt, seed=d)
    c.check(c.run())
    assert P.photon_get_last_device_error()[0] == 0


@pytest.mark.parametrize("dtype", [W.DTYPE_F32, W.DTYPE_F16])
def test_strides_in_place_and_without_a_norm(dtype):
    c = Case(T=19, hq=8, hkv=4, d=128, dtype=dtype, sections=[64], extra=4, seed=2)
    out = c.run()
    c.check(out)
    for a, b in zip(out, c.run(in_place=True)):
        assert np.array_equal(a, b)
    c = Case(T=19, hq=8, hkv=4, d=64, dtype=dtype, sections=[32], extra=1, seed=3, norm=False)
    c.check(c.run(in_place=True))
    c.w[0] = I.narrow(np.ones(64), dtype)     # a norm on q alone
    c.check(c.run())


def test_padding_and_positions_outside_the_table():
    c = Case(T=12, hq=4, hkv=2, d=64, dtype=W.DTYPE_F16, sections=[16, 16], seed=4)
    c.pos[0, [3, 11]] = -1          # padding: outputs as they were
    c.pos[1, 11] = -9
    got = c.run()
    assert P.photon_get_last_device_error()[0] == 0
    rows = np.setdiff1d(np.arange(12), [3, 11])
    c.check(got, rows)
    for g in got:
        assert (g[[3, 11]] == -1).all()
    c.pos[0, 5], c.pos[1, 6] = c.max_pos, -1   # outside: normed, not turned
    got = c.run()
    assert P.photon_get_last_device_error() == (6, 16)
    c.check(got, rows)
    # unturned is not turned by no angle: an infinity keeps to its own element
    c.w = [None, None]
    c.fused[5, 0, 3] = np.inf
    got = c.run()[0][5, 0]
    assert P.photon_get_last_device_error() == (6, 16)
    assert np.array_equal(got, I.to_f64(c.fused[5, 0], c.dtype))


@pytest.mark.parametrize("dtype,size", [(W.DTYPE_BF16, 2.0 ** 100), (W.DTYPE_F32, 2.0 ** 120),
                                        (W.DTYPE_BF16, 2.0 ** -100), (W.DTYPE_F32, 2.0 ** -80),
                                        (W.DTYPE_F16, 2.0 ** 13), (W.DTYPE_F16, 2.0 ** -12)])
def test_squares_that_leave_fp32(dtype, size):
    c = Case(T=6, hq=4, hkv=2, d=128, dtype=dtype, sections=[64], seed=6, size=size, eps=0.0)
    c.check(c.run())
    c.eps = 1e-6
    c.check(c.run())


def test_zero_rows_and_rows_that_are_not_finite():
    c = Case(T=4, hq=4, hkv=2, d=64, dtype=W.DTYPE_F32, sections=[32], seed=7)
    c.fused[1, 2] = 0.0
    c.fused[2, 0, 5] = np.nan
    got = c.run()
    assert not got[0][1, 2].any()
    bad = np.isnan(got[0]).any(-1)
    want = np.zeros((4, 4), bool)
    want[2, 0] = True
    assert np.array_equal(bad, want) and np.isfinite(got[1]).all()


def test_offsets_past_32_bits():
    """Rows 4 MB apart, in place: the last ones lie more than 4 GiB behind the first."""
    c = Case(T=1100, hq=4, hkv=2, d=64, dtype=W.DTYPE_F16, sections=[32], seed=9)
    stride, width = 1 << 21, 6 * 64
    big = torch.empty((c.T, stride), dtype=torch.float16, device="cuda")
    big[:, :width] = dev(c.fused).reshape(c.T, width)
    k = big[:, 4 * 64:]
    P.photon_qk_norm_rope(big, stride, k, stride, dev(c.w[0]), dev(c.w[1]), c.eps, dev(c.pos),
                          c.table, c.max_pos, P.RopeAxes.make([32]), c.T, big, stride, k, stride,
                          c.shape)
    got = I.to_f64(host(big[:, :width].reshape(c.T, 6, 64), c.fused), c.dtype)
    c.check([got[:, :4], got[:, 4:]])


def test_captured_and_on_another_stream():
    c = Case(T=9, hq=4, hkv=2, d=64, dtype=W.DTYPE_F16, sections=[32], seed=8)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = c.run()
    c.check(got)
    on, stride = dev(c.fused), c.fused.shape[1] * c.d
    qo = torch.zeros((9, 4, 64), dtype=on.dtype, device="cuda")
    ko = torch.zeros((9, 2, 64), dtype=on.dtype, device="cuda")
    w, pos = [dev(x) for x in c.w], dev(c.pos)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.photon_qk_norm_rope(on, stride, on[:, 4:], stride, *w, c.eps, pos, c.table, c.max_pos,
                              P.RopeAxes.make([32]), 9, qo, 0, ko, 0, c.shape)
    c.pos = (c.pos + 77) % c.max_pos
    pos.copy_(dev(c.pos))
    graph.replay()
    torch.cuda.synchronize()
    c.check([I.to_f64(host(t, c.fused[:, :n]), c.dtype) for t, n in ((qo, 4), (ko, 2))])
