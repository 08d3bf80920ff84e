"""photon_prompt_attention against causal softmax attention in 64 bits.

Bound, for finite inputs: with A = log2(e) |scale| sum |q| max |k|, a score is
off by at most 2^-22 A (fp32 accumulation of head_dim products, the tensor
cores keep at least 22 bits), which the weights' quotient turns into 2 ln 2
2^-22 A of the largest |v|; each weight is rounded to the storage type, half a
step, eps / 2 of itself, and the exponentials and sums add 2^-18; then one
rounding of the output, eps / 2 of it."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import int4_util as I
import paged_kv_attention_photon_gb300 as P
import workloads as W
from gpu_util import dev, host

pytestmark = pytest.mark.gpu
TYPES = [W.DTYPE_F16, W.DTYPE_BF16]


def attention(q, k, v, starts, scale, eps):
    """(out, bound) in 64 bits; rows of no prompt are NaN."""
    T, hq, d = q.shape
    G = hq // k.shape[1]
    out = np.full((T, hq, d), np.nan)
    bound = np.zeros((T, hq, 1))
    for s, e in zip(starts[:-1], starts[1:]):
        for h in range(hq if e > s else 0):
            kk, vv, qq = k[s:e, h // G], v[s:e, h // G], q[s:e, h]
            x = scale * (qq @ kk.T)
            x[np.triu_indices(e - s, 1)] = -np.inf
            p = np.exp(x - x.max(-1, keepdims=True))
            out[s:e, h] = (p @ vv) / p.sum(-1, keepdims=True)
            mag = 1.4427 * abs(scale) * np.abs(qq).sum(-1) * np.abs(kk).max()
            loss = 2 * np.log(2) * 2.0 ** -22 * mag + eps / 2 + 2.0 ** -18
            bound[s:e, h, 0] = loss * np.abs(vv).max()
    bound = bound + eps / 2 * (np.abs(np.nan_to_num(out)) + bound) + 2.0 ** -25
    return out, bound


class Case:
    def __init__(self, lens, hq, hkv, d, dtype, *, seed=0, tail=0, lead=0, fused=False, size=1.0):
        rng = np.random.default_rng(seed + sum(lens))
        self.starts = (lead + np.concatenate([[0], np.cumsum(lens)])).astype(np.int32)
        self.T = int(self.starts[-1]) + tail
        self.dtype, self.hq, self.hkv, self.d = dtype, hq, hkv, d
        self.all = I.narrow(rng.standard_normal((self.T, hq + 2 * hkv, d)) * size, dtype)
        self.fused, self.scale = fused, d ** -0.5
        self.longest = max(lens, default=0)
        self.shape = P.PagedShape.make(num_seqs=len(lens), num_q_heads=hq, num_kv_heads=hkv,
                                       head_dim=d, num_blocks=0, max_blocks_per_seq=1, dtype=dtype)
        self.up()

    def parts(self):
        h = self.hq
        return self.all[:, :h], self.all[:, h:h + self.hkv], self.all[:, h + self.hkv:]

    def up(self):
        if self.fused:
            on = dev(self.all)
            self.on = [on, on[:, self.hq:], on[:, self.hq + self.hkv:]]
            self.stride = self.all.shape[1] * self.d
        else:
            self.on = [dev(x) for x in self.parts()]
            self.stride = 0
        self.out = torch.full((self.T, self.hq, self.d), -1, dtype=torch.int16, device="cuda")
        self.on_starts = dev(self.starts)

    def run(self, stream=None, longest=None):
        q, k, v = self.on
        P.photon_prompt_attention(q, self.stride, k, self.stride, v, self.stride, self.on_starts,
                                  self.T, self.longest if longest is None else longest, self.scale,
                                  self.out, 0, self.shape, stream)

    def raw(self):
        return self.out.cpu().numpy()

    def check(self, starts=None, skip=()):
        """Every prompt's rows within the bound, every other row as it was."""
        st, bits = P.photon_get_last_device_error()
        assert st == 0, bits
        self.compare(self.starts if starts is None else starts, skip)

    def compare(self, starts, skip=()):
        q, k, v = (I.to_f64(x, self.dtype) for x in self.parts())
        want, bound = attention(q, k, v, starts, self.scale, I.EPS[self.dtype])
        got = I.to_f64(host(self.out, self.parts()[0]), self.dtype)
        mine = ~np.isnan(want).any((1, 2))
        for b in skip:
            mine[starts[b]:starts[b + 1]] = False
        assert np.isfinite(got[mine]).all()
        over = (np.abs(got - want) - bound)[mine]
        assert over.max(initial=-1) <= 0, f"{over.max()} over the bound"
        assert (self.raw()[~mine] == -1).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (8, 2), (8, 1)])
def test_one_prompt_of_each_length(dtype, d, hq, hkv):
    for n in (1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 400):
        c = Case([n], hq, hkv, d, dtype)
        c.run()
        c.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fused", [False, True])
def test_ragged(dtype, d, fused):
    c = Case([5, 0, 130, 1, 1, 300, 0, 64, 77, 0], 4, 2, d, dtype, tail=9, lead=3, fused=fused)
    c.run()
    c.check()
    c.run(longest=5000)     # only an upper bound
    c.check()


def test_many_prompts():
    """More prompts than lanes, more items than SMs, rounds of items per CTA."""
    rng = np.random.default_rng(1)
    lens = [int(x) for x in rng.integers(0, 60, 150)]
    lens[40:80] = [0] * 40
    lens[3] = 700
    c = Case(lens, 8, 4, 64, W.DTYPE_BF16, tail=1)
    c.run()
    c.check()


@pytest.mark.parametrize("d,dtype", [(64, W.DTYPE_F16), (128, W.DTYPE_BF16)])
def test_long_prompt(d, dtype):
    c = Case([2500], 4, 1, d, dtype)
    c.run()
    c.check()


def test_all_sms_busy():
    c = Case([1024] * 5 + [777], 16, 8, 64, W.DTYPE_F16, fused=True)
    c.run()
    c.check()


@pytest.mark.parametrize("scale", [0.0, -0.2, 2.0])
def test_scales(scale):
    c = Case([140, 40], 4, 2, 64, W.DTYPE_F16)
    c.scale = scale
    c.run()
    c.check()


def test_growing_scores():
    """Keys that grow along the prompt move the running maximum in every chunk."""
    c = Case([600], 4, 2, 128, W.DTYPE_F16)
    grow = np.linspace(0.01, 12, 600)[:, None, None]
    c.all[:, 4:6] = I.narrow(np.abs(I.to_f64(c.all[:, 4:6], c.dtype)) * grow, c.dtype)
    c.all[:, :4] = I.narrow(np.abs(I.to_f64(c.all[:, :4], c.dtype)), c.dtype)
    c.up()
    c.run()
    c.check()


def test_neighbours_that_are_not_finite():
    """NaN and infinite rows of q, k and v beside a prompt (another prompt, lead and tail rows)
    do not reach it."""
    c = Case([70, 33, 65], 4, 2, 128, W.DTYPE_F16, lead=4, tail=6)
    s = c.starts
    c.all[:s[0]] = np.nan
    c.all[s[3]:] = np.inf
    c.all[s[1]:s[2]] = np.nan
    c.up()
    c.run()
    assert P.photon_get_last_device_error()[0] == 0
    got = I.to_f64(host(c.out, c.parts()[0]), c.dtype)
    q, k, v = (np.nan_to_num(I.to_f64(x, c.dtype), posinf=0) for x in c.parts())
    want, bound = attention(q, k, v, s, c.scale, I.EPS[c.dtype])
    for b in (0, 2):
        rows = slice(s[b], s[b + 1])
        assert (np.abs(got - want) <= bound)[rows].all()
    assert np.isnan(got[s[1]:s[2]]).all()
    assert (c.raw()[:s[0]] == -1).all() and (c.raw()[s[3]:] == -1).all()


def test_rejected_prompts():
    c = Case([30, 40, 50], 4, 2, 64, W.DTYPE_F16)
    c.run(longest=40)       # the last one is longer
    assert P.photon_get_last_device_error() == (6, 32)
    c.compare(np.array([0, 30, 70], np.int32))
    for bad in ([0, 30, 70, 121], [-1, 30, 70, 120], [0, 30, 20, 20]):
        c.up()
        c.on_starts = dev(np.array(bad, np.int32))
        c.run()
        assert P.photon_get_last_device_error() == (6, 32), bad
    assert (c.raw()[30:] == -1).all()


def test_offsets_past_32_bits():
    """Rows 4 MB apart: the last ones lie more than 4 GiB behind the first."""
    c = Case([1000, 0, 110], 4, 2, 64, W.DTYPE_F16, fused=True)
    width, c.stride = c.all.shape[1] * c.d, 1 << 21
    big = torch.empty((c.T, c.stride), dtype=torch.float16, device="cuda")
    big[:, :width] = c.on[0].reshape(c.T, width)
    out = big[:, width:width + c.hq * c.d]
    out.fill_(0)
    at = [big, big[:, c.hq * c.d:], big[:, (c.hq + c.hkv) * c.d:]]
    P.photon_prompt_attention(at[0], c.stride, at[1], c.stride, at[2], c.stride, c.on_starts, c.T,
                              c.longest, c.scale, out, c.stride, c.shape)
    c.out.copy_(out.contiguous().view(torch.int16).reshape(c.out.shape))
    c.check()


def test_two_streams_at_once():
    cases = [Case([300, 90, 700], 8, 4, 128, W.DTYPE_F16), Case([500] * 4, 8, 2, 64, W.DTYPE_BF16)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, stream in zip(cases, streams):
            c.run(stream)
    torch.cuda.synchronize()
    for c in cases:
        c.check()


def test_captured_and_on_another_stream():
    c = Case([100, 60], 4, 2, 64, W.DTYPE_F16, tail=40)
    e = Case([90], 8, 1, 128, W.DTYPE_BF16)
    c.run(), e.run()
    c.longest = 200
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(), e.run()
    c.starts = np.array([0, 3, 200], np.int32)
    c.on_starts.copy_(dev(c.starts))
    c.out.fill_(-1)
    for _ in range(2):
        graph.replay()
    c.check()
    e.check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.out.fill_(-1)
        c.run()
    side.synchronize()
    c.check()


def test_equal_to_the_paged_prefill():
    """The same prompts through a paged 16-bit cache and photon_paged_multi_query."""
    lens, hq, hkv, d = [200, 64, 129], 8, 4, 128
    c = Case(lens, hq, hkv, d, W.DTYPE_F16)
    c.run()
    mbs = (max(lens) + 15) // 16
    nb = 3 * mbs
    bt = np.random.default_rng(0).permutation(nb).astype(np.int32).reshape(3, mbs)
    slots = np.concatenate([bt[b][np.arange(n) // 16].astype(np.int64) * 16 + np.arange(n) % 16
                            for b, n in enumerate(lens)])
    shape = P.PagedShape.make(num_seqs=3, num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                              num_blocks=nb, max_blocks_per_seq=mbs, dtype=W.DTYPE_F16)
    pools = [torch.zeros((nb, hkv, 16, d), dtype=torch.float16, device="cuda") for _ in range(2)]
    P.photon_cache_write(c.on[1], c.on[2], dev(slots), c.T, *pools, shape)
    nws = P.photon_paged_multi_query_workspace_size(shape, c.T, max(lens))
    ws = torch.empty(max(nws, 16), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(c.on[0])
    P.photon_paged_multi_query(c.on[0], *pools, dev(bt), dev(np.array(lens, np.int32)), c.on_starts,
                               c.T, max(lens), c.scale, out, ws, nws, shape)
    got = I.to_f64(host(c.out, c.parts()[0]), c.dtype)
    assert np.abs(got - out.double().cpu().numpy()).max() <= 4e-3


@pytest.mark.parametrize("longest", [None, 1 << 20])
@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 64), (8, 4, 128)])
def test_a_thousand_prompts(hq, hkv, d, longest):
    """Items found 32 prompts at a time over many rounds: short prompts, empty and rejected ones
    in long runs, and tile indices that only a few far apart prompts have."""
    rng = np.random.default_rng(12)
    lens = [int(x) for x in rng.integers(1, 40, 1100)]
    lens[64:200] = [0] * 136
    for b, n in ((0, 300), (33, 1500), (500, 700), (501, 700), (1099, 1100)):
        lens[b] = n
    c = Case(lens, hq, hkv, d, W.DTYPE_F16, tail=3)
    c.run(longest=longest)
    c.check()
    # all but the short ones are longer than the bound: rejected, their rows left as they were
    c.up()
    c.run(longest=299)
    assert P.photon_get_last_device_error() == (6, 32)
    keep = np.array([n < 300 for n in lens])
    q, k, v = (I.to_f64(x, c.dtype) for x in c.parts())
    want, bound = attention(q, k, v, c.starts, c.scale, I.EPS[c.dtype])
    mine = np.concatenate([np.repeat(keep, lens), [False] * 3])
    got = I.to_f64(host(c.out, c.parts()[0]), c.dtype)
    assert (np.abs(got - want) <= bound)[mine].all()
    assert (c.raw()[~mine] == -1).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("hq,hkv,d", [(2, 1, 64), (8, 2, 128)])
@pytest.mark.parametrize("nats", [12.0, 17.0, 17.75])
def test_many_keys_of_little_weight(dtype, hq, hkv, d, nats):
    """A prompt's first key holds nearly all of the weight and has a small v; each key behind it
    weighs e^-nats, next to what fp16 can hold, and has an ordinary v.

    Bound: a weight is rounded to the storage type, eps / 2 of itself, or where fp16 ends by half
    of 2^-24 below weights of 2^7 at least; exponentials, and sums of n / 16 products of 16 keys in
    fp32, 2^-22 a product; then the output's rounding."""
    n = 9000
    c = Case([n], hq, hkv, d, dtype)
    c.scale = 8.0 / d
    x = I.to_f64(c.all, dtype)
    x[:, :hq] = 1.0
    x[:, hq:hq + hkv] = 0.0
    x[0, hq:hq + hkv] = nats / 8                # exact: the scores are nats and 0
    x[0, hq + hkv:] *= 0.003
    x[1:, hq + hkv:] = np.abs(x[1:, hq + hkv:])
    c.all = I.narrow(x, dtype)
    c.up()
    c.run()
    assert P.photon_get_last_device_error()[0] == 0
    got = I.to_f64(host(c.out, c.parts()[0]), dtype)
    v = I.to_f64(c.all, dtype)[:, hq + hkv:]
    w = np.full((n, 1, 1), np.exp(-nats))
    w[0] = 1.0
    total, size = np.cumsum(w, 0), np.cumsum(w * np.abs(v), 0)
    want = np.cumsum(w * v, 0) / total
    keys = np.arange(1, n + 1)[:, None, None]
    eps = I.EPS[dtype] / 2
    bound = (eps + 2.0 ** -20 + keys / 16 * 2.0 ** -22) * 2 * size / total
    if dtype == W.DTYPE_F16:
        bound += keys * 2.0 ** -32 * np.abs(v).max()
    bound += eps * (np.abs(want) + bound) + 2.0 ** -25
    want, bound = (np.repeat(y, hq // hkv, 1) for y in (want, bound))
    assert (np.abs(got - want) <= bound).all(), (np.abs(got - want) / bound).max()


def test_repeated_calls_give_the_same_bits():
    for c in (Case([700, 1, 90, 400, 33] * 9, 8, 4, 128, W.DTYPE_F16),
              Case([513, 64, 2, 1000], 16, 4, 64, W.DTYPE_BF16)):
        c.run()
        c.check()
        first = c.out.clone()
        for _ in range(10):
            c.out.fill_(-1)
            c.run()
            assert torch.equal(c.out, first)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 64), (8, 1, 128)])
@pytest.mark.parametrize("size", [1e3, 2e5, 7e6, 3e7, 1e8, 1e9, 1e10])
def test_scores_far_from_zero(dtype, hq, hkv, d, size):
    """Scores of that size (log2 domain), so far apart that only the keys of the largest one so far
    weigh anything; those are equal, and a row is the mean of their v.  Constant k rows, so equal
    rows have equal scores whatever the products lose."""
    n = 400
    c = Case([n], hq, hkv, d, dtype)
    rng = np.random.default_rng(int(size) % 1000 + d)
    ladder = np.array([0.25, 0.5, 0.625, 0.75, 0.875, 1.0]) * 1.37
    pick = np.sort(rng.integers(0, len(ladder), n))
    pick[rng.integers(0, n, n // 3)] = 0
    x = I.to_f64(c.all, dtype)
    x[:, :hq] = 3.0 + np.arange(hq)[:, None] / 4
    x[:, hq:hq + hkv] = ladder[pick][:, None, None]
    c.all = I.narrow(x, dtype)
    v = np.repeat(I.to_f64(c.all, dtype)[:, hq + hkv:], hq // hkv, 1)
    for sign in (1, -1):     # a negative scale turns the ladder round
        c.scale = sign * size / (1.4427 * 1.37 * 3.0 * d)
        c.up()
        c.run()
        assert P.photon_get_last_device_error()[0] == 0
        got = I.to_f64(host(c.out, c.parts()[0]), dtype)
        for i in range(n):
            seen = pick[:i + 1]
            want = v[:i + 1][seen == (seen.max() if sign > 0 else seen.min())].mean(0)
            # equal weights, each rounded (eps / 2); sums of up to n of them, 2^-22 each
            tol = (I.EPS[dtype] / 2 + n * 2.0 ** -22) * np.abs(v).max()
            tol = tol + I.EPS[dtype] / 2 * (np.abs(want) + tol) + 2.0 ** -25
            assert (np.abs(got[i] - want) <= tol).all(), (sign, i, np.abs(got[i] - want).max())
