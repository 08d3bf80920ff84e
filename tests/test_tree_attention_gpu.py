"""photon_paged_tree_attention against softmax attention in 64 bits over the keys that each
node sees.  The bound stands with the definition in tree_util.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import int4_util as I
import paged_kv_attention_photon_gb300 as P
import tree_util as T
import workloads as W
from gpu_util import dev, host

pytestmark = pytest.mark.gpu
TYPES = [W.DTYPE_F16, W.DTYPE_BF16]


class Case:
    """Sequences of (tokens before the tree, nodes); what no context holds is NaN."""

    def __init__(self, seqs, hq, hkv, d, dtype, *, kind="tree", seed=0, tail=0, lead=0, scale=None,
                 size=1.0, spare=4):
        rng = np.random.default_rng(seed + 7 * len(seqs) + sum(a + b for a, b in seqs))
        self.hq, self.hkv, self.d, self.dtype = hq, hkv, d, dtype
        self.n = np.array([b for _, b in seqs], dtype=int)
        self.ctx = np.array([a + b for a, b in seqs], dtype=np.int32)
        self.starts = (lead + np.concatenate([[0], np.cumsum(self.n)])).astype(np.int32)
        self.T = int(self.starts[-1]) + tail
        self.longest = int(max(self.n, default=0))
        self.scale = d ** -0.5 if scale is None else scale
        self.parents = np.full(self.T, -5, dtype=np.int32)
        for s, n in zip(self.starts, self.n):
            self.parents[s:s + n] = T.random_parents(rng, n, kind)
        used = [-(-int(c) // 16) for c in self.ctx]
        self.mbs = max(max(used, default=1), 1)
        self.nb = sum(used) + spare
        order = rng.permutation(self.nb)
        self.tables = np.full((len(seqs), self.mbs), -1, dtype=np.int32)
        self.q = I.narrow(rng.standard_normal((self.T, hq, d)) * size, dtype)
        nan = I.narrow(np.array([np.nan]), dtype)[0]
        self.pools = [np.full((self.nb, hkv, 16, d), nan) for _ in range(2)]
        at = 0
        for b, u in enumerate(used):
            self.tables[b, :u] = order[at:at + u]
            at += u
            j = np.arange(self.ctx[b])
            for p in self.pools:
                p[self.tables[b, j // 16], :, j % 16] = I.narrow(
                    rng.standard_normal((len(j), hkv, d)) * size, dtype)
        self.up()

    def up(self):
        self.shape = P.PagedShape.make(num_seqs=len(self.n), num_q_heads=self.hq,
                                       num_kv_heads=self.hkv, head_dim=self.d, num_blocks=self.nb,
                                       max_blocks_per_seq=self.mbs, dtype=self.dtype)
        self.on = [dev(x) for x in (self.q, *self.pools, self.tables, self.ctx, self.starts,
                                    self.parents)]
        self.out = torch.full((self.T, self.hq, self.d), -1, dtype=torch.int16, device="cuda")
        self.bytes = P.photon_paged_tree_attention_workspace_size(self.shape, self.T, self.longest)
        self.ws = torch.full((max(self.bytes, 16),), 0xFF, dtype=torch.uint8, device="cuda")

    def run(self, stream=None, longest=None):
        P.photon_paged_tree_attention(*self.on, self.T, self.longest if longest is None else longest,
                                      self.scale, self.out, self.ws, self.bytes, self.shape, stream)

    def raw(self):
        return self.out.cpu().numpy()

    def values(self):
        raw = self.raw()
        return I.to_f64(raw.view(np.float16 if self.dtype == W.DTYPE_F16 else np.uint16), self.dtype)

    def want(self, b, **more):
        s, n, ctx = self.starts[b], self.n[b], self.ctx[b]
        k, v = (T.cached_rows(p, self.tables[b], ctx, self.dtype) for p in self.pools)
        return T.tree_attention(I.to_f64(self.q[s:s + n], self.dtype), k, v, self.parents[s:s + n],
                                self.scale, I.EPS[self.dtype], **more)

    def check(self, skip=(), only=None):
        got = self.values()
        for b in range(len(self.n)) if only is None else only:
            if b in skip or self.n[b] == 0:
                continue
            s, n = self.starts[b], self.n[b]
            want, bound = self.want(b)
            off = np.abs(got[s:s + n] - want)
            assert (off <= bound).all(), (b, int(n), int(self.ctx[b]), np.nanmax(off / bound))
        assert (self.raw()[:self.starts[0]] == -1).all()
        assert (self.raw()[self.starts[-1]:] == -1).all()

    def ok(self):
        assert P.photon_get_last_device_error() == (0, 0)


SHAPES = [(8, 8), (4, 2), (16, 4), (8, 1)]   # 1, 2, 4, 8 query heads a KV head


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", SHAPES)
def test_sizes_of_trees_and_contexts(hq, hkv, d, dtype):
    c = Case([(0, 1), (0, 5), (1, 1), (15, 2), (16, 8), (17, 16), (62, 2), (63, 9), (100, 31),
              (127, 1), (128, 32), (129, 33), (300, 64), (1000, 7), (70, 65), (511, 3)],
             hq, hkv, d, dtype, tail=3)
    c.run()
    c.check()
    c.ok()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", SHAPES)
def test_trees_of_more_rows_than_a_tile(hq, hkv, d, dtype):
    """Up to 256 nodes: two tiles, and with more heads several groups of them."""
    c = Case([(40, 127), (64, 128), (3, 129), (500, 200), (0, 255), (129, 256)], hq, hkv, d, dtype,
             seed=1)
    c.run()
    c.check()
    c.ok()


@pytest.mark.parametrize("kind", ["chain", "forest"])
@pytest.mark.parametrize("d", [64, 128])
def test_chains_and_forests(kind, d):
    c = Case([(7, 1), (30, 100), (90, 256), (0, 40), (257, 17)], 8, 2, d, W.DTYPE_BF16, kind=kind)
    c.run()
    c.check()
    c.ok()


@pytest.mark.parametrize("dtype", TYPES)
def test_one_long_context_over_every_sm(dtype):
    c = Case([(20011, 24)], 8, 2, 128, dtype)
    c.run()
    c.check()
    c = Case([(20011, 40)], 8, 1, 64, dtype)   # two tiles
    c.run()
    c.check()
    c.ok()


@pytest.mark.parametrize("seqs", [1, 3, 8, 19, 24, 40])
@pytest.mark.parametrize("d,ctx,n", [(128, 60, 9), (128, 400, 20), (64, 900, 33), (128, 1020, 4), (64, 1300, 70)])
def test_pairs_whole_and_split(seqs, d, ctx, n):
    """Fewer and more pairs than CTAs, contexts of 1 to 11 chunks: whole pairs, pairs over two
    CTAs, pairs over several, one and two rounds."""
    rng = np.random.default_rng(seqs)
    c = Case([(int(rng.integers(0, ctx + 1)), int(rng.integers(1, n + 1))) for _ in range(seqs - 1)] +
             [(ctx, n)], 16, 8, d, W.DTYPE_F16)
    c.run()
    c.check()
    c.ok()


@pytest.mark.parametrize("seqs", [4, 60])
@pytest.mark.parametrize("wider", [1, 60, 4000])
def test_tables_wider_than_any_context(seqs, wider):
    """A table of the longest context that there may be: any numbers behind a context's blocks."""
    rng = np.random.default_rng(wider)
    c = Case([(int(rng.integers(0, 300)), int(rng.integers(1, 20))) for _ in range(seqs)], 16, 8, 64,
             W.DTYPE_F16, seed=seqs)
    c.tables = np.concatenate([c.tables, rng.integers(-9, 2 ** 30, (seqs, wider), dtype=np.int32)], 1)
    c.mbs += wider
    c.up()
    c.run(longest=min(256, c.longest + wider))
    c.check()
    c.ok()


def test_many_short_sequences_and_empty_ones():
    rng = np.random.default_rng(3)
    seqs = [(int(rng.integers(0, 90)), int(rng.integers(0, 20))) for _ in range(400)]
    seqs[0] = seqs[399] = (50, 0)
    c = Case(seqs, 4, 2, 64, W.DTYPE_F16, lead=2, tail=9)
    c.run()
    c.check()
    c.ok()


def test_mixed_lengths_share_runs():
    rng = np.random.default_rng(4)
    seqs = [(int(np.exp(rng.uniform(0, 8.5))), int(rng.integers(1, 40))) for _ in range(40)]
    c = Case(seqs, 8, 2, 128, W.DTYPE_BF16)
    c.run()
    c.check()
    c.ok()
    first = c.raw()
    for _ in range(5):
        c.out.fill_(-1)
        c.run()
        assert np.array_equal(c.raw(), first)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ctx,lo,hi", [(60, 28, 40), (900, 28, 127)])
def test_items_of_one_tile_and_of_two_in_turn(d, ctx, lo, hi):
    """Each CTA has several items of few chunks: those of one tile's rows, which the other tile
    passes over, before and after those of both tiles' rows.  Calls in a row, on either of two
    batches."""
    rng = np.random.default_rng(ctx + d)
    both = []
    for _ in range(2):
        seqs = [(int(np.exp(rng.uniform(2, np.log(ctx)))), int(rng.integers(lo, hi + 1)))
                for _ in range(48)]
        both.append(Case(seqs, 24, 3, d, W.DTYPE_F16))
    firsts = []
    for c in both:
        c.run()
        c.ok()
        c.check()
        firsts.append(c.raw())
    for _ in range(8):
        for c in both:
            c.out.fill_(-1)
        for i in range(100):
            both[i % 2].run()
        for c, first in zip(both, firsts):
            c.ok()
            assert np.array_equal(c.raw(), first)


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0, 1e-30])
@pytest.mark.parametrize("dtype", TYPES)
def test_scales(scale, dtype):
    c = Case([(200, 12), (0, 3), (1500, 20)], 4, 2, 64, dtype, scale=scale)
    c.run()
    c.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale,size", [(0.125, 60.0), (40.0, 60.0), (3e4, 60.0)])
def test_scores_of_any_size(dtype, scale, size):
    """One key holds all the weight, or equal ones share it: rows are convex sums of v."""
    c = Case([(300, 9), (30, 2), (2000, 3)], 4, 1, 64, dtype, scale=scale, size=size)
    c.run()
    got = c.values()
    assert np.isfinite(got).all()
    for b in range(3):
        s, n = c.starts[b], c.n[b]
        want, bound = c.want(b)
        see = bound[..., 0] < np.abs(want).max() / 4
        assert (np.abs(got[s:s + n] - want) <= bound)[see].all()
        v = T.cached_rows(c.pools[1], c.tables[b], c.ctx[b], dtype)
        # weights and output each rounded once, the exponentials and sums 2^-18
        assert (np.abs(got[s:s + n]) <= np.abs(v).max() * (1 + 1.25 * I.EPS[dtype])).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale", [0.125, 40.0, -40.0, 3e4, -1e20, 1e30])
def test_the_largest_scores_share_a_row(scale, dtype, d):
    """Scores are exact (small integers in one element), and those below the largest lie 1200 |scale|
    and more below it: a row is the mean of the V of the keys that it sees with the largest one.
    Each such key's weight is rounded once, the exponentials and sums are off by 2^-18, and the
    output is rounded."""
    rng = np.random.default_rng(7)
    c = Case([(0, 1), (300, 9), (30, 2), (2000, 3), (9000, 20), (130, 90)], 4, 2, d, dtype, scale=scale)
    c.q[:] = I.narrow(np.zeros(1), dtype)[0]
    c.q[:, :, 5] = I.narrow(np.array([60.0]), dtype)[0]
    tops = []
    for b in range(len(c.n)):
        ctx, n = int(c.ctx[b]), int(c.n[b])
        first = rng.integers(-60, 41, ctx).astype(float)
        top = rng.random(ctx) < 3.0 / ctx                       # a few anywhere, some nodes, the root
        top[ctx - n:] |= rng.random(n) < 0.3
        top[ctx - n] = True
        first[top] = 60.0
        j = np.arange(ctx)
        k = I.narrow(np.sign(scale) * first, dtype)
        rows = c.pools[0][c.tables[b, j // 16], :, j % 16]
        rows[:, :, 5] = k[:, None]
        c.pools[0][c.tables[b, j // 16], :, j % 16] = rows
        tops.append(top)
    c.up()
    c.run()
    got = c.values()
    for b, top in enumerate(tops):
        s, n, ctx = c.starts[b], int(c.n[b]), int(c.ctx[b])
        v = T.cached_rows(c.pools[1], c.tables[b], c.ctx[b], dtype)
        see = np.ones((n, ctx), dtype=bool)
        see[:, ctx - n:] = T.sees(c.parents[s:s + n])
        w = (see & top).astype(float)
        want = np.repeat(np.einsum("nj,jhd->nhd", w / w.sum(-1, keepdims=True), v), 2, axis=1)
        off = (I.EPS[dtype] / 2 + 2.0 ** -18) * np.abs(v).max()
        assert (np.abs(got[s:s + n] - want) <= off + I.EPS[dtype] / 2 * (np.abs(want) + off) + 2.0 ** -25).all(), b
    c.ok()


def test_many_keys_of_little_weight():
    """What lies 2^-24 below the first key adds up (fp16 weights are lifted)."""
    c = Case([(9000, 1)], 1, 1, 64, W.DTYPE_F16, scale=1.0)
    c.q[:] = I.narrow(np.zeros(1), c.dtype)[0]
    c.q[0, 0, 0] = 1.0
    t = c.tables[0]
    c.pools[0][t] = 0.0
    c.pools[0][t[0], 0, 0, 0] = 17.0      # e^17 of the others
    c.pools[1][t] = 1.0
    c.pools[1][t[0], 0, 0] = 0.0
    c.up()
    c.run()
    want = 9000 * np.exp(-17) / (1 + 9000 * np.exp(-17))
    # lifted by 2^7 they are 2^-17.5, half a step of 2^-24 is 2^-7.5 of them; the output's rounding 2^-11
    assert np.abs(c.values()[0] - want).max() <= want * 2.0 ** -7


def test_nan_in_a_row_and_infinities_elsewhere():
    c = Case([(150, 4), (40, 6)], 4, 2, 64, W.DTYPE_BF16)
    c.q[c.starts[0] + 1, 2] = I.narrow(np.array([np.nan]), c.dtype)[0]
    c.up()
    c.run()
    bad = np.isnan(c.values()).any(-1)
    want = np.zeros_like(bad)
    want[c.starts[0] + 1, 2] = True
    assert np.array_equal(bad, want)
    # a key that only some nodes see: an infinite k of node 1 stays out of its siblings' rows
    c = Case([(33, 3)], 2, 1, 64, W.DTYPE_F16)
    c.parents[:3] = [-1, 0, 0]
    j = 33 + 1
    c.pools[0][c.tables[0, j // 16], :, j % 16] = np.inf
    c.up()
    c.run()
    c.pools[0][c.tables[0, j // 16], :, j % 16] = 0
    got, (want, bound) = c.values(), c.want(0)
    for i in (0, 2):
        assert (np.abs(got[i] - want[i]) <= bound[i]).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv,seqs", [
    (4, 2, [(30, 9), (7, 3), (200, 40)]),                       # an item each
    (8, 1, [(3, 16), (60, 2), (100, 33), (250, 64)]),           # rows of both tiles among others
    (4, 2, [(9000, 20)]),                                       # one context over every SM
    (2, 1, [(90 + i % 50, 1 + i % 13) for i in range(700)]),    # several items a CTA
    (4, 2, [(760, 30)] * 3 + [(120, 200)]),                     # both tiles' chunks in turn
])
def test_v_that_is_not_finite_reaches_the_rows_that_see_it(hq, hkv, seqs, d, dtype):
    """Infinities and NaN in V of some nodes: the rows that see one have it, the others none."""
    rng = np.random.default_rng(d + len(seqs))
    c = Case(seqs, hq, hkv, d, dtype, kind="forest", seed=3)
    odd = {}
    for b, n in enumerate(c.n):
        marks = odd[b] = np.zeros((n, hkv, d))
        for i in rng.choice(n, min(n, 1 + n // 6), replace=False):
            for h in range(hkv):
                marks[i, h, rng.choice(d, 3, replace=False)] = rng.choice([np.inf, -np.inf, np.nan], 3)
        if b % 3 == 1:
            marks[:] = 0                                        # a sequence without
    finite = c.pools[1].copy()
    wide = I.to_f64(c.pools[1], dtype)
    for b, n in enumerate(c.n):
        j = c.ctx[b] - n + np.arange(n)
        at = (c.tables[b, j // 16], slice(None), j % 16)
        hit = odd[b] != 0
        held = wide[at]
        wide[at] = np.where(hit, odd[b], held)
        even = finite[at]
        even[hit] = 0
        finite[at] = even
    c.pools[1] = I.narrow(wide, dtype)
    c.up()
    c.run()
    got = c.values()
    c.pools[1] = finite
    for b, n in enumerate(c.n):
        s = c.starts[b]
        want, bound = c.want(b)
        see = T.sees(c.parents[s:s + n])
        extra = np.zeros((n, hkv, d))
        for i in range(n):
            with np.errstate(invalid="ignore"):
                extra[i] = odd[b][see[i]].sum(0)                # inf - inf: NaN
        want = want + np.repeat(extra, hq // hkv, axis=1)
        rows, plain = got[s:s + n], np.isfinite(want)
        assert (np.abs(rows[plain] - want[plain]) <= bound[plain]).all(), b
        assert np.array_equal(rows[~plain], want[~plain], equal_nan=True), b
    c.ok()


def test_blocks_outside_the_pool_are_left_out():
    c = Case([(400, 20), (70, 3), (0, 2)], 4, 2, 128, W.DTYPE_F16)
    lost = {0: [0, 7, 11], 1: [2], 2: [0]}
    for b, blocks in lost.items():
        c.tables[b, blocks] = [c.nb, -1, 1 << 30][:len(blocks)]
    c.up()
    c.run()
    assert P.photon_get_last_device_error() == (6, 1)
    got = c.values()
    for b, blocks in lost.items():
        there = ~np.isin(np.arange(c.ctx[b]) // 16, blocks)
        held = c.tables[b].copy()
        held[blocks] = 0
        k, v = (np.where(there[:, None, None], T.cached_rows(p, held, c.ctx[b], c.dtype), 0) for p in c.pools)
        s, n = c.starts[b], c.n[b]
        want, bound = T.tree_attention(I.to_f64(c.q[s:s + n], c.dtype), k, v, c.parents[s:s + n],
                                       c.scale, I.EPS[c.dtype], there=there)
        assert (np.abs(got[s:s + n] - want) <= bound).all()
    assert not got[c.starts[2]:c.starts[3]].any()   # no key is left


def test_blocks_outside_the_pool_among_items_of_one_and_four_chunks():
    """Every CTA has several items, one tile's each: the other tile passes over them, and copies
    run as far ahead as they can.  Ids outside the pool in a third of the sequences."""
    rng = np.random.default_rng(11)
    for chunks in ((1, 4), (4, 4)):
        c = Case([(128 * chunks[i % 2] - int(rng.integers(4, 60)), int(rng.integers(1, 4)))
                  for i in range(900)], 2, 1, 64, W.DTYPE_F16)
        held = c.tables.copy()
        there = []
        for b in range(900):
            mask = np.ones(c.ctx[b], dtype=bool)
            if b % 3 == 0:
                used = -(-int(c.ctx[b]) // 16)
                lost = rng.choice(used, int(rng.integers(1, used)), replace=False)
                c.tables[b, lost] = rng.choice([c.nb, -1, 1 << 30], len(lost))
                held[b, lost] = 0
                mask = ~np.isin(np.arange(c.ctx[b]) // 16, lost)
            there.append(mask)
        c.up()
        c.run()
        assert P.photon_get_last_device_error() == (6, 1)
        first = c.raw()
        got = c.values()
        c.tables = held
        for b in range(900):
            s, n = c.starts[b], c.n[b]
            want, bound = c.want(b, there=there[b])
            assert (np.abs(got[s:s + n] - want) <= bound).all(), b
        for _ in range(40):
            c.run()
        assert np.array_equal(c.raw(), first)
        assert P.photon_get_last_device_error() == (6, 1)


def test_parents_outside_their_tree_count_as_roots():
    c = Case([(60, 10), (20, 5)], 4, 2, 64, W.DTYPE_F16)
    c.ok()
    c.parents[c.starts[0] + np.array([0, 3, 4, 6])] = [0, 3, -2, 9]
    c.up()
    c.run()
    assert P.photon_get_last_device_error() == (6, 64)
    c.parents[c.starts[0] + np.array([0, 3, 4, 6])] = -1
    c.check()


def test_rejected_sequences():
    c = Case([(30, 4), (20, 9), (5, 3), (40, 4)], 4, 2, 64, W.DTYPE_F16, tail=2)
    c.ctx[2] = 2                      # fewer tokens than nodes
    c.up()
    c.run(longest=8)                  # the second tree is larger than that
    assert P.photon_get_last_device_error() == (6, 36)
    c.check(skip=(1, 2))
    raw = c.raw()
    s = c.starts[1]
    assert (raw[s:s + 8] == 0).all() and (raw[s + 8] == -1).all()
    assert (raw[c.starts[2]:c.starts[3]] == 0).all()
    c.ctx[2], c.ctx[3] = 8, c.mbs * 16 + 1
    c.up()
    c.run()
    assert P.photon_get_last_device_error() == (6, 4)
    c.check(skip=(3,))
    assert (c.raw()[c.starts[3]:c.starts[4]] == 0).all()
    c.ctx[3] = 44
    c.up()
    c.on[5][3:] = c.T + 1              # rows behind the last token, and before the first
    c.run()
    assert P.photon_get_last_device_error() == (6, 32)
    raw = c.raw()
    assert (raw[c.starts[2]:] == -1).all()
    c.starts[3:] = [c.starts[2], c.starts[2]]
    c.n[2:] = 0
    c.check()


def test_a_chain_is_the_multi_query_call():
    c = Case([(500, 4), (33, 2), (1200, 3)], 4, 2, 128, W.DTYPE_F16, kind="chain")
    c.run()
    got = c.values()
    n = P.photon_paged_multi_query_workspace_size(c.shape, c.T, c.longest)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    other = torch.zeros_like(c.out)
    P.photon_paged_multi_query(*c.on[:6], c.T, c.longest, c.scale, other, ws, n, c.shape)
    other = I.to_f64(other.cpu().numpy().view(np.float16), c.dtype)
    for b in range(3):
        _, bound = c.want(b)
        s = c.starts[b]
        assert (np.abs(got - other)[s:s + c.n[b]] <= 2 * bound).all()


def test_pool_past_32_bits():
    """A pool of more than 4 GiB whose blocks lie at its end."""
    c = Case([(700, 13), (90, 30)], 8, 4, 128, W.DTYPE_F16, spare=0)
    NB = 300000                        # 16 KB a block: 4.9 GB
    pools = []
    for p in c.pools:
        big = torch.zeros((NB, 4, 16, 128), dtype=torch.float16, device="cuda")
        big[NB - c.nb:] = dev(p)
        pools.append(big)
    c.shape.num_blocks = NB
    c.on[1:3] = pools
    c.on[3] = dev(np.where(c.tables >= 0, c.tables + NB - c.nb, -1).astype(np.int32))
    c.run()
    c.check()
    c.ok()


def test_streams_at_once_and_a_captured_call():
    cases = [Case([(3000, 16)] * 6, 8, 2, 128, W.DTYPE_F16, seed=i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(4):
        for c, s in zip(cases, streams):
            c.run(stream=s)
    torch.cuda.synchronize()
    for c in cases:
        c.check(only=[0, 5])
    c = Case([(40, 8), (200, 20), (0, 1)], 4, 2, 64, W.DTYPE_BF16, spare=80)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    c.run()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        c.run()
    rng = np.random.default_rng(5)
    for step in range(3):
        # other trees, and contexts that are cut shorter
        c.ctx = np.maximum(c.n, c.ctx - 11).astype(np.int32)
        for s, n in zip(c.starts, c.n):
            c.parents[s:s + n] = T.random_parents(rng, n, "forest")
        c.on[4].copy_(dev(c.ctx))
        c.on[6].copy_(dev(c.parents))
        c.out.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        c.check()
    c.ok()
