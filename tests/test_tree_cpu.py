"""Host-side checks of a speculative step's entry points (sizes and refusals, none of which
reaches the device), and pins of the definitions that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest

import paged_kv_attention_photon_gb300 as P
import tree_util as T

FAKE, FAKE2 = 0x10000, 0x20000   # aligned non-null addresses that are never read
OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    P.build()
    return P._load()


def _shape(**over):
    base = dict(num_seqs=4, num_q_heads=16, num_kv_heads=8, head_dim=128, block_size=16,
                num_blocks=100, max_blocks_per_seq=8, dtype=P.F16, partition_size=0)
    base.update(over)
    return P.PagedShape.make(**base)


BAD_SHAPES = [(dict(head_dim=96), UNSUPPORTED), (dict(block_size=32), UNSUPPORTED),
              (dict(num_q_heads=40), UNSUPPORTED), (dict(num_q_heads=12), INVALID),
              (dict(num_seqs=-1), INVALID), (dict(dtype=7), UNSUPPORTED)]


def _append(lib, shape, q=FAKE, qs=0, k=FAKE, ks=0, v=FAKE, vs=0, positions=FAKE, table=FAKE,
            most=64, rotary=128, pairs=0, slots=FAKE, n=3, qo=FAKE2, qos=0, kc=FAKE2, vc=FAKE2):
    return lib.photon_rope_cache_append(q, qs, k, ks, v, vs, positions, table, most, rotary, pairs,
                                        slots, n, qo, qos, kc, vc, ctypes.byref(shape), None)


def test_append_refusals(lib):
    for over, want in BAD_SHAPES:
        assert _append(lib, _shape(**over)) == want
    s = _shape()
    assert _append(lib, s, n=-1) == INVALID
    assert _append(lib, s, n=0, k=None) == OK
    for name, bad in (("most", 0), ("rotary", 0), ("rotary", -16), ("rotary", 144), ("pairs", 2),
                      ("pairs", -1), ("qs", -16), ("ks", 1016), ("vs", 8), ("qos", 2040)):
        assert _append(lib, s, **{name: bad}) == INVALID, name
    assert _append(lib, s, rotary=24) == UNSUPPORTED
    assert _append(lib, s, ks=1028) == MISALIGNED
    for name in ("q", "k", "v", "positions", "table", "slots", "qo", "kc", "vc"):
        assert _append(lib, s, **{name: None}) == INVALID, name
    for name in ("q", "k", "v", "table", "slots", "qo", "kc", "vc"):
        assert _append(lib, s, **{name: FAKE + 4}) == MISALIGNED, name
    assert _append(lib, s, positions=FAKE + 2) == MISALIGNED


def _tree(lib, shape, q=FAKE, kc=FAKE, vc=FAKE, tables=FAKE, lens=FAKE, starts=FAKE, parents=FAKE,
          n=8, longest=4, scale=0.1, out=FAKE2, ws=FAKE2, size=None):
    if size is None:
        size = lib.photon_paged_tree_attention_workspace_size(ctypes.byref(shape), n, longest)
    return lib.photon_paged_tree_attention(q, kc, vc, tables, lens, starts, parents, n, longest,
                                           scale, out, ws, size, ctypes.byref(shape), None)


def test_tree_attention_refusals(lib):
    for over, want in BAD_SHAPES + [(dict(dtype=P.F32), UNSUPPORTED)]:
        assert _tree(lib, _shape(**over)) == want
        assert P.photon_paged_tree_attention_workspace_size(_shape(**over), 8, 4) == 0
    s = _shape()
    assert _tree(lib, s, n=-1) == INVALID
    assert _tree(lib, s, longest=-1) == INVALID
    assert _tree(lib, s, longest=257) == UNSUPPORTED
    assert _tree(lib, s, scale=float("inf")) == INVALID
    assert _tree(lib, s, scale=float("nan")) == INVALID
    for over in (dict(n=0), dict(longest=0)):
        assert _tree(lib, s, q=None, **over) == OK
    assert _tree(lib, _shape(num_seqs=0), q=None) == OK
    for name in ("q", "kc", "vc", "tables", "lens", "starts", "parents", "out"):
        assert _tree(lib, s, **{name: None}) == INVALID, name
        assert _tree(lib, s, **{name: FAKE + 2}) == MISALIGNED, name
    need = P.photon_paged_tree_attention_workspace_size(s, 8, 4)
    assert _tree(lib, s, size=need - 1) == WORKSPACE
    assert _tree(lib, s, ws=None) == WORKSPACE
    assert _tree(lib, s, ws=FAKE + 8) == MISALIGNED
    assert _tree(lib, _shape(num_seqs=65535, max_blocks_per_seq=1 << 20)) == UNSUPPORTED
    assert _tree(lib, _shape(num_blocks=1 << 26)) == UNSUPPORTED
    assert _tree(lib, s, n=1 << 27) == UNSUPPORTED


def test_tree_attention_workspace_grows_with_what_it_holds():
    size = P.photon_paged_tree_attention_workspace_size
    s = _shape()
    assert size(s, 8, 4) % 256 == 0
    # one more token: its 16 heads' maximum, sum and row
    assert size(s, 1024, 4) - size(s, 512, 4) == 512 * 16 * (8 + 128 * 4)
    assert size(s, 8, 0) == size(s, 0, 4) == size(_shape(num_seqs=0), 8, 4) == 0
    assert size(_shape(max_blocks_per_seq=9000), 8, 4) == size(s, 8, 4)


def _verify(lib, target=FAKE, ts=0, draft=FAKE, ds=0, vocab=100, dtype=0, tokens=FAKE, parents=FAKE,
            starts=FAKE, accept=FAKE, sample=FAKE, seqs=2, n=6, longest=4, path=FAKE2, count=FAKE2,
            following=FAKE2):
    return lib.photon_verify_tree(target, ts, draft, ds, vocab, dtype, tokens, parents, starts,
                                  accept, sample, seqs, n, longest, path, count, following, None)


def test_verify_refusals(lib):
    for name, bad in (("vocab", 0), ("seqs", -1), ("n", -1), ("longest", -1), ("ts", 99), ("ds", 50),
                      ("ts", -100)):
        assert _verify(lib, **{name: bad}) == INVALID, name
    for name, bad in (("vocab", (1 << 20) + 1), ("dtype", 3), ("longest", 257), ("seqs", 65536)):
        assert _verify(lib, **{name: bad}) == UNSUPPORTED, name
    assert _verify(lib, seqs=0, target=None) == OK
    names = ("target", "tokens", "parents", "starts", "accept", "sample", "path", "count", "following")
    for name in names:
        assert _verify(lib, **{name: None}) == INVALID, name
        assert _verify(lib, **{name: FAKE + 2}) == MISALIGNED, name
    assert _verify(lib, draft=FAKE + 2) == MISALIGNED
    assert _verify(lib, dtype=1, target=FAKE + 1) == MISALIGNED


def _compact(lib, shape, pools=(FAKE, FAKE2), tables=FAKE, lens=FAKE, starts=FAKE, path=FAKE,
             count=FAKE, n=8, longest=4, num=None):
    held = P.CachePools(pools)
    return lib.photon_cache_compact(held.data_ptr() if pools else None, len(held) if num is None else num,
                                    tables, lens, starts, path, count, n, longest,
                                    ctypes.byref(shape), None)


def test_compact_refusals(lib):
    for over, want in BAD_SHAPES:
        assert _compact(lib, _shape(**over)) == want
    s = _shape()
    for name in ("n", "longest", "num"):
        assert _compact(lib, s, **{name: -1}) == INVALID
    assert _compact(lib, s, longest=257) == UNSUPPORTED
    assert _compact(lib, s, pools=[FAKE] * 257) == UNSUPPORTED
    for over in (dict(n=0), dict(longest=0), dict(pools=())):
        assert _compact(lib, s, tables=None, **over) == OK
    assert _compact(lib, s, pools=(FAKE, 0)) == INVALID
    assert _compact(lib, s, pools=(FAKE, FAKE + 8)) == MISALIGNED
    assert _compact(lib, s, pools=(), num=2) == INVALID
    for name in ("tables", "lens", "starts", "path", "count"):
        assert _compact(lib, s, **{name: None}) == INVALID, name
        assert _compact(lib, s, **{name: FAKE + 2}) == MISALIGNED, name


# ------------------------------------------------------------------ the definitions
def test_sees():
    m = T.sees(np.array([-1, 0, 0, 1, -1, 3]))
    assert [list(np.flatnonzero(r)) for r in m] == [[0], [0, 1], [0, 2], [0, 1, 3], [4], [0, 1, 3, 5]]


def test_attention_of_a_chain_is_causal():
    """Against a triangular mask, and a tree's leaf against its own line of tokens alone."""
    rng = np.random.default_rng(1)
    n, ctx, hq, hkv, d = 5, 12, 4, 2, 8
    q, k, v = rng.standard_normal((n, hq, d)), rng.standard_normal((ctx, hkv, d)), rng.standard_normal((ctx, hkv, d))
    got, _ = T.tree_attention(q, k, v, T.random_parents(rng, n, "chain"), 0.3, 0.0)
    for i in range(n):
        for h in range(hq):
            e = ctx - n + i + 1
            w = np.exp(0.3 * k[:e, h // 2] @ q[i, h])
            assert np.allclose(got[i, h], w @ v[:e, h // 2] / w.sum(), atol=1e-12)
    parents = np.array([-1, 0, 0, 2, 1])
    got, _ = T.tree_attention(q, k, v, parents, 0.3, 0.0)
    line = list(range(ctx - n)) + [ctx - n + j for j in (0, 2, 3)]
    alone, _ = T.tree_attention(q[3:4], k[line], v[line], np.array([-1]), 0.3, 0.0)
    assert np.allclose(got[3], alone[0], atol=1e-12)


def test_verification_keeps_the_targets_distribution():
    """Over all drawn children and random numbers (a fine grid), the first token after node 0
    is distributed as the target's row says; drawn children, two of them."""
    p = np.array([0.5, 0.3, 0.2, 0.0])
    q = np.array([0.2, 0.2, 0.2, 0.4])
    grid = (np.arange(40) + 0.5) / 40
    got = np.zeros(4)
    for x in range(4):
        for y in range(4):
            for u in grid:
                for w in grid:
                    path, _ = T.verify(np.tile(p, (3, 1)), np.tile(q, (3, 1)), [0, x, y], [-1, 0, 0],
                                       [0, u, w], 0.0)
                    share = q[x] * q[y] / len(grid) ** 2
                    if len(path) > 1:
                        got[[x, y][path[1] - 1]] += share
                    else:
                        # what is left, whatever the sampling number
                        nexts = [T.verify(np.tile(p, (3, 1)), np.tile(q, (3, 1)), [0, x, y],
                                          [-1, 0, 0], [0, u, w], s)[1] for s in (0.1, 0.5, 0.9)]
                        for t in nexts:
                            got[t] += share / 3
    assert np.abs(got - p).max() < 0.03   # grid steps of 1/40, sampling steps of 1/3


def test_verification_of_chosen_children_keeps_the_distribution():
    p = np.array([0.45, 0.25, 0.2, 0.1])
    grid = (np.arange(60) + 0.5) / 60
    got = np.zeros(4)
    for u in grid:
        for w in grid:
            for s in grid[::6]:
                path, following = T.verify(np.tile(p, (3, 1)), None, [0, 1, 0], [-1, 0, 0], [0, u, w], s)
                got[[1, 0][path[1] - 1] if len(path) > 1 else following] += 1
    assert np.abs(got / got.sum() - p).max() < 0.02   # grid steps of 1/60 twice


def test_verification_by_hand():
    one = np.eye(4)
    # greedy: a target of ones and zeros follows exactly its own tokens
    p = one[[2, 1, 3, 0]]
    assert T.verify(p, None, [9, 2, 1, 0], [-1, 0, 1, 2], [0.9] * 4, 0.5) == ([0, 1, 2], 3)
    # the same token twice: the second one is not left; padding is passed over
    p = np.tile([0.5, 0.5, 0, 0], (4, 1))
    assert T.verify(p, None, [0, 0, 0, 1], [-1, 0, 0, 0], [0, 0.6, 0.0, 0.99], 0.3) == ([0, 3], 0)
    assert T.verify(p, None, [0, -1, 5, 1], [-1, 0, 0, 0], [0, 0, 0, 0.4], 0.3) == ([0, 3], 0)
    # p <= q everywhere else: nothing is left after the rejection but p's surplus
    p, q = np.tile([0.4, 0.6], (2, 1)), np.tile([0.7, 0.3], (2, 1))
    assert T.verify(p, q, [0, 0], [-1, 0], [0, 0.6], 0.0) == ([0], 1)
    assert T.verify(p, q, [0, 0], [-1, 0], [0, 0.5], 0.99) == ([0, 1], 1)
    # p == q and a child that q says is impossible: what is left is 0, so p is sampled
    assert T.verify(p, p * [0, 1] + [0.4, 0], [0, 0], [-1, 0], [0, 0.9999999], 0.0) == ([0, 1], 0)
    q = np.tile([0.5, 0.7], (2, 1))
    assert T.verify(p, q, [0, 0], [-1, 0], [0, 0.9], 0.5) == ([0], 1)
    assert T.verify(np.zeros((1, 3)), None, [0], [-1], [0], 0.5) == ([0], -1)


def test_compacted():
    rng = np.random.default_rng(0)
    pool = rng.standard_normal((6, 2, 16, 4))
    table = np.array([3, 1, 5])
    new = T.compacted(pool, table, 36, 20, [0, 2, 3, 17])
    flat = lambda p: np.concatenate([p[b].transpose(1, 0, 2) for b in table])
    want = flat(pool).copy()
    want[16:20] = want[[16, 18, 19, 33]]
    assert np.array_equal(flat(new), want)
    assert np.array_equal(new[[0, 2, 4]], pool[[0, 2, 4]])
