"""photon_verify_tree against a walk down each tree in 64 bits.  What comes out are whole
numbers: they are equal."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import int4_util as I
import paged_kv_attention_photon_gb300 as P
import tree_util as T
import workloads as W
from gpu_util import dev

pytestmark = pytest.mark.gpu
TYPES = [W.DTYPE_F32, W.DTYPE_F16, W.DTYPE_BF16]


def softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return e / e.sum(-1, keepdims=True)


class Case:
    def __init__(self, nodes, vocab, dtype=W.DTYPE_F32, *, drafted=True, kind="tree", seed=0,
                 spread=2.0, apart=1.0, pad=0, lead=0, tail=0):
        rng = np.random.default_rng(seed + sum(nodes) + vocab)
        self.n, self.vocab, self.dtype = np.array(nodes), vocab, dtype
        self.starts = (lead + np.concatenate([[0], np.cumsum(nodes)])).astype(np.int32)
        self.T = int(self.starts[-1]) + tail
        self.longest = int(max(nodes, default=0))
        x = spread * rng.standard_normal((self.T, vocab))
        y = x + apart * rng.standard_normal((self.T, vocab))
        self.p = I.narrow(softmax(x), dtype)
        q = softmax(y)
        self.q = I.narrow(q, dtype) if drafted else None
        self.parents = np.full(self.T, -1, dtype=np.int32)
        self.tokens = rng.integers(0, vocab, self.T).astype(np.int32)
        for s, n in zip(self.starts, nodes):
            self.parents[s:s + n] = T.random_parents(rng, n, kind)
            for i in range(1, n):
                up = s + self.parents[s + i]
                if self.parents[s + i] < 0:
                    continue
                if drafted:
                    at = np.searchsorted(np.cumsum(q[up]), rng.random() * q[up].sum(), side="right")
                    self.tokens[s + i] = min(at, vocab - 1)
                else:
                    self.tokens[s + i] = np.argsort(-q[up], kind="stable")[
                        min(vocab - 1, int((self.parents[s:s + i] == self.parents[s + i]).sum()))]
        self.accept = rng.random(self.T).astype(np.float32)
        self.sample = rng.random(len(nodes)).astype(np.float32)
        self.pad = pad

    def rows(self, x):
        """On the device, rows `pad` elements further apart, NaN between them."""
        if x is None:
            return None
        wide = np.full((self.T, self.vocab + self.pad), I.narrow(np.array([np.nan]), self.dtype)[0])
        wide[:, :self.vocab] = x
        return dev(wide)

    def up(self):
        self.on = [self.rows(self.p), self.rows(self.q), *[dev(x) for x in (
            self.tokens, self.parents, self.starts, self.accept, self.sample)]]
        self.got = [torch.full((k,), -7, dtype=torch.int32, device="cuda")
                    for k in (max(self.T, 1), len(self.n), len(self.n))]

    def run(self, stream=None, longest=None, stride=None):
        p, q, *rest = self.on
        stride = self.vocab + self.pad if stride is None else stride
        P.photon_verify_tree(p, stride, q, stride, self.vocab, self.dtype, *rest, len(self.n),
                             self.T, self.longest if longest is None else longest, *self.got, stream)

    def check(self, skip=()):
        path, count, following = [t.cpu().numpy() for t in self.got]
        p = I.to_f64(self.p, self.dtype)
        q = None if self.q is None else I.to_f64(self.q, self.dtype)
        accepted = 0
        for b, n in enumerate(self.n):
            s = self.starts[b]
            if b in skip:
                continue
            if n == 0:
                assert (count[b], following[b]) == (0, -1)
                continue
            rows = slice(s, s + n)
            line, token = T.verify(p[rows], None if q is None else q[rows], self.tokens[rows],
                                   self.parents[rows], self.accept[rows], self.sample[b])
            assert path[rows].tolist() == line + [-1] * (n - len(line)), (b, path[rows], line)
            assert (count[b], following[b]) == (len(line), token), b
            accepted += len(line) - 1
        assert (path[:self.starts[0]] == -7).all() and (path[self.starts[-1]:] == -7).all()
        return accepted

    def go(self, **more):
        self.up()
        self.run(**more)
        return self.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("vocab", [1, 2, 31, 1000, 4099, 32000, 100003])
def test_vocabularies(vocab, drafted, dtype):
    c = Case([1, 5, 9, 16, 3, 12], vocab, dtype, drafted=drafted, kind="tree", tail=1, lead=1)
    c.go()
    assert P.photon_get_last_device_error() == (0, 0)


@pytest.mark.parametrize("kind", ["chain", "tree", "forest"])
@pytest.mark.parametrize("drafted", [True, False])
def test_shapes_of_trees(kind, drafted):
    accepted = 0
    for seed in range(4):
        c = Case([0, 1, 2, 33, 64, 65, 5, 0, 17], 777, drafted=drafted, kind=kind, seed=seed,
                 spread=3.0, apart=0.5)
        accepted += c.go()
    assert accepted > 0   # some nodes are
    c = Case([256, 200], 300, drafted=drafted, kind=kind, spread=4.0, apart=0.3)
    c.go()


def test_no_rows_at_all():
    starts, sample = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(3, device="cuda")
    count, following = torch.full((3,), -7, device="cuda").int(), torch.full((3,), -7, device="cuda").int()
    P.photon_verify_tree(None, 0, None, 0, 100, W.DTYPE_F32, None, None, starts, None, sample, 3, 0, 5,
                         None, count, following)
    assert count.tolist() == [0] * 3 and following.tolist() == [-1] * 3


def test_all_accepted_and_none():
    c = Case([6, 6], 500, kind="chain", apart=0.0)     # p == q: every child is accepted
    assert c.go() == 10
    c.accept[:] = 0.999999
    c.q = I.narrow(np.tile(np.eye(500)[3], (12, 1)), c.dtype)
    c.tokens[:] = 3                                    # drawn for certain, hardly likely
    assert c.go() == 0


@pytest.mark.parametrize("pad", [0, 1, 4, 61])
@pytest.mark.parametrize("dtype", TYPES)
def test_strides_and_alignment(dtype, pad):
    """Rows on any element; what lies between them is NaN."""
    c = Case([7, 3, 20], 2001, dtype, pad=pad, seed=pad)
    c.go()
    if pad == 0:
        c.run(stride=0)
        c.check()
        # rows that begin on an odd element
        p = torch.empty(c.p.size + 1, dtype=c.on[0].dtype, device="cuda")
        p[1:] = c.on[0].reshape(-1)
        c.on[0] = p[1:]
        c.run()
        c.check()


def test_many_siblings():
    """Every node a child of node 0: a pass over the row for each rejection."""
    for drafted in (True, False):
        c = Case([40, 256], 5000, drafted=drafted, spread=1.0, apart=2.0)
        for s, n in zip(c.starts, c.n):
            c.parents[s + 1:s + n] = 0
        c.accept[:] = 0.99
        c.go()


@pytest.mark.parametrize("shrink", [0.25, 2.0 ** -6, 2.0 ** -12])
@pytest.mark.parametrize("before", [1, 2, 3, 5])
def test_chosen_children_that_leave_little(before, shrink):
    """Each child before the last takes all but a random share below `shrink` of what is left, and is
    rejected; the last one's probability is 0.2 % above or below what it is accepted from."""
    rng = np.random.default_rng(before)
    n = before + 2
    c = Case([n] * 200, 60, W.DTYPE_F32, drafted=False)
    c.p[:] = 0
    high = np.nextafter(np.float32(1), np.float32(0))
    for b, s in enumerate(c.starts[:-1]):
        c.parents[s + 1:s + n] = 0
        c.tokens[s + 1:s + n] = rng.permutation(60)[:n - 1]
        left = 1.0                                             # exact in 64 bits
        for i in range(before):
            x = np.float32(left * (1 - shrink * rng.uniform(0.1, 1)))
            c.p[s, c.tokens[s + 1 + i]] = x
            left -= float(x)
        c.accept[s + 1:s + n] = high
        c.accept[s + n - 1] = u = np.float32(rng.uniform(0.2, 0.9))
        c.p[s, c.tokens[s + n - 1]] = np.float32(float(u) * left * (1.002 if b % 2 else 0.998))
    assert c.go() == 100


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kinds,rejected", [([2, 1, 1, 0], n) for n in (1, 2, 20, 60, 80)] +
                         [([1.25, 1.25, 1.25, 0.25], n) for n in (1, 2, 9, 12, 13, 14, 18)])
def test_what_is_left_after_many_rejections(kinds, rejected, dtype):
    """Children that the target does not take: what is left comes ever closer to nothing in
    (p - L q)+, but stays where p / q is largest.  Every fourth entry is of one of four kinds of
    p / q, with q alike.  After the second rejection only the first kind is left, and each takes
    the same share from what L lacks to its p / q: 0.75 of it stays in the first case (2^-33 after
    80), 0.25 in the second (2^-36 after 18)."""
    vocab, n = 4096, rejected + 1
    c = Case([n] * 6, vocab, dtype)
    q = np.full(vocab, 2.0 ** -12)
    c.p[:], c.q[:] = I.narrow(np.tile(kinds, vocab // 4) * q, dtype), I.narrow(q, dtype)
    for s in c.starts[:-1]:
        c.parents[s + 1:s + n] = 0
        c.tokens[s + 1:s + n] = 4 * np.arange(rejected) + 3
    c.accept[:] = 0.9
    c.sample[:] = [0.0, 0.2502, 0.5003, 0.7204, 0.9305, 0.9994]
    # the last child of one sequence is of the first kind: accepted where it stands last
    c.tokens[c.starts[2] + n - 1] = 400
    assert c.go() == 1


@pytest.mark.parametrize("kinds,rejected", [([2, 1, 1, 0], 150), ([2, 1, 1, 0], 254),
                                            ([1.25, 1.25, 1.25, 0.25], 40), ([1.25, 1.25, 1.25, 0.25], 254)])
def test_rejections_that_leave_less_than_48_bits_tell(kinds, rejected):
    test_what_is_left_after_many_rejections(kinds, rejected, W.DTYPE_F32)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab,spread,apart", [(2, 1.0, 1.0), (3, 4.0, 1.0), (8, 3.0, 3.0), (40, 0.3, 1.0),
                                               (450, 6.0, 3.0), (5000, 2.0, 0.1)])
def test_siblings_of_the_same_tokens(vocab, spread, apart, dtype):
    """Drawn children that come again and again: what is left may be a sliver of p."""
    rng = np.random.default_rng(vocab)
    c = Case([60] * 24, vocab, dtype, spread=spread, apart=apart, seed=vocab)
    for s, n in zip(c.starts, c.n):
        c.parents[s + 1:s + n] = 0
        held = c.tokens[s + 1:s + n]
        c.tokens[s + 1:s + n] = rng.choice(held[:max(1, int(rng.integers(1, 30)))], n - 1)
        c.accept[s + 1:s + n] = rng.choice([0.5, 0.97, 0.999], n - 1)
    c.go()


def test_the_same_token_twice_and_padding():
    c = Case([8, 8], 60, drafted=False)
    c.parents[:] = np.tile([-1, 0, 0, 0, 0, 0, 0, 0], 2)
    c.tokens[:8] = [1, 4, 4, -1, 9, 4, 9, 2]
    c.accept[:] = 0.999
    c.go()
    assert P.photon_get_last_device_error() == (0, 0)
    c = Case([8, 8], 60)
    c.tokens[[2, 9]] = -3
    c.go()
    c.tokens[3] = 60
    c.go()
    assert P.photon_get_last_device_error() == (6, 64)


@pytest.mark.parametrize("drafted", [True, False])
def test_the_first_nodes_token_is_not_used(drafted):
    c = Case([4, 1, 7], 90, drafted=drafted)
    for first in (90, 1 << 30, -2, 0):
        c.tokens[c.starts[:-1]] = first
        c.go()
        assert P.photon_get_last_device_error() == (0, 0)


def test_sampling_numbers_at_the_borders():
    """0 and the largest float below 1; rows whose first or last entries are 0."""
    low, high = 0.0, float(np.nextafter(np.float32(1), np.float32(0)))
    for vocab in (50, 5000, 40000):
        c = Case([1] * 8, vocab, spread=1.0)
        c.p[:, 0] = c.p[:, -1] = 0
        c.p[2:4, : vocab // 2] = 0
        c.p[4:6, vocab // 2:] = 0
        c.p[6] = 0
        c.p[6, vocab - 7] = 0.25
        c.p[7] = 0
        c.sample[:] = [low, high] * 4
        c.go()


def test_nothing_is_left():
    """q covers p: the target's own row is sampled; a row of zeros has no token."""
    c = Case([3, 3, 2], 4100, kind="chain", apart=0.0)
    for s in c.starts[:-1]:
        c.q[s] = c.p[s]
        c.tokens[s + 1] = 11
        c.p[s, 11] = 0.0
    c.accept[:] = 0.5
    c.p[c.starts[2]] = 0.0
    c.go()


def test_entries_that_are_no_probabilities():
    c = Case([6, 9, 4], 900, seed=5)
    c.p[::2, 5] = np.nan
    c.q[1::2, 6] = np.nan
    c.p[1, 8] = np.inf
    c.p[3, 7], c.q[2, 9] = -0.5, -np.inf
    c.go()


def test_shares_below_what_32_bits_add_up():
    """One entry holds nearly all; numbers next to it decide among the rest."""
    vocab = 50000
    c = Case([1] * 6, vocab)
    rng = np.random.default_rng(0)
    c.p[:] = (rng.random((6, vocab)) * 2e-10).astype(np.float32)
    c.p[:, 20000] = 1.0
    sums = np.cumsum(c.p.astype(np.float64), -1)
    c.sample[:] = [np.float32(1e-7), np.float32(2e-6), 0.5, np.float32(0.9999985),
                   np.float32(0.9999999), 0.0]
    c.go()
    # entries all alike: the token is the number's share of the vocabulary
    c.p[:] = np.float32(1 / vocab)
    c.go()


def test_rejected_sequences_and_parents():
    c = Case([5, 9, 4], 700)
    c.up()
    c.run(longest=8)
    assert P.photon_get_last_device_error() == (6, 32)
    path, count, following = [t.cpu().numpy() for t in c.got]
    assert (count[1], following[1]) == (0, -1) and (path[5:14] == -7).all()
    c.check(skip=(1,))
    c.parents[c.starts[1] + 3] = 3
    c.parents[0] = 2
    c.up()
    c.run()
    assert P.photon_get_last_device_error() == (6, 64)
    c.parents[c.starts[1] + 3] = c.parents[0] = -1
    c.check()
    c.up()
    c.on[4][-1] = c.T + 1
    c.run()
    assert P.photon_get_last_device_error() == (6, 32)
    c.check(skip=(2,))


def test_large_vocabularies_and_batches():
    c = Case([2, 3], 1 << 18, drafted=True, spread=1.0)
    c.go()
    c = Case([2, 3], 300007, drafted=False, spread=1.0)
    c.go()
    for B in (9, 34, 40, 90, 160, 210, 300):     # one to eight CTAs a sequence, in one turn or two
        for drafted in (True, False):
            c = Case([3] * B, 9001, drafted=drafted, seed=B)
            c.go()
    c = Case([2] * 700, 1500, drafted=True)
    c.go()
    c = Case([3] * 700, 3000, drafted=False)
    c.go()


def test_rows_past_32_bits():
    """Rows 4 GiB and more behind the first."""
    c = Case([3, 3], 900, kind="chain", spread=3.0, apart=0.5)
    stride = (1 << 30) // 4
    on = []
    for x in (c.p, c.q):
        big = torch.full((6, stride), float("nan"), device="cuda")   # 6 GiB
        big[:, :900] = dev(x)
        on.append(big)
    c.up()
    c.on[:2] = on
    c.run(stride=stride)
    c.check()


def test_streams_and_a_captured_call():
    cases = [Case([9] * 30, 6000, seed=s, spread=3.0) for s in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    for c in cases:
        c.up()
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s in zip(cases, streams):
            c.run(stream=s)
    torch.cuda.synchronize()
    for c in cases:
        c.check()
    c, graph = cases[0], torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    rng = np.random.default_rng(1)
    for _ in range(3):
        c.accept = rng.random(c.T).astype(np.float32)
        c.sample = rng.random(30).astype(np.float32)
        c.on[5].copy_(dev(c.accept))
        c.on[6].copy_(dev(c.sample))
        graph.replay()
        torch.cuda.synchronize()
        c.check()
