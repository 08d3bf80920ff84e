"""photon_cache_compact bit for bit, and a speculative step as an engine runs it: drafted trees
turned and appended, attended to, verified, and their accepted rows moved together, each stage
against its definition on what the stage before it gave, the pools against a host mirror."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import int4_util as I
import paged_kv_attention_photon_gb300 as P
import tree_util as T
import workloads as W
from gpu_util import dev, host, rope_table

pytestmark = pytest.mark.gpu
TYPES = [W.DTYPE_F32, W.DTYPE_F16, W.DTYPE_BF16]


class Moves:
    def __init__(self, seqs, hkv, d, dtype, num_pools, seed=0, kind="any"):
        """seqs: (tokens before the tree, nodes, accepted nodes)."""
        rng = np.random.default_rng(seed)
        self.n = np.array([n for _, n, _ in seqs])
        self.ctx = np.array([a + n for a, n, _ in seqs], dtype=np.int32)
        self.starts = np.concatenate([[0], np.cumsum(self.n)]).astype(np.int32)
        self.T, self.longest = int(self.starts[-1]), int(max(self.n))
        used = [-(-int(c) // 16) for c in self.ctx]
        self.nb, self.mbs = sum(used) + 3, max(used)
        order = rng.permutation(self.nb)
        self.tables = np.full((len(seqs), self.mbs), -1, dtype=np.int32)
        self.path = np.full(self.T, -1, dtype=np.int32)
        self.count = np.array([m for _, _, m in seqs], dtype=np.int32)
        at = 0
        for b, (a, n, m) in enumerate(seqs):
            self.tables[b, :used[b]] = order[at:at + used[b]]
            at += used[b]
            if m:
                self.path[self.starts[b]:self.starts[b] + m] = [0] + sorted(
                    rng.choice(np.arange(1, n), m - 1, replace=False)) if kind == "any" else range(m)
        word = np.uint32 if dtype == W.DTYPE_F32 else np.uint16
        self.pools = [rng.integers(0, 2 ** (8 * word().itemsize), (self.nb, hkv, 16, d)).astype(word)
                      for _ in range(num_pools)]
        self.shape = P.PagedShape.make(num_seqs=len(seqs), num_q_heads=hkv, num_kv_heads=hkv,
                                       head_dim=d, num_blocks=self.nb, max_blocks_per_seq=self.mbs,
                                       dtype=dtype)

    def run(self, longest=None, stream=None):
        self.on = [dev(p.view(np.int32 if p.dtype == np.uint32 else np.uint16)) for p in self.pools]
        self.args = [dev(x) for x in (self.tables, self.ctx, self.starts, self.path, self.count)]
        P.photon_cache_compact(P.CachePools(self.on), *self.args, self.T,
                               self.longest if longest is None else longest, self.shape, stream)

    def check(self, skip=()):
        for on, pool in zip(self.on, self.pools):
            want = pool
            for b, m in enumerate(self.count):
                if b not in skip and m:
                    s = self.starts[b]
                    want = T.compacted(want, self.tables[b], int(self.ctx[b]), int(self.n[b]),
                                       self.path[s:s + m])
            assert np.array_equal(on.cpu().numpy().view(want.dtype), want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("hkv,d", [(1, 64), (8, 128), (5, 64), (24, 128)])
def test_rows_move_together(hkv, d, dtype):
    c = Moves([(0, 1, 1), (3, 5, 2), (15, 8, 8), (30, 16, 5), (100, 64, 9), (7, 40, 39), (9, 3, 0),
               (64, 128, 77), (0, 256, 30)], hkv, d, dtype, 3, seed=hkv)
    c.run()
    c.check()
    assert P.photon_get_last_device_error() == (0, 0)


def test_chains_stay_and_many_pools():
    c = Moves([(20, 6, 4), (31, 2, 2)], 2, 64, W.DTYPE_F16, 256, kind="chain")
    c.run()
    c.check()
    c = Moves([(20, 9, 4), (31, 30, 6)] * 3, 2, 64, W.DTYPE_F16, 256)
    c.run()
    c.check()
    c = Moves([(20 + b % 7, 6, 3) for b in range(2000)], 1, 64, W.DTYPE_F16, 2)
    c.run()
    c.check()


def test_what_is_refused_is_left_as_it_was():
    c = Moves([(20, 6, 4), (31, 5, 3), (40, 7, 3), (12, 4, 2), (6, 4, 2)], 2, 64, W.DTYPE_F16, 2)
    c.path[c.starts[0] + 2] = c.path[c.starts[0] + 1]     # does not rise
    c.path[c.starts[1] + 2] = 5                           # not a node
    c.count[2] = 8                                        # more than the nodes
    c.run()
    assert P.photon_get_last_device_error() == (6, 64)
    c.check(skip=(0, 1, 2))
    c = Moves([(20, 6, 4), (31, 5, 3), (40, 7, 3)], 2, 64, W.DTYPE_F16, 2)
    c.tables[0, 1] = c.nb
    c.ctx[1] = 4
    c.run(longest=6)
    assert P.photon_get_last_device_error() == (6, 37)
    c.check(skip=(0, 1, 2))


def test_what_is_wrong_shows_where_nothing_moves():
    """A sequence without nodes, and one of which nothing was accepted."""
    def one(bits, **change):
        c = Moves([(20, 6, 4), (31, 0, 0), (9, 5, 0)], 2, 64, W.DTYPE_F16, 2)
        for name, (b, value) in change.items():
            getattr(c, name)[b] = value
        c.run()
        assert P.photon_get_last_device_error() == ((6, bits) if bits else (0, 0)), change
        c.count[1:] = 0
        c.check()

    one(0)
    one(64, count=(1, 2))
    one(64, count=(1, -1))
    one(64, count=(2, -1))
    one(4, ctx=(2, 4))
    one(4, ctx=(2, -1))
    one(4, ctx=(2, 1 << 20))
    one(0, ctx=(1, -1))          # no nodes: its context is not looked at


def test_pool_past_32_bits():
    c = Moves([(40, 20, 6), (7, 9, 4)], 4, 128, W.DTYPE_F16, 1, seed=3)
    NB = 300000                        # 16 KB a block: 4.9 GB
    big = torch.zeros((NB, 4, 16, 128), dtype=torch.int16, device="cuda")
    big[NB - c.nb:] = dev(c.pools[0])
    far = np.where(c.tables >= 0, c.tables + NB - c.nb, -1).astype(np.int32)
    c.shape.num_blocks = NB
    P.photon_cache_compact(P.CachePools([big]), dev(far), dev(c.ctx), dev(c.starts), dev(c.path),
                           dev(c.count), c.T, c.longest, c.shape)
    c.on = [big[NB - c.nb:].contiguous()]
    c.check()


# ------------------------------------------------------------------ a step
HQ, HKV, D, VOCAB, MAX_POS, LAYERS = 8, 2, 64, 700, 512, 2


class Engine:
    """Sequences with their own trees; two layers' pools, mirrored on the host."""

    def __init__(self, seed, dtype, seqs, longest):
        self.rng = np.random.default_rng(seed)
        self.dtype, self.seqs, self.longest = dtype, seqs, longest
        self.mbs = 14
        self.nb = seqs * self.mbs + 2
        self.tables = self.rng.permutation(self.nb)[:seqs * self.mbs].reshape(seqs, self.mbs).astype(np.int32)
        self.before = self.rng.integers(0, 60, seqs).astype(np.int32)
        self.mirror = [I.narrow(self.rng.standard_normal((self.nb, HKV, 16, D)), dtype)
                       for _ in range(2 * LAYERS)]
        self.pools = [dev(p) for p in self.mirror]
        self.held = P.CachePools(self.pools)
        self.on_tables = dev(self.tables)
        self.table = rope_table(1e4, MAX_POS, D)
        self.shape = P.PagedShape.make(num_seqs=seqs, num_q_heads=HQ, num_kv_heads=HKV, head_dim=D,
                                       num_blocks=self.nb, max_blocks_per_seq=self.mbs, dtype=dtype)
        T_ = seqs * longest
        kind = self.pools[0].dtype
        self.t = dict(
            x=[torch.zeros((T_, HQ + 2 * HKV, D), dtype=kind, device="cuda") for _ in range(LAYERS)],
            q=torch.zeros((T_, HQ, D), dtype=kind, device="cuda"),
            out=[torch.zeros((T_, HQ, D), dtype=kind, device="cuda") for _ in range(LAYERS)],
            positions=torch.zeros(T_, dtype=torch.int32, device="cuda"),
            slots=torch.zeros(T_, dtype=torch.int64, device="cuda"),
            lens=torch.zeros(seqs, dtype=torch.int32, device="cuda"),
            starts=torch.zeros(seqs + 1, dtype=torch.int32, device="cuda"),
            parents=torch.zeros(T_, dtype=torch.int32, device="cuda"),
            tokens=torch.zeros(T_, dtype=torch.int32, device="cuda"),
            p=torch.zeros((T_, VOCAB), device="cuda"), qd=torch.zeros((T_, VOCAB), device="cuda"),
            accept=torch.zeros(T_, device="cuda"), sample=torch.zeros(seqs, device="cuda"),
            path=torch.zeros(T_, dtype=torch.int32, device="cuda"),
            count=torch.zeros(seqs, dtype=torch.int32, device="cuda"),
            following=torch.zeros(seqs, dtype=torch.int32, device="cuda"))
        self.T = T_
        n = P.photon_paged_tree_attention_workspace_size(self.shape, T_, longest)
        self.ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")

    def draw(self):
        """New trees, projections, probabilities and numbers, on the host and the device."""
        rng, h = self.rng, {}
        n = rng.integers(1, self.longest + 1, self.seqs)
        starts = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        rows = starts[-1]
        h["n"], h["starts"] = n, starts
        h["lens"] = (self.before + n).astype(np.int32)
        h["parents"] = np.full(self.T, -1, dtype=np.int32)
        h["positions"] = np.full(self.T, -1, dtype=np.int32)     # rows behind the last tree: padding
        h["slots"] = np.full(self.T, -1, dtype=np.int64)
        for b in range(self.seqs):
            s = slice(starts[b], starts[b + 1])
            h["parents"][s] = T.random_parents(rng, n[b])
            h["positions"][s] = self.before[b] + T.depths(h["parents"][s])
            j = self.before[b] + np.arange(n[b])
            h["slots"][s] = self.tables[b, j // 16].astype(np.int64) * 16 + j % 16
        h["x"] = [I.narrow(rng.standard_normal((self.T, HQ + 2 * HKV, D)), self.dtype) for _ in range(LAYERS)]
        logits = 2 * rng.standard_normal((self.T, VOCAB))
        near = logits + rng.standard_normal((self.T, VOCAB))
        soft = lambda z: (np.exp(z) / np.exp(z).sum(-1, keepdims=True)).astype(np.float32)
        h["p"], h["qd"] = soft(logits), soft(near)
        h["tokens"] = np.zeros(self.T, dtype=np.int32)
        for b in range(self.seqs):
            for i in range(1, n[b]):
                row = h["qd"][starts[b] + h["parents"][starts[b] + i]].astype(np.float64)
                h["tokens"][starts[b] + i] = rng.choice(VOCAB, p=row / row.sum())
        h["accept"] = rng.random(self.T).astype(np.float32)
        h["sample"] = rng.random(self.seqs).astype(np.float32)
        for name in ("lens", "starts", "parents", "positions", "slots", "tokens", "p", "qd", "accept", "sample"):
            self.t[name].copy_(dev(h[name]))
        for on, x in zip(self.t["x"], h["x"]):
            on.copy_(dev(x))
        self.rows = rows
        return h

    def step(self):
        t, stride = self.t, (HQ + 2 * HKV) * D
        for layer in range(LAYERS):
            x, (k, v) = t["x"][layer], self.pools[2 * layer:2 * layer + 2]
            P.photon_rope_cache_append(x, stride, x[:, HQ:], stride, x[:, HQ + HKV:], stride,
                                       t["positions"], self.table, MAX_POS, D, 0, t["slots"], self.T,
                                       x, stride, k, v, self.shape)
            t["q"].copy_(x[:, :HQ])
            P.photon_paged_tree_attention(t["q"], k, v, self.on_tables, t["lens"], t["starts"],
                                          t["parents"], self.T, self.longest, D ** -0.5,
                                          t["out"][layer], self.ws, self.ws.numel(), self.shape)
        P.photon_verify_tree(t["p"], 0, t["qd"], 0, VOCAB, P.F32, t["tokens"], t["parents"],
                             t["starts"], t["accept"], t["sample"], self.seqs, self.T, self.longest,
                             t["path"], t["count"], t["following"])
        P.photon_cache_compact(self.held, self.on_tables, t["lens"], t["starts"], t["path"],
                               t["count"], self.T, self.longest, self.shape)

    def check(self, h):
        """Every stage; then the contexts are as long as what was accepted."""
        eps, starts, n = I.EPS[self.dtype], h["starts"], h["n"]
        path, count, following = (self.t[k].cpu().numpy() for k in ("path", "count", "following"))
        lines = []
        for b in range(self.seqs):
            s = slice(starts[b], starts[b + 1])
            line, token = T.verify(h["p"][s], h["qd"][s], h["tokens"][s], h["parents"][s],
                                   h["accept"][s], h["sample"][b])
            assert path[s].tolist() == line + [-1] * (n[b] - len(line))
            assert (count[b], following[b]) == (len(line), token)
            lines.append(line)
        table = self.table.cpu().numpy().astype(np.float64)
        for layer in range(LAYERS):
            x = I.to_f64(h["x"][layer], self.dtype)
            back = host(self.t["x"][layer], h["x"][layer])[:, :HQ]
            cos, sin = (table[np.maximum(h["positions"], 0)][:, None, :, i] for i in (0, 1))
            a, c = x[..., :D // 2], x[..., D // 2:]
            z = np.concatenate([a * cos - c * sin, c * cos + a * sin], -1)
            bound = 3 * 2.0 ** -24 * np.tile(np.abs(a) + np.abs(c), 2)
            bound = bound + eps / 2 * (np.abs(z) + bound) + 2.0 ** -25
            rows = np.arange(starts[-1])
            assert (np.abs(I.to_f64(back, self.dtype) - z[:, :HQ]) <= bound[:, :HQ])[rows].all()
            out = I.to_f64(host(self.t["out"][layer], back), self.dtype)
            held = [host(p, m) for p, m in zip(self.pools[2 * layer:2 * layer + 2],
                                               self.mirror[2 * layer:2 * layer + 2])]
            for which, mirror in enumerate(self.mirror[2 * layer:2 * layer + 2]):
                part = slice(HQ + which * HKV, HQ + (which + 1) * HKV)
                for t in rows:
                    slot = h["slots"][t]
                    mirror[slot // 16, :, slot % 16] = h["x"][layer][t, part] if which else \
                        I.narrow(z[t, part], self.dtype)
            # The attention against what it read: V from the mirror, K as the device rounded
            # it, from where the rows are now.  A rejected node's row that an accepted one
            # has taken the place of is gone; nodes that see it are left out here.
            for b in range(self.seqs):
                s, ctx, line = slice(starts[b], starts[b + 1]), int(h["lens"][b]), lines[b]
                mirrors = self.mirror[2 * layer:2 * layer + 2]
                v = T.cached_rows(mirrors[1], self.tables[b], ctx, self.dtype)
                now = T.cached_rows(held[0], self.tables[b], ctx, self.dtype)
                k, first, known = now.copy(), ctx - n[b], np.arange(n[b]) >= len(line)
                k[first + np.array(line)] = now[first:first + len(line)]
                known[line] = True
                want, off = T.tree_attention(I.to_f64(back[s], self.dtype), k, v, h["parents"][s],
                                             D ** -0.5, eps)
                fine = ~(T.sees(h["parents"][s]) & ~known).any(1)
                assert fine[line].all() and (np.abs(out[s] - want) <= off)[fine].all()
            for which in range(2):
                m = self.mirror[2 * layer + which]
                for b in range(self.seqs):
                    m = T.compacted(m, self.tables[b], int(h["lens"][b]), int(n[b]), lines[b])
                if which == 0:   # keys were rounded on the device: within one step, then as there
                    off = np.abs(I.to_f64(held[0], self.dtype) - I.to_f64(m, self.dtype))
                    assert (off <= eps * np.abs(I.to_f64(m, self.dtype)) + 2.0 ** -24).all()
                    m = held[0].copy()
                else:
                    assert np.array_equal(held[1].view(np.uint8), np.ascontiguousarray(m).view(np.uint8))
                self.mirror[2 * layer + which] = m
        self.before = (self.before + count).astype(np.int32)
        return int(count.sum()) - self.seqs


@pytest.mark.parametrize("dtype", [W.DTYPE_F16, W.DTYPE_BF16])
def test_speculative_steps(dtype):
    e = Engine(1, dtype, 5, 14)
    accepted = 0
    for _ in range(6):
        h = e.draw()
        e.step()
        assert P.photon_get_last_device_error() == (0, 0)
        accepted += e.check(h)
    assert accepted > 5


def test_a_step_as_one_graph():
    """Captured once on a stream of its own and replayed over new trees and growing contexts."""
    e = Engine(2, W.DTYPE_F16, 4, 12)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    e.draw()
    kept = [p.clone() for p in e.pools]
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        e.step()
    stream.synchronize()
    for p, k in zip(e.pools, kept):
        p.copy_(k)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        e.step()
    for _ in range(8):
        h = e.draw()
        graph.replay()
        torch.cuda.synchronize()
        assert P.photon_get_last_device_error() == (0, 0)
        e.check(h)
