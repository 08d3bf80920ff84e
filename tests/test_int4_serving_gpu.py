"""The 4-bit path as an engine runs it: one fused projection per token, its q
and k normed and rotated, whole prompts attending over their own rows, every new
row quantised into the paged cache at the scheduler's slots, and decode steps
over that cache.  Each stage is checked against its formula in 64 bits on what
the stage before it produced, the pools bit for bit on a host mirror."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import int4_util as I
import paged_kv_attention_photon_gb300 as P
import workloads as W
from gpu_util import dev, host, rope_table
from test_prompt_attention_gpu import attention
from test_qk_norm_rope_gpu import formula

pytestmark = pytest.mark.gpu

HQ, HKV, D, EPS = 8, 4, 64, 1e-6
MAX_POS = 256


class Engine:
    def __init__(self, seed, dtype, num_blocks, mbs):
        self.rng = np.random.default_rng(seed)
        self.dtype, self.mbs, self.nb = dtype, mbs, num_blocks
        rec = I.record_bytes(D)
        self.host = [np.full((num_blocks, HKV, rec), 0xFF, dtype=np.uint8) for _ in range(2)]
        self.pool = [dev(p) for p in self.host]
        self.w = [I.narrow(1 + 0.1 * self.rng.standard_normal(D), dtype) for _ in range(2)]
        self.on_w = [dev(x) for x in self.w]
        self.table = rope_table(1e4, MAX_POS, D)
        self.axes = P.RopeAxes.make([D // 2])

    def shape(self, seqs):
        return P.PagedShape.make(num_seqs=seqs, num_q_heads=HQ, num_kv_heads=HKV, head_dim=D,
                                 num_blocks=self.nb, max_blocks_per_seq=self.mbs, dtype=self.dtype)

    def project(self, positions):
        """A fused projection of those tokens, on the host and the device."""
        x = I.narrow(self.rng.standard_normal((len(positions), HQ + 2 * HKV, D)), self.dtype)
        return x, dev(x)

    def turn(self, x, on, positions):
        """q and k normed and rotated in place; checked."""
        stride = x.shape[1] * D
        P.photon_qk_norm_rope(on, stride, on[:, HQ:], stride, *self.on_w, EPS,
                              dev(np.asarray([positions], dtype=np.int32)), self.table, MAX_POS,
                              self.axes, len(positions), on, stride, on[:, HQ:], stride,
                              self.shape(0))
        back = host(on, x)
        assert np.array_equal(back[:, HQ + HKV:].view(np.uint16), x[:, HQ + HKV:].view(np.uint16))
        f = I.to_f64(x, self.dtype)
        for part, w in ((slice(0, HQ), self.w[0]), (slice(HQ, HQ + HKV), self.w[1])):
            z, b = formula(f[:, part], I.to_f64(w, self.dtype), EPS, np.asarray([positions]),
                           self.table.cpu().numpy().astype(np.float64), [D // 2], False, MAX_POS)
            got = I.to_f64(back[:, part], self.dtype)
            assert (np.abs(got - z) <= b + I.EPS[self.dtype] / 2 * (np.abs(z) + b) + 2.0 ** -25).all()
        return back

    def write(self, x, on, slots):
        stride = x.shape[1] * D
        P.photon_cache_write_int4(on[:, HQ:], stride, on[:, HQ + HKV:], stride, dev(slots),
                                  len(slots), *self.pool, self.shape(1))
        self.mirror(x, slots)

    def mirror(self, x, slots):
        for which, part in enumerate((x[:, HQ:HQ + HKV], x[:, HQ + HKV:])):
            codes, step, lo = I.quantise(part, self.dtype)
            for t, s in enumerate(slots):
                for h in range(HKV):
                    I.store_row(self.host[which], which == 0, D, s // 16, h, s % 16, codes[t, h],
                                step[t, h], lo[t, h])

    def check_pools(self):
        for p, h in zip(self.pool, self.host):
            assert np.array_equal(p.cpu().numpy(), h)


@pytest.mark.parametrize("dtype,num_blocks,max_new", [(W.DTYPE_F16, 200, 12),
                                                      (W.DTYPE_BF16, 10, 40)])
def test_scheduler_drives_the_4_bit_path(dtype, num_blocks, max_new):
    """Whole prompts and decode rows of a request trace; the small pool preempts and recomputes."""
    max_prompt = 60
    mbs = (max_prompt + max_new + 15) // 16
    e = Engine(3, dtype, num_blocks, mbs)
    trace = W.request_trace(9, 14, max_prompt=max_prompt, max_new=max_new,
                            pool_tokens=num_blocks * 16, arrivals_per_step=1.5)
    sched = P.Scheduler(num_blocks=num_blocks, block_size=16, max_blocks_per_seq=mbs, max_seqs=8,
                        max_step_tokens=8 * (max_prompt + max_new))
    nxt = steps = decoded = prompts = preempted = 0
    while steps < 300:
        while nxt < len(trace) and trace[nxt][0] <= steps:
            sched.add_request(*trace[nxt][1:])
            nxt += 1
        st = sched.schedule()
        preempted += st["num_preempted"]
        n_of, ctx = st["query_lens"].copy(), st["context_lens"].astype(np.int32)
        tables = np.ascontiguousarray(st["block_tables"]).astype(np.int32)
        slots = st["slot_mapping"].astype(np.int64).copy()
        first = np.concatenate([[0], np.cumsum(n_of)]).astype(int)
        whole = [r for r in range(len(n_of)) if n_of[r] == ctx[r]]
        one = [r for r in range(len(n_of)) if n_of[r] == 1 and ctx[r] > 1]
        assert sorted(whole + one) == list(range(len(n_of)))
        if whole:
            pos = np.concatenate([np.arange(ctx[r]) for r in whole]).astype(np.int32)
            x, on = e.project(pos)
            x = e.turn(x, on, pos)
            starts = np.concatenate([[0], np.cumsum(ctx[whole])]).astype(np.int32)
            out = torch.empty((len(pos), HQ, D), dtype=on.dtype, device="cuda")
            stride = x.shape[1] * D
            P.photon_prompt_attention(on, stride, on[:, HQ:], stride, on[:, HQ + HKV:], stride,
                                      dev(starts), len(pos), int(ctx[whole].max()), D ** -0.5, out, 0,
                                      e.shape(len(whole)))
            e.write(x, on, np.concatenate([slots[first[r]:first[r + 1]] for r in whole]))
            f = I.to_f64(x, dtype)
            want, bound = attention(f[:, :HQ], f[:, HQ:HQ + HKV], f[:, HQ + HKV:], starts, D ** -0.5,
                                    I.EPS[dtype])
            assert (np.abs(I.to_f64(host(out, x[:, :HQ]), dtype) - want) <= bound).all()
            prompts += len(whole)
        if one:
            pos = (ctx[one] - 1).astype(np.int32)
            x, on = e.project(pos)
            x = e.turn(x, on, pos)
            e.write(x, on, slots[first[one]])
            q = on[:, :HQ].contiguous()
            shape = e.shape(len(one))
            n = P.photon_paged_decode_int4_workspace_size(shape)
            ws = torch.empty(n, dtype=torch.uint8, device="cuda")
            out = torch.empty_like(q)
            P.photon_paged_decode_int4(q, *e.pool, dev(tables[one]), dev(ctx[one]), D ** -0.5, out, ws,
                                       n, shape)
            want, bound = I.decode(x[:, :HQ], *e.host, tables[one], ctx[one], D ** -0.5, dtype)
            assert (np.abs(I.to_f64(host(out, x[:, :HQ]), dtype) - want) <= bound).all()
            decoded += len(one)
        st_, bits = P.photon_get_last_device_error()
        assert st_ == 0, bits
        sched.update()
        steps += 1
        s = sched.stats()
        if nxt == len(trace) and s["running"] == 0 and s["waiting"] == 0:
            break
    e.check_pools()
    assert sched.stats()["finished"] == len(trace) and decoded > 0 and prompts >= len(trace)
    if num_blocks < 100:
        assert preempted > 0


def test_decode_steps_as_one_graph():
    """Norm and rotation, cache write and decode captured once and replayed over growing
    contexts, on a stream of its own."""
    dtype, B, mbs = W.DTYPE_BF16, 5, 4
    e = Engine(5, dtype, B * mbs + 2, mbs)
    tables = np.random.default_rng(1).permutation(B * mbs + 2)[:B * mbs].astype(np.int32)
    tables = tables.reshape(B, mbs)
    ctx = np.array([1, 14, 30, 16, 0], dtype=np.int32)   # rows before the first step
    for b in range(B):
        if ctx[b]:
            pos = np.arange(ctx[b])
            x, on = e.project(pos)
            x = e.turn(x, on, pos)
            e.write(x, on, tables[b][pos // 16].astype(np.int64) * 16 + pos % 16)
    x, on = e.project(np.zeros(B))
    stride, shape = x.shape[1] * D, e.shape(B)
    n = P.photon_paged_decode_int4_workspace_size(shape)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    q = torch.empty((B, HQ, D), dtype=on.dtype, device="cuda")
    k = torch.empty((B, HKV, D), dtype=on.dtype, device="cuda")
    out = torch.empty_like(q)
    pos, lens, slots = dev(ctx[None].copy()), dev(ctx), dev(np.zeros(B, dtype=np.int64))
    on_tables = dev(tables)
    held = [p.clone() for p in e.pool]
    stream = torch.cuda.Stream()

    def step():
        P.photon_qk_norm_rope(on, stride, on[:, HQ:], stride, *e.on_w, EPS, pos, e.table, MAX_POS,
                              e.axes, B, q, 0, k, 0, shape)
        P.photon_cache_write_int4(k, 0, on[:, HQ + HKV:], stride, slots, B, *e.pool, shape)
        P.photon_paged_decode_int4(q, *e.pool, on_tables, lens, D ** -0.5, out, ws, n, shape)

    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    for p, h in zip(e.pool, held):
        p.copy_(h)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    for _ in range(18):
        x, fresh = e.project(np.zeros(B))
        where = tables[np.arange(B), ctx // 16].astype(np.int64) * 16 + ctx % 16
        on.copy_(fresh)
        pos.copy_(dev(ctx[None].copy()))
        slots.copy_(dev(where))
        ctx += 1
        lens.copy_(dev(ctx))
        graph.replay()
        torch.cuda.synchronize()
        assert P.photon_get_last_device_error()[0] == 0
        turned = x.copy()
        turned[:, :HQ] = host(q, x[:, :HQ])
        turned[:, HQ:HQ + HKV] = host(k, x[:, HQ:HQ + HKV])
        e.mirror(turned, where)
        want, bound = I.decode(turned[:, :HQ], *e.host, tables, ctx, D ** -0.5, dtype)
        assert (np.abs(I.to_f64(host(out, x[:, :HQ]), dtype) - want) <= bound).all()
    e.check_pools()


def test_binding_takes_the_current_stream():
    side = torch.cuda.Stream()
    assert P._stream(None) == torch.cuda.current_stream().cuda_stream
    with torch.cuda.stream(side):
        assert P._stream(None) == side.cuda_stream == torch.cuda.current_stream().cuda_stream
    assert P._stream(side) == side.cuda_stream and P._stream(17) == 17
