"""Measured cases of a speculative step from trees of drafted tokens: what such a step does
around the model's projections and its logits.

Four operators, named by a case's "op":

* "append": q and k of new tokens turned by their positions, k and v stored at their slots
  of the paged cache (photon_rope_cache_append);
* "tree": attention of each sequence's drafted tokens over its cached context and their
  own ancestors (photon_paged_tree_attention);
* "verify": drafted tokens accepted or rejected against the target's probabilities from
  given random numbers, and the token that follows (photon_verify_tree);
* "compact": the accepted tokens' cached rows moved together behind the context, in every
  layer's pools (photon_cache_compact).

A sequence's tree has nodes 0 .. n - 1; parents[i] < i is node i's parent, -1 for a node
that follows the context.  The nodes' rows lie in the cache in that order, the last n of
context_lens.  Node i attends to the context before the tree, to its ancestors and to
itself.

Verification begins at node 0, which is certain.  At node c with the target's probabilities
p and the draft's q (rows of c), r = p and Z = 1; its children in their order: x is accepted
if r(x) > u Z q(x), and the walk goes on there; else r becomes max(0, r / Z - q) and Z its
sum.  Without draft probabilities a child was certain: it is accepted if r(x) > u Z, else
Z loses r(x), and r(x) becomes 0.  Where no child is left, the next token is the first one
whose cumulated r passes the sampling number times the sum of r (of p, where r is all 0).
"""
import math
import random

import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_ROPE_BASE = 1e6


# ------------------------------------------------------------------ cases
def listed():
    qwen = dict(q_heads=16, kv_heads=8, head_dim=128)   # the library's long-context decode shape
    llama = dict(q_heads=32, kv_heads=8, head_dim=64)   # its batch sweep and its batch-256 mix
    return [
        # the drafted trees of one step of 64 sequences
        dict(name="append_tree_b64", op="append", seqs=64, lo=16, hi=16, past=8192, chain=False,
             salt=1, pad=0, interleaved=False, rotary=128, dtype="f16", **qwen),
        # whole prompts on their way into the cache
        dict(name="append_16x1024", op="append", seqs=16, lo=1024, hi=1024, past=0, chain=True,
             salt=2, pad=0, interleaved=False, rotary=128, dtype="bf16", **qwen),
        # ragged chunks of prompts in a padded batch, half of each head turned, neighbours paired
        dict(name="append_ragged", op="append", seqs=24, lo=1, hi=2048, past=4096, chain=True,
             salt=3, pad=13, interleaved=True, rotary=32, dtype="f32", **llama),
        # a small batch: latency counts
        dict(name="tree_b4", op="tree", seqs=4, lo=64, hi=2048, long=0.0, nodes_lo=8, nodes_hi=8,
             chain=False, salt=4, dtype="f16", **llama),
        # 64 long contexts in a fragmented pool, sixteen nodes each
        dict(name="tree_b64", op="tree", seqs=64, lo=128, hi=8192, long=0.0, nodes_lo=16,
             nodes_hi=16, chain=False, salt=5, dtype="f16", **qwen),
        # a serving mix: four short contexts to each long one, trees of every size
        dict(name="tree_mix_b256", op="tree", seqs=256, lo=32, hi=512, long=0.2, nodes_lo=1,
             nodes_hi=32, chain=False, salt=6, dtype="bf16", **llama),
        # wide trees: 256 rows of q for each row of the cache
        dict(name="tree_wide_b32", op="tree", seqs=32, lo=512, hi=8192, long=0.0, nodes_lo=64,
             nodes_hi=64, chain=False, salt=7, dtype="bf16", **llama),
        # four drafted tokens in a row
        dict(name="verify_chain_b4", op="verify", seqs=4, nodes_lo=5, nodes_hi=5, chain=True,
             drafted=True, vocab=32000, salt=8, dtype="f32"),
        # a step of 64 sequences, children drawn from the draft's distribution
        dict(name="verify_tree_b64", op="verify", seqs=64, nodes_lo=16, nodes_hi=16, chain=False,
             drafted=True, vocab=128256, salt=9, dtype="f32"),
        # children that are the draft's most likely tokens; an odd vocabulary
        dict(name="verify_top_b32", op="verify", seqs=32, nodes_lo=1, nodes_hi=48, chain=False,
             drafted=False, vocab=99991, salt=10, dtype="f32"),
        # one layer of a small batch
        dict(name="compact_b4", op="compact", seqs=4, lo=64, hi=512, nodes_lo=8, nodes_hi=8,
             chain=False, pools=2, salt=11, dtype="f16", **llama),
        # sixteen layers of a step
        dict(name="compact_b64", op="compact", seqs=64, lo=16, hi=128, nodes_lo=16, nodes_hi=16,
             chain=False, pools=32, salt=12, dtype="bf16", **qwen),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "tree", "tree", "verify", "compact"])
    c = dict(op=op, salt=rng.randrange(1 << 20))
    if op == "verify":
        c["dtype"] = rng.choice(["f32", "f32", "f16", "bf16"])
        c["vocab"] = _log_int(rng, 1000, 160000)
        c["chain"] = rng.random() < 0.4
        c["drafted"] = rng.random() < 0.6
        c["nodes_hi"] = _log_int(rng, 1, 12 if c["chain"] else 64)
        c["nodes_lo"] = _log_int(rng, 1, c["nodes_hi"])
        most = 64 * 16 * 128256 // (c["vocab"] * c["nodes_hi"])
        c["seqs"] = max(1, min(_log_int(rng, 1, 256), most))
        return c
    q_heads, kv_heads = rng.choice([(16, 8), (32, 8), (16, 16), (8, 1), (4, 2), (24, 3), (32, 4)])
    d = rng.choice([64, 128])
    c.update(q_heads=q_heads, kv_heads=kv_heads, head_dim=d, chain=rng.random() < 0.25,
             dtype=rng.choice(["f16", "bf16"]))
    if op == "append":
        c["dtype"] = rng.choice(["f16", "bf16", "f32"])
        c["interleaved"] = rng.random() < 0.5
        c["rotary"] = rng.choice([d, d, d // 2, d // 4])
        c["pad"] = rng.choice([0, 0, 2, 31])
        c["past"] = _log_int(rng, 1, 16384)
        c["hi"] = _log_int(rng, 1, 4096 if c["chain"] else 64)
        c["lo"] = _log_int(rng, 1, c["hi"])
        width = (q_heads + 2 * kv_heads) * d * (2 if c["dtype"] == "f32" else 1)
        most = 16384 * 32 * 128 // width // c["hi"]
        c["seqs"] = max(1, min(_log_int(rng, 1, 256), most))
        return c
    c["nodes_hi"] = _log_int(rng, 1, 128 if op == "tree" else 48)
    c["nodes_lo"] = _log_int(rng, 1, c["nodes_hi"])
    if op == "tree":
        c["hi"] = _log_int(rng, 1, 16384)
        c["lo"] = _log_int(rng, 1, c["hi"])
        c["long"] = 0.0
        most = min(64 * 8192 * 8 * 128 // (kv_heads * d),
                   32 * 4096 * 64 * 32 * 64 // (c["nodes_hi"] * q_heads * d)) // c["hi"]
        c["seqs"] = max(1, min(_log_int(rng, 1, 256), most))
        return c
    c["dtype"] = rng.choice(["f16", "bf16", "f32"])
    c["hi"] = _log_int(rng, 1, 512)
    c["lo"] = _log_int(rng, 1, c["hi"])
    c["pools"] = 2 * _log_int(rng, 1, 32)
    width = kv_heads * d * (2 if c["dtype"] == "f32" else 1)
    most = 64 * 32 * 16 * 512 * 8 * 128 // (width * c["pools"] * 16 * (c["hi"] + c["nodes_hi"]))
    c["seqs"] = max(1, min(_log_int(rng, 1, 256), most))
    return c


def _nodes(c):
    """Nodes of each sequence's tree (new tokens of each sequence, for an append)."""
    lo, hi = (c["lo"], c["hi"]) if c["op"] == "append" else (c["nodes_lo"], c["nodes_hi"])
    r = random.Random("nodes %d %d %d %d" % (c["salt"], c["seqs"], lo, hi))
    return [_log_int(r, lo, hi) for _ in range(c["seqs"])]


def _past(c):
    """Tokens before them: log-uniform; a `long` share of a serving mix uniform in [4096, 16384]."""
    lo, hi = (1, c["past"]) if c["op"] == "append" else (c["lo"], c["hi"])
    r = random.Random("past %d %d %d %d" % (c["salt"], c["seqs"], lo, hi))
    if hi == 0:
        return [0] * c["seqs"]
    n = [_log_int(r, lo, hi) for _ in range(c["seqs"])]
    if c.get("long"):
        n = [r.randint(4096, 16384) if r.random() < c["long"] else x for x in n]
    return n


def _paths(c):
    """The accepted nodes of each sequence's tree, the root first; of a chain the first ones."""
    r = random.Random("paths %d %d" % (c["salt"], c["seqs"]))
    lines = []
    for n in _nodes(c):
        m = _log_int(r, 1, min(n, 8))
        lines.append(list(range(m)) if c["chain"] else [0] + sorted(r.sample(range(1, n), m - 1)))
    return lines


def work(c):
    size = 4 if c["dtype"] == "f32" else 2
    n = _nodes(c)
    if c["op"] == "verify":
        # one row of each kind for every sequence; each node's token, parent and number
        rows = c["seqs"] * (2 if c["drafted"] else 1)
        return {"bytes": rows * c["vocab"] * size + 16 * sum(n) + 12 * c["seqs"],
                "flops": 3 * rows * c["vocab"]}
    d, hkv = c["head_dim"], c["kv_heads"]
    row = d * size
    if c["op"] == "append":
        t, heads = sum(n), c["q_heads"] + 2 * hkv
        table = min(t, max(n) + max(_past(c))) * c["rotary"] * 4
        return {"bytes": 2 * t * heads * row + 12 * t + table,
                "flops": 3 * t * (c["q_heads"] + hkv) * c["rotary"]}
    past = _past(c)
    if c["op"] == "compact":
        moved = sum(i != j for line in _paths(c) for j, i in enumerate(line))
        return {"bytes": 2 * moved * c["pools"] * hkv * row + 8 * sum(n) + 12 * c["seqs"], "flops": 0}
    keys = sum(a + b for a, b in zip(past, n))
    return {"bytes": 2 * keys * hkv * row + 2 * sum(n) * c["q_heads"] * row + 4 * sum(n)
            + 4 * sum(-(-(a + b) // 16) for a, b in zip(past, n)) + 8 * c["seqs"],
            "flops": 4 * c["q_heads"] * d * sum(b * (a + 1) for a, b in zip(past, n))}


# ------------------------------------------------------------------ inputs
def _trees(c, g, n):
    """parents of all nodes, packed: chains, or each node below any earlier one."""
    i = torch.cat([torch.arange(x) for x in n]).cuda()
    if c["chain"]:
        return (i - 1).to(torch.int32)
    below = (torch.rand(len(i), generator=g, device="cuda") * i).long().clamp(max=i - 1)
    return torch.where(i == 0, -1, below).to(torch.int32)


def _within(lens):
    """[b][longest]: which cells are there, and their packed rows (0 where not)."""
    starts = torch.cumsum(lens, 0) - lens
    cell = torch.arange(int(lens.max()), device="cuda")
    there = cell < lens[:, None]
    return there, torch.where(there, starts[:, None] + cell, 0)


def _reach(parents, lens):
    """[b][i][j]: node j is node i or one of its ancestors."""
    there, row = _within(lens)
    n = row.shape[1]
    up = parents[row].long().masked_fill(~there, -1)
    step = (torch.arange(n, device="cuda") == up[:, :, None]).float()
    reach = step + torch.eye(n, device="cuda")
    for _ in range(max(1, n - 1).bit_length()):
        reach = (reach @ reach).clamp(max=1)
    return reach > 0


def _tables(c, g, lens):
    """Block tables in a random order, and how many blocks the pool has."""
    used = [-(-x // 16) for x in lens]
    blocks = sum(used) + 5 + sum(used) // 8
    order = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    held = torch.arange(max(max(used), 1), device="cuda") < torch.tensor(used, device="cuda")[:, None]
    table = torch.full(held.shape, -1, dtype=torch.int32, device="cuda")
    table[held] = order[:sum(used)]
    return table, blocks


def _pool(c, g, blocks, lead=()):
    shape = (*lead, blocks, c["kv_heads"], 16, c["head_dim"])
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(_TYPES[c["dtype"]])


def _slots(table, lens, n):
    """Slots of each sequence's last n positions, packed, and those positions."""
    seq = torch.repeat_interleave(torch.arange(len(n), device="cuda"), n)
    at = torch.arange(len(seq), device="cuda") - torch.repeat_interleave(torch.cumsum(n, 0) - n, n)
    pos = (lens - n)[seq] + at
    return table[seq, pos // 16].long() * 16 + pos % 16, pos


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, n = _TYPES[c["dtype"]], _nodes(c)
    t = sum(n)
    s = dict(c=c, dt=dt, t=t, longest=max(n), n=torch.tensor(n, device="cuda"))
    starts = [0]
    for x in n:
        starts.append(starts[-1] + x)
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    s["parents"] = _trees(c, g, n)
    if c["op"] == "verify":
        _prepare_verify(s, g)
    else:
        past = _past(c)
        lens = [a + b for a, b in zip(past, n)]
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["table"], s["blocks"] = _tables(c, g, lens)
        d, hq, hkv = c["head_dim"], c["q_heads"], c["kv_heads"]
    if c["op"] == "append":
        pad = c["pad"]
        # one projection's output, q, k and v side by side in a token's row
        x = torch.randn((t + pad, hq + 2 * hkv, d), generator=g, device="cuda").to(dt)
        s["q"], s["k"], s["v"] = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        slots, pos = _slots(s["table"], s["lens"].long(), s["n"])
        if not c["chain"]:
            depth = (_reach(s["parents"], s["n"]).sum(-1) - 1)[_within(s["n"])[0]]
            pos = torch.repeat_interleave(s["lens"].long() - s["n"], s["n"]) + depth
        gone = torch.full((pad,), -1, device="cuda")
        s["slots"] = torch.cat([slots, gone]).contiguous()
        s["positions"] = torch.cat([pos, gone]).to(torch.int32).contiguous()
        s["t"], s["max_positions"] = t + pad, max(lens)
        pairs = c["rotary"] // 2
        angle = (torch.arange(max(lens), device="cuda", dtype=torch.float64)[:, None]
                 * _ROPE_BASE ** (-torch.arange(pairs, device="cuda", dtype=torch.float64) / pairs))
        s["cos_sin"] = torch.stack([angle.cos(), angle.sin()], -1).float().contiguous()
        # blocks of earlier tokens are there as well, but what they hold is not read
        s["k_cache"], s["v_cache"] = _small_pools(s, g)
        s["q_out"] = torch.zeros((t + pad, hq, d), dtype=dt, device="cuda")
    elif c["op"] == "tree":
        s["q"] = torch.randn((t, hq, d), generator=g, device="cuda").to(dt)
        s["k_cache"], s["v_cache"] = _pool(c, g, s["blocks"]), _pool(c, g, s["blocks"])
        # what belongs to no sequence may hold anything
        everywhere = torch.ones(s["blocks"] * 16, dtype=torch.bool, device="cuda")
        everywhere[_slots(s["table"], s["lens"].long(), s["lens"].long())[0]] = False
        lost = everywhere.view(-1, 1, 16, 1)
        s["k_cache"].masked_fill_(lost, math.nan)
        s["v_cache"].masked_fill_(lost, math.nan)
        s["out"] = torch.zeros((t, hq, d), dtype=dt, device="cuda")
    elif c["op"] == "compact":
        s["pools"] = _pool(c, g, s["blocks"], (c["pools"],))
        lines = _paths(c)
        path = [x for a, line in zip(n, lines) for x in line + [-1] * (a - len(line))]
        s["path"] = torch.tensor(path, dtype=torch.int32, device="cuda")
        s["path_len"] = torch.tensor([len(x) for x in lines], dtype=torch.int32, device="cuda")
    if own:
        import paged_kv_attention_photon_gb300 as P
        s["lib"] = P
        if c["op"] != "verify":
            s["shape"] = P.PagedShape.make(
                num_seqs=c["seqs"], num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                num_blocks=s["blocks"], max_blocks_per_seq=s["table"].shape[1],
                dtype={"f32": P.F32, "f16": P.F16, "bf16": P.BF16}[c["dtype"]])
        if c["op"] == "tree":
            s["ws_bytes"] = P.photon_paged_tree_attention_workspace_size(s["shape"], t, s["longest"])
            s["ws"] = torch.empty(max(s["ws_bytes"], 16), dtype=torch.uint8, device="cuda")
        if c["op"] == "compact":
            s["layers"] = P.CachePools(list(s["pools"]))
        if c["op"] == "verify":
            s["type"] = {"f32": P.F32, "f16": P.F16, "bf16": P.BF16}[c["dtype"]]
    return s


def _small_pools(s, g):
    """Pools with the blocks of the new tokens alone; slots and tables follow."""
    c = s["c"]
    kept = s["slots"][s["slots"] >= 0]
    used, at = torch.unique(kept // 16, return_inverse=True)
    order = torch.randperm(len(used) + 3, generator=g, device="cuda")
    s["slots"][s["slots"] >= 0] = order[at] * 16 + kept % 16
    s["blocks"] = len(used) + 3
    return _pool(c, g, s["blocks"]), _pool(c, g, s["blocks"])


def _prepare_verify(s, g):
    c, t, v = s["c"], s["t"], s["c"]["vocab"]
    # the target's logits, and the draft's, which are near them
    logits = 4 * torch.randn((t, v), generator=g, device="cuda")
    near = logits + 1.5 * torch.randn((t, v), generator=g, device="cuda")
    s["target"] = torch.softmax(logits, -1).to(s["dt"])
    draft = torch.softmax(near, -1).to(s["dt"])
    first = s["starts"][:-1].long()
    above = torch.repeat_interleave(first, s["n"]) + s["parents"].long()
    root = s["parents"] < 0
    above = torch.where(root, 0, above)
    s["tokens"] = torch.zeros(t, dtype=torch.int32, device="cuda")
    if c["drafted"]:
        # each child drawn from its parent's distribution
        race = torch.empty((t, v), device="cuda").exponential_(generator=g)
        s["tokens"] = (draft[above].float() / race).argmax(-1).to(torch.int32)
        s["draft"] = draft
    else:
        # the children of a node are its most likely tokens in order
        rank = (above[:, None] == above[None]) & ~root[:, None] & ~root[None]
        rank = torch.tril(rank, -1).sum(-1)
        top = draft.topk(int(rank.max()) + 1, dim=-1).indices
        s["tokens"] = top[above, rank].to(torch.int32)
    s["accept"] = torch.rand(t, generator=g, device="cuda")
    s["sample"] = torch.rand(c["seqs"], generator=g, device="cuda")
    s["path"] = torch.zeros(t, dtype=torch.int32, device="cuda")
    s["path_len"] = torch.zeros(c["seqs"], dtype=torch.int32, device="cuda")
    s["next"] = torch.zeros(c["seqs"], dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ one pass
def run(s):
    c = s["c"]
    if own:
        P = s["lib"]
        if c["op"] == "append":
            P.photon_rope_cache_append(s["q"], s["q"].stride(0), s["k"], s["k"].stride(0), s["v"],
                                       s["v"].stride(0), s["positions"], s["cos_sin"],
                                       s["max_positions"], c["rotary"], int(c["interleaved"]),
                                       s["slots"], s["t"], s["q_out"], 0, s["k_cache"],
                                       s["v_cache"], s["shape"])
            return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        if c["op"] == "tree":
            P.photon_paged_tree_attention(s["q"], s["k_cache"], s["v_cache"], s["table"],
                                          s["lens"], s["starts"], s["parents"], s["t"],
                                          s["longest"], c["head_dim"] ** -0.5, s["out"], s["ws"],
                                          s["ws_bytes"], s["shape"])
            return s["out"]
        if c["op"] == "verify":
            P.photon_verify_tree(s["target"], 0, s.get("draft"), 0, c["vocab"], s["type"],
                                 s["tokens"], s["parents"], s["starts"], s["accept"], s["sample"],
                                 c["seqs"], s["t"], s["longest"], s["path"], s["path_len"],
                                 s["next"])
            return {"path": s["path"], "path_len": s["path_len"], "next": s["next"]}
        P.photon_cache_compact(s["layers"], s["table"], s["lens"], s["starts"], s["path"],
                               s["path_len"], s["t"], s["longest"], s["shape"])
        return s["pools"]
    return {"append": _append, "tree": _tree, "verify": _verify, "compact": _compact}[c["op"]](s)


def _turned(s, x):
    """x [t][heads][d] turned by the positions, in 32 bits."""
    c, half = s["c"], s["c"]["rotary"] // 2
    x = x.float()
    turn = s["cos_sin"][s["positions"].long().clamp(min=0)][:, None]
    cos, sin = turn[..., 0], turn[..., 1]
    rest = x[..., 2 * half:]
    if c["interleaved"]:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, rest], -1).to(s["dt"])


def _append(s):
    kept = s["slots"] >= 0
    slot = s["slots"][kept]
    s["k_cache"][slot // 16, :, slot % 16] = _turned(s, s["k"])[kept]
    s["v_cache"][slot // 16, :, slot % 16] = s["v"][kept]
    there = (s["positions"] >= 0)[:, None, None]
    s["q_out"].copy_(torch.where(there, _turned(s, s["q"]), s["q_out"]))
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _dense(s, pool):
    """The contexts' rows in 32 bits, [b][hkv][rows][d], zero behind each one's end."""
    x = pool[s["table"].long().clamp(min=0)].float()                    # [b][blocks][hkv][16][d]
    x = x.transpose(1, 2).flatten(2, 3)
    behind = torch.arange(x.shape[2], device="cuda") >= s["lens"][:, None]
    return x.masked_fill_(behind[:, None, :, None], 0)


def _tree(s):
    c = s["c"]
    hq, hkv, d = c["q_heads"], c["kv_heads"], c["head_dim"]
    there, row = _within(s["n"])
    b, n = row.shape
    k, v = _dense(s, s["k_cache"]), _dense(s, s["v_cache"])
    rows = k.shape[2]
    first = (s["lens"] - s["n"])[:, None]                               # the tree's first row
    cell = torch.arange(rows, device="cuda") - first
    seen = _reach(s["parents"], s["n"])                                 # [b][n][n]
    seen = seen.gather(2, cell.clamp(0, n - 1)[:, None].expand(b, n, rows).long())
    seen = seen & (cell < s["n"][:, None])[:, None] | (cell < 0)[:, None]
    q = s["q"][row].float().view(b, n, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).flatten(2, 3)
    p = torch.matmul(q, k.transpose(2, 3)).mul_(d ** -0.5)              # [b][hkv][g n][rows]
    p.unflatten(2, (-1, n)).masked_fill_(~seen[:, None, None], -math.inf)
    p.sub_(p.amax(-1, keepdim=True)).exp_()
    p.div_(p.sum(-1, keepdim=True))
    o = torch.matmul(p, v).unflatten(2, (-1, n)).permute(0, 3, 1, 2, 4).reshape(b, n, hq, d)
    return o[there].to(s["dt"])


def _verify(s):
    c = s["c"]
    at, n = s["starts"][:-1].long(), s["n"]
    seqs = torch.arange(len(n), device="cuda")
    drafted = c["drafted"]
    # r = max(0, scale p - less q); without a draft, p but for the tokens that are out
    scale = torch.ones(len(n), dtype=torch.float64, device="cuda")
    less, total = torch.zeros_like(scale), torch.ones_like(scale)
    out = torch.zeros((len(n), c["vocab"]), dtype=torch.bool, device="cuda")
    cur, count = at.clone(), torch.ones_like(at)
    path = torch.full((s["t"],), -1, dtype=torch.int32, device="cuda")
    path[at] = 0

    def left():
        p = s["target"][cur].double()
        if drafted:
            return (scale[:, None] * p - less[:, None] * s["draft"][cur].double()).clamp(min=0)
        return p.masked_fill(out, 0)

    for i in range(1, s["longest"]):
        row = torch.where(i < n, at + i, at)
        asked = (i < n) & (at + s["parents"][row] == cur)
        x = s["tokens"][row].long()
        p = s["target"][cur, x].double()
        if drafted:
            q = s["draft"][cur, x].double()
            r = (scale * p - less * q).clamp(min=0)
        else:
            q = 1.0
            r = p.masked_fill(out[seqs, x], 0)
        yes = asked & (r > s["accept"][row].double() * total * q)
        no = asked & ~yes
        # the walk goes on at node i
        place = torch.where(yes, at + count, at)
        path[place] = torch.where(yes, i, path[place]).to(torch.int32)
        count = count + yes
        cur = torch.where(yes, row, cur)
        if drafted:
            safe = torch.where(total > 0, total, 1.0)
            scale = torch.where(no, scale / safe, scale)
            less = torch.where(no, less / safe + 1, less)
            total = torch.where(no, left().sum(-1), total)
        else:
            total = torch.where(no, (total - r).clamp(min=0), total)
            out[seqs, x] |= no
            out &= ~yes[:, None]
        scale, total = torch.where(yes, 1.0, scale), torch.where(yes, 1.0, total)
        less = torch.where(yes, 0.0, less)
    r = left()
    r = torch.where((r.sum(-1) > 0)[:, None], r, s["target"][cur].double())
    sums = torch.cumsum(r, -1)
    passed = sums > s["sample"].double()[:, None] * sums[:, -1:]
    return {"path": path, "path_len": count.to(torch.int32),
            "next": passed.to(torch.uint8).argmax(-1).to(torch.int32)}


def _compact(s):
    """Every path's rows, read before any is written."""
    seq = torch.repeat_interleave(torch.arange(len(s["n"]), device="cuda"), s["n"])
    place = torch.arange(s["t"], device="cuda") - s["starts"][seq].long()
    kept = s["path"] >= 0
    seq, place, node = seq[kept], place[kept], s["path"][kept].long()
    first = (s["lens"].long() - s["n"])[seq]

    def slot(pos):
        return s["table"][seq, pos // 16].long(), pos % 16

    (a, i), (b, j) = slot(first + node), slot(first + place)
    s["pools"][:, b, :, j] = s["pools"][:, a, :, i]
    return s["pools"]


# ------------------------------------------------------------------ in 64 bits
def exact(c, seed):
    s = prepare(c, seed)
    return {"append": _exact_append, "tree": _exact_tree, "verify": _exact_verify,
            "compact": _exact_compact}[c["op"]](s)


def _exact_append(s):
    c, r = s["c"], s["c"]["rotary"]
    pairs = torch.arange(r // 2, device="cuda")
    one = 2 * pairs if c["interleaved"] else pairs
    two = one + 1 if c["interleaved"] else pairs + r // 2
    turn = s["cos_sin"].double()[s["positions"].long().clamp(min=0)]
    z = torch.complex(turn[..., 0], turn[..., 1])[:, None]

    def turned(x):
        x = x.double()
        w = torch.complex(x[..., one], x[..., two]) * z
        y = x.clone()
        y[..., one], y[..., two] = w.real, w.imag
        return y

    q = torch.where((s["positions"] >= 0)[:, None, None], turned(s["q"]), 0.0)
    pools = []
    for pool, x in ((s["k_cache"], turned(s["k"])), (s["v_cache"], s["v"].double())):
        flat = pool.double().transpose(1, 2).reshape(-1, c["kv_heads"], c["head_dim"])
        kept = s["slots"] >= 0
        flat[s["slots"][kept]] = x[kept]
        pools.append(flat.view(-1, 16, c["kv_heads"], c["head_dim"]).transpose(1, 2).contiguous())
    return {"q": q, "k_cache": pools[0], "v_cache": pools[1]}


def _ancestors(parents):
    """For each node of one tree (a list of parents) itself and its ancestors, root first."""
    lines = []
    for i, up in enumerate(parents):
        lines.append((lines[up] if up >= 0 else []) + [i])
    return lines


def _exact_tree(s):
    c = s["c"]
    hq, hkv, d = c["q_heads"], c["kv_heads"], c["head_dim"]
    out = torch.zeros((s["t"], hq, d), dtype=torch.float64, device="cuda")
    first = s["starts"].tolist()
    for b, (n, length) in enumerate(zip(s["n"].tolist(), s["lens"].tolist())):
        j = torch.arange(length, device="cuda")
        block = s["table"][b, j // 16].long()
        k = s["k_cache"][block, :, j % 16].double()                     # [len][hkv][d]
        v = s["v_cache"][block, :, j % 16].double()
        seen = torch.zeros((n, length), dtype=torch.bool)
        seen[:, :length - n] = True
        for i, line in enumerate(_ancestors(s["parents"][first[b]:first[b + 1]].tolist())):
            seen[i, [length - n + x for x in line]] = True
        q = s["q"][first[b]:first[b + 1]].double().view(n, hkv, hq // hkv, d)
        score = torch.einsum("nhgd,jhd->hgnj", q, k) / math.sqrt(d)
        w = torch.softmax(score.masked_fill(~seen.cuda(), -math.inf), -1)
        out[first[b]:first[b + 1]] = torch.einsum("hgnj,jhd->nhgd", w, v).reshape(n, hq, d)
    return out


def _exact_verify(s):
    """A walk down each tree."""
    tokens, parents, u = s["tokens"].tolist(), s["parents"].tolist(), s["accept"].double().tolist()
    path = torch.full((s["t"],), -1, dtype=torch.int32)
    lengths, nexts = [], []
    first = s["starts"].tolist()
    for b, n in enumerate(s["n"].tolist()):
        node, line = 0, [0]
        while True:
            row = first[b] + node
            p = s["target"][row].double()
            r, z, down = p, 1.0, None
            for i in range(node + 1, n):
                if parents[first[b] + i] != node:
                    continue
                x = tokens[first[b] + i]
                if s["c"]["drafted"]:
                    q = s["draft"][row].double()
                    if float(r[x]) > u[first[b] + i] * z * float(q[x]):
                        down = i
                        break
                    r = torch.clamp(r / z - q if z > 0 else torch.zeros_like(r), min=0)
                    z = float(r.sum())
                else:
                    if float(r[x]) > u[first[b] + i] * z:
                        down = i
                        break
                    z = max(z - float(r[x]), 0.0)
                    r = r.clone()
                    r[x] = 0
            if down is None:
                break
            node = down
            line.append(down)
        if not float(r.sum()) > 0:
            r = p
        path[first[b]:first[b] + len(line)] = torch.tensor(line, dtype=torch.int32)
        lengths.append(len(line))
        sums = torch.cumsum(r, 0)
        nexts.append(int(torch.searchsorted(sums, float(s["sample"][b]) * float(sums[-1]), right=True)))
    return {"path": path, "path_len": torch.tensor(lengths, dtype=torch.int32),
            "next": torch.tensor(nexts, dtype=torch.int32)}


def _exact_compact(s):
    pools = s["pools"].double()
    held = pools.clone()
    first = s["starts"].tolist()
    for b, (n, length) in enumerate(zip(s["n"].tolist(), s["lens"].tolist())):
        table = s["table"][b].tolist()
        for j, node in enumerate(s["path"][first[b]:first[b] + int(s["path_len"][b])].tolist()):
            to, of = length - n + j, length - n + node
            pools[:, table[to // 16], :, to % 16] = held[:, table[of // 16], :, of % 16]
    return pools
