"""Measured cases of the 4-bit serving path: what a prompt and a decode step
do with q, k and v between the projections and the attention's output.

Four operators, named by a case's "op":

* "qk": per-head RMS norm of q and k, with the position rotation (one axis, or
  several: time, height, width) in the same pass (photon_qk_norm_rope);
* "prompt": causal attention of whole prompts, packed one after another, over
  their own K and V rows (photon_prompt_attention);
* "write": the K/V rows of new tokens quantised to 4 bits into the paged cache
  (photon_cache_write_int4), and the rows of the contexts read back as values
  (photon_paged_gather_int4);
* "decode": attention of one new token per sequence over the 4-bit paged cache
  (photon_paged_decode_int4).

The 4-bit cache.  A row of head_dim elements of one (token, KV head) has two
numbers in the storage type: lo, its smallest element, and step = (largest -
smallest) / 15, rounded to that type.  Element x is held as the code
n = clamp(round_half_even((x - lo) / step), 0, 15) (0 where step is 0) and
stands for lo + n * step.  A pool has one record per (block, KV head), of 8 *
head_dim + 64 bytes: the codes of 16 rows, then 16 pairs (step, lo).  K codes:
row by row, two elements a byte, the lower one in the low nibble.  V codes:
rows in pairs; of a pair, four elements (two bytes) of the even row, then the
same four of the odd row, and so on along the row.
"""
import math
import random

import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_ROPE_BASE = 1e6
_EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    qwen = dict(q_heads=16, kv_heads=8, head_dim=128)   # the library's long-context decode shape
    llama = dict(q_heads=32, kv_heads=8, head_dim=64)   # its batch sweep and its batch-256 mix
    return [
        # the new tokens of one decode step of 64 sequences: latency counts
        dict(name="qk_step_b64", op="qk", seqs=64, lo=128, hi=8192, step=True, salt=1, pad=0,
             axes=1, dealt=False, rotary=128, dtype="f16", **qwen),
        # sixteen prompts of 1024 tokens, as the prefill benchmark has them
        dict(name="qk_prompt_16x1024", op="qk", seqs=16, lo=1024, hi=1024, step=False, salt=2,
             pad=0, axes=1, dealt=False, rotary=128, dtype="bf16", **qwen),
        # prompts with images: three axes dealt in turn, a padded batch, 32-bit activations
        dict(name="qk_image_ragged", op="qk", seqs=11, lo=37, hi=2048, step=False, salt=3, pad=5,
             axes=3, dealt=True, rotary=64, dtype="f32", **llama),
        dict(name="prompt_16x1024", op="prompt", seqs=16, lo=1024, hi=1024, salt=4, pad=0,
             dtype="f16", **qwen),
        # a batch of chat prompts of every length, one of them empty, rows behind the last
        dict(name="prompt_ragged", op="prompt", seqs=24, lo=1, hi=2048, salt=5, pad=7,
             dtype="bf16", **llama),
        # one long document
        dict(name="prompt_1x16384", op="prompt", seqs=1, lo=16384, hi=16384, salt=6, pad=0,
             dtype="bf16", **qwen),
        # one new row per sequence, into blocks that hold earlier ones
        dict(name="write_step_b64", op="write", seqs=64, lo=1, hi=16, step=True, salt=7, pad=0,
             dtype="f16", **qwen),
        dict(name="write_prompt_16x1024", op="write", seqs=16, lo=1024, hi=1024, step=False,
             salt=8, pad=0, dtype="bf16", **qwen),
        # ragged prompts in a padded batch
        dict(name="write_ragged", op="write", seqs=24, lo=1, hi=2048, step=False, salt=9, pad=13,
             dtype="f16", **llama),
        # a small batch: the library's sweep at batch 4
        dict(name="decode_b4", op="decode", seqs=4, lo=64, hi=2048, salt=10, long=0.0,
             dtype="f16", **llama),
        # 64 long contexts in a fragmented pool
        dict(name="decode_b64", op="decode", seqs=64, lo=128, hi=8192, salt=11, long=0.0,
             dtype="f16", **qwen),
        # a serving mix: four short contexts to each long one
        dict(name="decode_mix_b256", op="decode", seqs=256, lo=32, hi=512, salt=12, long=0.2,
             dtype="bf16", **llama),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qk", "prompt", "write", "decode"])
    q_heads, kv_heads = rng.choice([(16, 8), (32, 8), (16, 16), (8, 1), (4, 2), (24, 3), (32, 4)])
    head_dim = rng.choice([64, 128])
    c = dict(op=op, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim,
             dtype=rng.choice(["f16", "bf16"]), salt=rng.randrange(1 << 20))
    if op == "qk":
        c["dtype"] = rng.choice(["f16", "bf16", "f32"])
        c["axes"] = rng.choice([1, 1, 2, 3, 4])
        c["dealt"] = c["axes"] > 1 and rng.random() < 0.5
        c["rotary"] = rng.choice([head_dim, head_dim, head_dim // 2])
        c["step"] = rng.random() < 0.3
        c["pad"] = rng.choice([0, 0, 3, 17])
        if c["step"]:
            c.update(seqs=_log_int(rng, 1, 512), lo=1, hi=_log_int(rng, 16, 16384))
        else:
            c["hi"] = _log_int(rng, 2, 8192)
            c["lo"] = _log_int(rng, 1, c["hi"])
            width = (q_heads + kv_heads) * head_dim * (2 if c["dtype"] == "f32" else 1)
            most = 16384 * 24 * 128 // width
            c["seqs"] = max(1, min(_log_int(rng, 1, 64), most // c["hi"]))
    elif op == "prompt":
        c["hi"] = _log_int(rng, 2, 8192)
        c["lo"] = _log_int(rng, 1, c["hi"])
        most = 16384 * 16384 * 16 * 128 // (q_heads * head_dim) // c["hi"] ** 2
        c["seqs"] = max(1, min(_log_int(rng, 1, 64), most))
        c["pad"] = rng.choice([0, 0, 1, 19])
    elif op == "write":
        c["step"] = rng.random() < 0.3
        c["pad"] = rng.choice([0, 0, 2, 31])
        if c["step"]:
            c.update(seqs=_log_int(rng, 1, 512), lo=1, hi=16)
        else:
            c["hi"] = _log_int(rng, 2, 8192)
            c["lo"] = _log_int(rng, 1, c["hi"])
            most = 16384 * 8 * 128 // (kv_heads * head_dim) // c["hi"]
            c["seqs"] = max(1, min(_log_int(rng, 1, 64), most))
    else:
        c["hi"] = _log_int(rng, 17, 16384)
        c["lo"] = _log_int(rng, 1, c["hi"])
        c["long"] = 0.0
        most = 64 * 8192 * 8 * 128 // (kv_heads * head_dim) // c["hi"]
        c["seqs"] = max(1, min(_log_int(rng, 1, 256), most))
    return c


def _lengths(c):
    """The sequences' lengths: log-uniform in [lo, hi]; a `long` share of a serving mix
    uniform in [4096, 16384]; in a ragged prompt batch of over 20 one empty prompt."""
    r = random.Random("%d %d %d %d" % (c["salt"], c["seqs"], c["lo"], c["hi"]))
    n = [_log_int(r, c["lo"], c["hi"]) for _ in range(c["seqs"])]
    if c.get("long"):
        n = [r.randint(4096, 16384) if r.random() < c["long"] else x for x in n]
    if c["op"] == "prompt" and c["seqs"] > 20:
        n[7] = 0
    return n


def _tokens(c):
    """Rows of the call: one per sequence in a decode step, and the padding behind them."""
    return (c["seqs"] if c.get("step") else sum(_lengths(c))) + c.get("pad", 0)


def _record(c):
    return 8 * c["head_dim"] + 64


def work(c):
    size = 4 if c["dtype"] == "f32" else 2
    d, hq, hkv, n = c["head_dim"], c["q_heads"], c["kv_heads"], _lengths(c)
    row = d * size
    if c["op"] == "qk":
        t = c["seqs"] if c["step"] else sum(n)
        table = min(t, max(n)) * c["rotary"] * 4
        return {"bytes": 2 * t * (hq + hkv) * row + 4 * c["axes"] * t + table + 2 * row,
                "flops": t * (hq + hkv) * d * 8}
    if c["op"] == "prompt":
        t = sum(n)
        return {"bytes": t * (2 * hq + 2 * hkv) * row + 4 * (c["seqs"] + 1),
                "flops": 4 * hq * d * sum(x * (x + 1) // 2 for x in n)}
    if c["op"] == "write":
        t = c["seqs"] if c["step"] else sum(n)
        blocks = sum(-(-x // 16) for x in n)
        dense = c["seqs"] * -(-max(n) // 16) * 16
        held = d // 2 + 4
        return {"bytes": 2 * hkv * (t * (row + held) + sum(n) * held + dense * row) + 8 * t + 4 * blocks,
                "flops": 2 * hkv * d * (4 * t + 2 * sum(n))}
    return {"bytes": sum(n) * hkv * (d + 8) + 2 * c["seqs"] * hq * row + 4 * c["seqs"]
            + 4 * sum(-(-x // 16) for x in n),
            "flops": 4 * sum(n) * hq * d}


# ------------------------------------------------------------------ inputs
def _sections(c):
    """Pairs of each axis: the first axis takes what is left over."""
    pairs, a = c["rotary"] // 2, c["axes"]
    each = pairs // (a + 1) if a > 1 else 0
    return [pairs - (a - 1) * each] + [each] * (a - 1)


def _starts(n):
    s = [0]
    for x in n:
        s.append(s[-1] + x)
    return s


def _rows(g, shape, dtype, spread):
    """Activations: normal, with a few channels that are several times larger."""
    x = torch.randn(shape, generator=g, device="cuda")
    channel = 1 + spread * (torch.rand(shape[-1], generator=g, device="cuda") > 0.95)
    return (x * channel).to(dtype)


def _pool_of(c, g, blocks):
    """A pool of that many blocks: codes with a bell-shaped spread, steps and minima as
    normal rows have them; then the records of blocks that no table names."""
    rec, d, hkv = _record(c), c["head_dim"], c["kv_heads"]
    spare = 5 + blocks // 8
    pool = torch.full((blocks + spare, hkv, rec), 255, dtype=torch.uint8, device="cuda")
    r = [torch.randint(0, 256, (blocks, hkv, 8 * d), dtype=torch.uint8, generator=g, device="cuda")
         for _ in range(3)]
    pool[:blocks, :, :8 * d] = (r[0] & 0x77) + (r[1] & 0x77) + (r[2] & 0x11)
    step = 0.25 + 0.25 * torch.rand(blocks, hkv, 16, generator=g, device="cuda")
    lo = -7.5 * step * (0.8 + 0.4 * torch.rand(blocks, hkv, 16, generator=g, device="cuda"))
    pairs = torch.stack([step, lo], -1).to(_TYPES[c["dtype"]]).contiguous()
    pool[:blocks, :, 8 * d:] = pairs.view(torch.uint8).view(blocks, hkv, 64)
    return pool


def _paged(c, g):
    """Pools, block tables in a random order, and the contexts' lengths; what a pool holds
    behind a context's end is garbage."""
    n = _lengths(c)
    used = [-(-x // 16) for x in n]
    blocks, most = sum(used), max(max(used), 1)
    k, v = _pool_of(c, g, blocks), _pool_of(c, g, blocks)
    order = torch.randperm(k.shape[0], generator=g, device="cuda")
    k, v = k[torch.argsort(order)], v[torch.argsort(order)]     # record i now sits at order[i]
    count = torch.tensor(used, device="cuda")
    cell = torch.arange(most, device="cuda")
    held = cell < count[:, None]
    table = torch.full((c["seqs"], most), -1, dtype=torch.int32, device="cuda")
    table[held] = order[:blocks].to(torch.int32)
    lens = torch.tensor(n, dtype=torch.int32, device="cuda")
    last = torch.tensor([x - 1 for x in used], device="cuda").clamp(min=0)
    at = table.gather(1, last[:, None]).long().squeeze(1)
    pos = last[:, None] * 16 + torch.arange(16, device="cuda")
    behind = (pos >= lens[:, None])[:, None, :, None].expand(-1, c["kv_heads"], -1, 4)
    for pool in (k, v):
        pairs = pool[at][:, :, 8 * c["head_dim"]:].reshape(c["seqs"], c["kv_heads"], 16, 4)
        pairs = torch.where(behind, torch.full_like(pairs, 255), pairs)
        full = pool[at]
        full[:, :, 8 * c["head_dim"]:] = pairs.reshape(c["seqs"], c["kv_heads"], 64)
        pool[at] = full
    return dict(k_cache=k, v_cache=v, table=table, lens=lens)


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, n = _TYPES[c["dtype"]], _lengths(c)
    d, hq, hkv, t = c["head_dim"], c["q_heads"], c["kv_heads"], _tokens(c)
    s = dict(c=c, dt=dt, t=t)

    def fused():
        """One projection's output, q, k and v side by side in a token's row."""
        x = _rows(g, (t, hq + 2 * hkv, d), dt, 4.0)
        return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]

    if c["op"] == "qk":
        s["q"], s["k"], _ = fused()
        s["q_weight"] = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(dt)
        s["k_weight"] = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(dt)
        if c["step"]:
            pos = torch.tensor([x - 1 for x in n], device="cuda")
        else:
            pos = torch.cat([torch.arange(x, device="cuda") for x in n])
        pos = torch.cat([pos, torch.full((c["pad"],), -1, device="cuda")])
        # the first axis counts on, the others walk rows and columns of an image
        pos = torch.stack([pos if a == 0 else torch.where(pos < 0, pos, pos // 7 ** (a - 1) % 29)
                           for a in range(c["axes"])])
        s["positions"] = pos.to(torch.int32).contiguous()
        s["max_positions"] = max(max(n), 29)
        pairs = c["rotary"] // 2
        angle = (torch.arange(s["max_positions"], device="cuda", dtype=torch.float64)[:, None]
                 * _ROPE_BASE ** (-torch.arange(pairs, device="cuda", dtype=torch.float64) / pairs))
        s["cos_sin"] = torch.stack([angle.cos(), angle.sin()], -1).float().contiguous()
        axis = torch.zeros(pairs, dtype=torch.long)
        left = _sections(c)
        at = left[0]
        for a in range(1, c["axes"]):
            if c["dealt"]:
                axis[a:a + c["axes"] * left[a]:c["axes"]] = a
            else:
                axis[at:at + left[a]] = a
                at += left[a]
        s["axis"] = axis.cuda()
        s["q_out"] = torch.zeros((t, hq, d), dtype=dt, device="cuda")
        s["k_out"] = torch.zeros((t, hkv, d), dtype=dt, device="cuda")
    elif c["op"] == "prompt":
        _, _, s["v"] = fused()
        s["q"] = torch.randn((t, hq, d), generator=g, device="cuda").to(dt)
        s["k"] = torch.randn((t, hkv, d), generator=g, device="cuda").to(dt)
        starts = _starts(n)
        s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        s["longest"] = max(n)
        s["out"] = torch.zeros((t, hq, d), dtype=dt, device="cuda")
    else:
        s.update(_paged(c, g))
        if c["op"] == "decode":
            s["q"] = torch.randn((c["seqs"], hq, d), generator=g, device="cuda").to(dt)
            s["out"] = torch.zeros((c["seqs"], hq, d), dtype=dt, device="cuda")
        else:
            _, k, s["v"] = fused()
            s["k"] = k.contiguous()
            seq = torch.arange(c["seqs"], device="cuda")
            lens = s["lens"].long()
            if c["step"]:
                pos = lens - 1
            else:
                seq = torch.repeat_interleave(seq, lens)
                pos = torch.cat([torch.arange(x, device="cuda") for x in n])
            slots = s["table"][seq, pos // 16].long() * 16 + pos % 16
            s["slots"] = torch.cat([slots, torch.full((c["pad"],), -1, device="cuda")]).contiguous()
            shape = (c["seqs"], hkv, s["table"].shape[1] * 16, d)
            s["k_dense"] = torch.zeros(shape, dtype=dt, device="cuda")
            s["v_dense"] = torch.zeros(shape, dtype=dt, device="cuda")
    if own:
        import paged_kv_attention_photon_gb300 as P
        s["lib"] = P
        cache = "k_cache" in s
        s["shape"] = P.PagedShape.make(
            num_seqs=c["seqs"], num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
            num_blocks=s["k_cache"].shape[0] if cache else 0,
            max_blocks_per_seq=s["table"].shape[1] if cache else 1,
            dtype={"f32": P.F32, "f16": P.F16, "bf16": P.BF16}[c["dtype"]])
        if c["op"] == "qk":
            s["rope_axes"] = P.RopeAxes.make(_sections(c), interleaved=c["dealt"])
        if c["op"] == "decode":
            s["ws_bytes"] = P.photon_paged_decode_int4_workspace_size(s["shape"])
            s["ws"] = torch.empty(max(s["ws_bytes"], 16), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    c = s["c"]
    if own:
        P = s["lib"]
        if c["op"] == "qk":
            P.photon_qk_norm_rope(s["q"], s["q"].stride(0), s["k"], s["k"].stride(0),
                                  s["q_weight"], s["k_weight"], _EPS, s["positions"],
                                  s["cos_sin"], s["max_positions"], s["rope_axes"], s["t"],
                                  s["q_out"], 0, s["k_out"], 0, s["shape"])
            return {"q": s["q_out"], "k": s["k_out"]}
        if c["op"] == "prompt":
            P.photon_prompt_attention(s["q"], 0, s["k"], 0, s["v"], s["v"].stride(0), s["starts"],
                                      s["t"], s["longest"], c["head_dim"] ** -0.5, s["out"], 0,
                                      s["shape"])
            return s["out"]
        if c["op"] == "write":
            P.photon_cache_write_int4(s["k"], 0, s["v"], s["v"].stride(0), s["slots"], s["t"],
                                      s["k_cache"], s["v_cache"], s["shape"])
            P.photon_paged_gather_int4(s["k_cache"], s["v_cache"], s["table"], s["lens"],
                                       s["k_dense"], s["v_dense"], s["shape"])
            return {"k": s["k_dense"], "v": s["v_dense"]}
        P.photon_paged_decode_int4(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                                   c["head_dim"] ** -0.5, s["out"], s["ws"], s["ws_bytes"],
                                   s["shape"])
        return s["out"]
    if c["op"] == "qk":
        return {"q": _norm_rope(s, s["q"], s["q_weight"]), "k": _norm_rope(s, s["k"], s["k_weight"])}
    if c["op"] == "prompt":
        return _prompt(s)
    if c["op"] == "write":
        _write(s, s["k"], s["k_cache"], True)
        _write(s, s["v"], s["v_cache"], False)
        k, v = _held(s)
        return {"k": k.to(s["dt"]).transpose(1, 2).contiguous(),
                "v": v.to(s["dt"]).transpose(1, 2).contiguous()}
    return _decode(s)


def _norm_rope(s, x, weight):
    x = x.float()
    half = s["c"]["rotary"] // 2
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS) * weight.float()
    pos = s["positions"].long()
    at = pos[s["axis"]].clamp(min=0).T                                  # [t][pairs]
    turn = s["cos_sin"][at, torch.arange(half, device="cuda")]          # [t][pairs][2]
    cos, sin = turn[:, None, :, 0], turn[:, None, :, 1]
    a, b = y[..., :half], y[..., half:2 * half]
    y = torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., 2 * half:]], -1)
    return torch.where((pos[0] >= 0)[:, None, None], y, 0.0).to(s["dt"])


def _prompt(s):
    c, n = s["c"], s["longest"]
    hq, hkv, d = c["q_heads"], c["kv_heads"], c["head_dim"]
    starts = s["starts"].long()
    lens = starts[1:] - starts[:-1]
    cell = torch.arange(n, device="cuda")
    there = cell < lens[:, None]                                        # [b][n]
    row = torch.where(there, starts[:-1, None] + cell, 0)
    q = s["q"][row].float().view(-1, n, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    k = s["k"][row].float().permute(0, 2, 3, 1)[:, :, None]             # [b][hkv][1][d][n]
    v = s["v"][row].float().transpose(1, 2)[:, :, None]                 # [b][hkv][1][n][d]
    p = torch.matmul(q, k).mul_(d ** -0.5)                              # [b][hkv][g][n][n]
    p.masked_fill_(cell[None, :] > cell[:, None], -math.inf)
    p.sub_(p.amax(-1, keepdim=True)).exp_()
    p.div_(p.sum(-1, keepdim=True))
    o = torch.matmul(p, v).permute(0, 3, 1, 2, 4).reshape(-1, n, hq, d)
    out = torch.zeros((s["t"], hq, d), dtype=s["dt"], device="cuda")
    out[row[there]] = o[there].to(s["dt"])
    return out


def _round_once(x, dtype):
    """64-bit values rounded to a 16-bit type with one rounding: first to 32 bits towards
    zero with the rest in the last bit, which the second rounding then sees."""
    f = x.float()
    off = f.double() != x
    bits = f.view(torch.int32)
    bits = torch.where(off & (f.double().abs() > x.abs()), bits - 1, bits)
    return torch.where(off, bits | 1, bits).view(torch.float32).to(dtype)


def _codes_of(pool, d, keys):
    """The pool's codes as bytes of two elements, [blocks][hkv][16 rows ...][d / 2]."""
    codes = pool[:, :, :8 * d]
    return codes.view(*codes.shape[:2], 16, d // 2) if keys else codes.view(*codes.shape[:2], 8, d // 4, 2, 2)


def _write(s, x, pool, keys):
    """Rows quantised in 64 bits (a code next to a border goes by the last bits) and stored."""
    d, dt = s["c"]["head_dim"], s["dt"]
    kept = s["slots"] >= 0
    slot, x = s["slots"][kept], x[kept].double()
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    step = _round_once((hi - lo) / 15, dt)
    n = torch.where(step == 0, 0.0, (x - lo) / step.double()).round().clamp(0, 15).to(torch.uint8)
    packed = n[..., ::2] | (n[..., 1::2] << 4)
    block, row = slot // 16, slot % 16
    if keys:
        _codes_of(pool, d, True)[block, :, row] = packed
    else:
        _codes_of(pool, d, False)[block, :, row // 2, :, row % 2] = packed.view(*packed.shape[:2], d // 4, 2)
    pairs = torch.cat([step, lo.to(dt)], -1)                            # [t][hkv][2]
    pool[:, :, 8 * d:].view(dt).view(*pool.shape[:2], 16, 2)[block, :, row] = pairs


def _held(s):
    """The contexts' K and V in 32 bits, [b][rows][hkv][d], zero behind each context's end."""
    c, dt = s["c"], s["dt"]
    d, hkv = c["head_dim"], c["kv_heads"]
    table = s["table"].long().clamp(min=0)
    b, most = table.shape
    rows = most * 16
    there = (torch.arange(rows, device="cuda") < s["lens"][:, None])[:, :, None, None]

    def values(pool, keys):
        blocks = pool[table.view(-1)]
        codes = _codes_of(blocks, d, keys)
        codes = codes if keys else codes.transpose(3, 4).reshape(-1, hkv, 16, d // 2)
        n = torch.stack([codes & 15, codes >> 4], -1).view(-1, hkv, 16, d)
        pairs = blocks[:, :, 8 * d:].contiguous().view(dt).view(-1, hkv, 16, 2).float()
        x = n * pairs[..., :1] + pairs[..., 1:]
        x = x.transpose(1, 2).reshape(b, rows, hkv, d)
        return torch.where(there, x, 0.0)

    return values(s["k_cache"], True), values(s["v_cache"], False)


def _decode(s):
    c = s["c"]
    hq, hkv, d = c["q_heads"], c["kv_heads"], c["head_dim"]
    k, v = _held(s)
    q = s["q"].float().view(-1, hkv, hq // hkv, d)
    p = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(d ** -0.5)          # [b][hkv][g][rows]
    behind = torch.arange(p.shape[-1], device="cuda") >= s["lens"][:, None]
    p.masked_fill_(behind[:, None, None], -math.inf)
    p.sub_(p.amax(-1, keepdim=True)).exp_()
    p.div_(p.sum(-1, keepdim=True))
    return torch.matmul(p, v.transpose(1, 2)).view(-1, hq, d).to(s["dt"])


# ------------------------------------------------------------------ in 64 bits
def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "qk":
        return {"q": _exact_turned(s, s["q"], s["q_weight"]),
                "k": _exact_turned(s, s["k"], s["k_weight"])}
    d, hq, hkv = c["head_dim"], c["q_heads"], c["kv_heads"]
    group, n = hq // hkv, _lengths(c)
    if c["op"] == "prompt":
        out = torch.zeros((s["t"], hq, d), dtype=torch.float64, device="cuda")
        first = 0
        for length in n:
            for a in range(first, first + length, 2048):
                z = min(a + 2048, first + length)
                for h in range(hq):
                    score = s["q"][a:z, h].double() @ s["k"][first:z, h // group].double().T
                    seen = (torch.arange(first, z, device="cuda")[None]
                            <= torch.arange(a, z, device="cuda")[:, None])
                    w = torch.softmax(torch.where(seen, score / math.sqrt(d), -math.inf), -1)
                    out[a:z, h] = w @ s["v"][first:z, h // group].double()
            first += length
        return out
    if c["op"] == "write":
        # the rows written, by position, over what a record held before
        k, v = _exact_rows(s)
        for x, dense in ((s["k"], k), (s["v"], v)):
            t = 0
            for b, length in enumerate(n):
                count = 1 if c["step"] else length
                rows = x[t:t + count].double()
                low = rows.min(-1, keepdim=True).values
                step = _nearest((rows.max(-1, keepdim=True).values - low) / 15, s["dt"])
                code = torch.round((rows - low) / torch.where(step > 0, step, 1.0)).clamp(0, 15)
                code = torch.where(step > 0, code, 0.0)
                dense[b, :, length - count:length] = (low + code * step).transpose(0, 1)
                t += count
        return {"k": k, "v": v}
    k, v = _exact_rows(s)
    out = torch.zeros((c["seqs"], hq, d), dtype=torch.float64, device="cuda")
    for b, length in enumerate(n):
        q = s["q"][b].double().view(hkv, group, d)
        w = torch.softmax(torch.einsum("hgd,hjd->hgj", q, k[b, :, :length].double()) / math.sqrt(d), -1)
        out[b] = torch.einsum("hgj,hjd->hgd", w, v[b, :, :length].double()).reshape(hq, d)
    return out


def _nearest(x, dtype):
    """The value of `dtype` that is nearest to x >= 0 (64 bits), ties to the even one."""
    low = x.float().to(dtype)
    tick = low.view(torch.int16)
    near = torch.stack([(tick + k).clamp(min=0).view(dtype).double() for k in (-1, 0, 1)])
    gap = (near - x).abs()
    even = torch.stack([((tick + k) & 1) for k in (-1, 0, 1)])
    best = gap == gap.amin(0)
    best = torch.where(best.sum(0) > 1, best & (even == 0), best)
    return (near * best).sum(0)


def _exact_rows(s):
    """What the records of each context stand for, element by element of the definition."""
    c, d, hkv = s["c"], s["c"]["head_dim"], s["c"]["kv_heads"]
    shape = (c["seqs"], hkv, s["table"].shape[1] * 16, d)
    out = []
    e = torch.arange(d, device="cuda")
    for pool, keys in ((s["k_cache"], True), (s["v_cache"], False)):
        dense = torch.zeros(shape, dtype=torch.float64, device="cuda")
        for b, length in enumerate(_lengths(c)):
            j = torch.arange(length, device="cuda")
            record = pool[s["table"][b, j // 16].long()]                # [len][hkv][bytes]
            r = (j % 16)[:, None]
            byte = (r * (d // 2) + e // 2) if keys else ((r // 2 * (d // 4) + e // 4) * 4 + r % 2 * 2 + e % 4 // 2)
            code = record.gather(2, byte[:, None, :].expand(-1, hkv, -1)) >> (e % 2 * 4).to(torch.uint8)
            pair = record[:, :, 8 * d:].contiguous().view(s["dt"]).double().view(length, hkv, 16, 2)
            pair = pair[torch.arange(length, device="cuda"), :, j % 16]  # [len][hkv][2]
            dense[b, :, :length] = (pair[..., 1:] + (code & 15).double() * pair[..., :1]).transpose(0, 1)
        out.append(dense)
    return out


def _exact_turned(s, x, weight):
    c = s["c"]
    half, sections = c["rotary"] // 2, _sections(c)
    y = x.double()
    y = y / (y.pow(2).mean(-1, keepdim=True) + _EPS).sqrt() * weight.double()
    z = y.clone()
    first = 0
    for a in range(c["axes"]):
        if not c["dealt"]:
            pairs = list(range(first, first + sections[a]))
            first += sections[a]
        elif a:
            pairs = [a + c["axes"] * i for i in range(sections[a])]
        else:
            taken = {i + c["axes"] * j for i in range(1, c["axes"]) for j in range(sections[i])}
            pairs = [p for p in range(half) if p not in taken]
        pairs = torch.tensor(pairs, dtype=torch.long, device="cuda")
        turn = s["cos_sin"].double()[s["positions"][a].long().clamp(min=0)][:, pairs]
        cos, sin = turn[:, None, :, 0], turn[:, None, :, 1]
        one, two = y[..., pairs], y[..., pairs + half]
        z[..., pairs] = one * cos - two * sin
        z[..., pairs + half] = two * cos + one * sin
    z[s["positions"][0] < 0] = 0
    return z
