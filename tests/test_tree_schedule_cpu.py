"""How far the tree attention's copies run ahead of a softmax warp that is held up, on a model
of one CTA's roles: what a chunk's softmax still reads has to be there then.  Sizes are read
from the kernel's source."""
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "paged_kv_attention_photon_gb300", "csrc", "tree_attention.cu")


def constant(name, text=None):
    text = open(SOURCE).read() if text is None else text
    return int(re.search(r"constexpr int %s = (\d+);" % name, text).group(1))


def stages(name, d):
    wide, narrow = re.search(r"%s = D == 128 \? (\d+) : (\d+);" % name, open(SOURCE).read()).groups()
    return int(wide if d == 128 else narrow)


def takers(items, one_tile):
    """For each chunk of a CTA's items (chunks, more rows than a tile) the tiles that take it."""
    line = []
    for m, (chunks, apart) in enumerate(items):
        for c in range(chunks):
            line.append((0, 1) if apart else ((m + (c if chunks > one_tile else 0)) & 1,))
    return line


def published(line, k_stages, v_stages, held_tile, held):
    """Chunks whose K copies have begun when nothing moves any more, with the softmax of one tile
    held up before chunk `held`.  Copies wait for both tiles to hand a stage back; a tile's
    issuer of S hands a chunk back when its S is done or the other tile takes it, and its next S
    waits for the last one's P V, which waits for softmax and V."""
    n = len(line)
    k = v = 0
    s_at, s_own, soft, pv_at, pv_own = [0, 0], [0, 0], [0, 0], [0, 0], [0, 0]
    own = [[c for c in range(n) if t in line[c]] for t in (0, 1)]
    moved = True
    while moved:
        moved = False
        if k < n and (k < k_stages or min(s_at) > k - k_stages):
            k, moved = k + 1, True
        if v < n and (v < v_stages or min(pv_at) > v - v_stages):
            v, moved = v + 1, True
        for t in (0, 1):
            c = s_at[t]
            if c < k and (t not in line[c] or pv_own[t] == s_own[t]):
                s_own[t] += t in line[c]
                s_at[t], moved = c + 1, True
            if soft[t] < s_own[t] and not (t == held_tile and own[t][soft[t]] == held):
                soft[t], moved = soft[t] + 1, True
            c = pv_at[t]
            if c < v and (t not in line[c] or soft[t] > pv_own[t]):
                pv_own[t] += t in line[c]
                pv_at[t], moved = c + 1, True
    return k


def furthest(items, d, one_tile):
    line = takers(items, one_tile)
    return max(published(line, stages("kKStages", d), stages("kVStages", d), t, c) - 1 - c
               for c in range(len(line)) for t in line[c])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("one_tile", [1, constant("kOneTile")])
def test_missing_blocks_are_remembered_until_softmax_has_read_them(d, one_tile):
    rng = random.Random(d + one_tile)
    lists = [[(4, False)] * 6, [(1, False), (4, False)] * 3, [(6, False), (4, False), (5, False)],
             [(8, True), (4, False), (1, False), (4, False)]]
    lists += [[(rng.choice([1, 1, 2, 3, 4, 4, 5, 6, 9]), rng.random() < 0.2)
               for _ in range(rng.randint(2, 7))] for _ in range(400)]
    most = max(furthest(items, d, one_tile) for items in lists)
    assert most >= stages("kKStages", d)          # the model runs ahead at all
    assert most < constant("kGoneRing")


def test_every_chunk_ends_where_nothing_is_held_up():
    for one_tile in (1, 4):
        for items in ([(4, False)] * 5, [(1, False), (9, False), (2, True)]):
            line = takers(items, one_tile)
            assert published(line, 2, 2, 0, -1) == len(line)
