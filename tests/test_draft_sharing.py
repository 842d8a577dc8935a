"""The block manager's prefix cache when sequences that hold drafts share
blocks: a block found by its ids holds those ids' rows, whoever wrote to it."""

import random

import pytest

import paged_kv_cache_473_b200 as pa


def _forked_draft():
    """Two sequences of block size 4 that know ids 1 .. 5 and share three drafted positions, which fill block 1."""
    bm = pa.BlockManager(8, 4)
    bm.add_sequence(1, 5, [1, 2, 3, 4, 5])
    for _ in range(3):
        bm.append_slots([1])
    bm.fork(1, 2)
    return bm


@pytest.mark.parametrize("child_first", (True, False))
def test_a_block_held_in_part_is_not_found_once_its_holder_writes_to_it(child_first):
    """One holder learns the ids of the whole block, the other keeps part of it and, left alone, appends there."""
    bm = _forked_draft()
    if child_first:
        bm.truncate(2, 6, [6])
    bm.truncate(1, 8, [6, 7, 8])
    if not child_first:
        bm.truncate(2, 6, [6])
    bm.free(1)
    slots, cow = bm.append_slots([2], [99])
    assert cow.numel() == 0
    written = int(slots[0]) // 4
    assert bm.add_sequence(3, 8, list(range(1, 9))) == 4
    assert written not in [int(s) // 4 for s in bm.slots(3, 0, 8)]


@pytest.mark.parametrize("ids", (None, [20, 30, 40]))
def test_a_block_whose_rows_a_commit_moved_is_not_found_by_other_ids(ids):
    """One holder learns ids 6, 7, 8 of the shared drafts and leaves; the other, alone, commits another path."""
    bm = _forked_draft()
    bm.truncate(1, 8, [6, 7, 8])
    bm.free(1)
    for _ in range(4):
        bm.append_slots([2])  # more of its tree, whose nodes 1, 3 and 5 are moved to positions 5, 6, 7
    moved = [int(s) // 4 for s in bm.slots(2, 5, 3)]
    assert all(bm.ref_count(b) == 1 for b in moved)
    bm.truncate(2, 8, ids)
    assert bm.add_sequence(3, 8, list(range(1, 9))) == 4
    assert not set(moved) & {int(s) // 4 for s in bm.slots(3, 0, 8)}
    if ids:
        assert bm.add_sequence(4, 8, [1, 2, 3, 4, 5, *ids]) == 8


def test_ids_learned_by_the_only_holder_are_found():
    bm = _forked_draft()
    bm.free(1)
    bm.truncate(2, 8, [6, 7, 8])
    assert bm.add_sequence(3, 8, list(range(1, 9))) == 8


@pytest.mark.parametrize("seed", range(24))
def test_random_books_with_forks_inside_a_drafting_step(seed):
    """As the serving loop does, with forks between a draft's append and its cut; a row stands for
    the whole text before it.  Rows are moved only in blocks that no other sequence holds."""
    rng = random.Random(1000 + seed)
    bs, nb = rng.choice((1, 2, 3, 4, 8)), 48
    bm = pa.BlockManager(nb, bs)
    rows = [None] * (nb * bs)
    text, draft, next_id = {}, {}, 0
    seen = [[]]  # texts that some sequence had: prompts ask for them again

    def append(s, tok, prefix, known):
        slot, cow = bm.append_slots([s], [tok] if known else None)
        for a, b in cow.tolist():
            rows[b * bs:(b + 1) * bs] = rows[a * bs:(a + 1) * bs]
        rows[int(slot[0])] = tuple(prefix) + (tok,)

    for _ in range(4000):
        what = rng.choice(("add", "append", "draft", "draft", "settle", "settle", "settle", "cut", "fork", "fork", "free"))
        ids = list(text)
        if len(ids) > 4:
            what = "free"
        s = rng.choice(ids) if ids else None
        try:
            if what == "add" or not ids:
                toks = rng.choice(seen[-12:]) + [rng.randrange(2) for _ in range(rng.randrange(0, 4))]
                cached = bm.add_sequence(next_id, len(toks), toks if rng.random() < 0.8 else None)
                for p, slot in enumerate(bm.slots(next_id, 0, len(toks)).tolist()):
                    if p >= cached:
                        rows[slot] = tuple(toks[:p + 1])
                text[next_id], draft[next_id] = toks, []
                next_id += 1
            elif what == "append" and not draft[s]:
                tok = rng.randrange(2)
                append(s, tok, text[s], rng.random() < 0.9)
                text[s] = text[s] + [tok]
            elif what == "draft":
                for _ in range(rng.randrange(1, 9)):
                    tok = rng.randrange(2)
                    append(s, tok, text[s] + draft[s], False)
                    draft[s] = draft[s] + [tok]
            elif what == "settle" and draft[s]:
                base, n = len(text[s]), len(draft[s])
                slots = bm.slots(s, base, n).tolist()
                take = rng.randrange(0, n + 1)
                path = list(range(take))
                if all(bm.ref_count(x // bs) == 1 for x in slots):
                    path = sorted(rng.sample(range(n), take))
                new = text[s] + [draft[s][j] for j in path]
                if path != list(range(take)):
                    for i in range(take):
                        rows[slots[i]] = tuple(new[:base + i + 1])
                bm.truncate(s, base + take, new[base:] if rng.random() < 0.7 else None)
                text[s], draft[s] = new, []
                seen.append(new)
            elif what == "cut" and not draft[s]:
                n = rng.randrange(0, len(text[s]) + 1)
                bm.truncate(s, n)
                text[s] = text[s][:n]
            elif what == "fork":
                bm.fork(s, next_id)
                text[next_id], draft[next_id] = list(text[s]), list(draft[s])
                next_id += 1
            elif what == "free" or len(text[s]) > 20:
                bm.free(s)
                del text[s], draft[s]
        except pa.PagedAttnError:
            continue  # the pool is full
        for s, toks in text.items():
            all_of = toks + draft[s]
            assert bm.length(s) == len(all_of)
            got = [rows[x] for x in bm.slots(s, 0, len(all_of)).tolist()]
            assert got == [tuple(all_of[:p + 1]) for p in range(len(all_of))], (what, s)
    for s in list(text):
        bm.free(s)
    assert bm.num_free == nb
