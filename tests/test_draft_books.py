"""The drafting step on a machine without a GPU: the host-side checks of its
calls, the binding's checks of its arguments, the 64-bit forms the GPU tests
use, and the block manager's truncation."""

import random

import pytest
import torch

import paged_kv_cache_473_b200 as pa
from paged_kv_cache_473_b200 import _binding as bnd
from tests import draft_reference as ref

A = 0x10000   # 16-byte aligned fake device address: every call below fails its checks before a launch
OK, INVALID, UNSUPPORTED, WORKSPACE = bnd.PA_OK, bnd.PA_ERR_INVALID, bnd.PA_ERR_UNSUPPORTED, bnd.PA_ERR_WORKSPACE


def _call(name, order, defaults, kw):
    a = dict(defaults)
    a.update(kw)
    return getattr(bnd.lib, name)(*[a[k] for k in order.split()])


ROPE = ("q qs k ks qw kw eps inv rd inter pos n hq hkv d qo qos ko kos dt stream",
        dict(q=A, qs=1024, k=A, ks=1024, qw=None, kw=None, eps=1e-6, inv=A, rd=128, inter=0, pos=A, n=4, hq=8, hkv=2,
             d=128, qo=A, qos=1024, ko=A, kos=256, dt=bnd.PA_BF16, stream=None))
APPEND = ("q qs k ks v vs qw kw eps inv rd inter pos slots n hq hkv d qo kc vc nb bs dt stream",
          dict(ROPE[1], v=A, vs=1024, slots=A, kc=A, vc=A, nb=8, bs=16))


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(qo=None), INVALID), (dict(q=A + 8), INVALID),
    (dict(k=A + 2), INVALID), (dict(qs=-8), INVALID), (dict(qs=1025), INVALID), (dict(ks=1028), INVALID),
    (dict(qw=A + 4), INVALID), (dict(kw=A + 8), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(inv=None), INVALID), (dict(pos=None), INVALID), (dict(pos=A + 2), INVALID),
    (dict(inv=A + 1), INVALID), (dict(rd=-16), INVALID), (dict(rd=144), INVALID), (dict(rd=24), UNSUPPORTED),
    (dict(n=-1), INVALID), (dict(hq=0), INVALID), (dict(hkv=-1), INVALID), (dict(d=0), INVALID),
    (dict(d=96, rd=96), UNSUPPORTED), (dict(dt=5), INVALID), (dict(hq=70000, qs=0, qos=70000 * 128), UNSUPPORTED),
    (dict(n=0, q=None, k=None), OK)])
def test_rotation_host_checks(kw, status):
    assert _call("pa_qk_norm_rope", *ROPE, kw) == status
    assert _call("pa_rope_append", *APPEND, kw) == status
    assert pa.last_launch_count() == 0


@pytest.mark.parametrize("kw", [dict(ko=None), dict(ko=A + 8), dict(kos=128), dict(kos=260), dict(qos=1016)])
def test_rotation_output_checks(kw):
    assert _call("pa_qk_norm_rope", *ROPE, kw) == INVALID


@pytest.mark.parametrize("kw", [dict(v=None), dict(v=A + 8), dict(vs=-8), dict(vs=4), dict(kc=None), dict(vc=A + 4),
                                dict(slots=None), dict(slots=A + 4), dict(nb=0), dict(bs=-1)])
def test_append_checks(kw):
    assert _call("pa_rope_append", *APPEND, kw) == INVALID


TREE = ("q k v bt cl tl mask ms B T hq hkv d bs mb nb scale cap win out dt maxL ws wsb stream",
        dict(q=A, k=A, v=A, bt=A, cl=A, tl=None, mask=A, ms=16, B=2, T=16, hq=8, hkv=2, d=128, bs=16, mb=4, nb=8,
             scale=0.1, cap=0.0, win=0, out=A, dt=bnd.PA_BF16, maxL=64, ws=A, wsb=1 << 32, stream=None))


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(out=A + 8), INVALID), (dict(mask=None), INVALID), (dict(mask=A + 4), INVALID),
    (dict(tl=A + 2), INVALID), (dict(ms=15), INVALID), (dict(ms=-1), INVALID), (dict(T=0), INVALID),
    (dict(T=65, ms=65), UNSUPPORTED), (dict(maxL=0), INVALID), (dict(hq=9), INVALID), (dict(hq=32), UNSUPPORTED),
    (dict(d=96), UNSUPPORTED), (dict(bs=8), UNSUPPORTED), (dict(bs=24), UNSUPPORTED), (dict(dt=3), INVALID),
    (dict(cap=float("nan")), INVALID), (dict(B=70000), UNSUPPORTED), (dict(nb=1 << 27), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(ws=A + 8), WORKSPACE), (dict(wsb=1000), WORKSPACE), (dict(B=0, q=None), OK)])
def test_tree_host_checks(kw, status):
    assert _call("pa_decode_tree", *TREE, kw) == status
    assert pa.last_launch_count() == 0


def test_tree_workspace_size():
    """Two partials per CTA: grows with the tree's rows up to 128 per kv head, not with batch or context."""
    one = pa.decode_tree_workspace_size(1, 1, 32, 128, 1024, 8)
    assert 256 * 1024 < one < pa.decode_tree_workspace_size(1, 8, 32, 128, 1024, 8)
    most = pa.decode_tree_workspace_size(1, 32, 32, 128, 1024, 8)
    assert pa.decode_tree_workspace_size(500, 64, 32, 128, 1 << 20, 8) <= 2 * most < 256 << 20
    for bad in ((0, 4, 8, 64, 10, 2), (1, 0, 8, 64, 10, 2), (1, 65, 8, 64, 10, 2), (1, 4, 9, 64, 10, 2), (1, 4, 18, 64, 10, 2)):
        assert pa.decode_tree_workspace_size(*bad) == 0
    args = dict(TREE[1], wsb=pa.decode_tree_workspace_size(2, 16, 8, 128, 64, 2) - 1)
    assert _call("pa_decode_tree", TREE[0], args, {}) == WORKSPACE


COMMIT = ("k v layers bt cl tl T acc ma al B hkv d bs mb nb new dt stream",
          dict(k=A, v=A, layers=2, bt=A, cl=A, tl=None, T=16, acc=A, ma=5, al=A, B=2, hkv=2, d=128, bs=16, mb=4, nb=8,
               new=2 * A, dt=bnd.PA_BF16, stream=None))


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INVALID), (dict(v=A + 8), INVALID), (dict(layers=0), INVALID), (dict(bt=None), INVALID),
    (dict(cl=A + 1), INVALID), (dict(tl=A + 1), INVALID), (dict(T=0), INVALID), (dict(T=65), UNSUPPORTED),
    (dict(acc=None), INVALID), (dict(ma=0), INVALID), (dict(al=None), INVALID), (dict(B=-1), INVALID),
    (dict(d=100), UNSUPPORTED), (dict(bs=24), UNSUPPORTED), (dict(new=A), INVALID), (dict(new=A + 2), INVALID),
    (dict(dt=9), INVALID), (dict(nb=1 << 28), UNSUPPORTED), (dict(B=70000), UNSUPPORTED), (dict(B=0, k=None), OK)])
def test_commit_host_checks(kw, status):
    assert _call("pa_commit_tree", *COMMIT, kw) == status
    assert pa.last_launch_count() == 0


def test_binding_refuses_mismatched_tensors():
    """Shapes, types, strides and devices are looked at before the library is called."""
    bf, f32 = torch.bfloat16, torch.float32
    q, k = torch.zeros(4, 8, 64, dtype=bf), torch.zeros(4, 2, 64, dtype=bf)
    pos, inv = torch.zeros(4, dtype=torch.int32), torch.ones(32)
    kc = torch.zeros(2, 2, 16, 64, dtype=bf)
    slots = torch.zeros(4, dtype=torch.int64)
    for bad in (dict(k=k[:3]), dict(k=k.float()), dict(inv=inv.double()), dict(pos=pos.long()), dict(pos=pos[:3]),
                dict(inv=None, rotary_dim=64), dict(q_weight=torch.ones(32)), dict(k_weight=torch.ones(64, dtype=bf)), {}):
        a = dict(q=q, k=k, pos=pos, inv=inv)
        a.update(bad)
        with pytest.raises(ValueError):  # the last one: nothing wrong but the device
            pa.qk_norm_rope(a.pop("q"), a.pop("k"), a.pop("pos"), a.pop("inv"), **a)
    for bad in (dict(v=k.float()), dict(slots=slots.int()), dict(slots=slots[:2]), dict(kc=kc.float()),
                dict(kc=kc[:, :1]), {}):
        a = dict(v=k, slots=slots, kc=kc)
        a.update(bad)
        with pytest.raises(ValueError):
            pa.rope_append(q, k, a["v"], pos, a["slots"], inv, a["kc"], a["kc"].clone())
    qt, bt, cl = torch.zeros(3, 5, 8, 64, dtype=bf), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    mask = torch.zeros(3, 5, dtype=torch.int64)
    for bad in (dict(mask=mask[:2]), dict(mask=mask.int()), dict(bt=bt[:2]), dict(cl=cl.long()),
                dict(tree_lens=cl[:1]), dict(out=qt[:2]), dict(kc=kc.float()), dict(kc=kc[..., :32]), {}):
        a = dict(mask=mask, bt=bt, cl=cl, kc=kc)
        a.update(bad)
        x = a.pop("kc")
        with pytest.raises(ValueError):
            pa.decode_tree(qt, x, x, a.pop("bt"), a.pop("cl"), a.pop("mask"), 0.1, max_context_len=32, **a)
    acc = torch.zeros(3, 4, dtype=torch.int32)
    for bad in (dict(acc=acc[:2]), dict(acc=acc.long()), dict(al=cl[:2]), dict(bt=bt[0]), dict(new_lens=cl[:2]),
                dict(kc=kc[0]), {}):
        a = dict(acc=acc, al=cl, bt=bt, kc=kc)
        a.update(bad)
        with pytest.raises(ValueError):
            pa.commit_tree(a["kc"], a["kc"], a["bt"], cl, a["acc"], a["al"], tree_len=5, new_lens=a.get("new_lens"))


# ---- the 64-bit forms the GPU tests compare with ---------------------------------------------


def test_reference_rotation_closed_forms():
    x = torch.zeros(2, 1, 64, dtype=torch.float64)
    x[:, 0, 0], x[:, 0, 1] = 1.0, 2.0
    inv = torch.full((32,), 0.5)
    pos = torch.tensor([0, 3], dtype=torch.int32)
    import math

    y, _ = ref.norm_rope(x, None, 0.0, pos, inv, True)
    assert torch.equal(y[0], x[0])
    c, s = math.cos(1.5), math.sin(1.5)
    assert abs(float(y[1, 0, 0]) - (c - 2 * s)) < 1e-15 and abs(float(y[1, 0, 1]) - (2 * c + s)) < 1e-15
    y, _ = ref.norm_rope(x, None, 0.0, pos, inv, False)  # pairs (0, 32) and (1, 33)
    assert abs(float(y[1, 0, 32]) - s) < 1e-15 and abs(float(y[1, 0, 33]) - 2 * s) < 1e-15
    w = torch.full((64,), 3.0)
    y, _ = ref.norm_rope(x, w, 0.0, None, None, False)
    assert abs(float(y[0, 0, 1]) - 2 / math.sqrt(5 / 64) * 3) < 1e-12


def test_reference_tree_is_causal_attention_on_a_chain_and_follows_paths():
    """A chain against the causal oracle; a tree's node against the chain of its own path."""
    import oracle

    g = torch.Generator().manual_seed(1)
    lens = [9, 40, 64]
    kc, vc, tables, cl = ref.pool(g, lens, 2, 64, 16, torch.float32, device="cpu")
    q = torch.randn((3, 9, 4, 64), generator=g)
    chain, _ = ref.random_trees(g, 3, 9, chain=True)
    for cap, window in ((0.0, 0), (3.0, 0), (0.0, 11), (0.0, 2)):
        out, _ = ref.tree(q, kc, vc, tables, cl, chain, 0.125, cap, window)
        want = torch.from_numpy(oracle.decode_multi(q, kc, vc, tables, cl, 0.125, cap, window))
        assert (out - want).abs().max() < 1e-12
    mask, _ = ref.random_trees(g, 3, 9)
    for window in (0, 3, 30):
        out, _ = ref.tree(q, kc, vc, tables, cl, mask, 0.125, 0.0, window)
        for b, n in enumerate(lens):
            bt = tables[b].long()
            k = kc[bt[bt >= 0]].transpose(1, 2).reshape(-1, 2, 64)[:n]
            v = vc[bt[bt >= 0]].transpose(1, 2).reshape(-1, 2, 64)[:n]
            for j in range(9):
                path = [i for i in range(9) if (ref.words(mask[b])[j] >> i) & 1]
                at = list(range(n - 9)) + [n - 9 + i for i in path]
                lo = max(0, len(at) - window) if window else 0
                s = torch.einsum("hd,thd->ht", q[b, j].double(), k[at[lo:]].double().repeat_interleave(2, 1)) * 0.125
                o = torch.einsum("ht,thd->hd", torch.softmax(s, -1), v[at[lo:]].double().repeat_interleave(2, 1))
                assert (o - out[b, j]).abs().max() < 1e-12


# ---- truncation -------------------------------------------------------------------------------


def test_truncate_after_a_draft():
    bm = pa.BlockManager(16, 4)
    bm.add_sequence(1, 6, [1, 2, 3, 4, 5, 6])
    free = bm.num_free
    for _ in range(7):  # the drafts' slots, without ids
        bm.append_slots([1])
    assert bm.length(1) == 13 and bm.num_free == free - 2
    bm.truncate(1, 9, [7, 8, 9])  # three accepted
    assert bm.length(1) == 9 and bm.num_free == free - 1
    assert bm.add_sequence(2, 8, [1, 2, 3, 4, 5, 6, 7, 8]) == 8  # the second block was filled by accepted tokens
    bm.append_slots([1], [10])
    bm.append_slots([1], [11])
    bm.append_slots([1], [12])
    assert bm.add_sequence(3, 12, [1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12]) == 12  # ids went on from there


def test_truncate_into_a_known_block_takes_it_out_of_the_prefix_cache():
    bm = pa.BlockManager(8, 4)
    bm.add_sequence(1, 8, list(range(8)))
    bm.truncate(1, 6)
    assert bm.add_sequence(2, 8, list(range(8))) == 4  # only the first block
    slots, cow = bm.append_slots([1], [60])
    assert cow.numel() == 0 and bm.length(1) == 7
    bm.truncate(1, 4)
    bm.append_slots([1], [4])
    bm.truncate(1, 0)
    assert bm.length(1) == 0
    bm.free(1)
    bm.free(2)
    assert bm.num_free == 8


def test_truncate_of_a_shared_block_copies_on_write():
    bm = pa.BlockManager(8, 4)
    bm.add_sequence(1, 8, list(range(8)))
    bm.fork(1, 2)
    bm.truncate(2, 7)
    slots, cow = bm.append_slots([2], [70])
    assert cow.shape == (1, 2) and bm.ref_count(int(cow[0, 0])) == 1


def test_truncate_refusals_change_nothing():
    bm = pa.BlockManager(8, 4)
    bm.add_sequence(1, 5, list(range(5)))
    bm.append_slots([1])
    for args in ((1, 7), (1, -1), (9, 0), (1, 6, [5, 6]), (1, 5, [9])):
        with pytest.raises(pa.PagedAttnError):
            bm.truncate(*args)
        assert bm.length(1) == 6
    assert bnd.lib.pa_bm_truncate(None, 1, 0, None, 0) == INVALID
    assert bnd.lib.pa_bm_truncate(bm._h, 1, 6, None, 1) == INVALID
    assert bnd.lib.pa_bm_truncate(bm._h, 1, 6, None, -1) == INVALID
    bm.truncate(1, 6, [5])
    bm.truncate(1, 6)


@pytest.mark.parametrize("seed", range(20))
def test_random_books_against_a_simulated_pool(seed):
    """Random prompts, appends, drafts, truncations, forks and frees, with the rows written to a
    simulated pool: every sequence reads its own text back, prefix-cache hits included, no block is lost."""
    rng = random.Random(seed)
    bs, nb = rng.choice((1, 2, 4, 8)), 40
    bm = pa.BlockManager(nb, bs)
    rows = [None] * (nb * bs)  # what the pool holds
    text, next_id = {}, 0

    def write(slot, token, pos):
        rows[slot] = (token, pos)

    def copy(cow):
        for a, b in cow.tolist():
            rows[b * bs:(b + 1) * bs] = rows[a * bs:(a + 1) * bs]

    for _ in range(400):
        what = rng.choice(("add", "append", "append", "draft", "draft", "cut", "fork", "free"))
        ids = list(text)
        if what == "add" or not ids:
            n = rng.randrange(0, 14)
            toks = [rng.randrange(3) for _ in range(n)]
            known = rng.random() < 0.8
            try:
                cached = bm.add_sequence(next_id, n, toks if known else None)
            except pa.PagedAttnError:
                continue
            text[next_id] = toks
            for p, slot in enumerate(bm.slots(next_id, 0, n).tolist()):
                if p >= cached:
                    write(slot, toks[p], p)
            next_id += 1
        elif what == "append":
            s = rng.choice(ids)
            tok = rng.randrange(3)
            try:
                slots, cow = bm.append_slots([s], [tok] if rng.random() < 0.9 else None)
            except pa.PagedAttnError:
                continue
            copy(cow)
            write(int(slots[0]), tok, len(text[s]))
            text[s] = text[s] + [tok]
        elif what == "draft":
            s = rng.choice(ids)
            base, slots = len(text[s]), []
            for i in range(rng.randrange(1, 9)):
                try:
                    slot, cow = bm.append_slots([s])
                except pa.PagedAttnError:
                    break
                copy(cow)
                write(int(slot[0]), -1, -1)
                slots.append(int(slot[0]))
            take = rng.randrange(0, len(slots) + 1)
            toks = [rng.randrange(3) for _ in range(take)]
            for i, tok in enumerate(toks):  # what the commit leaves there
                write(slots[i], tok, base + i)
            bm.truncate(s, base + take, toks if rng.random() < 0.8 else None)
            text[s] = text[s] + toks
        elif what == "cut":
            s = rng.choice(ids)
            n = rng.randrange(0, len(text[s]) + 1)
            bm.truncate(s, n)
            text[s] = text[s][:n]
        elif what == "fork":
            s = rng.choice(ids)
            bm.fork(s, next_id)
            text[next_id] = list(text[s])
            next_id += 1
        else:
            s = rng.choice(ids)
            bm.free(s)
            del text[s]
        for s, toks in text.items():
            assert bm.length(s) == len(toks)
            got = [rows[x] for x in bm.slots(s, 0, len(toks)).tolist()]
            assert got == [(t, p) for p, t in enumerate(toks)], (what, s)
    for s in list(text):
        bm.free(s)
    assert bm.num_free == nb
