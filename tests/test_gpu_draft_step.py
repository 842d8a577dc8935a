"""Moving an accepted path's rows (pa_commit_tree), and the whole drafting step:
rotate and append a tree's tokens, verify them, commit the accepted path, go on
decoding, with the block manager keeping the books."""

import pytest
import torch

import paged_kv_cache_473_b200 as pa
from tests import draft_reference as ref
from tests.gpu_helpers import bits

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clear_device_errors():
    pa.device_errors()
    yield


def _moved(cache, tables, lens, counts, paths):
    """The move in plain indexing; cache [layers, nb, hkv, bs, d] on the CPU."""
    out = cache.clone()
    bs = cache.shape[3]
    for b, path in enumerate(paths):
        base = lens[b] - counts[b]
        for i, node in enumerate(path):
            s, t = base + node, base + i
            out[:, tables[b, t // bs], :, t % bs] = cache[:, tables[b, s // bs], :, s % bs]
    return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layers,heads,block", [(1, (2, 64), 16), (5, (8, 128), 16), (2, (4, 256), 128), (3, (3, 80), 8),
                                                (1, (1, 16), 1)])
def test_commit(layers, heads, block, dtype):
    """Overlapping moves (a row that is a source and a place), whole chains, empty paths, ragged trees, all layers."""
    hkv, d = heads
    g = torch.Generator().manual_seed(layers * 100 + d)
    T = 64
    lens = [64, 200, 70, 10, 0, 99, 130]
    counts = [64, 64, 20, 10, 0, 33, 0]
    paths = [[0, 2, 3, 5, 7, 8, 63], list(range(64)), [0, 1, 5, 6, 7], [9], [], list(range(1, 33)), []]
    kc, vc, tables, cl = ref.pool(g, lens, hkv, d, block, dtype, fill=1.25)
    kc, vc = (torch.stack([c + i for i in range(layers)]).contiguous() for c in (kc, vc))
    accepted = torch.full((len(lens), 64), 77, dtype=torch.int32)
    for b, p in enumerate(paths):
        accepted[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
    want = [_moved(c.cpu(), tables.cpu(), lens, counts, paths) for c in (kc, vc)]
    if layers == 1:
        kc, vc = kc[0], vc[0]
    new = pa.commit_tree(kc, vc, tables, cl, accepted.cuda(), torch.tensor([len(p) for p in paths], dtype=torch.int32).cuda(),
                         tree_len=T, tree_lens=torch.tensor(counts, dtype=torch.int32).cuda())
    assert new.tolist() == [n - c + len(p) for n, c, p in zip(lens, counts, paths)]
    for got, w in zip((kc, vc), want):
        assert torch.equal(bits(got.reshape(w.shape)), bits(w))
    assert pa.device_errors() == 0 and pa.last_launch_count() == 1


def test_commit_refuses_bad_paths_and_lengths():
    """Reported; nothing of the sequence moves, its length stays; the others are committed."""
    g = torch.Generator().manual_seed(2)
    lens = [20, 20, 20, 20, 20, 20, 5, 20]
    kc, vc, tables, cl = ref.pool(g, lens, 2, 64, 16, torch.bfloat16, fill=0.0)
    before = kc.clone()
    bad = [[0, 3, 3], [0, 8], [-1, 2], [2, 1], [0, 2, 5]]
    accepted = torch.zeros((8, 3), dtype=torch.int32)
    for b, p in enumerate(bad):
        accepted[b, :len(p)] = torch.tensor(p)
    take = torch.tensor([3, 2, 2, 2, 3, 4, 1, -1], dtype=torch.int32)  # row 5: more than max_accept; row 6: L < n
    new = pa.commit_tree(kc, vc, tables, cl, accepted.cuda(), take.cuda(), tree_len=8)
    assert pa.device_errors() == pa.DEVERR_CONTEXT
    assert new.tolist() == [20, 20, 20, 20, 15, 20, 5, 20]
    want = _moved(before[None].cpu(), tables.cpu(), lens, [8] * 8, [[], [], [], [], [0, 2, 5], [], [], []])[0]
    assert torch.equal(bits(kc), bits(want))


def test_commit_block_ids_outside_the_pool():
    g = torch.Generator().manual_seed(3)
    kc, vc, tables, cl = ref.pool(g, [40], 2, 64, 16, torch.bfloat16, fill=0.0)
    before = kc.clone()
    tables[0, 2] = kc.shape[0]
    accepted = torch.tensor([[0, 2, 12]], dtype=torch.int32).cuda()  # node 12 is position 36, in the bad block
    pa.commit_tree(kc, vc, tables, cl, accepted, torch.tensor([3], dtype=torch.int32).cuda(), tree_len=16)
    assert pa.device_errors() == pa.DEVERR_BLOCK
    t = tables.cpu()
    want = before.clone()
    want[t[0, 25 // 16], :, 25 % 16] = before[t[0, 26 // 16], :, 26 % 16]
    assert torch.equal(bits(kc), bits(want))


def test_commit_in_a_graph_and_on_another_stream():
    g = torch.Generator().manual_seed(5)
    lens = [50, 33]
    kc, vc, tables, cl = ref.pool(g, lens, 2, 64, 16, torch.bfloat16, fill=0.0)
    first = kc.clone()
    accepted = torch.tensor([[0, 4, 9], [0, 2, 3]], dtype=torch.int32).cuda()
    take = torch.tensor([3, 2], dtype=torch.int32).cuda()
    new = torch.zeros(2, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    pa.commit_tree(kc, vc, tables, cl, accepted, take, tree_len=16, new_lens=new, stream=side)
    side.synchronize()
    want = _moved(first[None].cpu(), tables.cpu(), lens, [16, 16], [[0, 4, 9], [0, 2]])[0]
    assert torch.equal(bits(kc), bits(want)) and new.tolist() == [37, 19]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.commit_tree(kc, vc, tables, cl, accepted, take, tree_len=16, new_lens=new)
    kc.copy_(first)
    accepted.copy_(torch.tensor([[1, 2, 3], [0, 5, 15]], dtype=torch.int32))
    take.fill_(3)
    graph.replay()
    torch.cuda.synchronize()
    want = _moved(first[None].cpu(), tables.cpu(), lens, [16, 16], [[1, 2, 3], [0, 5, 15]])[0]
    assert torch.equal(bits(kc), bits(want)) and new.tolist() == [37, 20]


def _weights(gen, hq, hkv, d, vocab):
    """A one-layer stand-in for a model: a token's query, key and value rows come from a table."""
    w = torch.randn((vocab, (hq + 2 * hkv) * d), generator=gen)
    return w.to(torch.bfloat16).cuda()


@pytest.mark.parametrize("heads", [(32, 8, 128), (32, 4, 64), (8, 4, 256)])
def test_drafting_steps_follow_plain_decoding(heads):
    """Three drafting steps with the block manager against one-token-at-a-time
    decoding of the accepted tokens: the same cache rows bit for bit, the same
    attention within the bound, and the plain decode goes on from the result."""
    hq, hkv, d = heads
    gen = torch.Generator().manual_seed(d + hq)
    block, T, B, vocab, layers = 16, 13, 3, 50, 2
    table = _weights(gen, hq, hkv, d, vocab)
    inv = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).float().cuda()
    qw, kw = (1 + 0.2 * torch.randn((2, d), generator=gen)).cuda()
    scale = d ** -0.5

    def rows(tokens):
        x = table[torch.tensor(tokens, device="cuda")]
        q, k, v = x.split((hq * d, hkv * d, hkv * d), 1)
        return q.view(-1, hq, d), k.view(-1, hkv, d), v.view(-1, hkv, d)

    def append(tokens, positions, slots, kc, vc):
        q, k, v = rows(tokens)
        return pa.rope_append(q, k, v, torch.tensor(positions, dtype=torch.int32).cuda(), slots.cuda(), inv, kc, vc,
                              q_weight=qw, k_weight=kw)

    def caches():
        return [torch.zeros((layers, 64, hkv, block, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    bm, plain = pa.BlockManager(64, block), pa.BlockManager(64, block)
    kc, vc = caches()
    pk, pv = caches()
    prompts = [torch.randint(0, vocab, (n,), generator=gen).tolist() for n in (20, 47, 1)]
    text = [list(p) for p in prompts]
    for m, (a, b) in ((bm, (kc, vc)), (plain, (pk, pv))):
        for i, p in enumerate(prompts):
            m.add_sequence(i, len(p), p)
            for layer in range(layers):
                append(p, list(range(len(p))), m.slots(i, 0, len(p)), a[layer], b[layer])
    for step in range(3):
        mask, parent = ref.random_trees(gen, B, T)
        drafts = torch.randint(0, vocab, (B, T), generator=gen).tolist()
        slots = []
        for _ in range(T):
            got, cow = bm.append_slots(range(B))
            assert cow.numel() == 0
            slots.append(got)
        slots = torch.stack(slots, 1)
        tables, lens = bm.block_tables(range(B), 16)
        tables, lens = tables.cuda(), lens.cuda()
        positions = [len(text[b]) + x for b in range(B) for x in ref.depths(ref.words(mask[b]), T)]
        for layer in range(layers):
            q = append([t for r in drafts for t in r], positions, slots.flatten(), kc[layer], vc[layer])
        out = pa.decode_tree(q.view(B, T, hq, d), kc[-1], vc[-1], tables, lens, mask.cuda(), scale, max_context_len=256)
        # the accepted path: from the root to some node
        paths = []
        for b in range(B):
            node = int(torch.randint(0, T, (1,), generator=gen))
            paths.append([i for i in range(T) if (ref.words(mask[b])[node] >> i) & 1])
        accepted = torch.zeros((B, T), dtype=torch.int32)
        for b, p in enumerate(paths):
            accepted[b, :len(p)] = torch.tensor(p)
        take = torch.tensor([len(p) for p in paths], dtype=torch.int32)
        new = pa.commit_tree(kc, vc, tables, lens, accepted.cuda(), take.cuda(), tree_len=T)
        for b, p in enumerate(paths):
            tokens = [drafts[b][i] for i in p]
            text[b] += tokens
            bm.truncate(b, len(text[b]), tokens)
        assert new.tolist() == [len(t) for t in text] == [bm.length(b) for b in range(B)]
        # the same tokens one at a time
        for b, p in enumerate(paths):
            for i, node in enumerate(p):
                at = len(text[b]) - len(p) + i
                slot, _ = plain.append_slots([b], [drafts[b][node]])
                for layer in range(layers):
                    q1 = append([drafts[b][node]], [at], slot, pk[layer], pv[layer])
                pt, pl = plain.block_tables([b], 16)
                args = (pk[-1], pv[-1], pt.cuda(), pl.cuda())
                one, err = ref.tree(q1[:, None], *args, torch.ones((1, 1), dtype=torch.int64), scale)
                ref.assert_near(out[b, node][None, None], one, err, f"step {step} sequence {b} node {node}")
    for b in range(B):
        n = len(text[b])
        s, t = bm.slots(b, 0, n), plain.slots(b, 0, n)
        for x, y in ((kc, pk), (vc, pv)):
            assert torch.equal(bits(x[:, s // block, :, s % block]), bits(y[:, t // block, :, t % block]))
    # and the plain fused decode step goes on from the committed cache
    tokens = [7, 8, 9]
    slots, _ = bm.append_slots(range(B), tokens)
    tables, lens = bm.block_tables(range(B), 16)
    q, k, v = rows(tokens)
    pos = (lens - 1).cuda()
    q, k = pa.qk_norm_rope(q, k, pos, inv, q_weight=qw, k_weight=kw)
    got = pa.decode_step(q, k, v.contiguous(), kc[-1], vc[-1], tables.cuda(), lens.cuda(), scale, split=True,
                         max_context_len=256)
    want, err = ref.tree(q[:, None], kc[-1], vc[-1], tables, lens, torch.ones((B, 1), dtype=torch.int64), scale)
    ref.assert_near(got[:, None], want, err, "decode step after the commits")
    assert pa.device_errors() == 0
