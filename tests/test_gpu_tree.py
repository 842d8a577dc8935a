"""Attention of drafted trees over the paged cache (pa_decode_tree) against a
plain 64-bit form: head layouts, tree and context sizes, windows, the softcap,
ragged and empty trees, what stands in masked places, schedules and workspaces."""

import pytest
import torch

import oracle
import paged_kv_cache_473_b200 as pa
from tests import draft_reference as ref
from tests.gpu_helpers import bits

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _clear_device_errors():
    pa.device_errors()
    yield


def _case(lens, nodes, heads, dtype=BF, block=16, seed=0, q_scale=2.0, shared=False, fill=float("nan")):
    hq, hkv, d = heads
    g = torch.Generator().manual_seed(seed * 7919 + nodes * 31 + sum(lens) + d)
    kc, vc, tables, cl = ref.pool(g, lens, hkv, d, block, dtype, fill=fill)
    q = (torch.randn((len(lens), nodes, hq, d), generator=g) * q_scale).to(dtype).cuda()
    mask, _ = ref.random_trees(g, 1 if shared else len(lens), nodes)
    return {"q": q, "k_cache": kc, "v_cache": vc, "tables": tables, "lens": cl,
            "mask": (mask[0] if shared else mask).cuda(), "scale": d ** -0.5}


def _run(c, **kw):
    args = dict(kw)
    if "max_context_len" not in args:
        args["max_context_len"] = max(1, int(c["lens"].max()))
    return pa.decode_tree(c["q"], c["k_cache"], c["v_cache"], c["tables"], c["lens"], c["mask"],
                          args.pop("scale", c["scale"]), args.pop("softcap", 0.0), args.pop("window", 0), **args)


def _ref(c, **kw):
    return ref.tree(c["q"], c["k_cache"], c["v_cache"], c["tables"], c["lens"], c["mask"],
                    kw.pop("scale", c["scale"]), **kw)


def _check(c, what, **kw):
    out = _run(c, **kw)
    kw.pop("max_context_len", None)
    ref.assert_near(out, *_ref(c, **kw), what)
    assert pa.device_errors() == 0
    return out


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("heads", [(8, 2, 64), (32, 4, 64), (8, 4, 256), (32, 8, 128), (6, 2, 128), (7, 1, 64),
                                   (1, 1, 256), (5, 1, 128)])
@pytest.mark.parametrize("nodes", [1, 2, 5, 16, 31, 64])
def test_head_layouts_and_tree_sizes(heads, nodes, dtype):
    """Contexts from the bare tree over tile and block edges; one row to 512 rows per kv head."""
    lens = [nodes, nodes + 1, nodes + 63, 128, 129 + nodes, 300]
    _check(_case(lens, nodes, heads, dtype, seed=1), f"{heads} nodes={nodes}")


@pytest.mark.parametrize("block", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype,heads", [(BF, (32, 8, 128)), (F32, (8, 2, 64))])
def test_block_sizes(block, dtype, heads):
    lens = [9, block - 1 + 9, block + 9, 3 * block + 5, 511]
    _check(_case(lens, 9, heads, dtype, block, seed=2), f"block={block}")


@pytest.mark.parametrize("window", [1, 2, 7, 40, 63, 64, 65, 100, 200, 2 ** 31 - 1])
@pytest.mark.parametrize("dtype,heads,nodes", [(BF, (32, 8, 128), 12), (BF, (32, 4, 64), 40), (BF, (8, 4, 256), 64),
                                               (F32, (8, 2, 64), 33)])
def test_windows(window, dtype, heads, nodes):
    """Each node's window ends at its own depth; small windows cut the tree itself."""
    lens = [nodes, nodes + 5, 130 + nodes, 321, 64 + nodes]
    _check(_case(lens, nodes, heads, dtype, seed=3), f"window={window}", window=window)


def test_window_on_a_deep_chain():
    """A chain of 64: the last node's window leaves the first nodes, and the context, out."""
    for dtype in (BF, F32):
        c = _case([64, 200, 90], 64, (8, 2, 64), dtype, seed=4)
        g = torch.Generator().manual_seed(9)
        c["mask"] = ref.random_trees(g, 3, 64, chain=True)[0].cuda()
        for window in (1, 10, 63, 64, 80):
            _check(c, f"chain window={window}", window=window)


@pytest.mark.parametrize("softcap", [0.5, 5.0, 50.0, float("inf")])
@pytest.mark.parametrize("dtype,heads", [(BF, (8, 4, 256)), (BF, (32, 4, 64)), (F32, (8, 2, 64))])
def test_softcap(softcap, dtype, heads):
    c = _case([12, 40, 333], 12, heads, dtype, seed=5, q_scale=6.0)
    out = _run(c, softcap=softcap)
    ref.assert_near(out, *_ref(c, softcap=softcap if softcap < 1e30 else 0.0), f"softcap={softcap}")


@pytest.mark.parametrize("scale", [0.0, -0.125, 1.0])
def test_scale_of_any_sign(scale):
    for dtype in (BF, F32):
        c = _case([10, 75, 200], 10, (8, 2, 64), dtype, seed=6, q_scale=1.0)
        for softcap in (0.0, 20.0):
            _check(c, f"scale={scale} softcap={softcap}", scale=scale, softcap=softcap)


@pytest.mark.parametrize("dtype,heads", [(BF, (32, 8, 128)), (BF, (7, 1, 64)), (BF, (8, 4, 256)), (F32, (6, 2, 128))])
def test_ragged_and_empty(dtype, heads):
    """Trees of fewer nodes, none, empty sequences: their rows are zero, bits past a tree are ignored."""
    lens = [40, 0, 64, 33, 5, 200, 150, 64]
    counts = torch.tensor([40, 7, 1, 0, 5, 39, 17, 64], dtype=torch.int32)
    c = _case(lens, 64, heads, dtype, seed=7)
    tl = counts.cuda()
    out = torch.full_like(c["q"], float("nan"))
    _run(c, tree_lens=tl, out=out)
    ref.assert_near(out, *_ref(c, tree_lens=counts), "ragged")
    assert pa.device_errors() == 0
    for b, n in enumerate(counts.tolist()):
        assert torch.count_nonzero(out[b, (n if lens[b] else 0):]).item() == 0
    c["mask"] |= -1 << 41  # bits of nodes that only the last tree has
    c["mask"][7] = _case(lens, 64, heads, dtype, seed=7)["mask"][7]
    again = _run(c, tree_lens=tl)
    assert torch.equal(bits(again), bits(out))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_that_attend_nothing(dtype):
    """An empty mask word: the context alone; without a context, a zero row."""
    c = _case([6, 90], 6, (32, 8, 128), dtype, seed=8)
    c["mask"][:, 2] = 0
    c["mask"][:, 4] = 0
    out = _check(c, "empty words")
    assert torch.count_nonzero(out[0, 2]).item() == 0 and torch.count_nonzero(out[0, 4]).item() == 0
    assert torch.count_nonzero(out[1, 2]).item() > 0
    c["mask"][:] = 0
    _check(c, "all words empty")
    _check(c, "all words empty, window", window=1)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_lengths_that_do_not_fit(dtype):
    """Reported, zero rows, the other sequences as ever."""
    c = _case([30, 30, 30, 30, 30], 8, (8, 2, 64), dtype, seed=9)
    good = _run(c)
    lens = c["lens"].clone()
    c["lens"] = torch.tensor([30, 7, -1, 33, 30], dtype=torch.int32).cuda()  # below n, negative, past the table
    out = _run(c, max_context_len=64)
    assert pa.device_errors() == pa.DEVERR_CONTEXT
    c["lens"] = lens
    assert torch.equal(bits(out[[0, 4]]), bits(good[[0, 4]])) and torch.count_nonzero(out[1:4]).item() == 0
    out = _run(c, max_context_len=29)  # above the bound
    assert pa.device_errors() == pa.DEVERR_CONTEXT and torch.count_nonzero(out).item() == 0
    tl = torch.tensor([8, -1, 9, 8, 2 ** 31 - 1], dtype=torch.int32).cuda()
    out = _run(c, tree_lens=tl)
    assert pa.device_errors() == pa.DEVERR_CONTEXT
    assert torch.equal(bits(out[[0, 3]]), bits(good[[0, 3]])) and torch.count_nonzero(out[[1, 2, 4]]).item() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("bad_id", [-1, 10 ** 6, -(2 ** 31)])
def test_block_ids_outside_the_pool(dtype, bad_id):
    c = _case([64, 128], 4, (8, 2, 64), dtype, seed=10)
    good = _run(c)
    c["tables"][1, 2] = bad_id
    out = _run(c)
    assert pa.device_errors() == pa.DEVERR_BLOCK
    assert torch.equal(bits(out[0]), bits(good[0])) and torch.isfinite(out).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("heads", [(32, 8, 128), (8, 4, 256), (32, 4, 64)])
@pytest.mark.parametrize("junk", [float("nan"), float("inf"), -float("inf")])
def test_masked_places_reach_no_row(dtype, heads, junk):
    """Keys and values that only some rows attend (or none), not finite: the others are as without them."""
    nodes = 12
    lens = [12, 70, 150, 61]
    c = _case(lens, nodes, heads, dtype, seed=11)
    bs = c["k_cache"].shape[2]
    hit = []
    for b, n in enumerate(lens):  # node 5's value row, and (where there is a context) node 7's whole key and value
        for node, (in_k, in_v) in ((5, (False, True)), (7, (True, True))):
            t = n - nodes + node
            blk, off = int(c["tables"][b, t // bs]), t % bs
            if in_v:
                c["v_cache"][blk, :, off, 3::7] = junk
            if in_k:
                c["k_cache"][blk, :, off, 1] = junk
        hit.append(t)
    out = _run(c)
    want, err = _ref(c)
    assert pa.device_errors() == 0
    mask = c["mask"].cpu()
    touched = ((mask >> 5) & 1).bool() | ((mask >> 7) & 1).bool()
    clean = ~touched
    assert clean.any() and touched.any()
    ref.assert_near(out[clean.cuda()], want[clean], err[clean], "rows that do not attend them")
    only5 = ((mask >> 5) & 1).bool() & ~((mask >> 7) & 1).bool()
    ref.assert_near(out[only5.cuda()], want[only5], err[only5], "rows that attend the value")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window", [3, 50])
def test_values_before_some_windows_reach_only_the_others(dtype, window):
    """Not-finite rows at and before the windows' starts."""
    c = _case([30, 140, 203], 24, (32, 8, 128), dtype, seed=12)
    c["mask"] = ref.random_trees(torch.Generator().manual_seed(1), 3, 24, chain=True)[0].cuda()
    bs = c["k_cache"].shape[2]
    for b, n in enumerate([30, 140, 203]):
        for t in (n - 24 + 1 - window, n - 24 + 4 - window, n - 24 - window - 9):
            if 0 <= t:
                c["v_cache"][int(c["tables"][b, t // bs]), :, t % bs, ::5] = float("inf")
                c["k_cache"][int(c["tables"][b, t // bs]), :, t % bs, 0] *= 3
    out = _run(c, window=window)
    ref.assert_near(out, *_ref(c, window=window), "window starts")


def test_one_tree_for_all_sequences():
    for dtype in (BF, F32):
        c = _case([20, 77, 140, 16], 16, (8, 2, 64), dtype, seed=13, shared=True)
        out = _check(c, "shared tree")
        c["mask"] = c["mask"].expand(4, 16).contiguous()
        assert torch.equal(bits(_run(c)), bits(out))


@pytest.mark.parametrize("heads,nodes", [((32, 8, 128), 4), ((8, 4, 256), 20), ((32, 4, 64), 8)])
def test_a_chain_is_the_causal_multi_query_call(heads, nodes):
    """Against the C oracle's causal rows and pa_decode_multi."""
    c = _case([nodes, 65, 200, 130], nodes, heads, seed=14, q_scale=1.0)
    c["mask"] = ref.random_trees(torch.Generator(), 4, nodes, chain=True)[0].cuda()
    out = _run(c)
    want = torch.from_numpy(oracle.decode_multi(c["q"], c["k_cache"], c["v_cache"], c["tables"], c["lens"], c["scale"]))
    _, err = _ref(c)
    ref.assert_near(out, want, err, "chain against the oracle")
    multi = pa.decode_multi(c["q"], c["k_cache"], c["v_cache"], c["tables"], c["lens"], c["scale"], max_context_len=200)
    assert (multi.float() - out.float()).abs().max().item() <= 2e-2


@pytest.mark.parametrize("dtype", [BF, F32])
def test_where_the_blocks_lie_does_not_matter(dtype):
    """The same bits for another placement, for a repeated call and whatever the workspace holds behind its counters."""
    c = _case([100, 333, 64, 17], 10, (32, 8, 128), dtype, seed=15)
    out = _run(c)
    nb = c["k_cache"].shape[0]
    perm = torch.randperm(nb, generator=torch.Generator().manual_seed(3)).cuda()
    moved = dict(c)
    for name in ("k_cache", "v_cache"):
        moved[name] = torch.empty_like(c[name])
        moved[name][perm] = c[name]
    t = c["tables"].clone()
    t[t >= 0] = perm[t[t >= 0].long()].int()
    moved["tables"] = t
    assert torch.equal(bits(_run(moved)), bits(out))
    need = pa.decode_tree_workspace_size(4, 10, 32, 128, 333, 8)
    ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")
    ws[:256 * 1024] = 0
    for _ in range(3):
        assert torch.equal(bits(_run(c, workspace=ws)), bits(out))
    assert torch.count_nonzero(ws[:256 * 1024]).item() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_tensors_aligned_to_16_bytes_only(dtype):
    """q, out and the caches 16 bytes off a larger alignment: the same bits."""
    c = _case([100, 333, 64, 17], 10, (32, 8, 128), dtype, seed=25)
    want = _run(c)
    skip = 16 // c["q"].element_size()

    def off(t):
        flat = torch.empty(t.numel() + 64, dtype=t.dtype, device="cuda")
        view = flat[skip:skip + t.numel()].view(t.shape)
        assert view.data_ptr() % 32 == 16
        return view.copy_(t)

    moved = dict(c, q=off(c["q"]), k_cache=off(c["k_cache"]), v_cache=off(c["v_cache"]))
    out = off(torch.zeros_like(c["q"]))
    assert torch.equal(bits(_run(moved, out=out)), bits(want))


def test_many_short_sequences():
    """More sequences than threads in a CTA, most of them a tile or less, some empty."""
    g = torch.Generator().manual_seed(4)
    lens = torch.randint(3, 90, (700,), generator=g).tolist()
    for b in (0, 5, 333, 699):
        lens[b] = 0
    _check(_case(lens, 3, (8, 2, 64), seed=16), "many short")
    _check(_case([0] * 40 + [50] + [0] * 300, 2, (32, 4, 64), seed=17), "one of many")
    c = _case([0, 0, 0], 4, (32, 8, 128), seed=18)
    assert torch.count_nonzero(_run(c, max_context_len=16)).item() == 0


@pytest.mark.parametrize("heads,nodes", [((8, 4, 256), 44), ((8, 4, 256), 64), ((8, 4, 256), 24), ((16, 2, 256), 64),
                                         ((32, 8, 128), 16), ((32, 8, 128), 31), ((32, 8, 128), 64), ((32, 4, 64), 8),
                                         ((32, 4, 64), 40)])
def test_many_tiles_in_flight(heads, nodes):
    """Every multiprocessor goes through many units of a few tiles, the last ones
    masked: loads, products and the mending of V at every stage of the rings."""
    g = torch.Generator().manual_seed(nodes + heads[2])
    for spread in ((64, 400), (250, 900)):
        lens = torch.randint(*spread, (96,), generator=g).tolist()
        c = _case(lens, nodes, heads, seed=32 + spread[0])
        want = _ref(c)
        outs = [_run(c) for _ in range(3)]
        for out in outs:
            ref.assert_near(out, *want, f"{heads} {nodes} {spread}")
    assert pa.device_errors() == 0


@pytest.mark.parametrize("heads,nodes,lens", [((32, 8, 128), 64, [5000, 70]), ((8, 4, 256), 7, [9000]),
                                              ((32, 4, 64), 24, [12345, 300, 4000]), ((1, 1, 64), 2, [20000]),
                                              ((32, 8, 128), 1, [64 * 200 + 1])])
def test_long_contexts_in_pieces(heads, nodes, lens):
    """Few sequences over all SMs: many pieces per (sequence, kv head), joined."""
    _check(_case(lens, nodes, heads, seed=19), f"{heads} long")
    _check(_case(lens, nodes, heads, seed=20), f"{heads} long, window", window=1000)


def test_large_scores_and_one_dominant_key():
    """Scores in the thousands: the running maximum moves, earlier sums vanish."""
    for dtype in (BF, F32):
        c = _case([400, 150], 6, (8, 2, 64), dtype, seed=21, q_scale=40.0)
        c["k_cache"][int(c["tables"][0, 20])] *= 8
        _check(c, "large scores", scale=1.0)


def test_strided_pool_offsets_past_32_bits():
    """Blocks that start past 2^31 elements."""
    hkv, d, block = 8, 128, 16
    nb = 2 ** 31 // (hkv * block * d) + 40
    small = _case([200, 90], 8, (32, hkv, d), seed=22)
    out = _run(small)
    c = dict(small)
    k = small["k_cache"].shape[0]
    for name in ("k_cache", "v_cache"):
        c[name] = torch.empty((nb, hkv, block, d), dtype=BF, device="cuda")
        c[name][nb - k:] = small[name]
    t = small["tables"].clone()
    t[t >= 0] += nb - k
    c["tables"] = t
    assert torch.equal(bits(_run(c)), bits(out))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_other_stream_and_captured_graph(dtype):
    c = _case([100, 333, 64, 17], 10, (32, 8, 128), dtype, seed=23, fill=0.5)
    want = _run(c)
    ws = torch.zeros(max(16, pa.decode_tree_workspace_size(4, 10, 32, 128, 333, 8)), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    _run(c, out=out, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(bits(out), bits(want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _run(c, out=out, workspace=ws, max_context_len=333)
    for step in (1, 2):  # lengths and trees change in place, the replay follows
        c["lens"].copy_(torch.tensor([100 - step, 300 + step, 64, 10], dtype=torch.int32))
        c["mask"].copy_(ref.random_trees(torch.Generator().manual_seed(step), 4, 10)[0])
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        ref.assert_near(out, *_ref(c), f"replay {step}")
    assert pa.device_errors() == 0


def test_a_workspace_shared_with_the_split_decode():
    """The counter region stays zero: the dynamic schedule before and after gives the same bits."""
    c = _case([700, 1500, 90], 5, (32, 8, 128), seed=24)
    need = max(pa.decode_tree_workspace_size(3, 5, 32, 128, 1500, 8), pa.decode_splitk_workspace_size(3, 32, 128, 1500, 0, 8))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    q1 = c["q"][:, 0].contiguous()

    def step():
        return pa.decode_splitk(q1, c["k_cache"], c["v_cache"], c["tables"], c["lens"], c["scale"],
                                max_context_len=1500, workspace=ws)

    first, tree = step(), _run(c, workspace=ws)
    for _ in range(3):
        assert torch.equal(bits(step()), bits(first))
        assert torch.equal(bits(_run(c, workspace=ws)), bits(tree))
    assert torch.count_nonzero(ws[:256 * 1024]).item() == 0


@pytest.mark.parametrize("heads", [(4, 1, 64), (4, 2, 128), (2, 1, 256)])
@pytest.mark.parametrize("window", [0, 37])
def test_fp32_ranges_shared_by_a_cluster(heads, window):
    """fp32: the bound on the contexts decides how many CTAs share a range; one to eight here, some without a token."""
    c = _case([90, 7, 41], 7, heads, F32, seed=33)
    want = _ref(c, window=window)
    for most in (90, 100, 200, 400, 800, 100000):
        ref.assert_near(_run(c, window=window, max_context_len=most), *want, f"{heads} at most {most}")
    c = _case([1500], 40, heads, F32, seed=34)
    ref.assert_near(_run(c, window=window), *_ref(c, window=window), f"{heads} long")
    assert pa.device_errors() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_calls_in_a_row_without_a_wait(dtype):
    """Each call's launches may begin while those before still run: forty in a
    row, of four shapes in turn on one workspace, give what each gives alone."""
    shapes = [([300, 45, 900], 9, (32, 8, 128)), ([64, 65], 33, (32, 8, 128)), ([2000] * 5, 8, (32, 4, 64)),
              ([130, 700], 50, (8, 4, 256))]
    cases = [_case(lens, nodes, heads, dtype, seed=35 + i) for i, (lens, nodes, heads) in enumerate(shapes)]
    alone = [_run(c) for c in cases]
    need = max(pa.decode_tree_workspace_size(len(lens), nodes, h[0], h[2], max(lens), h[1]) for lens, nodes, h in shapes)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    outs = [torch.full_like(alone[i % 4], 7.0) for i in range(40)]
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        _run(cases[i % 4], out=out, workspace=ws, max_context_len=max(shapes[i % 4][0]))
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        assert torch.equal(bits(out), bits(alone[i % 4])), i
    assert torch.count_nonzero(ws[:256 * 1024]).item() == 0 and pa.device_errors() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_two_streams_at_once(dtype):
    """Calls on two streams, each with its own workspace and output."""
    cases = [_case([800, 333, 1200], 12, (32, 8, 128), dtype, seed=41), _case([500] * 6, 40, (32, 4, 64), dtype, seed=42)]
    want = [_run(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    spaces = [torch.zeros(max(16, pa.decode_tree_workspace_size(6, 64, 32, 128, 1200, 8)), dtype=torch.uint8, device="cuda")
              for _ in cases]
    outs = [[torch.empty_like(w) for _ in range(8)] for w in want]
    torch.cuda.synchronize()
    for k in range(8):
        for i, c in enumerate(cases):
            _run(c, out=outs[i][k], workspace=spaces[i], stream=streams[i], max_context_len=1200)
    torch.cuda.synchronize()
    for i, w in enumerate(want):
        for out in outs[i]:
            if dtype is F32:  # the bound on the contexts may change how a range is shared, and so the sums' order
                ref.assert_near(out, *_ref(cases[i]), f"stream {i}")
            else:
                assert torch.equal(bits(out), bits(w)), i


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("heads", [(32, 8, 128), (32, 4, 64), (8, 4, 256)])
def test_a_captured_batch_that_empties(dtype, heads):
    """One captured call whose batch is padded differently at each replay; rows of sequences without a tree are zero."""
    lens, nodes = [70, 300, 129, 64, 500], 20
    c = _case(lens, nodes, heads, dtype, seed=43)
    tl = torch.full((5,), nodes, dtype=torch.int32, device="cuda")
    ws = torch.zeros(max(16, pa.decode_tree_workspace_size(5, nodes, heads[0], heads[2], 512, heads[1])), dtype=torch.uint8,
                     device="cuda")
    out = torch.full_like(c["q"], 7.0)
    _run(c, out=out, workspace=ws, tree_lens=tl, max_context_len=512)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _run(c, out=out, workspace=ws, tree_lens=tl, max_context_len=512)
    for now, trees in (([0, 300, 0, 64, 500], [20, 1, 0, 20, 7]), ([0] * 5, [0] * 5), (lens, [20] * 5), ([1, 0, 0, 0, 0], [1, 0, 0, 0, 0])):
        c["lens"].copy_(torch.tensor(now, dtype=torch.int32))
        tl.copy_(torch.tensor(trees, dtype=torch.int32))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        ref.assert_near(out, *_ref(c, tree_lens=tl), f"{now}")
        for b, n in enumerate(trees):
            assert torch.count_nonzero(out[b, n if now[b] else 0:]).item() == 0
    assert pa.device_errors() == 0


@pytest.mark.parametrize("heads,nodes", [((32, 8, 128), 9), ((32, 8, 128), 40), ((8, 4, 256), 60), ((32, 4, 64), 8)])
def test_what_a_workspace_holds_before_does_not_matter(heads, nodes):
    """Any bytes in it give the same result, and the split decode's counters are left as they are."""
    lens = [90, 1700, 400]
    c = _case(lens, nodes, heads, seed=44)
    want = _run(c)
    ref.assert_near(want, *_ref(c), f"{heads}")
    need = pa.decode_tree_workspace_size(3, nodes, heads[0], heads[2], 1700, heads[1])
    for fill in (0xA5, 0x7F, 0xFF):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(bits(_run(c, workspace=ws)), bits(want))
        assert torch.equal(ws[:256 * 1024], torch.full((256 * 1024,), fill, dtype=torch.uint8, device="cuda"))
    with pytest.raises(pa.PagedAttnError):
        _run(c, workspace=torch.zeros(need - 1, dtype=torch.uint8, device="cuda"))
    assert pa.device_errors() == 0
