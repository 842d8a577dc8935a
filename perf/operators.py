"""The operators of a drafting step over the paged cache, as cases to measure.

A serving engine that drafts a tree of tokens and verifies it in one pass runs,
per layer: the norm and rotation of the new queries and keys with their append
(``rope_append``, or ``norm_rope`` where another call appends), the attention of
the drafted tree over the cache (``tree``), and, once the accepted path is
known, the move of its rows to their places (``commit``).

``own`` is false: ``run`` computes the operators with elementary torch
operations in 32 bits (angles in 64), rounded once at the end.  ``own`` is true:
``run`` makes the calls a user makes of this package.
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}

# (query heads, kv heads, head_dim) of this repository's decode workloads, and
# two odd group sizes (3 and 7).
_HEADS = ((8, 2, 64), (32, 4, 64), (8, 4, 256), (32, 8, 128), (6, 2, 128), (7, 1, 64))


# ---- cases ---------------------------------------------------------------------------


def _rope(op, tokens, heads, dtype="bf16", norm=False, interleaved=False, rotary=0, pad=0, block=16, far=8192):
    hq, hkv, d = heads
    return {"op": op, "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "dtype": dtype, "norm": norm,
            "interleaved": interleaved, "rotary": rotary or d, "pad": pad, "block": block, "far": far}


def _tree(batch, nodes, heads, lo, hi, dtype="bf16", block=16, softcap=0.0, window=0, ragged=False):
    hq, hkv, d = heads
    return {"op": "tree", "batch": batch, "nodes": nodes, "hq": hq, "hkv": hkv, "d": d, "lo": lo, "hi": hi,
            "dtype": dtype, "block": block, "softcap": softcap, "window": window, "ragged": ragged}


def _commit(batch, nodes, path, layers, heads, lo, hi, dtype="bf16", block=16):
    hq, hkv, d = heads
    return {"op": "commit", "batch": batch, "nodes": nodes, "path": path, "layers": layers, "hkv": hkv, "d": d,
            "lo": lo, "hi": hi, "dtype": dtype, "block": block}


def listed():
    return [
        # One decode step's rotation and append for 64 sequences, rows of a fused projection.
        dict(_rope("rope_append", 64, (32, 4, 64)), name="append decode 64"),
        # The same for a whole prefill of 16 prompts of 1024 tokens.
        dict(_rope("rope_append", 16384, (32, 8, 128)), name="append prefill 16K"),
        # fp32, odd count, padded rows of a captured batch, norms, interleaved pairs on half of the head.
        dict(_rope("rope_append", 37, (8, 2, 64), "f32", True, True, 32, 5), name="append fp32 odd"),
        # Norm and rotation ahead of the fused decode step, one token for each of 128 sequences.
        dict(_rope("norm_rope", 128, (32, 8, 128), norm=True), name="norm_rope decode 128"),
        # A prefill chunk of odd length with norms, wide heads, far positions, three quarters rotated.
        dict(_rope("norm_rope", 8191, (8, 4, 256), norm=True, rotary=192, far=131072), name="norm_rope prefill 8K"),
        # A small tree on the fp32 cache: latency.
        dict(_tree(4, 5, (8, 2, 64), 8, 100, "f32"), name="tree fp32 4x5"),
        # Eight drafted tokens for each of 64 sequences, contexts up to 2048.
        dict(_tree(64, 8, (32, 4, 64), 128, 2048), name="tree 64x8 d64"),
        # Sixteen drafted tokens for each of 128 sequences, contexts spread over 256 to 8192.
        dict(_tree(128, 16, (32, 8, 128), 256, 8192), name="tree 128x16 d128"),
        # Wide heads with the logit softcap, large pages, a ragged batch of trees.
        dict(_tree(256, 24, (8, 4, 256), 129, 1024, block=128, softcap=50.0, ragged=True), name="tree 256x24 d256"),
        # The largest trees on long contexts: arithmetic as much as bandwidth.
        dict(_tree(8, 64, (32, 8, 128), 16384, 131072), name="tree 8x64 long"),
        # The accepted paths of 64 sequences moved in every layer's cache at once.
        dict(_commit(64, 16, 5, 22, (32, 4, 64), 128, 2048), name="commit 64 in 22 layers"),
        # One layer's cache, large trees.
        dict(_commit(128, 64, 9, 1, (32, 8, 128), 256, 2048), name="commit 128 in a layer"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope_append", "norm_rope", "tree", "tree", "tree", "commit"))
    heads = rng.choice(_HEADS)
    hq, hkv, d = heads
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    block = rng.choice((16, 16, 32, 64, 128, 256))
    if op in ("rope_append", "norm_rope"):
        n = _log(rng, 1, 16384 * 48 * 128 // ((hq + 2 * hkv) * d * (2 if dtype == "f32" else 1)))
        pad = rng.randrange(0, min(n, 9)) if op == "rope_append" and rng.random() < 0.3 else 0
        return _rope(op, n, heads, dtype, rng.random() < 0.5, rng.random() < 0.3, rng.randrange(1, d // 16 + 1) * 16,
                     pad, block, _log(rng, 64, 1 << 20))
    if op == "commit":
        nodes = rng.randrange(3, 65)
        return _commit(_log(rng, 1, 256), nodes, rng.randrange(1, (nodes + 1) // 2 + 1), rng.choice((1, 1, 2, 5, 22)),
                       heads, 64, _log(rng, 128, 1024), dtype, block)
    nodes = rng.randrange(1, 65)
    if dtype == "f32":  # the fp32 cache serves checks and small models
        batch, hi = _log(rng, 1, 16), _log(rng, 128, 2048)
    else:
        batch = _log(rng, 1, 256)
        # no more work than the largest listed case, and a plain form that fits
        room = 8 * 131072 * 8 * 128 // (batch * hkv * d)
        hi = _log(rng, 128, min(131072, max(256, min(room, 8 * 131072 * 32 * 64 // (batch * hq * nodes)) // 2)))
    lo = max(nodes, hi // rng.choice((1, 4, 16)))
    return _tree(batch, nodes, heads, lo, max(lo, hi), dtype, block, 50.0 if rng.random() < 0.25 else 0.0,
                 _log(rng, 8, 4096) if rng.random() < 0.25 else 0, rng.random() < 0.4)


# ---- sizes that follow from a case alone (a seed only changes their order) -------------


def _lengths(c):
    """Context lengths, drafted nodes included: evenly spread over the logarithm of [lo, hi]."""
    b, lo, hi = c["batch"], math.log(c["lo"]), math.log(c["hi"])
    return [min(c["hi"], max(c["lo"], int(round(math.exp(lo + (hi - lo) * (i + 0.5) / b))))) for i in range(b)]


def _tree_lens(c):
    n, b = c["nodes"], c["batch"]
    return [n if not c.get("ragged") else max(1, n - (i * 7) % (n // 2 + 1)) for i in range(b)]


def _paths(c):
    return [1 + (i % c["path"]) for i in range(c["batch"])]


# ---- inputs --------------------------------------------------------------------------


def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _pool(c, g, cpu, lens):
    """Block tables over a shuffled pool with some blocks of others in between."""
    bs = c["block"]
    need = [-(-n // bs) for n in lens]
    nb = sum(need) + max(1, sum(need) // 16)
    ids = torch.randperm(nb, generator=cpu).to(torch.int32)
    tables = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
    at = 0
    for b, k in enumerate(need):
        tables[b, :k] = ids[at:at + k]
        at += k
    return tables.cuda(), nb


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    dt, d, hkv = _DT[c["dtype"]], c["d"], c["hkv"]
    if c["op"] in ("rope_append", "norm_rope"):
        n, hq, rd = c["tokens"], c["hq"], c["rotary"]
        rows = _randn(g, (n, (hq + 2 * hkv) * d), dt)  # the fused projection's output
        q, k, v = rows.split((hq * d, hkv * d, hkv * d), dim=1)
        s = {"op": c["op"], "q": q.view(n, hq, d), "k": k.view(n, hkv, d), "v": v.view(n, hkv, d),
             "positions": torch.randint(0, c["far"], (n,), generator=cpu, dtype=torch.int32).cuda(),
             "inv_freq": (10000.0 ** (-torch.arange(0, rd, 2, dtype=torch.float64) / rd)).float().cuda(),
             "q_weight": None, "k_weight": None, "eps": 1e-6, "interleaved": c["interleaved"], "rotary": rd,
             "q_out": torch.empty((n, hq, d), dtype=dt, device="cuda")}
        if c["norm"]:
            s["q_weight"] = 1 + 0.2 * torch.randn((d,), generator=g, device="cuda")
            s["k_weight"] = 1 + 0.2 * torch.randn((d,), generator=g, device="cuda")
        if c["op"] == "norm_rope":
            s["k_out"] = torch.empty((n, hkv, d), dtype=dt, device="cuda")
            return s
        bs = c["block"]
        nb = -(-n // bs) + 1 + n // (8 * bs)
        slots = torch.randperm(nb * bs, generator=cpu)[:n]
        if n > 1024:  # a prefill fills whole blocks, a decode step one row of each
            blocks = torch.randperm(nb, generator=cpu)
            at = torch.arange(n)
            slots = blocks[at // bs] * bs + at % bs
        if c["pad"]:  # the padded rows of a captured batch are its last ones
            slots[n - c["pad"]:] = -1
            s["q_out"].zero_()  # padded rows stay as they were
        s["slots"] = slots.cuda()
        s["k_cache"] = _randn(g, (nb, hkv, bs, d), dt)
        s["v_cache"] = _randn(g, (nb, hkv, bs, d), dt)
        return s
    order = torch.randperm(c["batch"], generator=cpu).tolist()
    lens = [_lengths(c)[i] for i in order]
    s = {"op": c["op"], "nodes": c["nodes"], "max_len": max(lens),
         "lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    s["tables"], nb = _pool(c, g, cpu, lens)
    if c["op"] == "commit":
        s["k_cache"] = _randn(g, (c["layers"], nb, hkv, c["block"], d), dt)
        s["v_cache"] = _randn(g, (c["layers"], nb, hkv, c["block"], d), dt)
        take = [_paths(c)[i] for i in order]
        path = torch.zeros((c["batch"], c["path"]), dtype=torch.int32)
        for b, a in enumerate(take):
            # The root, then one node of each deeper level.  A tree's levels lie one
            # after the other, so these are behind the first a places, and the same
            # pass again moves the same rows.
            path[b, 1:a] = torch.sort(torch.randperm(c["nodes"] - a, generator=cpu)[:a - 1])[0].to(torch.int32) + a
        s["path"] = path.cuda()
        s["take"] = torch.tensor(take, dtype=torch.int32, device="cuda")
        s["new_lens"] = torch.empty((c["batch"],), dtype=torch.int32, device="cuda")
        return s
    s["k_cache"] = _randn(g, (nb, hkv, c["block"], d), dt)
    s["v_cache"] = _randn(g, (nb, hkv, c["block"], d), dt)
    s["q"] = _randn(g, (c["batch"], c["nodes"], c["hq"], d), dt, 2.0)
    s["scale"], s["softcap"], s["window"] = d ** -0.5, c["softcap"], c["window"]
    bit = torch.ones((c["batch"],), dtype=torch.int64)
    mask = torch.zeros((c["batch"], c["nodes"]), dtype=torch.int64)
    for j in range(c["nodes"]):  # node j hangs below an earlier node: that node's ancestors and itself
        if j:
            parent = (torch.rand((c["batch"],), generator=cpu) * j).long()
            mask[:, j] = mask.gather(1, parent[:, None])[:, 0]
        mask[:, j] |= bit << j
    s["mask"] = mask.cuda()
    s["tree_lens"] = None
    if c["ragged"]:
        s["tree_lens"] = torch.tensor([_tree_lens(c)[i] for i in order], dtype=torch.int32, device="cuda")
    s["out"] = torch.empty_like(s["q"])
    return s


# ---- the plain forms -------------------------------------------------------------------


def _rotated(x, weight, s):
    """Norm over each head, then the rotation of the first ``rotary`` elements by position * inv_freq."""
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + s["eps"]) * weight
    rd = s["rotary"]
    angle = (s["positions"].double()[:, None] * s["inv_freq"].double())[:, None, :]
    cos, sin = angle.cos().float(), angle.sin().float()
    y, rest = y[..., :rd], y[..., rd:]
    if s["interleaved"]:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = y[..., :rd // 2], y[..., rd // 2:]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, rest), -1).to(x.dtype)


def _plain_norm_rope(s):
    s["q_out"].copy_(_rotated(s["q"], s["q_weight"], s))
    s["k_out"].copy_(_rotated(s["k"], s["k_weight"], s))


def _plain_append(s):
    bs = s["k_cache"].shape[2]
    live = s["slots"] >= 0
    slots = s["slots"][live]
    s["q_out"][live] = _rotated(s["q"], s["q_weight"], s)[live]
    s["k_cache"][slots // bs, :, slots % bs] = _rotated(s["k"], s["k_weight"], s)[live]
    s["v_cache"][slots // bs, :, slots % bs] = s["v"][live]


def _depths(mask):
    """Nodes that each node attends besides itself: its distance below the root."""
    n = mask.shape[1]
    bits = (mask[:, :, None] >> torch.arange(n, device=mask.device)) & 1
    return bits.sum(-1) - torch.diagonal(bits, dim1=1, dim2=2)


def _plain_tree(s):
    q, mask, window = s["q"], s["mask"], s["window"]
    batch, n, hq, d = q.shape
    hkv, bs = s["k_cache"].shape[1:3]
    pages = s["tables"].clamp(min=0).long()
    length = pages.shape[1] * bs
    k = s["k_cache"][pages].transpose(1, 2).reshape(batch, hkv, length, d).float()
    x = q.float().view(batch, n, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(batch, hkv, -1, d)
    x = (x @ k.transpose(2, 3)) * s["scale"]
    del k
    if s["softcap"] > 0:
        x = s["softcap"] * torch.tanh(x / s["softcap"])
    x = x.view(batch, hkv, n, hq // hkv, length)

    lens = s["lens"].long()[:, None]
    count = torch.full_like(lens, n) if s["tree_lens"] is None else s["tree_lens"].long()[:, None]
    base = lens - count
    t = torch.arange(length, device=q.device)[None]
    node = t - base
    in_tree = (node >= 0) & (node < count)
    node = node.clamp(0, n - 1)
    keep = ((mask[:, :, None] >> node[:, None]) & 1).bool() & in_tree[:, None] | (t < base)[:, None]
    keep &= (torch.arange(n, device=q.device) < count)[:, :, None]
    if window > 0:
        depth = _depths(mask)
        at = torch.where(t < base, t, base + depth.gather(1, node))
        keep &= at[:, None] > (base + depth)[:, :, None] - window
    x = x.masked_fill(~keep[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = x.sum(-1)
    v = s["v_cache"][pages].transpose(1, 2).reshape(batch, hkv, length, d).float()
    o = (x.view(batch, hkv, -1, length) @ v).view(batch, hkv, n, hq // hkv, d)
    o = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
    s["out"].copy_(o.permute(0, 2, 1, 3, 4).reshape(batch, n, hq, d))


def _plain_commit(s):
    bs = s["k_cache"].shape[3]
    base = s["lens"].long()[:, None] - s["nodes"]
    i = torch.arange(s["path"].shape[1], device=base.device)[None]
    real = i < s["take"].long()[:, None]
    src = base + torch.where(real, s["path"].long(), 0)  # behind a path's end: the root onto itself
    dst = base + torch.where(real, i, 0)
    tables = s["tables"].long()
    from_block, to_block = tables.gather(1, src // bs), tables.gather(1, dst // bs)
    k = s["k_cache"][:, from_block, :, src % bs]
    v = s["v_cache"][:, from_block, :, src % bs]
    s["k_cache"][:, to_block, :, dst % bs] = k
    s["v_cache"][:, to_block, :, dst % bs] = v
    s["new_lens"].copy_(s["lens"] - s["nodes"] + s["take"])


_PLAIN = {"rope_append": _plain_append, "norm_rope": _plain_norm_rope, "tree": _plain_tree, "commit": _plain_commit}


# ---- the framework's calls ---------------------------------------------------------------


def _own_norm_rope(s):
    import paged_kv_cache_473_b200 as pa

    pa.qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                    eps=s["eps"], interleaved=s["interleaved"], q_out=s["q_out"], k_out=s["k_out"])


def _own_append(s):
    import paged_kv_cache_473_b200 as pa

    pa.rope_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["inv_freq"], s["k_cache"], s["v_cache"],
                   q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"], interleaved=s["interleaved"],
                   q_out=s["q_out"])


def _own_tree(s):
    import paged_kv_cache_473_b200 as pa

    if "workspace" not in s:  # kept from step to step
        b, n, hq, d = s["q"].shape
        need = pa.decode_tree_workspace_size(b, n, hq, d, s["max_len"], s["k_cache"].shape[1])
        s["workspace"] = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")
    pa.decode_tree(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["mask"], s["scale"], s["softcap"],
                   s["window"], max_context_len=s["max_len"], tree_lens=s["tree_lens"], out=s["out"],
                   workspace=s["workspace"])


def _own_commit(s):
    import paged_kv_cache_473_b200 as pa

    pa.commit_tree(s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["path"], s["take"], tree_len=s["nodes"],
                   new_lens=s["new_lens"])


_OWN = {"rope_append": _own_append, "norm_rope": _own_norm_rope, "tree": _own_tree, "commit": _own_commit}

_OUTPUTS = {"rope_append": ("q_out", "k_cache", "v_cache"), "norm_rope": ("q_out", "k_out"), "tree": ("out",),
            "commit": ("k_cache", "v_cache", "new_lens")}


def run(state):
    (_OWN if own else _PLAIN)[state["op"]](state)
    return {name: state[name] for name in _OUTPUTS[state["op"]]}


# ---- what a pass cannot do without ---------------------------------------------------------


def work(case):
    c = case
    size = 4 if c["dtype"] == "f32" else 2
    if c["op"] in ("rope_append", "norm_rope"):
        n = c["tokens"] - c["pad"]
        heads = c["hq"] + c["hkv"] * (2 if c["op"] == "rope_append" else 1)
        index = 12 if c["op"] == "rope_append" else 4
        turned = (c["hq"] + c["hkv"]) * (3 * c["rotary"] + (4 * c["d"] if c["norm"] else 0))
        return {"bytes": n * (2 * heads * c["d"] * size + index) + 2 * c["rotary"] + (8 * c["d"] if c["norm"] else 0),
                "flops": n * turned}
    lens = _lengths(c)
    if c["op"] == "commit":
        moved = sum(a - 1 for a in _paths(c))
        row = c["layers"] * 2 * c["hkv"] * c["d"] * size
        return {"bytes": 2 * moved * row + 4 * (sum(_paths(c)) + 3 * c["batch"]), "flops": 0}
    counts = _tree_lens(c)
    # Positions before the tree that some node attends (its window starts no earlier than the root's).
    before = [a - n if c["window"] <= 0 else min(a - n, c["window"]) for a, n in zip(lens, counts)]
    keys = sum(before) + sum(counts)
    pairs = sum(n * (a + 1) for a, n in zip(before, counts))
    rows = c["batch"] * c["nodes"] * c["hq"] * c["d"]
    return {"bytes": size * (2 * keys * c["hkv"] * c["d"] + 2 * rows) + 4 * (keys // c["block"]) + 8 * c["batch"] * c["nodes"],
            "flops": 4 * pairs * c["hq"] * c["d"]}


# ---- the definitions, in 64 bits -------------------------------------------------------------


def _exact_rows(x, weight, s):
    """One complex product for each pair of elements."""
    x = x.double()
    if weight is not None:
        rms = torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + s["eps"])
        x = x / rms * weight.double()
    rd = s["rotary"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device).expand(x.shape[0], rd // 2),
                       torch.outer(s["positions"].double(), s["inv_freq"].double()))[:, None]
    out = x.clone()
    first = torch.arange(rd // 2, device=x.device) * (2 if s["interleaved"] else 1)
    second = first + (1 if s["interleaved"] else rd // 2)
    z = torch.complex(x[..., first], x[..., second]) * turn
    out[..., first], out[..., second] = z.real, z.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "norm_rope":
        return {"q_out": _exact_rows(s["q"], s["q_weight"], s), "k_out": _exact_rows(s["k"], s["k_weight"], s)}
    if s["op"] == "rope_append":
        nb, hkv, bs, d = s["k_cache"].shape
        q, live = s["q_out"].double(), torch.nonzero(s["slots"] >= 0)[:, 0]
        q[live] = _exact_rows(s["q"], s["q_weight"], s)[live]
        got = {"q_out": q}
        for name, rows in (("k_cache", _exact_rows(s["k"], s["k_weight"], s)), ("v_cache", s["v"].double())):
            flat = s[name].double().transpose(1, 2).reshape(nb * bs, hkv, d)  # by slot
            flat[s["slots"][live]] = rows[live]
            got[name] = flat.view(nb, bs, hkv, d).transpose(1, 2).contiguous()
        return got
    lens, tables = s["lens"].tolist(), s["tables"].long()
    bs = s["k_cache"].shape[-2]
    if s["op"] == "commit":
        layers, nb, hkv, _, d = s["k_cache"].shape
        place, source = [], []
        for b, (path, a) in enumerate(zip(s["path"].tolist(), s["take"].tolist())):
            slots = (tables[b][:, None] * bs + torch.arange(bs, device=tables.device)).flatten().tolist()
            base = lens[b] - s["nodes"]
            place += [slots[base + i] for i in range(a)]
            source += [slots[base + node] for node in path[:a]]
        got = {"new_lens": torch.tensor([n - s["nodes"] + a for n, a in zip(lens, s["take"].tolist())], dtype=torch.int32)}
        for name in ("k_cache", "v_cache"):
            flat = s[name].transpose(2, 3).reshape(layers, nb * bs, hkv, d).double()
            flat[:, place] = flat[:, source].clone()
            got[name] = flat.view(layers, nb, bs, hkv, d).transpose(2, 3).contiguous()
        return got
    batch, nodes, hq, d = s["q"].shape
    hkv = s["k_cache"].shape[1]
    masks = s["mask"].tolist()
    counts = [nodes] * batch if s["tree_lens"] is None else s["tree_lens"].tolist()
    out = torch.zeros((batch, nodes, hq, d), dtype=torch.float64, device="cuda")
    for b in range(batch):
        n, base = counts[b], lens[b] - counts[b]
        sees = torch.tensor([[(masks[b][j] >> i) & 1 for i in range(n)] for j in range(n)], dtype=torch.float64)
        deep = (sees.sum(1) - sees.diagonal()).cuda()
        sees = sees.cuda().bool()
        rows = tables[b][:-(-lens[b] // bs)]
        where = torch.cat((torch.arange(base, device="cuda").double(), base + deep))  # positions, the nodes' by depth
        keep = torch.cat((torch.ones((n, base), dtype=torch.bool, device="cuda"), sees), 1)
        if s["window"] > 0:
            keep &= where[None] > (base + deep)[:, None] - s["window"]
        for g in range(hkv):
            k = s["k_cache"][rows, g].reshape(-1, d)[:lens[b]].double()
            v = s["v_cache"][rows, g].reshape(-1, d)[:lens[b]].double()
            heads = slice(g * (hq // hkv), (g + 1) * (hq // hkv))
            x = torch.einsum("jhd,td->hjt", s["q"][b, :n, heads].double(), k) * s["scale"]
            if s["softcap"] > 0:
                x = s["softcap"] * torch.tanh(x / s["softcap"])
            w = torch.softmax(x.masked_fill(~keep, -math.inf), -1).nan_to_num(0.0)
            out[b, :n, heads] = torch.einsum("hjt,td->jhd", w, v)
    return {"out": out}
