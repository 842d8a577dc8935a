"""Plain 64-bit forms of the drafting step's operators (CPU, torch fp64), with
elementwise error bounds derived from the kernels' arithmetic.

Each bound counts roundings of at most half a step (``eps / 2`` relative):
2^-8 for bf16 values, 2^-24 for fp32 operations.
"""

from __future__ import annotations

import math

import torch

H32 = 2.0 ** -24  # one fp32 rounding
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: H32}  # the rounding at a store


def norm_rope(x, weight, eps, positions, inv_freq, interleaved):
    """Rows ``[N, H, D]`` normed (weight given) and rotated; returns (y, bound on |error| before the store)."""
    x = x.detach().cpu().double()
    if weight is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + float(torch.tensor(eps, dtype=torch.float32)))
        x = x * weight.detach().cpu().double()
    # The norm: a sum of D squares held by D / 8 lanes (8 + 5 additions and the products), halved by the
    # root; the root, the quotient and two products: under 16 roundings.
    out, err = x.clone(), x.abs() * 16 * H32
    rd = 0 if inv_freq is None else 2 * inv_freq.numel()
    if rd:
        t = positions.detach().cpu().double()[:, None] * inv_freq.detach().cpu().double()[None]
        cos, sin = torch.cos(t)[:, None], torch.sin(t)[:, None]
        i = torch.arange(rd // 2)
        a_at, b_at = (2 * i, 2 * i + 1) if interleaved else (i, i + rd // 2)
        a, b = x[..., a_at], x[..., b_at]
        out[..., a_at], out[..., b_at] = a * cos - b * sin, b * cos + a * sin
        # cos and sin: the angle in half turns rounded once (its error in radians is pi times that),
        # two units in the last place of sincospif; the products and the sum: under 12 roundings more.
        e = (a.abs() + b.abs()) * 28 * H32
        err[..., a_at], err[..., b_at] = e, e
    return out, err


def depths(mask, n):
    """Nodes each of the first n nodes attends besides itself."""
    return [bin(mask[j] & ((1 << n) - 1) & ~(1 << j)).count("1") for j in range(n)]


def words(mask):
    """Python ints (64 bits, unsigned) of an int64 mask row."""
    return [int(w) & (2 ** 64 - 1) for w in mask]


def tree(q, k_cache, v_cache, tables, lens, mask, scale, softcap=0.0, window=0, tree_lens=None):
    """``[B, T, Hq, D]`` attention of drafted trees, and a bound on each element's error."""
    dt = q.dtype
    q, k_cache, v_cache = (x.detach().cpu() for x in (q, k_cache, v_cache))
    tables, lens, mask = tables.cpu().long(), lens.cpu().tolist(), mask.cpu()
    B, T, hq, d = q.shape
    hkv, bs = k_cache.shape[1:3]
    G = hq // hkv
    scale = float(torch.tensor(scale, dtype=torch.float32))
    out, err = torch.zeros(B, T, hq, d, dtype=torch.float64), torch.zeros(B, T, hq, d, dtype=torch.float64)
    counts = [T] * B if tree_lens is None else tree_lens.cpu().tolist()
    for b in range(B):
        L, n = lens[b], counts[b]
        if L <= 0 or not 0 < n <= T or n > L:
            continue
        base, w = L - n, words(mask[b] if mask.dim() == 2 else mask)
        depth = torch.tensor(depths(w, n))
        at = torch.cat((torch.arange(base), base + depth))  # logical positions
        sees = torch.tensor([[bool((w[j] >> i) & 1) for i in range(n)] for j in range(n)])
        keep = torch.cat((torch.ones(n, base, dtype=torch.bool), sees), 1)
        if window > 0:
            keep &= at[None] > (base + depth)[:, None] - window
        rows = tables[b, : -(-L // bs)]
        for g in range(hkv):
            k = k_cache[rows, g].reshape(-1, d)[:L].double()
            v = v_cache[rows, g].reshape(-1, d)[:L].double()
            x = q[b, :n, g * G:(g + 1) * G].double().permute(1, 0, 2)  # [G, n, d]
            s = x @ k.T * scale
            size = x.abs() @ k.abs().T * abs(scale)
            if softcap > 0:
                s = softcap * torch.tanh(s / softcap)
            s, size = s.masked_fill(~keep, -math.inf), size.masked_fill(~keep, 0.0)
            any_ = keep.any(1)
            p = torch.softmax(s, -1)
            p[:, ~any_] = 0.0
            # A masked place weighs nothing, whatever stands there.
            vz = torch.where(keep.any(0)[:, None], v, 0.0)
            if torch.isfinite(vz).all():
                o, a = p @ vz, p @ vz.abs()
            else:
                pv = torch.where(keep[None, :, :, None], p[..., None] * vz[None, None], 0.0)
                o, a = pv.sum(2), pv.abs().sum(2)
            top = size.nan_to_num(0.0, 0.0, 0.0).amax(-1, keepdim=True)
            # Score: D products summed in fp32 (two roundings each on the tensor cores, which may truncate),
            # scaled to the base-2 domain (|s| log2 e, one more), the cap's tanh (four roundings of 2 cap),
            # the exponential (four).  A weight is off by that relatively, and so is their sum.
            delta = (2 * d * H32 + 4 * H32) * top + (16 * H32 * softcap if softcap > 0 else 0.0) + 8 * H32
            # Sums over the L keys in steps of 16, joined over pieces.
            delta = 2 * delta + (L / 8 + 64) * H32
            if dt == torch.bfloat16:
                delta = delta + HALF[dt]  # the weights are rounded to bf16 for the second product
            out[b, :n, g * G:(g + 1) * G] = o.permute(1, 0, 2)
            err[b, :n, g * G:(g + 1) * G] = (a * delta).permute(1, 0, 2)
    return out, err


def assert_near(got, ref, err, what=""):
    """got is within the bound and half a step of its type of ref; NaN and infinities in the same places."""
    g = got.detach().cpu().double()
    assert g.shape == ref.shape
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isnan(g), torch.isnan(ref)), f"{what}: NaN in other places"
    assert torch.equal(g[~fine & ~torch.isnan(ref)], ref[~fine & ~torch.isnan(ref)]), f"{what}: infinities differ"
    tol = ref.abs() * HALF[got.dtype] * (1 + 2.0 ** -8) + err
    over = ((g - ref).abs() - tol)[fine]
    if over.numel():
        worst = float(over.max())
        assert worst <= 0, f"{what}: {worst:.3g} over the bound (largest error {float((g - ref).abs()[fine].max()):.3g})"


def random_trees(gen, batch, nodes, chain=False):
    """int64 mask words ``[batch, nodes]`` of random trees (node j below an earlier node), and the parents."""
    parent = torch.zeros(batch, nodes, dtype=torch.int64)
    mask = torch.zeros(batch, nodes, dtype=torch.int64)
    for b in range(batch):
        for j in range(nodes):
            up = 0
            if j:
                i = j - 1 if chain else int(torch.randint(0, j, (1,), generator=gen))
                parent[b, j] = i
                up = int(mask[b, i])
            w = (up & (2 ** 64 - 1)) | (1 << j)
            mask[b, j] = w - 2 ** 64 if w >> 63 else w
    return mask, parent


def pool(gen, lens, hkv, d, block, dtype, extra=3, fill=float("nan"), device="cuda"):
    """A paged pool with random rows for each sequence's positions and canaries everywhere else."""
    need = [-(-n // block) for n in lens]
    nb = sum(need) + extra
    ids = torch.randperm(nb, generator=gen)
    tables = torch.full((len(lens), max(1, max(need, default=0))), -1, dtype=torch.int32)
    kc = torch.full((nb, hkv, block, d), fill, dtype=dtype)
    vc = torch.full((nb, hkv, block, d), fill, dtype=dtype)
    at = 0
    for b, n in enumerate(lens):
        for i in range(need[b]):
            blk = int(ids[at])
            at += 1
            tables[b, i] = blk
            m = min(block, n - i * block)
            kc[blk, :, :m] = torch.randn((hkv, m, d), generator=gen).to(dtype)
            vc[blk, :, :m] = torch.randn((hkv, m, d), generator=gen).to(dtype)
    return (kc.to(device), vc.to(device), tables.to(device),
            torch.tensor(list(lens), dtype=torch.int32, device=device))
