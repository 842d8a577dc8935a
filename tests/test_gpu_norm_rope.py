"""Norm and rotation of queries and keys (pa_qk_norm_rope) and the same with the
paged append (pa_rope_append), against a plain 64-bit form."""

import pytest
import torch

import paged_kv_cache_473_b200 as pa
from tests import draft_reference as ref
from tests.gpu_helpers import bits

pytestmark = pytest.mark.gpu

HEADS = [(8, 2, 64), (32, 4, 64), (32, 8, 128), (6, 2, 128), (8, 4, 256), (7, 1, 64), (1, 1, 256), (5, 3, 128)]


@pytest.fixture(autouse=True)
def _clear_device_errors():
    pa.device_errors()
    yield


def _inputs(n, heads, dtype, rotary, norm, seed=0, fused=True, far=5000):
    hq, hkv, d = heads
    g = torch.Generator().manual_seed(seed * 1000 + n * 7 + d + hq)
    rows = torch.randn((n, (hq + 2 * hkv) * d), generator=g).to(dtype).cuda()
    q, k, v = (t.view(n, h, d) for t, h in zip(rows.split((hq * d, hkv * d, hkv * d), 1), (hq, hkv, hkv)))
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    positions = torch.randint(0, far, (n,), generator=g, dtype=torch.int32).cuda()
    inv_freq = (10000.0 ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / max(rotary, 1))).float().cuda()
    qw = (1 + 0.3 * torch.randn((d,), generator=g)).cuda() if norm else None
    kw = (1 + 0.3 * torch.randn((d,), generator=g)).cuda() if norm else None
    return q, k, v, positions, inv_freq, qw, kw


def _check(got, x, w, positions, inv_freq, interleaved, what, eps=1e-6):
    assert_args = ref.norm_rope(x, w, eps, positions, inv_freq, interleaved)
    ref.assert_near(got, *assert_args, what)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("n", [1, 3, 37, 300])
def test_norm_rope(heads, dtype, n):
    """Every head layout and row split; rows of a fused projection; norm, interleaving and partial rotation."""
    d = heads[2]
    for rotary, norm, interleaved in ((d, False, False), (d, True, True), (16, True, False), (d - 16, False, True),
                                      (d // 2, True, False), (48, False, False)):
        q, k, v, pos, inv, qw, kw = _inputs(n, heads, dtype, rotary, norm)
        q_in, k_in = q.clone(), k.clone()
        qo, ko = pa.qk_norm_rope(q, k, pos, inv, q_weight=qw, k_weight=kw, interleaved=interleaved)
        what = f"{heads} n={n} rotary={rotary} norm={norm} interleaved={interleaved}"
        _check(qo, q_in, qw, pos, inv, interleaved, what + " q")
        _check(ko, k_in, kw, pos, inv, interleaved, what + " k")
        assert torch.equal(q, q_in) and torch.equal(k, k_in)
        assert pa.last_launch_count() == 1


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_in_place_on_a_fused_projection(dtype):
    """q_out = q and k_out = k, strided: the same bits as out of place, v's columns untouched."""
    q, k, v, pos, inv, qw, kw = _inputs(77, (32, 8, 128), dtype, 96, True)
    qo, ko = pa.qk_norm_rope(q, k, pos, inv, q_weight=qw, k_weight=kw)
    v_in = v.clone()
    pa.qk_norm_rope(q, k, pos, inv, q_weight=qw, k_weight=kw, q_out=q, k_out=k)
    assert torch.equal(bits(q), bits(qo)) and torch.equal(bits(k), bits(ko)) and torch.equal(v, v_in)


def test_norm_only_and_one_weight():
    q, k, v, pos, inv, qw, kw = _inputs(20, (8, 4, 256), torch.bfloat16, 0, True)
    qo, ko = pa.qk_norm_rope(q, k, None, None, q_weight=qw)
    _check(qo, q, qw, None, None, False, "norm only")
    assert torch.equal(bits(ko), bits(k))  # neither normed nor rotated


def test_far_and_negative_positions():
    """Angles of positions up to 2^31 - 1 in either direction keep their accuracy."""
    q, k, v, pos, inv, qw, kw = _inputs(64, (8, 2, 64), torch.float32, 64, False)
    pos = torch.tensor([2 ** 31 - 1 - i for i in range(32)] + [-(2 ** 31) + i for i in range(16)] +
                       [10 ** 6 + i for i in range(16)], dtype=torch.int32).cuda()
    qo, ko = pa.qk_norm_rope(q, k, pos, inv)
    _check(qo, q, None, pos, inv, False, "far")


def test_norm_of_tiny_large_and_zero_heads():
    """eps decides at zero; squares of 1e15 stay finite in fp32."""
    q, k, v, pos, inv, qw, kw = _inputs(6, (8, 2, 64), torch.float32, 64, True, fused=False)
    q[0] = 0
    q[1] *= 1e-12
    q[2] *= 1e15
    qo, _ = pa.qk_norm_rope(q, k, pos, inv, q_weight=qw, k_weight=kw, eps=1e-5)
    _check(qo, q, qw, pos, inv, False, "extremes", eps=1e-5)
    assert torch.count_nonzero(qo[0]).item() == 0


def test_nan_and_infinity_stay_in_their_head():
    q, k, v, pos, inv, qw, kw = _inputs(9, (8, 2, 64), torch.bfloat16, 64, True)
    clean, _ = pa.qk_norm_rope(q, k, pos, inv, q_weight=qw, k_weight=kw)
    q[4, 3, 17] = float("nan")
    q[5, 0, 2] = float("inf")
    got, _ = pa.qk_norm_rope(q, k, pos, inv, q_weight=qw, k_weight=kw)
    hit = torch.zeros(9, 8, dtype=torch.bool)
    hit[4, 3] = hit[5, 0] = True
    assert torch.equal(got[~hit.cuda()], clean[~hit.cuda()])
    assert torch.isnan(got[4, 3]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("heads,block,n", [((8, 2, 64), 16, 1), ((32, 8, 128), 16, 53), ((8, 4, 256), 128, 200),
                                           ((7, 1, 64), 24, 90), ((5, 3, 128), 1, 33)])
def test_rope_append(heads, block, n, dtype):
    """Rotated keys and bit-exact values at their slots, every other slot untouched, padding tokens skipped."""
    hq, hkv, d = heads
    q, k, v, pos, inv, qw, kw = _inputs(n, heads, dtype, d // 2, True, seed=3)
    nb = -(-n // block) + 3
    g = torch.Generator().manual_seed(n)
    slots = torch.randperm(nb * block, generator=g)[:n]
    pad = torch.arange(n) % 5 == 4
    slots[pad] = -1 - torch.arange(int(pad.sum()))
    kc = torch.full((nb, hkv, block, d), float("nan"), dtype=dtype, device="cuda")
    vc = torch.full_like(kc, float("nan"))
    q_out = torch.full((n, hq, d), 7.0, dtype=dtype, device="cuda")
    got = pa.rope_append(q, k, v, pos, slots.cuda(), inv, kc, vc, q_weight=qw, k_weight=kw, q_out=q_out)
    assert got is q_out and pa.device_errors() == 0
    live = ~pad
    assert torch.all(q_out[pad.cuda()] == 7.0)
    y, err = ref.norm_rope(q, qw, 1e-6, pos, inv, False)
    ref.assert_near(q_out[live.cuda()], y[live], err[live], "q")
    y, err = ref.norm_rope(k, kw, 1e-6, pos, inv, False)
    blk, off = slots[live] // block, slots[live] % block
    ref.assert_near(kc[blk, :, off], y[live], err[live], "k")
    assert torch.equal(bits(vc[blk, :, off]), bits(v[live.cuda()]))
    for c in (kc, vc):  # the canaries of all other slots
        c[blk, :, off] = float("nan")
        assert torch.isnan(c).all()


def test_rope_append_equals_its_parts():
    """The fused call and qk_norm_rope followed by write_kv give the same bits."""
    for heads, dtype in (((32, 8, 128), torch.bfloat16), ((8, 2, 64), torch.float32)):
        hq, hkv, d = heads
        q, k, v, pos, inv, qw, kw = _inputs(130, heads, dtype, d, True, seed=5)
        slots = torch.randperm(160, generator=torch.Generator().manual_seed(1))[:130].cuda()
        caches = [torch.zeros((10, hkv, 16, d), dtype=dtype, device="cuda") for _ in range(4)]
        q1 = pa.rope_append(q, k, v, pos, slots, inv, *caches[:2], q_weight=qw, k_weight=kw)
        q2, k2 = pa.qk_norm_rope(q, k, pos, inv, q_weight=qw, k_weight=kw)
        pa.write_kv(k2, v.contiguous(), slots, *caches[2:])
        assert torch.equal(bits(q1), bits(q2))
        assert torch.equal(bits(caches[0]), bits(caches[2])) and torch.equal(bits(caches[1]), bits(caches[3]))


def test_rope_append_slot_outside_the_pool():
    q, k, v, pos, inv, qw, kw = _inputs(4, (8, 2, 64), torch.bfloat16, 64, False)
    kc = torch.zeros((2, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    slots = torch.tensor([3, 32, 2 ** 40, 5]).cuda()
    q_out = pa.rope_append(q, k, v, pos, slots, inv, kc, vc)
    assert pa.device_errors() == pa.DEVERR_SLOT
    y, err = ref.norm_rope(q, None, 1e-6, pos, inv, False)
    ref.assert_near(q_out, y, err, "q of skipped rows too")
    written = torch.nonzero(vc.abs().sum((1, 3)).flatten())[:, 0].tolist()
    assert written == [3, 5]


def test_rope_append_past_32_bit_offsets():
    """A pool whose last block starts past 2^31 elements (and 2^32 bytes)."""
    hkv, d, block = 8, 128, 16
    nb = 2 ** 31 // (hkv * block * d) + 64
    kc = torch.empty((nb, hkv, block, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    q, k, v, pos, inv, qw, kw = _inputs(3, (8, hkv, d), torch.bfloat16, d, False)
    last = (nb - 1) * block
    kc[0].fill_(3.0)
    slots = torch.tensor([last, last + 15, last - 1]).cuda()
    pa.rope_append(q, k, v, pos, slots, inv, kc, vc)
    assert pa.device_errors() == 0
    y, err = ref.norm_rope(k, None, 1e-6, pos, inv, False)
    ref.assert_near(torch.stack([kc[nb - 1, :, 0], kc[nb - 1, :, 15], kc[nb - 2, :, 15]]), y, err, "far rows")
    assert torch.equal(vc[nb - 1, :, 15], v[1]) and torch.all(kc[0] == 3.0)


def test_other_stream_and_captured_graph():
    q, k, v, pos, inv, qw, kw = _inputs(40, (32, 4, 64), torch.bfloat16, 64, False)
    slots = torch.arange(40).cuda()
    want_k = torch.zeros((3, 4, 16, 64), dtype=torch.bfloat16, device="cuda")
    want_v = torch.zeros_like(want_k)
    want_q = pa.rope_append(q, k, v, pos, slots, inv, want_k, want_v)
    kc, vc, q_out = torch.zeros_like(want_k), torch.zeros_like(want_k), torch.zeros_like(want_q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    pa.rope_append(q, k, v, pos, slots, inv, kc, vc, q_out=q_out, stream=side)
    side.synchronize()
    assert torch.equal(bits(kc), bits(want_k)) and torch.equal(bits(q_out), bits(want_q))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.rope_append(q, k, v, pos, slots, inv, kc, vc, q_out=q_out)
    for shift in (3, 11):  # new positions in place: the replay sees them
        pos += shift
        kc.zero_(), q_out.zero_()
        graph.replay()
        want_q = pa.rope_append(q, k, v, pos, slots, inv, want_k, want_v)
        torch.cuda.synchronize()
        assert torch.equal(bits(kc), bits(want_k)) and torch.equal(bits(q_out), bits(want_q))


def test_no_tokens():
    q = torch.empty((0, 8, 64), dtype=torch.bfloat16, device="cuda")
    k = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    pos = torch.empty((0,), dtype=torch.int32, device="cuda")
    inv = torch.ones(32, device="cuda")
    qo, ko = pa.qk_norm_rope(q, k, pos, inv)
    assert qo.shape == q.shape and ko.shape == k.shape and pa.last_launch_count() == 0
