"""Calls on another stream than the current one that make their outputs (and
workspaces) themselves: the memory comes from the launch stream's pool, so that no
work queued on the current stream still uses it."""

import pytest
import torch

import paged_kv_cache_473_b200 as pa
from tests import draft_reference as ref

pytestmark = pytest.mark.gpu

D, HQ, HKV, BLOCK = 64, 8, 2, 16
LENS = [40, 7, 133]


@pytest.fixture(autouse=True)
def _clear_device_errors():
    pa.device_errors()
    yield
    assert pa.device_errors() == 0


def _pool_of(t):
    """The stream whose pool a tensor's memory is from."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not torch's memory")


def _inputs(dtype):
    g = torch.Generator().manual_seed(4)
    kc, vc, tables, cl = ref.pool(g, LENS, HKV, D, BLOCK, dtype, fill=0.0)
    s = {"kc": kc, "vc": vc, "tables": tables, "cl": cl, "max": max(LENS)}
    B = len(LENS)

    def rows(*shape):
        return torch.randn((*shape, D), generator=g).to(dtype).cuda()

    s["q"], s["qt"], s["k"], s["v"] = rows(B, HQ), rows(B, 5, HQ), rows(B, HKV), rows(B, HKV)
    s["mask"] = ref.random_trees(g, B, 5)[0].cuda()
    s["pos"] = (cl - 1).contiguous()
    s["inv"] = torch.rand(D // 2, generator=g).cuda()
    s["slots"] = torch.full((B,), -1, dtype=torch.int64).cuda()
    s["slots"][1] = int(tables[1, 0]) * BLOCK + 6
    s["accepted"] = torch.tensor([[0, 1]] * B, dtype=torch.int32).cuda()
    s["take"] = torch.full((B,), 2, dtype=torch.int32).cuda()
    s["cu"] = torch.arange(B + 1, dtype=torch.int32).cuda()
    return s


def _norm_rope(s, stream):
    return pa.qk_norm_rope(s["q"], s["k"], s["pos"], s["inv"], stream=stream)


def _append(s, stream):
    kc, vc = s["kc"].clone(), s["vc"].clone()  # (rows of padding tokens are not written)
    torch.cuda.current_stream().synchronize()
    out = pa.rope_append(s["q"], s["k"], s["v"], s["pos"], s["slots"], s["inv"], kc, vc, stream=stream)
    torch.cuda.synchronize()
    return out[1:2]


def _tree(s, stream):
    return pa.decode_tree(s["qt"], s["kc"], s["vc"], s["tables"], s["cl"], s["mask"], D ** -0.5,
                          max_context_len=s["max"], stream=stream)


def _commit(s, stream):
    return pa.commit_tree(s["kc"], s["vc"], s["tables"], s["cl"], s["accepted"], s["take"], tree_len=5, stream=stream)


def _args(s, q="q"):
    return s[q], s["kc"], s["vc"], s["tables"], s["cl"], D ** -0.5


def _decode(s, stream):
    return pa.decode(*_args(s), stream=stream)


def _splitk(s, stream):
    return pa.decode_splitk(*_args(s), max_context_len=s["max"], stream=stream)


def _splitk_parts(s, stream):
    return pa.decode_splitk(*_args(s), max_context_len=s["max"], partition_tokens=64, stream=stream)


def _step(s, stream):
    kc, vc = s["kc"].clone(), s["vc"].clone()
    torch.cuda.current_stream().synchronize()
    out = pa.decode_step(s["q"], s["k"], s["v"], kc, vc, s["tables"], s["cl"], D ** -0.5, max_context_len=s["max"],
                         stream=stream)
    torch.cuda.synchronize()
    return out


def _multi(s, stream):
    return pa.decode_multi(*_args(s, "qt"), max_context_len=s["max"], stream=stream)


def _cascade(s, stream):
    return pa.decode_cascade(*_args(s), n_sharers=0, prefix_len=0, max_context_len=s["max"], stream=stream)


def _prefill(s, stream):
    return pa.prefill(s["q"], None, None, None, s["cu"], s["kc"], s["vc"], s["tables"], s["cl"], D ** -0.5, max_q_len=1,
                      stream=stream)


DRAFT = [_norm_rope, _append, _tree, _commit]


def _check(call, dtype):
    s = _inputs(dtype)
    want = call(s, None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, torch.cuda.ExternalStream(side.cuda_stream)):
        out = call(s, stream)
        side.synchronize()
        for got, w in zip(out if isinstance(out, tuple) else (out,), want if isinstance(want, tuple) else (want,)):
            assert _pool_of(got) == side.cuda_stream
            assert torch.equal(got, w)
    with torch.cuda.stream(side):  # the current stream: its own pool, as ever
        out = call(s, None)
        assert _pool_of(out[0] if isinstance(out, tuple) else out) == side.cuda_stream
    with torch.cuda.stream(side):  # and the default stream, by its handle, from another one
        out = call(s, 0)
    torch.cuda.synchronize()
    for got, w in zip(out if isinstance(out, tuple) else (out,), want if isinstance(want, tuple) else (want,)):
        assert _pool_of(got) == 0 and torch.equal(got, w)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("call", DRAFT)
def test_outputs_of_the_drafting_step(call, dtype):
    _check(call, dtype)


@pytest.mark.parametrize("dtype,call", [(torch.float32, c) for c in (_decode, _splitk, _splitk_parts)] +
                         [(torch.bfloat16, c) for c in (_decode, _splitk, _splitk_parts, _step, _multi, _cascade, _prefill)])
def test_outputs_of_the_other_calls(dtype, call):
    _check(call, dtype)


@pytest.mark.parametrize("call", [_splitk, _splitk_parts, _multi, _step])
def test_a_workspace_is_zero_where_the_call_runs(call):
    """With the current stream busy, and memory that is not zero in the launch stream's pool."""
    s = _inputs(torch.bfloat16)
    want = call(s, None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        held = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in (1 << 10, 1 << 16, 1 << 20, 8 << 20)]
    side.synchronize()
    del held
    if call is not _step:  # (which waits for the current stream before the call)
        torch.cuda._sleep(100_000_000)
    out = call(s, side)
    side.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("call", [_norm_rope, _tree, _splitk])
def test_an_output_is_not_given_away_while_the_current_stream_uses_it(call):
    """Dropped by the caller with its use queued on the current stream, its memory is not reused before that has run."""
    s = _inputs(torch.bfloat16)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = call(s, side)
    out = out[0] if isinstance(out, tuple) else out
    side.synchronize()
    at, want = out.data_ptr(), out.clone()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # the current stream is busy for a tenth of a second
    copy = out.clone()
    shape, dtype = out.shape, out.dtype
    del out
    with torch.cuda.stream(side):
        other = torch.empty(shape, dtype=dtype, device="cuda")
        assert other.data_ptr() != at
        other.zero_()
    torch.cuda.synchronize()
    assert torch.equal(copy, want)


@pytest.mark.parametrize("call", [_norm_rope, _tree, _commit, _splitk_parts, _multi])
def test_outputs_on_a_forked_stream_of_a_capture(call):
    """Captured on a stream that joins the current one; an output that is kept, and one that is dropped."""
    s = _inputs(torch.bfloat16)
    want = call(s, None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        current = torch.cuda.current_stream()
        side.wait_stream(current)
        call(s, side)
        out = call(s, side)
        current.wait_stream(side)
    for _ in range(2):
        for x in out if isinstance(out, tuple) else (out,):
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for got, w in zip(out if isinstance(out, tuple) else (out,), want if isinstance(want, tuple) else (want,)):
            assert torch.equal(got, w)
    del graph, out
