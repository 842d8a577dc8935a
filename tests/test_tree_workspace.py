"""Tree attention's workspace: one sized for the largest tree serves the smaller ones."""

import pytest
import torch

import paged_kv_cache_473_b200 as pa
from tests import draft_reference as ref


def _size(nodes, group, d):
    return pa.decode_tree_workspace_size(3, nodes, 2 * group, d, 500, 2)


def test_size_never_falls_as_a_shape_grows():
    dims = (64, 128, 256)
    for d in dims:
        for group in range(1, 9):
            for nodes in range(1, 65):
                here = _size(nodes, group, d)
                assert here > 256 * 1024
                assert nodes == 1 or _size(nodes - 1, group, d) <= here, (nodes, group, d)
                assert group == 1 or _size(nodes, group - 1, d) <= here, (nodes, group, d)
                assert d == 64 or _size(nodes, group, d // 2) <= here, (nodes, group, d)


@pytest.mark.gpu
def test_one_workspace_for_all_smaller_trees():
    """Sizes around those whose plans have the most records: one, two and three row tiles."""
    pa.device_errors()
    g = torch.Generator().manual_seed(11)
    ws = {d: torch.empty(pa.decode_tree_workspace_size(3, 48, 16, d, 500, 2), dtype=torch.uint8, device="cuda")
          for d in (64, 128, 256)}
    for d in (64, 128, 256):
        for group, nodes in ((8, 48), (8, 32), (8, 17), (8, 16), (8, 1), (7, 36), (7, 19), (5, 48), (5, 26), (1, 48)):
            lens = [nodes + 3, 300, 500]
            kc, vc, tables, cl = ref.pool(g, lens, 2, d, 16, torch.bfloat16)
            q = torch.randn((3, nodes, 2 * group, d), generator=g).to(torch.bfloat16)
            mask, _ = ref.random_trees(g, 3, nodes)
            args = (q.cuda(), kc, vc, tables, cl, mask.cuda(), d ** -0.5)
            own = pa.decode_tree(*args, max_context_len=500)
            for held in dict.fromkeys((d, 256)):
                out = pa.decode_tree(*args, max_context_len=500, workspace=ws[held])
                assert torch.equal(out, own), (d, group, nodes)
    assert pa.device_errors() == 0
