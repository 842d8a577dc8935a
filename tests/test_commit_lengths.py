"""Commit of a tree's path: the new lengths lie in memory of their own.  (One CTA
writes a sequence's while others still read its lengths, path and table.)"""

import pytest

import paged_kv_cache_473_b200 as pa
from paged_kv_cache_473_b200 import _binding as bnd

B, A, MB = 8, 5, 4
AT = dict(k=0x1000000, v=0x2000000, bt=0x10000, cl=0x20000, tl=0x30000, acc=0x40000, al=0x50000)
SIZE = dict(bt=4 * B * MB, cl=4 * B, tl=4 * B, acc=4 * B * A, al=4 * B)


@pytest.mark.parametrize("what", ["bt", "cl", "tl", "acc", "al"])
@pytest.mark.parametrize("where", ["start", "before", "inside"])
def test_new_lengths_over_an_input_are_refused(what, where):
    at = {"start": AT[what], "before": AT[what] - 4 * B + 4, "inside": AT[what] + SIZE[what] - 4}[where]
    st = bnd.lib.pa_commit_tree(AT["k"], AT["v"], 1, AT["bt"], AT["cl"], AT["tl"], 16, AT["acc"], A, AT["al"], B, 2, 128,
                                16, MB, 8, at, bnd.PA_BF16, None)
    assert st == bnd.PA_ERR_INVALID
    assert pa.last_launch_count() == 0
