"""Rotation in place: the same rows, or none at all.  (An output that starts where
its input does, with rows another distance apart, would be written over rows of
other tokens that are still to be read.)"""

import pytest

import paged_kv_cache_473_b200 as pa
from paged_kv_cache_473_b200 import _binding as bnd

Q, K, V, IO, KC, VC = 0x100000, 0x200000, 0x300000, 0x400000, 0x500000, 0x600000
HQ, HKV, D = 8, 2, 128


def _rope(n=4, qs=HQ * D, ks=HKV * D, qo=Q, qos=HQ * D, ko=K, kos=HKV * D):
    return bnd.lib.pa_qk_norm_rope(Q, qs, K, ks, None, None, 1e-6, IO, D, 0, IO, n, HQ, HKV, D, qo, qos, ko, kos,
                                   bnd.PA_BF16, None)


@pytest.mark.parametrize("kw", [dict(qs=HQ * D + 8), dict(qs=0), dict(qos=12 * D), dict(qs=12 * D), dict(ks=12 * D),
                                dict(kos=12 * D), dict(ks=0), dict(n=2, qs=12 * D, qos=14 * D)])
def test_the_same_start_with_another_stride_is_refused(kw):
    assert _rope(**kw) == bnd.PA_ERR_INVALID
    assert pa.last_launch_count() == 0


def test_append_from_a_fused_projection_onto_itself_is_refused():
    def call(n, qs):
        return bnd.lib.pa_rope_append(Q, qs, K, 12 * D, V, 12 * D, None, None, 1e-6, IO, D, 0, IO, IO, n, HQ, HKV, D, Q,
                                      KC, VC, 8, 16, bnd.PA_BF16, None)

    assert call(2, 12 * D) == bnd.PA_ERR_INVALID
    assert pa.last_launch_count() == 0
