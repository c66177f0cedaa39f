"""How the attention of one token gives a cache's rows to CTAs (host side, no GPU)."""
import ctypes

import pytest

import chunked_gated_delta_10_gb300 as kda
from tests.test_serve_abi import _cache, lib  # noqa: F401

WHOLE, CLUSTER, PARTS, SHARES = range(4)
ROOM = {2: 1.0, 4: 0.96, 8: 0.89, 16: 0.74}  # of the places of all SMs, what clusters of this size were measured to find


def cache(HKV, K, V, page, dtype):
    return _cache(HKV=HKV, K=K, V=V, page_size=page, dtype=dtype, k_page=HKV * page * K, k_head=page * K, k_row=K,
                  v_page=HKV * page * V, v_head=page * V, v_row=V)


def plan(lib, HQ, HKV, K, V, dtype, N, rows, window=0, page=1):  # noqa: F811
    out = (ctypes.c_int32 * 4)()
    c = cache(HKV, K, V, page, dtype)
    assert lib.kda_debug_attend_plan(ctypes.byref(c), HQ, N, -(-rows // page), window, out) == 0
    return tuple(out)


def places(group, K, V, dtype):
    """CTAs of the attention kernels that 152 SMs hold."""
    if dtype == kda.DTYPE_BF16:
        return 152 * ((5 if K + V == 128 else 3) - (group > 8))
    ht = 1 if group == 1 else 4 if group <= 4 else 8
    return 152 * ((4 if ht == 1 else 3) + ((K + V < 256) if ht == 4 else (V == 64)))


def test_no_cluster_waits_for_another(lib):  # noqa: F811
    """All clusters of a launch fit at once, whatever the number of units."""
    seen = set()
    for dtype in (kda.DTYPE_BF16, kda.DTYPE_F32):
        for K, V in ((64, 64), (64, 128), (128, 64), (128, 128)):
            for group in (1, 4, 8, 16):
                for units in list(range(1, 60, 7)) + list(range(60, 420, 1 if group in (1, 8) else 9)):
                    for rows in (130, 260, 700, 1024, 3000):
                        split, parts, _, of = plan(lib, group, 1, K, V, dtype, units, rows)
                        if split == CLUSTER:
                            seen.add(parts)
                            assert of * parts <= places(group, K, V, dtype) * ROOM[parts], (dtype, K, V, group, units, rows)
    assert seen == set(ROOM)


@pytest.mark.parametrize("N, HQ", [(12, 16), (191, 1), (193, 1)])
def test_units_just_above_the_room_take_no_clusters_of_four(lib, N, HQ):  # noqa: F811
    """About 192 units of the fp32 kernel for heads of 64 are as many clusters of four as there are places, not room."""
    assert plan(lib, HQ, HQ, 64, 64, kda.DTYPE_F32, N, 1500, window=1024, page=20)[:2] != (CLUSTER, 4)


def test_plan_of_refused_sizes(lib):  # noqa: F811
    out = (ctypes.c_int32 * 4)()
    c = cache(2, 64, 64, 16, 0)
    assert lib.kda_debug_attend_plan(ctypes.byref(c), 3, 1, 4, 0, out) == 1
    assert lib.kda_debug_attend_plan(ctypes.byref(c), 4, 1, 4, 0, None) == 1
    assert lib.kda_debug_attend_plan(None, 4, 1, 4, 0, out) == 1
    assert lib.kda_debug_attend_plan(ctypes.byref(c), 4, 0, 4, 0, out) == 0
