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


def plan(lib, HQ, HKV, K, V, dtype, N, rows, window=0, page=1, sms=152, cluster=16):  # noqa: F811
    out = (ctypes.c_int32 * 4)()
    c = cache(HKV, K, V, page, dtype)
    assert lib.kda_debug_attend_plan(ctypes.byref(c), HQ, N, -(-rows // page), window, sms, cluster, out) == 0
    return tuple(out)


def places(group, K, V, dtype, sms=152):
    """CTAs of the attention kernels that the SMs hold."""
    if dtype == kda.DTYPE_BF16:
        return sms * (4 if K + V == 128 else 2 if group > 8 else 3)
    ht = 1 if group == 1 else 4 if group <= 4 else 8
    return sms * ((4 if ht == 1 else 3) + ((K + V < 256) if ht == 4 else (V == 64)))


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
    assert lib.kda_debug_attend_plan(ctypes.byref(c), 3, 1, 4, 0, 152, 16, out) == 1
    assert lib.kda_debug_attend_plan(ctypes.byref(c), 4, 1, 4, 0, 152, 16, None) == 1
    assert lib.kda_debug_attend_plan(None, 4, 1, 4, 0, 152, 16, out) == 1
    assert lib.kda_debug_attend_plan(ctypes.byref(c), 4, 0, 4, 0, 152, 16, out) == 0


def test_part_of_a_gpu(lib):  # noqa: F811
    """A device with fewer SMs, or one that cannot place the largest clusters, gets plans that it can run at once."""
    sizes = [(8, 1, 1, 2048, 0), (8, 1, 1, 65536, 0), (8, 8, 1, 2048, 0), (16, 4, 6, 900, 0), (4, 1, 64, 3000, 1), (8, 1, 64, 8192, 0)]
    for sms in (152, 76, 36, 18, 8):
        for cluster in (16, 8, 4, 1):
            for HQ, HKV, N, rows, dtype in sizes:
                split, parts, _, units = plan(lib, HQ, HKV, 128, 128, dtype, N, rows, sms=sms, cluster=cluster)
                fit = places(HQ // HKV, 128, 128, dtype, sms)
                if split == CLUSTER:
                    assert parts <= cluster and units * parts <= fit * ROOM[parts]
                if split == SHARES:
                    assert parts == fit
                if split == PARTS and N == 1:
                    assert units * parts <= fit
    one = [plan(lib, 8, 8, 128, 128, 0, 1, 2048, cluster=c)[:2] for c in (16, 8, 1)]
    assert one[0] == (CLUSTER, 16) and one[1] == (CLUSTER, 8) and one[2][0] != CLUSTER


def test_plan_without_a_device_is_a_gb300s(lib):  # noqa: F811
    import torch
    if torch.cuda.is_available():
        pytest.skip("the present device's plan")
    for N, rows in ((1, 2048), (1, 65536), (64, 8192), (300, 40)):
        assert plan(lib, 32, 8, 128, 128, 0, N, rows, sms=0) == plan(lib, 32, 8, 128, 128, 0, N, rows)


def places8(group, K, V, sms=152):
    """CTAs of the attention kernel over a cache in 8 bits that the SMs hold."""
    return sms * ((5 if K + V == 128 else 4) - (2 if group > 8 else 1))


def test_no_cluster_waits_for_another_in_8_bits(lib):  # noqa: F811
    seen = set()
    for K, V in ((64, 64), (64, 128), (128, 64), (128, 128)):
        for group in (1, 8, 16):
            for units in list(range(1, 60, 7)) + list(range(60, 420, 5)):
                for rows in (130, 260, 700, 1024, 3000):
                    split, parts, _, of = plan(lib, group, 1, K, V, kda.DTYPE_E4M3, units, rows)
                    if split == CLUSTER:
                        seen.add(parts)
                        assert of * parts <= places8(group, K, V) * ROOM[parts], (K, V, group, units, rows)
    assert {4, 8} <= seen <= set(ROOM)


@pytest.mark.parametrize("heads", [1, 2, 3, 5, 7, 8, 12, 31, 48, 50, 97, 152])
def test_shares_of_heads_together(lib, heads):  # noqa: F811
    """As many CTAs as there are places, or nearly, in whole bundles of heads that make up a sequence's."""
    split, ctas, _, _ = plan(lib, heads, heads, 128, 128, kda.DTYPE_E4M3, 64, 8192)
    assert split == SHARES
    assert 0.97 * places8(1, 128, 128) <= ctas <= places8(1, 128, 128)
    assert any(heads % t == 0 and ctas % t == 0 for t in range(min(heads, 2), heads + 1)) or ctas == places8(1, 128, 128)
