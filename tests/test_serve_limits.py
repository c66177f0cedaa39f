"""Sizes that the single-token operators refuse because their kernels count in 32 bits (no GPU)."""
import pytest

from tests.test_serve_abi import A, UNSUPPORTED, _append, _cache, lib  # noqa: F401


@pytest.mark.parametrize("HQ, HKV", [(2 ** 26 - 17, 8), (2 ** 26 - 32 - 16, 8), (1, 2 ** 25 - 16), (2 ** 30, 1)])
def test_append_refuses_rows_of_too_many_heads(lib, HQ, HKV):  # noqa: F811
    cache = _cache(HKV=HKV, k_page=HKV * 64 * 128, v_page=HKV * 64 * 64)
    assert _append(lib, cache, HQ=HQ, q_stride=HQ * 128, k_stride=HKV * 128, v_stride=HKV * 64) == UNSUPPORTED
