"""Host-side tests of the single-token operators' C ABI (no GPU): every refusal is returned before any CUDA call."""
import ctypes

import pytest
import torch

import chunked_gated_delta_10_gb300 as kda

A = 1 << 20  # a 16-byte aligned fake device address (never dereferenced: validation fails first)
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    kda.build()
    return kda.load()


def _step(lib, ptr=None, **dim):
    d = dict(N=2, T=1, H=2, HV=4, K=64, V=128, num_slots=2, dtype=0, scale=0.1)
    d.update(dim)
    p = dict(q=A, k=A, v=A, g=A, beta=A, state=A, slots=None, o=A, status=None, stream=None)
    p.update(ptr or {})
    return lib.kda_step(kda.StepDims(**d), *p.values())


@pytest.mark.parametrize("dim, code", [
    (dict(N=-1), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(HV=3), INVALID), (dict(dtype=2), INVALID),
    (dict(num_slots=1), INVALID), (dict(num_slots=-1), INVALID), (dict(K=96), UNSUPPORTED), (dict(V=256), UNSUPPORTED),
    (dict(N=2**30, num_slots=2**30), UNSUPPORTED)])
def test_step_refuses_sizes(lib, dim, code):
    assert _step(lib, **dim) == code


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta", "state", "o"])
def test_step_refuses_pointers(lib, name):
    assert _step(lib, {name: None}) == INVALID
    assert _step(lib, {name: A + 8}) == INVALID


def test_step_refuses_the_rest(lib):
    assert lib.kda_step(None, *([None] * 10)) == INVALID
    assert _step(lib, dict(slots=A + 2)) == INVALID
    assert _step(lib, dict(status=A + 2)) == INVALID
    assert _step(lib, dict(q=None, o=None), N=0) == 0   # nothing to do
    assert _step(lib, dict(q=None, o=None), T=0) == 0


def _cache(**kw):
    c = dict(k=A, v=A, k_page=8 * 64 * 128, k_row=128, k_head=64 * 128, v_page=8 * 64 * 64, v_row=64, v_head=64 * 64,
             num_pages=10, page_size=64, HKV=8, K=128, V=64, dtype=0)
    c.update(kw)
    return kda.Cache(**c)


BAD_CACHES = [(dict(num_pages=0), INVALID), (dict(page_size=0), INVALID), (dict(HKV=0), INVALID), (dict(dtype=3), INVALID),
              (dict(K=32), UNSUPPORTED), (dict(V=192), UNSUPPORTED), (dict(k_row=132), INVALID),
              (dict(v_page=-64), INVALID), (dict(k=A + 2), INVALID), (dict(v=None), INVALID)]


def _append(lib, cache=None, **kw):
    a = dict(k=A, k_stride=1024, v=A, v_stride=512, q=A, q_stride=2048, q_out=2 * A, HQ=16, N=2, R=4, cu=None, rope=A,
             rope_len=100, rope_dim=64, interleaved=0, table=A, table_stride=5, max_pages=5, lens=A, status=None,
             stream=None)
    a.update(kw)
    return lib.kda_cache_append(cache or _cache(), *a.values())


@pytest.mark.parametrize("bad, code", BAD_CACHES)
def test_append_and_attend_refuse_caches(lib, bad, code):
    assert _append(lib, _cache(**bad)) == code
    assert _attend(lib, _cache(**bad)) == code
    assert lib.kda_cache_attend_workspace_bytes(_cache(**bad), 16, 2, 5, 0) == 0


@pytest.mark.parametrize("bad", [
    dict(N=-1), dict(N=0), dict(R=-1), dict(R=5), dict(HQ=0), dict(HQ=-1), dict(q=None), dict(q_out=None),
    dict(q=None, q_out=None), dict(k=None), dict(v=None), dict(k=A + 8), dict(v=A + 8), dict(q=A + 8), dict(q_out=A + 8),
    dict(k_stride=1000), dict(k_stride=1028), dict(v_stride=504), dict(q_stride=2040), dict(q_stride=2052),
    dict(q_out=A, q_stride=4096), dict(rope=None), dict(rope_dim=0), dict(rope_dim=24), dict(rope_dim=144),
    dict(rope_len=-1), dict(rope=A + 4), dict(table=None), dict(table=A + 2), dict(table_stride=-1), dict(max_pages=-1),
    dict(lens=None), dict(lens=A + 1), dict(status=A + 2), dict(cu=A + 4)])
def test_append_refuses(lib, bad):
    assert _append(lib, **bad) == INVALID


def test_append_of_nothing(lib):
    assert lib.kda_cache_append(None, *([None, 0] * 3), None, 0, 0, 0, None, None, 0, 0, 0, None, 0, 0, None, None,
                                None) == INVALID
    assert _append(lib, R=0, k=None, v=None) == 0
    assert _append(lib, R=0, N=0, k=None, v=None) == 0
    assert _append(lib, R=2**31, N=2) == UNSUPPORTED


def _attend(lib, cache=None, **kw):
    a = dict(q=A, q_stride=2048, HQ=16, N=2, table=A, table_stride=5, max_pages=5, lens=A, window=0, scale=0.1, o=A,
             lse=A, status=None, ws=A, ws_bytes=1 << 30, stream=None)
    a.update(kw)
    return lib.kda_cache_attend(cache or _cache(), *a.values())


@pytest.mark.parametrize("bad, code", [
    (dict(N=-1), INVALID), (dict(HQ=0), INVALID), (dict(HQ=12), INVALID), (dict(max_pages=-1), INVALID),
    (dict(window=-1), INVALID), (dict(q=None), INVALID), (dict(q=A + 8), INVALID), (dict(q_stride=2040), INVALID),
    (dict(q_stride=2052), INVALID), (dict(o=None), INVALID), (dict(o=A + 4), INVALID), (dict(lse=A + 2), INVALID),
    (dict(table=None), INVALID), (dict(table=A + 2), INVALID), (dict(table_stride=-5), INVALID), (dict(lens=None), INVALID),
    (dict(lens=A + 2), INVALID), (dict(status=A + 1), INVALID), (dict(ws=None), WORKSPACE), (dict(ws=A + 8), WORKSPACE),
    (dict(ws_bytes=8), WORKSPACE), (dict(max_pages=2**26), UNSUPPORTED), (dict(N=2**28), UNSUPPORTED)])
def test_attend_refuses(lib, bad, code):
    assert _attend(lib, **bad) == code


def test_attend_of_nothing(lib):
    assert _attend(lib, N=0, q=None, o=None) == 0
    assert lib.kda_cache_attend_workspace_bytes(_cache(), 16, 2, 5, 0) > 0
    assert lib.kda_cache_attend_workspace_bytes(_cache(), 16, 0, 5, 0) > 0
    assert lib.kda_cache_attend_workspace_bytes(None, 16, 2, 5, 0) == 0


def test_binding_refuses_what_is_not_on_the_gpu():
    x = torch.zeros(2, 1, 2, 64)
    with pytest.raises(ValueError):
        kda.step(x, x, x, x, x[..., 0], torch.zeros(2, 2, 64, 64))
    with pytest.raises(ValueError):
        kda.cache_attend(x[:, 0], x, x, torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))


def test_structures_match_the_header():
    """The sizes that a C compiler gives the two structures."""
    assert ctypes.sizeof(kda.StepDims) == 9 * 4
    assert ctypes.sizeof(kda.Cache) == 8 * 8 + 6 * 4


def _sinks(lib, cache=None, **kw):
    a = dict(q=A, q_stride=2048, HQ=16, N=2, table=A, table_stride=5, max_pages=5, lens=A, window=8, sinks=2, scale=0.1, o=A,
             lse=A, status=None, ws=A, ws_bytes=1 << 30, stream=None)
    a.update(kw)
    return lib.kda_cache_attend_sinks(cache or _cache(), *a.values())


@pytest.mark.parametrize("bad, code", [(dict(sinks=-1), INVALID), (dict(window=-1), INVALID), (dict(q=None), INVALID),
                                       (dict(ws_bytes=8), WORKSPACE), (dict(N=2**28), UNSUPPORTED)])
def test_attend_sinks_refuses(lib, bad, code):
    assert _sinks(lib, **bad) == code
    assert _sinks(lib, N=0, q=None, o=None) == 0
    assert lib.kda_cache_attend_sinks_workspace_bytes(_cache(), 16, 2, 5, 8, -1) == 0


def _cache8(cache=None, **kw):
    c = dict(cache=_cache(**{**dict(dtype=2, k_page=8 * 64 * 128, v_page=8 * 64 * 64), **(cache or {})}), k_scale=A, v_scale=A,
             k_scale_page=32, k_scale_block=1, k_scale_head=4, v_scale_page=32, v_scale_block=1, v_scale_head=4, block=16,
             dtype=0)
    c.update(kw)
    return kda.Cache8(**c)


BAD_CACHES8 = [(dict(cache=b), code) for b, code in BAD_CACHES if b != dict(k_row=132)] + [
    (dict(cache=dict(dtype=0)), INVALID), (dict(cache=dict(k_row=136)), INVALID), (dict(block=0), INVALID), (dict(block=-16), INVALID),
    (dict(block=24), INVALID), (dict(block=128), INVALID), (dict(k_scale=None), INVALID), (dict(v_scale=A + 2), INVALID),
    (dict(k_scale_page=-1), INVALID), (dict(v_scale_block=-1), INVALID), (dict(v_scale_head=-4), INVALID), (dict(dtype=2), INVALID),
    (dict(dtype=-1), INVALID)]


def _append8(lib, cache=None, **kw):
    a = dict(k=A, k_stride=1024, v=A, v_stride=512, q=A, q_stride=2048, q_out=2 * A, HQ=16, N=2, R=4, cu=None, rope=A,
             rope_len=100, rope_dim=64, interleaved=0, table=A, table_stride=5, max_pages=5, lens=A, status=None,
             stream=None)
    a.update(kw)
    return lib.kda_cache8_append(cache or _cache8(), *a.values())


def _attend8(lib, cache=None, **kw):
    a = dict(q=A, q_stride=2048, HQ=16, N=2, table=A, table_stride=5, max_pages=5, lens=A, window=0, sinks=0, scale=0.1, o=A,
             lse=A, status=None, ws=A, ws_bytes=1 << 30, stream=None)
    a.update(kw)
    return lib.kda_cache8_attend(cache or _cache8(), *a.values())


@pytest.mark.parametrize("bad, code", BAD_CACHES8)
def test_cache8_refused(lib, bad, code):
    assert _append8(lib, _cache8(**bad)) == code
    assert _attend8(lib, _cache8(**bad)) == code
    assert lib.kda_cache8_attend_workspace_bytes(_cache8(**bad), 16, 2, 5, 0, 0) == 0


@pytest.mark.parametrize("bad", [
    dict(N=-1), dict(N=0), dict(R=-1), dict(R=5), dict(HQ=0), dict(q=None), dict(q_out=None), dict(k=None), dict(v=A + 8),
    dict(k_stride=1000), dict(k_stride=1028), dict(q_out=A, q_stride=4096), dict(rope=None), dict(rope_dim=24),
    dict(rope_dim=144), dict(table=None), dict(lens=None), dict(status=A + 2), dict(cu=A + 4)])
def test_append8_refuses(lib, bad):
    assert _append8(lib, **bad) == INVALID


def test_append8_refuses_shared_scales(lib):
    for name in ("k_scale_page", "v_scale_block", "v_scale_head"):
        assert _append8(lib, _cache8(**{name: 0})) == INVALID


def test_cache8_of_nothing(lib):
    assert _append8(lib, R=0, k=None, v=None) == 0
    assert _append8(lib, R=2**31, N=2) == UNSUPPORTED
    assert _append8(lib, R=2**31 - 2, N=2**30, cu=A, HQ=0, q=None, q_out=None) == UNSUPPORTED  # too many CTAs
    assert lib.kda_cache8_append(None, *([None, 0] * 3), None, 0, 0, 0, None, None, 0, 0, 0, None, 0, 0, None, None,
                                 None) == INVALID
    assert _attend8(lib, N=0, q=None, o=None) == 0
    assert lib.kda_cache8_attend_workspace_bytes(_cache8(), 16, 2, 5, 0, 0) > 0


@pytest.mark.parametrize("bad, code", [
    (dict(N=-1), INVALID), (dict(HQ=12), INVALID), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(q=None), INVALID),
    (dict(q_stride=2052), INVALID), (dict(o=A + 4), INVALID), (dict(ws=None), WORKSPACE), (dict(ws_bytes=8), WORKSPACE),
    (dict(max_pages=2**26), UNSUPPORTED), (dict(N=2**28), UNSUPPORTED)])
def test_attend8_refuses(lib, bad, code):
    assert _attend8(lib, **bad) == code


def test_the_structure_of_a_cache_in_8_bits():
    assert ctypes.sizeof(kda.Cache8) == 8 * 8 + 6 * 4 + 8 * 8 + 2 * 4


def _resize(lib, **kw):
    a = dict(table=A, table_stride=8, max_pages=8, N=2, page_size=16, lens=A, wanted=A, free=A, num_pages=16, count=A, cu=A,
             slots=A, rows=9000, granted=A, status=A, ws=A, ws_bytes=1 << 20, stream=None)
    a.update(kw)
    return lib.kda_cache_resize(*a.values())


@pytest.mark.parametrize("bad, code", [
    (dict(max_pages=-1), INVALID), (dict(N=-1), INVALID), (dict(page_size=0), INVALID), (dict(num_pages=-1), INVALID),
    (dict(rows=-1), INVALID), (dict(table_stride=-8), INVALID), (dict(table_stride=7), INVALID), (dict(lens=None), INVALID),
    (dict(wanted=None), INVALID), (dict(table=None), INVALID), (dict(free=None), INVALID), (dict(count=None), INVALID),
    (dict(table=A + 2), INVALID), (dict(lens=A + 1), INVALID), (dict(wanted=A + 2), INVALID), (dict(free=A + 2), INVALID),
    (dict(count=A + 2), INVALID), (dict(cu=A + 4), INVALID), (dict(slots=A + 4), INVALID), (dict(granted=A + 2), INVALID),
    (dict(status=A + 1), INVALID), (dict(ws=None), WORKSPACE), (dict(ws=A + 8), WORKSPACE), (dict(ws_bytes=16), WORKSPACE),
    (dict(N=65536), UNSUPPORTED), (dict(rows=2**31), UNSUPPORTED),
    (dict(max_pages=2**30, table_stride=2**30), UNSUPPORTED)])
def test_resize_refuses(lib, bad, code):
    assert _resize(lib, **bad) == code


def test_resize_workspace(lib):
    need = lib.kda_cache_resize_workspace_bytes
    assert need(1, 1, 1) == 0 and need(0, 0, 0) == 0 and need(-1, 1, 1) == 0  # one CTA, no workspace
    assert need(2, 8, 9000) == 3 * 8 + 4 * 4 and need(2000, 1, 0) > 0


def test_granted_lengths_refused(lib):
    """The appends with granted lengths make the checks of those without, and of the lengths' alignment."""
    a16 = [A, 1024, A, 512, A, 2048, 2 * A, 16, 2, 4, None, A, 100, 64, 0, A, 5, 5, A]
    for call, cache in ((lib.kda_cache_append_granted, _cache()), (lib.kda_cache8_append_granted, _cache8())):
        assert call(cache, *a16, A + 2, None, None) == INVALID
        assert call(cache, *a16, A, A + 2, None) == INVALID
        assert call(None, *a16, A, None, None) == INVALID
        assert call(cache, None, 1024, None, 512, None, 2048, None, 16, 2, 0, *a16[10:], None, None, None) == 0  # no rows


def test_resize_of_many_sequences_or_pages_is_no_work_of_one_cta(lib):
    need = lib.kda_cache_resize_workspace_bytes
    assert need(256, 512, 4096) == 0 and need(1, 1 << 17, 0) == 0
    for N, pages, rows in ((257, 1, 0), (1000, 16, 0), (1024, 128, 4096), (256, 513, 0), (16, 8193, 0), (1, 1, 4097)):
        assert need(N, pages, rows) == 8 * (N + 1) + 4 * (N + 2)
