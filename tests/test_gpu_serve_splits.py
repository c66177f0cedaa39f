"""Attention of one token per sequence with each way of giving a cache's rows to CTAs: a CTA or a cluster per unit, parts,
and equal shares, chosen by the sizes; ragged and empty sequences among them. Reference and bounds are those of
test_gpu_serve.py."""
import math

import pytest
import torch

from tests.test_gpu_serve import DT, _gen, attend_ref, check_attend, kda, make_cache, make_table, run_attend  # noqa: F401

pytestmark = pytest.mark.gpu


def lengths(gen, kind, N, longest):
    some = torch.randint(0, longest + 1, (N,), generator=gen).tolist()
    if kind == "ragged":
        return some
    if kind == "equal":
        return [longest] * N
    if kind == "one long":
        return [longest if n == N // 2 else n % 3 for n in range(N)]
    if kind == "short":  # fewer turns in all than CTAs
        return [x % 70 for x in some]
    if kind == "mostly short":
        return [longest if n % 20 == 7 else some[n] % 70 for n in range(N)]
    if kind == "empty":
        return [0] * N
    return [some[n] if n % 4 else 0 for n in range(N)]  # "gaps"


CASES = [
    # split, N, longest, lengths, HQ, HKV, K, V, page, window
    ("cache_attend", 5, 60, "ragged", 8, 2, 128, 128, 16, 0),
    ("cache_attend", 300, 30, "gaps", 4, 4, 64, 64, 7, 0),
    ("cache_attend_cluster", 3, 1000, "ragged", 16, 4, 64, 128, 32, 0),
    ("cache_attend_cluster", 2, 900, "empty", 8, 8, 64, 64, 16, 0),
    ("cache_attend_cluster", 4, 1500, "one long", 6, 3, 128, 64, 20, 700),
    ("cache_attend_parts", 1, 9000, "equal", 8, 2, 128, 128, 16, 0),
    ("cache_attend_parts", 1, 12000, "empty", 4, 1, 64, 64, 64, 0),
    ("cache_attend_parts", 2, 7000, "gaps", 5, 1, 128, 128, 27, 0),
    ("cache_attend_parts", 1, 9000, "ragged", 32, 2, 64, 64, 100, 8000),
    ("cache_attend_parts", 3, 6000, "one long", 16, 1, 128, 128, 64, 0),
    ("cache_attend_shares", 40, 3000, "ragged", 8, 8, 64, 64, 64, 0),
    ("cache_attend_shares", 40, 2500, "gaps", 32, 8, 64, 128, 16, 0),
    ("cache_attend_shares", 300, 2000, "one long", 6, 2, 64, 64, 128, 0),
    ("cache_attend_shares", 300, 2000, "empty", 4, 4, 128, 64, 50, 0),
    ("cache_attend_shares", 130, 1500, "gaps", 16, 4, 128, 128, 13, 1400),
    ("cache_attend_shares", 64, 3000, "equal", 16, 4, 64, 64, 64, 0),
    ("cache_attend_shares", 90, 2500, "ragged", 32, 2, 128, 128, 32, 0),
    ("cache_attend_shares", 200, 3000, "mostly short", 16, 4, 128, 128, 64, 0),
    ("cache_attend_shares", 160, 4000, "mostly short", 40, 4, 64, 64, 20, 0),
    ("cache_attend_shares", 20, 16000, "short", 8, 2, 128, 128, 64, 0),
    ("cache_attend_shares", 30, 20032, "short", 16, 1, 64, 64, 32, 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_splits(kda, case, dtype):  # noqa: F811
    split, N, longest, kind, HQ, HKV, K, V, size, window = CASES[case]
    gen = _gen(100 + case)
    lens = lengths(gen, kind, N, longest)
    pages = sum(-(-x // size) for x in lens) + 2
    kc, vc = make_cache(gen, pages, size, HKV, K, V, dtype, "heads first")
    width = -(-longest // size)
    table = make_table(gen, lens, size, pages, spare=width)[:, :width]
    own = torch.zeros(pages, size, dtype=torch.bool)
    for n, m in enumerate(lens):
        pos = torch.arange(max(0, m - window) if window else 0, m)
        own[table[n, pos // size].long(), pos % size] = True
    kc[~own], vc[~own] = math.nan, math.nan
    q = (2 * torch.randn(N, HQ, K, generator=gen)).to(DT[dtype])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_attend(kda, q, kc, vc, table, lens, window=window, status=status)
    if dtype == "bf16":  # (fp32 takes other tiles, and may split otherwise)
        assert kda.load().kda_launch_name(0).decode() == split
    assert int(status) == 0
    again = run_attend(kda, q, kc, vc, table, lens, window=window)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    few = torch.randperm(N, generator=gen)[:24].tolist() + [N // 2]  # the reference's sequences
    pick = lambda t: t[few]  # noqa: E731
    ref = attend_ref(pick(q), kc, vc, pick(table), [lens[n] for n in few], K ** -0.5, window, size)
    check_attend(dtype, (got[0][few], got[1][few]), ref)
    rest = torch.tensor(lens) <= 0
    assert not got[0].cpu()[rest].any() and (got[1].cpu()[rest] == -math.inf).all()


@pytest.mark.parametrize("split, N, room", [("cache_attend", 300, 32), ("cache_attend_cluster", 2, 512),
                                            ("cache_attend_parts", 1, 8192), ("cache_attend_shares", 64, 4096)])
def test_lengths_beyond_the_table(kda, split, N, room):  # noqa: F811
    """A length that the table has no pages for is cut there and flagged, with a window too, whatever the split."""
    gen = _gen(5)
    size = 64 if room >= 64 else 1
    kc, vc = make_cache(gen, room // size, size, 4, 64, 64, "bf16", "heads first")
    table = torch.arange(room // size, dtype=torch.int32).expand(N, -1)
    q = torch.randn(N, 4, 64, generator=gen).bfloat16()
    for window in (0, 40):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        lens = [2 ** 31 - 1] + [room + 3] * (N - 1)
        got = run_attend(kda, q, kc, vc, table, lens, window=window, status=status)
        if not window:
            assert kda.load().kda_launch_name(0).decode() == split
        assert int(status) == 1
        ref = attend_ref(q[:2], kc, vc, table[:2], lens[:2], 0.125, window, size)
        check_attend("bf16", (got[0][:2], got[1][:2]), ref)
