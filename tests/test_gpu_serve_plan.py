"""The plan of the attention of one token on the present device, and the forms of its splits that ordinary sizes take."""
import ctypes

import pytest
import torch

from tests.test_gpu_serve import DT, _gen, attend_ref, check_attend, kda, make_cache, make_table, run_attend  # noqa: F401
from tests.test_serve_plan import CLUSTER, PARTS, SHARES, WHOLE, plan

pytestmark = pytest.mark.gpu


def test_the_device_is_asked(kda):  # noqa: F811
    """Without a given device the plan is for the present one's SMs; a whole GB300 places clusters of 16."""
    lib, sms = kda.load(), torch.cuda.get_device_properties(0).multi_processor_count
    lib.kda_debug_attend_plan.restype = ctypes.c_int
    for dtype in (0, 1):
        for K in (64, 128):
            for HQ, HKV in ((4, 4), (16, 4), (16, 2), (20, 2)):
                for N, rows in ((1, 900), (1, 2048), (2, 9000), (1, 65536), (64, 8192), (300, 40)):
                    assert plan(lib, HQ, HKV, K, K, dtype, N, rows, sms=0) == plan(lib, HQ, HKV, K, K, dtype, N, rows, sms=sms)


# Every way in which the plan gives rows to CTAs: a cluster of each size, parts and shares with each number of groups that
# join them, for each number of heads that a CTA takes.
FORMS = [
    # dtype, split, CTAs of the cluster or groups of the join, N, longest, HQ, HKV, K, V
    ("bf16", WHOLE, 0, 48, 130, 1, 1, 64, 64),
    ("bf16", WHOLE, 0, 24, 130, 20, 1, 64, 64),
    ("bf16", CLUSTER, 2, 33, 511, 16, 8, 64, 64),
    ("bf16", CLUSTER, 2, 48, 260, 20, 1, 64, 64),
    ("bf16", CLUSTER, 4, 1, 130, 1, 1, 64, 64),
    ("bf16", CLUSTER, 4, 1, 130, 20, 1, 64, 64),
    ("bf16", CLUSTER, 8, 1, 260, 1, 1, 64, 64),
    ("bf16", CLUSTER, 8, 1, 260, 20, 1, 64, 64),
    ("bf16", CLUSTER, 16, 1, 700, 1, 1, 64, 64),
    ("bf16", CLUSTER, 16, 1, 700, 20, 1, 64, 64),
    ("bf16", PARTS, 1, 64, 2500, 1, 1, 64, 128),
    ("bf16", PARTS, 1, 48, 1500, 20, 1, 64, 128),
    ("bf16", PARTS, 4, 24, 4502, 1, 1, 64, 128),
    ("bf16", PARTS, 4, 2, 4502, 32, 16, 128, 64),
    ("bf16", PARTS, 4, 5, 4502, 20, 1, 64, 128),
    ("bf16", PARTS, 32, 1, 2500, 1, 1, 64, 64),
    ("bf16", PARTS, 32, 1, 2500, 20, 1, 64, 64),
    ("bf16", SHARES, 1, 64, 1500, 2, 2, 64, 128),
    ("bf16", SHARES, 1, 24, 4502, 20, 1, 64, 128),
    ("bf16", SHARES, 4, 24, 9000, 1, 1, 64, 128),
    ("bf16", SHARES, 4, 5, 12000, 20, 1, 64, 128),
    ("bf16", SHARES, 32, 9, 40000, 1, 1, 64, 64),
    ("bf16", SHARES, 32, 3, 20000, 20, 1, 64, 128),
    ("f32", WHOLE, 0, 64, 130, 2, 2, 64, 64),
    ("f32", WHOLE, 0, 64, 130, 4, 2, 64, 64),
    ("f32", WHOLE, 0, 64, 130, 32, 2, 64, 128),
    ("f32", CLUSTER, 2, 5, 130, 16, 16, 64, 64),
    ("f32", CLUSTER, 2, 5, 130, 32, 16, 64, 64),
    ("f32", CLUSTER, 2, 64, 130, 20, 1, 64, 64),
    ("f32", CLUSTER, 4, 5, 130, 4, 4, 64, 64),
    ("f32", CLUSTER, 4, 5, 130, 16, 4, 64, 64),
    ("f32", CLUSTER, 4, 8, 130, 20, 1, 64, 64),
    ("f32", CLUSTER, 8, 1, 130, 1, 1, 64, 64),
    ("f32", CLUSTER, 8, 1, 130, 4, 2, 64, 64),
    ("f32", CLUSTER, 8, 2, 130, 20, 1, 64, 64),
    ("f32", CLUSTER, 16, 1, 260, 1, 1, 64, 64),
    ("f32", CLUSTER, 16, 1, 260, 4, 2, 64, 64),
    ("f32", CLUSTER, 16, 1, 130, 20, 1, 64, 64),
    ("f32", PARTS, 1, 48, 1500, 2, 2, 64, 64),
    ("f32", PARTS, 1, 9, 1500, 16, 8, 64, 64),
    ("f32", PARTS, 1, 24, 700, 20, 1, 64, 64),
    ("f32", PARTS, 4, 9, 2500, 4, 4, 64, 64),
    ("f32", PARTS, 4, 16, 2500, 4, 2, 64, 64),
    ("f32", PARTS, 4, 5, 1500, 20, 1, 64, 64),
    ("f32", PARTS, 32, 1, 1500, 1, 1, 64, 64),
    ("f32", PARTS, 32, 1, 1500, 4, 2, 64, 64),
    ("f32", PARTS, 32, 1, 700, 20, 1, 64, 64),
]


@pytest.mark.parametrize("case", range(len(FORMS)))
def test_every_form(kda, case):  # noqa: F811
    dtype, split, width, N, longest, HQ, HKV, K, V = FORMS[case]
    gen, size = _gen(200 + case), 1
    took = plan(kda.load(), HQ, HKV, K, V, 0 if dtype == "bf16" else 1, N, longest, sms=0)
    if torch.cuda.get_device_properties(0).multi_processor_count == 152:
        assert took[0] == split and (took[1] if split == CLUSTER else took[2]) == width
    lens = torch.randint(0, longest + 1, (N,), generator=gen).tolist()
    lens[N // 2] = longest
    pages = sum(lens) + 1
    kc, vc = make_cache(gen, pages, size, HKV, K, V, dtype, "heads first")
    table = make_table(gen, lens, size, pages, spare=longest)[:, :longest]
    q = (2 * torch.randn(N, HQ, K, generator=gen)).to(DT[dtype])
    got = run_attend(kda, q, kc, vc, table, lens)
    again = run_attend(kda, q, kc, vc, table, lens)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    few = torch.randperm(N, generator=gen)[:3].tolist() + [N // 2]  # the reference's sequences
    ref = attend_ref(q[few], kc, vc, table[few], [lens[n] for n in few], K ** -0.5, 0, size)
    check_attend(dtype, (got[0][few], got[1][few]), ref)
