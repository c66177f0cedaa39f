"""kda_cache_append at sizes that its first tests leave out."""
import pytest
import torch

from tests.test_gpu_serve import kda  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("turned", [False, True])
@pytest.mark.parametrize("HQ, HKV", [(2 ** 24 + 1, 1), (1, 2 ** 24 + 1)])
def test_rows_beyond_32_bits(kda, HQ, HKV, turned):  # noqa: F811
    """Heads whose channels lie more than 2^31 elements into a row, copied, and turned by an angle of 0."""
    D = 128
    q, k, v = (torch.randn(1, n, D, dtype=torch.bfloat16, device="cuda") for n in (HQ, HKV, HKV))
    kc, vc = kda.new_cache(1, 1, HKV, D, D)
    rope = torch.cat([torch.ones(1, 32), torch.zeros(1, 32)], 1).cuda() if turned else None
    table, lens = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((1, 1), (1,)))
    out = kda.cache_append(k, v, kc, vc, table, lens, q=q, rope=rope)
    assert torch.equal(out, q) and torch.equal(kc[0], k) and torch.equal(vc[0], v)
