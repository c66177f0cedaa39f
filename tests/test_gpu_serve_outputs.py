"""What the single-token calls take and return: strides that say nothing, workspaces, and outputs of their own, that live,
are saved and are freed apart from each other."""
import io

import pytest
import torch

from tests.test_gpu_serve import _gen, kda  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N, L", [(2, 50), (1, 9000)])  # without a workspace of the kernels' own, and with one
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attend_outputs_are_tensors_of_their_own(kda, N, L, dtype):  # noqa: F811
    gen = _gen(41)
    width = -(-L // 16)
    kc, vc = kda.new_cache(N * width, 16, 2, 64, 64, dtype=dtype)
    table = torch.arange(N * width, dtype=torch.int32, device="cuda").view(N, width)
    q = torch.randn(N, 4, 64, generator=gen).to(dtype).cuda()
    lens = torch.full((N,), L, dtype=torch.int32, device="cuda")
    own = torch.empty(N, 4, 64, dtype=dtype, device="cuda")
    for out in (None, own):
        o, lse = kda.cache_attend(q, kc, vc, table, lens, out=out)
        assert o.untyped_storage().data_ptr() != lse.untyped_storage().data_ptr()
        for t in (o, lse):
            assert t.storage_offset() == 0 and t.untyped_storage().nbytes() == t.numel() * t.element_size()
        file = io.BytesIO()
        torch.save((o, lse), file)
        file.seek(0)
        again = torch.load(file)
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)


@pytest.mark.parametrize("N, L", [(2, 50), (1, 9000)])
def test_attend_workspace(kda, N, L):  # noqa: F811
    """A workspace of the size that is asked for serves, one that is too small is not touched, and the results are the same."""
    gen = _gen(42)
    width = -(-L // 16)
    kc, vc = (torch.randn(N * width, 16, 2, 64, generator=gen).bfloat16().cuda() for _ in range(2))
    table = torch.arange(N * width, dtype=torch.int32, device="cuda").view(N, width)
    q, lens = torch.randn(N, 4, 64, generator=gen).bfloat16().cuda(), torch.full((N,), L, dtype=torch.int32, device="cuda")
    need = kda.cache_attend_workspace_bytes(q, kc, vc, table)
    want = kda.cache_attend(q, kc, vc, table, lens)
    assert "parts" in kda.load().kda_launch_name(0).decode() or L < 9000
    for size in (need, need + 64, need - 1):
        ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        got = kda.cache_attend(q, kc, vc, table, lens, ws=ws)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        used = not bool((ws == 255).all())
        assert used == (size >= need and L == 9000)
    assert kda.cache_attend_workspace_bytes(q, kc, vc, table, window=10) <= need
    with pytest.raises(kda.KdaError):
        kda.cache_attend_workspace_bytes(q[:, :3], kc, vc, table)
    with pytest.raises(TypeError):
        kda.cache_attend_workspace_bytes(q.half(), kc.half(), vc.half(), table)


def test_strides_of_dimensions_of_one(kda):  # noqa: F811
    """A cache of one page, one row a page or one head may have any stride there."""
    gen = _gen(43)
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    for pages, rows, heads in ((1, 16, 2), (16, 1, 2), (4, 4, 1), (1, 16, 1), (16, 1, 1)):
        plain = [torch.randn(pages, rows, heads, 64, generator=gen).bfloat16().cuda() for _ in range(2)]
        odd = [t.clone().as_strided(t.shape, [3 if n == 1 else s for n, s in zip(t.shape, t.stride())]) for t in plain]
        table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
        k, v = (torch.randn(5, heads, 64, generator=gen).bfloat16().cuda() for _ in range(2))
        q = torch.randn(1, 2 * heads, 64, generator=gen).bfloat16().cuda()
        got = []
        for kc, vc in (plain, odd):
            kda.cache_append(k, v, kc, vc, table, z(1) + 11)
            got.append(kda.cache_attend(q, kc, vc, table, z(1) + 16) + (kc, vc))
            assert kda.cache_attend_workspace_bytes(q, kc, vc, table) > 0
        assert all(torch.equal(x, y) for x, y in zip(*got))
