"""kda_cache_append at sizes that its first tests leave out."""
import pytest
import torch

from tests.test_gpu_serve import DT, ROUND, U, _gen, kda, make_cache, make_table, rope_table, to_gpu, turn  # noqa: F401

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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens, T, HQ, HKV, K, V, size, rot, inter, layout", [
    ([4, 0], 3, 2, 1, 64, 64, 4, 64, False, "heads first"),  # several rows to a CTA
    ([0, 31, 5], 40, 8, 2, 128, 64, 16, 64, False, "rows first"),
    ([100, 7, 0, 63, 64], 129, 16, 4, 64, 128, 27, 32, True, "shared pool"),
    ([11] * 30, 70, 6, 3, 128, 128, 64, 0, False, "heads first"),
])
def test_as_many_rows_for_each_sequence(kda, lens, T, HQ, HKV, K, V, size, rot, inter, layout, dtype):  # noqa: F811
    """Without cu_seqlens R / N rows belong to each sequence; and the same rows with cu_seqlens, into a cache of their own."""
    gen, dt, N = _gen(51), DT[dtype], len(lens)
    reach = [x + T for x in lens]
    pages = sum(-(-x // size) for x in reach) + 2
    kc, vc = make_cache(gen, pages, size, HKV, K, V, dtype, layout)
    table = make_table(gen, reach, size, pages)
    q, k, v = (torch.randn(N * T, h, d, generator=gen).to(dt) for h, d in ((HQ, K), (HKV, K), (HKV, V)))
    rope = rope_table(max(reach), rot) if rot else None
    n = torch.arange(N * T) // T
    pos = torch.tensor(lens)[n] + torch.arange(N * T) % T
    page = table[n, pos // size].long()
    wq, size_q = turn(q, pos, rope, inter)
    wk, size_k = turn(k, pos, rope, inter)
    bound = lambda want, mag: (3 * U * mag + ROUND[dtype] * want.abs() * (mag > 0)) * 1.01  # noqa: E731
    for cu in (None, (torch.arange(N + 1) * T).cuda()):
        gk, gv = to_gpu(kc), to_gpu(vc)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = kda.cache_append(k.cuda(), v.cuda(), gk, gv, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                               q=q.cuda(), rope=None if rope is None else rope.cuda(), interleaved=inter, cu_seqlens=cu,
                               status=status)
        assert int(status) == 0
        assert ((out.double().cpu() - wq).abs() <= bound(wq, size_q)).all()
        assert ((gk.cpu()[page, pos % size].double() - wk).abs() <= bound(wk, size_k)).all()
        assert torch.equal(gv.cpu()[page, pos % size], v)
        for now, before in ((gk.cpu(), kc), (gv.cpu(), vc)):
            keep = torch.ones(pages, size, dtype=torch.bool)
            keep[page, pos % size] = False
            assert torch.equal(now[keep], before[keep])


@pytest.mark.parametrize("cu, kept", [([0, 2, 5], [0, 1, 2, 3, 4]), ([0, 2, 4], [0, 1, 2, 3]), ([1, 2, 5], [1, 2, 3, 4]),
                                      ([0, 0, 0], []), ([0, 2, 2], [0, 1])])
def test_rows_outside_the_packed_sequences(kda, cu, kept):  # noqa: F811
    """Rows before the first sequence or behind the last one belong to none: not appended, their queries 0, and flagged."""
    gen = _gen(52)
    k, v, q = (torch.randn(5, 2, 64, generator=gen).bfloat16().cuda() for _ in range(3))
    kc, vc = kda.new_cache(4, 8, 2, 64, 64)
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    lens, status = torch.tensor([6, 7], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = kda.cache_append(k, v, kc, vc, table, lens, q=q, cu_seqlens=torch.tensor(cu, device="cuda"), status=status)
    assert int(status) == (len(kept) < 5)
    want_k, want_q = torch.zeros_like(kc), torch.zeros_like(q)
    for r in kept:
        n = 0 if r < cu[1] else 1
        pos = int(lens[n]) + r - cu[n]
        want_k[table[n, pos // 8].long(), pos % 8] = k[r]
        want_q[r] = q[r]
    assert torch.equal(kc, want_k) and torch.equal(out, want_q) and int((vc != 0).flatten(2).any(2).sum()) == len(kept)
