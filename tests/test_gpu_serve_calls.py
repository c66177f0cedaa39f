"""The single-token operators as calls: refusals of the Python entry points, and captured graphs of every split."""
import pytest
import torch

from tests.test_gpu_serve import _gen, attend_ref, check_attend, kda, make_cache, rope_table, to_gpu  # noqa: F401

pytestmark = pytest.mark.gpu


def _step_args(**change):
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    a = dict(q=z(2, 1, 2, 64), k=z(2, 1, 2, 64), v=z(2, 1, 4, 128), g=z(2, 1, 4, 64, dt=torch.float32), beta=z(2, 1, 4),
             state=z(2, 4, 64, 128, dt=torch.float32))
    a.update(change)
    return a


def test_step_refuses(kda):  # noqa: F811
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    assert kda.step(**_step_args()).shape == (2, 1, 4, 128)
    for bad in (dict(k=z(2, 1, 2, 128)), dict(v=z(2, 1, 4, 128, dt=torch.float32)), dict(g=z(2, 1, 4, 64)),
                dict(beta=z(2, 1, 2)), dict(state=z(2, 4, 64, 128)), dict(state=z(2, 4, 64, 64, dt=torch.float32)),
                dict(q=z(2, 1, 2, 128)[..., ::2]), dict(q=torch.zeros(2, 1, 2, 64, dtype=torch.bfloat16)),
                dict(slots=z(2, dt=torch.int64)), dict(slots=z(3, dt=torch.int32)), dict(out=z(2, 1, 4, 64)),
                dict(status=z(2, dt=torch.int32)), dict(q=z(2, 2, 64))):
        with pytest.raises(ValueError):
            kda.step(**_step_args(**bad))
    with pytest.raises(TypeError):
        kda.step(**{n: (t if n in ("g", "state") else t.half()) for n, t in _step_args().items()})
    with pytest.raises(TypeError):
        kda.step(**_step_args(q=None))
    with pytest.raises(kda.KdaError, match="KDA_ERR_INVALID_ARG"):  # two sequences, one state
        kda.step(**_step_args(state=z(1, 4, 64, 128, dt=torch.float32)))
    odd = _step_args(q=z(2, 1, 2, 96), k=z(2, 1, 2, 96), g=z(2, 1, 4, 96, dt=torch.float32),
                     state=z(2, 4, 96, 128, dt=torch.float32))
    with pytest.raises(kda.KdaError, match="KDA_ERR_UNSUPPORTED"):
        kda.step(**odd)


def test_cache_calls_refuse(kda):  # noqa: F811
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    kc, vc = kda.new_cache(6, 16, 2, 64, 128)
    table, lens = z(3, 2, dt=torch.int32), z(3, dt=torch.int32)
    append = lambda **c: kda.cache_append(**{**dict(k=z(3, 2, 64), v=z(3, 2, 128), k_cache=kc, v_cache=vc,  # noqa: E731
                                                    page_table=table, kv_lens=lens), **c})
    attend = lambda **c: kda.cache_attend(**{**dict(q=z(3, 4, 64), k_cache=kc, v_cache=vc, page_table=table,  # noqa: E731
                                                    kv_lens=lens), **c})
    assert append() is None and attend()[0].shape == (3, 4, 128)
    both = [dict(v_cache=vc.float()), dict(v_cache=vc[:5]), dict(k_cache=kc.transpose(2, 3)), dict(page_table=table.long()),
            dict(page_table=table.t().contiguous().t()), dict(kv_lens=lens.long()), dict(kv_lens=z(2, dt=torch.int32)),
            dict(status=z(1)), dict(page_table=table.cpu())]
    for bad in both + [dict(k=z(3, 2, 128)), dict(k=z(3, 2, 64, dt=torch.float32)), dict(k=z(3, 64, 2).transpose(1, 2)),
                       dict(v=z(4, 2, 128)), dict(q=z(3, 4, 128)), dict(q=z(3, 4, 64), q_out=z(3, 4, 128)),
                       dict(q_out=z(3, 4, 64)), dict(rope=z(16, 64)), dict(cu_seqlens=z(4, dt=torch.int32)),
                       dict(cu_seqlens=z(3, dt=torch.int64))]:
        with pytest.raises(ValueError):
            append(**bad)
    for bad in both + [dict(q=z(3, 4, 128)), dict(q=z(2, 4, 64)), dict(q=z(3, 4, 64, dt=torch.float32)),
                       dict(out=z(3, 4, 64)), dict(ws=z(512)), dict(window=2 ** 31)]:
        with pytest.raises(ValueError):
            attend(**bad)
    for bad in (dict(q=z(3, 3, 64)), dict(window=-1)):
        with pytest.raises(kda.KdaError, match="KDA_ERR_INVALID_ARG"):
            attend(**bad)
    with pytest.raises(kda.KdaError, match="KDA_ERR_INVALID_ARG"):  # four rows for three sequences
        append(k=z(4, 2, 64), v=z(4, 2, 128))
    with pytest.raises(kda.KdaError, match="KDA_ERR_INVALID_ARG"):  # a rotation wider than the keys
        append(rope=rope_table(8, 128).cuda())
    with pytest.raises(TypeError):
        attend(k_cache=kc.half(), v_cache=vc.half(), q=z(3, 4, 64).half())
    out, ws = z(3, 4, 128), z(1 << 20, dt=torch.uint8)
    assert attend(out=out, ws=ws)[0] is out


@pytest.mark.parametrize("split, N, longest", [("cache_attend", 4, 50), ("cache_attend_cluster", 2, 900),
                                               ("cache_attend_parts", 1, 9000), ("cache_attend_shares", 48, 3000)])
def test_graph_of_each_split(kda, split, N, longest):  # noqa: F811
    """A captured call follows the lengths and rows that its buffers hold at each replay."""
    gen, size, heads = _gen(21), 64, 8 if N > 4 else 2
    width = -(-longest // size)
    kc, vc = make_cache(gen, N * width, size, heads, 64, 64, "bf16", "heads first")
    table = torch.randperm(N * width, generator=gen).to(torch.int32).view(N, width)
    q = torch.randn(N, 2 * heads, 64, generator=gen).bfloat16()
    gk, gv, gq, gt = to_gpu(kc), to_gpu(vc), q.cuda(), table.cuda()
    lens = torch.full((N,), longest, dtype=torch.int32, device="cuda")
    kda.cache_attend(gq, gk, gv, gt, lens)
    assert kda.load().kda_launch_name(0).decode() == split
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        o, lse = kda.cache_attend(gq, gk, gv, gt, lens)
    for turn in range(4):
        now = torch.randint(0, longest + 1, (N,), generator=gen)
        lens.copy_(now)
        q = torch.randn(N, 2 * heads, 64, generator=gen).bfloat16()
        gq.copy_(q)
        graph.replay()
        torch.cuda.synchronize()
        few = list(range(min(N, 6)))
        ref = attend_ref(q[few], kc, vc, table[few], now[few].tolist(), 0.125, 0, size)
        check_attend("bf16", (o[few], lse[few]), ref)
        eager = kda.cache_attend(gq, gk, gv, gt, lens)
        assert torch.equal(eager[0], o) and torch.equal(eager[1], lse)
