"""What attention of one token does with particular values: weights as precise as the sums, infinite and very large values."""
import math

import pytest
import torch

from tests.test_gpu_serve import DT, U, _gen, kda, run_attend  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_weights_are_as_precise_as_the_sums(kda, dtype):  # noqa: F811
    """Two rows whose weighted values cancel to some 2^-15 of themselves, so that the result's own rounding (2^-8 of what
    is left) hides nothing: what remains is the weights' error.

    A row's score is one product, so a weight errs by what the scaling to log2 units does to the score (|s| <= 0.51 log2
    units: 3 u |s|, less than 2^-23), by its exponential (2^-22) and by what the product with V holds of it (2^-21.9); the
    sum of two terms may be truncated at 2^-23 each. In all less than 2^-20 of the terms' magnitudes."""
    gen, dt, N, H, D = _gen(31), DT[dtype], 4, 64, 64
    x = -(torch.rand(N, H, generator=gen) * 0.3 + 0.05).to(torch.bfloat16).double()
    kc, vc = torch.zeros(N, 2, H, D, dtype=dt), torch.zeros(N, 2, H, D, dtype=dt)
    kc[:, 1, :, 0] = x.to(dt)
    b = torch.arange(128, 256, dtype=torch.float64).expand(N, H, -1)
    a = (x.exp()[..., None] * b).round()
    best = (a - x.exp()[..., None] * b).abs().argsort(-1)[..., :D]
    a, b = a.gather(-1, best), b.gather(-1, best)  # whole numbers below 256: bf16 holds them
    vc[:, 0], vc[:, 1] = (-a).to(dt), b.to(dt)
    q = torch.zeros(N, H, D, dtype=dt)
    q[..., 0] = 1.0
    o, _ = run_attend(kda, q, kc, vc, torch.arange(N, dtype=torch.int32)[:, None], [2] * N, scale=1.0)
    p1 = torch.sigmoid(x)[..., None]
    want, size = p1 * b - (1 - p1) * a, p1 * b + (1 - p1) * a
    rounding = (2.0 ** -8 if dtype == "bf16" else U) * want.abs()
    assert ((o.double().cpu() - want).abs() <= 2.0 ** -20 * size + 1.01 * rounding).all()


def same_kind(got, ref, bound):
    """Equal infinities and NaNs, and the finite values within the bound."""
    got = got.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    assert torch.equal(torch.isinf(got), torch.isinf(ref)) and torch.equal(got[torch.isinf(ref)], ref[torch.isinf(ref)])
    some = torch.isfinite(ref)
    assert ((got - ref).abs() <= bound)[some].all()


# split of the bf16 kernel, N, rows, heads
SPLITS = [("cache_attend", 300, 60, 4), ("cache_attend_cluster", 2, 900, 4), ("cache_attend_parts", 1, 9000, 2),
          ("cache_attend_shares", 48, 3000, 8)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("split, N, L, H", SPLITS)
def test_values_that_are_not_finite(kda, split, N, L, H, D, dtype):  # noqa: F811
    """An infinite value makes its channel infinite, two of opposite sign or a NaN make it NaN, and the other channels
    are what they are without them; at the row of the greatest weight as at the others."""
    gen, dt = _gen(32), DT[dtype]
    size, some = 20, 3
    width = -(-L // size)
    kc, vc = (torch.randn(some * width, size, H, D, generator=gen).to(dt) for _ in range(2))
    table = (torch.arange(N)[:, None] % some * width + torch.arange(width)).to(torch.int32)
    q = torch.randn(some, H, D, generator=gen).to(dt)
    flat_k, flat_v = (t.view(some, width * size, H, D)[:, :L] for t in (kc, vc))
    scores = torch.einsum("nhd,nthd->nht", q.double(), flat_k.double()) * D ** -0.5
    top = scores.argmax(-1)
    n, h = torch.meshgrid(torch.arange(some), torch.arange(H), indexing="ij")
    flat_v[n, top, h, 3] = math.inf
    flat_v[n, top, h, 5] = -math.inf
    flat_v[n, (top + 7) % L, h, 17] = math.inf
    flat_v[n, (top + L // 2) % L, h, D - 1] = -math.inf
    flat_v[n, (top + 1) % L, h, 33] = math.nan
    flat_v[n, top, h, 40], flat_v[n, (top + 3) % L, h, 40] = math.inf, -math.inf
    got, _ = run_attend(kda, q[torch.arange(N) % some], kc, vc, table, [L] * N)
    if dtype == "bf16":
        assert kda.load().kda_launch_name(0).decode() == split
    p = torch.softmax(scores, -1)
    ref = torch.einsum("nht,nthd->nhd", p, flat_v.double())
    # scores err by (K + 4) 2u sum |q k| scale, at most 24 here; the sums by 2 (L + 16) u
    bound = (2 * 24 * (D + 4) * 2 * U + 2.0 ** -20 + 2 * (L + 16) * U) * torch.einsum(
        "nht,nthd->nhd", p, flat_v.double().abs()) + 1.01 * (2.0 ** -8 if dtype == "bf16" else U) * ref.abs()
    for i in range(min(N, 6)):
        same_kind(got[i], ref[i % some], bound[i % some])
    assert torch.equal(got[-1].isnan(), got[(N - 1) % some].isnan())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("split, N, L, H", SPLITS)
def test_very_large_values(kda, split, N, L, H, dtype):  # noqa: F811
    """Values of 2^127 whose row has the greatest weight, with scores that rise along the rows: the weighted mean is
    finite and so is every sum of weights of at most one times them."""
    gen, dt, D, size = _gen(33), DT[dtype], 64, 20
    width = -(-L // size)
    kc, vc = (torch.zeros(width, size, 1, D, dtype=dt) for _ in range(2))
    flat_k, flat_v = (t.view(width * size, D)[:L] for t in (kc, vc))
    flat_k[:, 0] = (torch.arange(L) / L * 5.0).to(dt)  # up to 7.2 in log2 units
    q = torch.zeros(N, H, D, dtype=dt)
    q[..., 0] = 1.0
    s = flat_k[:, 0].double()
    flat_v[int(s.argmax()), : D // 2] = 2.0 ** 127
    flat_v[:, D // 2:] = torch.randn(L, D // 2, generator=gen).to(dt)
    one = lambda t: t.expand(-1, -1, H, -1).contiguous()  # noqa: E731
    o, lse = run_attend(kda, q, one(kc), one(vc), torch.arange(width, dtype=torch.int32).expand(N, -1), [L] * N, scale=1.0)
    p = torch.softmax(s, 0)
    want, mag = p @ flat_v.double(), p @ flat_v.double().abs()
    w = 2 * 5 * 68 * 2 * U + 2.0 ** -20 + 2 * (L + 16) * U
    o = o.double().cpu()
    assert torch.isfinite(o).all()
    assert ((o - want).abs() <= w * mag + 1.01 * (2.0 ** -8 if dtype == "bf16" else U) * want.abs()).all()
    assert ((lse.double().cpu() - torch.logsumexp(s, 0)).abs() <= w + 4 * U * 15).all()
