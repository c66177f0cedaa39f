"""What attention of one token does with particular values: weights as precise as the sums."""
import pytest
import torch

from tests.test_gpu_serve import DT, U, _gen, kda, run_attend  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_weights_are_as_precise_as_the_sums(kda, dtype):  # noqa: F811
    """Two rows whose weighted values cancel to some 2^-15 of themselves, so that the result's own rounding (2^-8 of what
    is left) hides nothing: what remains is the weights' error.

    A row's score is one product, so a weight errs by what the scaling to log2 units does to the score (|s| <= 0.51 log2
    units: 3 u |s|, less than 2^-23), by its exponential (2^-22) and by what the product with V holds of it (2^-22); the
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
