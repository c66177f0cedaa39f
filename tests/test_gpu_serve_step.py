"""kda_step against 64 bits element by element, with bounds that products in fewer bits than fp32's do not keep."""
import pytest
import torch

from tests.test_gpu_serve import ROUND, U, _rel, kda, run_step, step_inputs, step_ref  # noqa: F401

pytestmark = pytest.mark.gpu


def step_bounds(x, scale):
    """The error bounds of o (before its rounding) and of the new state for one token.

    e^g errs by (4 + 2 |g|) u (the exponential, and its argument's two roundings), so S' = e^g S by (5 + 2 |g|) u. A product
    with S' sums chains of K / 16 terms and joins 16 of them in 5 steps: with a = K / 16 + 10 + 2 max |g|,
      k S' errs by a u A, A = sum |k S'|;   q S' by a u C, C = sum |q S'|;   q k (9 sums of 1) by 9 u B, B = sum |q k|;
      d = beta (v - k S') by u beta (a A + 2 |v| + 2 A), and |d| <= beta (|v| + A);
      o = scale (q S' + (q k) d), three more roundings, by scale u ((a + 4) C + (a + 15) B beta (|v| + A));
      S' + k d by (6 + 2 |g|) u |S'| + u |k| beta ((a + 4) A + 4 |v|)."""
    q, k, v, g, beta, S = (x[n].double() for n in ("q", "k", "v", "g", "beta", "state"))
    rep = v.shape[2] // q.shape[2]
    q, k = (t[:, 0].repeat_interleave(rep, 1).abs() for t in (q, k))
    v, g, beta = v[:, 0].abs(), g[:, 0], beta[:, 0, :, None]
    S = (g.exp()[..., None] * S).abs()
    a = q.shape[-1] / 16 + 10 + 2 * float(g.abs().max())
    A, C = torch.einsum("nhk,nhkv->nhv", k, S), torch.einsum("nhk,nhkv->nhv", q, S)
    B = (q * k).sum(-1, keepdim=True)
    o = scale * U * ((a + 4) * C + (a + 15) * B * beta * (v + A))
    state = (6 + 2 * g.abs())[..., None] * U * S + U * k[..., None] * (beta * ((a + 4) * A + 4 * v))[:, :, None]
    return o, state


SIZES = [(1, 1, 1, 128, 128), (3, 2, 6, 64, 128), (2, 3, 3, 128, 64), (5, 2, 4, 64, 64), (40, 4, 8, 128, 128), (160, 1, 1, 128, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,H,HV,K,V", SIZES)
def test_step_element_by_element(kda, N, H, HV, K, V, dtype):  # noqa: F811
    x = step_inputs(N + 7, N, 1, H, HV, K, V, dtype)
    o, state = run_step(kda, x)
    ro, rs = step_ref(x, K ** -0.5)
    bo, bs = step_bounds(x, K ** -0.5)
    assert ((o.double().cpu() - ro).abs()[:, 0] <= 1.01 * (bo + ROUND[dtype] * ro.abs()[:, 0])).all()
    assert ((state.double().cpu() - rs).abs() <= 1.01 * bs).all()
