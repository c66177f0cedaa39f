"""The bounds of the KDA step's element test tell fp32 from products in half its bits (on the CPU, a plain form for the kernel)."""
import pytest
import torch

from tests.test_gpu_serve import step_inputs, step_ref
from tests.test_gpu_serve_step import SIZES, step_bounds


def plain(x, scale, bits):
    """One token in fp32, the factors of every product with the state rounded to so many bits."""
    def cut(t):
        if bits >= 24:
            return t
        m, e = torch.frexp(t)
        return torch.ldexp(torch.round(m * 2 ** bits) / 2 ** bits, e)

    q, k, v, g, beta, S = (x[n].float() for n in ("q", "k", "v", "g", "beta", "state"))
    rep = v.shape[2] // q.shape[2]
    q, k = (t[:, 0].repeat_interleave(rep, 1) for t in (q, k))
    S = g[:, 0].exp()[..., None] * S
    d = beta[:, 0, :, None] * (v[:, 0] - (cut(k)[..., None] * cut(S)).sum(2))
    S = S + k[..., None] * d[:, :, None]
    return scale * (cut(q)[..., None] * cut(S)).sum(2), S


@pytest.mark.parametrize("N,H,HV,K,V", [s for s in SIZES if s[0] <= 5])
def test_bounds(N, H, HV, K, V):
    x = step_inputs(N + 7, N, 1, H, HV, K, V, "f32")
    ro, rs = step_ref(x, K ** -0.5)
    bo, bs = step_bounds(x, K ** -0.5)
    for bits, keeps in ((24, True), (12, False), (11, False), (8, False)):
        o, state = plain(x, K ** -0.5, bits)
        kept = ((o.double() - ro[:, 0]).abs() <= bo + 2.0 ** -24 * ro[:, 0].abs()).all()
        kept = kept and ((state.double() - rs).abs() <= bs).all()
        assert bool(kept) == keeps, bits
