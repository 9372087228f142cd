"""The SwiGLU producer's backward pass where the sigmoid leaves binary32's
normal range: gates from -80 to -110, gradients and up values from one to very
large, against the 64-bit formula.

Bound, with u = 2^-24: e = exp(-|g|) is within two units in the last place, 4 u
of itself or, below the normal range, 2^-148; r = 1 / (1 + e) within 4 u (the
sum's rounding, a reciprocal of one unit in the last place); so sg = e r is
within 10 u of itself and 2^-147, 1 - sg = r within 4 u, 1 + g (1 - sg) within
4 u |g| + u of its value, and each further product adds u of itself and half
the smallest subnormal.  dh up of bf16 values is exact.  Doubled, and half a
step of bf16 at the end."""
import pytest
import torch

import fp4_quantization_block_b200 as fa
import rows_ref as R
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dh,up", [(1.0, 1.0), (-3.0, 0.5), (1024.0, -2.0), (2.0 ** 40, 2.0 ** 30)],
                         ids=lambda v: f"{v:g}")
def test_gates_far_below_zero(dh, up):
    need_gpu()
    g = torch.linspace(-110.0, -80.0, 4096).bfloat16().view(-1, 64)
    z = torch.cat([g, torch.full_like(g, up)], 1)
    d = torch.full_like(g, dh)
    gd, a, b = g.double(), abs(dh * up), abs(dh)
    sg, om = torch.sigmoid(gd), torch.sigmoid(-gd)
    f = 1.0 + gd * om
    want = torch.cat([dh * up * sg * f, dh * gd * sg], 1)
    e_dg = a * (sg * (4 * R.U * gd.abs() + R.U) + (sg * f).abs() * 12 * R.U
                + f.abs() * 2.0 ** -147 + 2.0 ** -149)
    e_du = b * (gd.abs() * (10 * R.U * sg + 2.0 ** -147) + 2 * R.U * (gd * sg).abs() + 2.0 ** -149)
    R.check("dz", fa.swiglu_bwd(z.cuda(), d.cuda()), want, 2 * torch.cat([e_dg, e_du], 1), torch.bfloat16)


def test_ordinary_gates_beside_far_ones():
    """A channel's result is the same bits whatever its neighbours' gates are,
    in place too."""
    need_gpu()
    g = torch.Generator().manual_seed(0)
    z = torch.randn(64, 512, generator=g).mul_(4).bfloat16().cuda()
    dh = torch.randn(64, 256, generator=g).bfloat16().cuda()
    want = fa.swiglu_bwd(z, dh)
    far = torch.rand(64, 256, generator=g).cuda() < 0.2
    z2 = z.clone()
    z2[:, :256][far] = -95.0
    got = fa.swiglu_bwd(z2, dh)
    near = ~far.repeat(1, 2)
    assert torch.equal(got[near], want[near])
    fa.swiglu_bwd(z2, dh, out=z2)
    assert torch.equal(z2, got)
