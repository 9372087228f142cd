"""The MLP half of a training block, forward and backward, through the public
calls in the order a training step makes them: dropout + residual + norm, the
gate+up linear, the SwiGLU producer, the down projection, dropout into the
residual stream, and back.  Every new operator's output is checked against the
64-bit form of the very inputs it had in the run; the run is captured into a
graph and replayed under a new step."""
import pytest
import torch

import fp4_quantization_block_b200 as fa
import rows_ref as R
from gpu_util import need_gpu
from test_gpu_norm import SEED, check_bwd, check_fwd

pytestmark = pytest.mark.gpu

MASK = 0x2545F491
P = 0.1


class Mlp:
    def __init__(self, T, H, F, fmt):
        g = torch.Generator().manual_seed(T + H + F)
        n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.T, self.H, self.F, self.fmt = T, H, F, fmt
        bf = torch.bfloat16
        self.attn, self.resid = n(T, H).to(bf).cuda(), n(T, H).to(bf).cuda()
        self.dout = (n(T, H) * 1e-2).to(bf).cuda()
        self.w, self.b = (1 + 0.1 * n(H)).cuda(), (0.1 * n(H)).cuda()
        wgu, wd = (n(2 * F, H) * 0.05).to(bf).cuda(), (n(H, F) * 0.05).to(bf).cuda()
        self.gu, self.gu_col = fa.quantize(wgu, fmt), fa.quantize(wgu, fmt, orient=fa.COLWISE)
        self.dn, self.dn_col = fa.quantize(wd, fmt), fa.quantize(wd, fmt, orient=fa.COLWISE)
        self.step = torch.zeros(1, dtype=torch.int64, device="cuda")

    def run(self):
        v = {}
        v["y"], v["s"], v["mean"], v["rstd"] = fa.dropout_add_layer_norm_fwd(
            self.attn, self.resid, self.w, self.b, P, SEED, step=self.step)
        v["z"], xcol = fa.linear_fwd_save(v["y"], self.gu, self.fmt, MASK)
        hq, hcol = fa.swiglu_quantize(v["z"], self.fmt, col=True, sign_mask=MASK)
        v["o"] = fa.gemm(hq, self.dn, out_dtype=torch.bfloat16)
        v["out"] = fa.dropout_fwd(v["o"], P, SEED + (1 << 32), step=self.step, residual=v["s"])
        # backward: dout reaches s through the residual and through the MLP
        v["do"] = fa.dropout_bwd(self.dout, P, SEED + (1 << 32), step=self.step)
        v["dh"], v["dwd"] = fa.linear_bwd(v["do"], self.dn_col, hcol, self.fmt, seed=3, sign_mask=MASK)
        v["dz"] = fa.swiglu_bwd(v["z"], v["dh"])
        v["dy"], v["dwgu"] = fa.linear_bwd(v["dz"], self.gu_col, xcol, self.fmt, seed=4, sign_mask=MASK)
        v["dattn"], v["dresid"], v["dw"], v["db"] = fa.dropout_add_layer_norm_bwd(
            v["dy"], self.dout, v["s"], self.w, v["mean"], v["rstd"], P, SEED, step=self.step)
        return v


def check(m, v, step):
    bf = torch.bfloat16
    mask, scale = R.kept(m.T, m.H, P, SEED, step)
    mask2, _ = R.kept(m.T, m.H, P, SEED + (1 << 32), step)
    d, bd = R.drop(m.attn.cpu(), mask, scale)
    s = m.resid.cpu().double() + d
    R.check("s", v["s"], s, bd + R.U * s.abs(), bf)
    check_fwd(v["s"], m.w, m.b, True, v["y"], v["mean"], v["rstd"])
    d, bd = R.drop(v["o"].cpu(), mask2, scale)
    out = v["s"].cpu().double() + d
    R.check("out", v["out"], out, bd + R.U * out.abs(), bf)
    d, bd = R.drop(m.dout.cpu(), mask2, scale)
    R.check("do", v["do"], d, bd, bf)
    dz, bz = R.swiglu_bwd(v["z"].cpu(), v["dh"].cpu())
    R.check("dz", v["dz"], dz, bz, bf)
    check_bwd(v["dy"], v["s"], m.w, v["mean"], v["rstd"], True, m.dout, v["dresid"], v["dw"], v["db"])
    (full, _, _), (bound, _, _) = R.norm_bwd(v["dy"].cpu(), v["s"].cpu(), m.w.cpu(), v["mean"].cpu(),
                                             v["rstd"].cpu(), True, m.dout.cpu())
    want, b3 = R.drop(full, mask, scale)
    R.check("dattn", v["dattn"], want, torch.where(mask, bound * scale, 0.0) + b3, bf)
    for k in ("z", "o", "dh", "dy", "dwgu", "dwd"):
        assert torch.isfinite(v[k]).all() and v[k].abs().max() > 0


@pytest.mark.parametrize("fmt", [fa.MXFP4, fa.NVFP4_CTA], ids=["mx", "nvc"])
@pytest.mark.parametrize("T,H,F", [(128, 256, 384), (96, 160, 224)], ids=["aligned", "ragged"])
def test_mlp_half_of_a_block(T, H, F, fmt):
    need_gpu()
    m = Mlp(T, H, F, fmt)
    m.step.fill_(7)
    check(m, m.run(), 7)


def test_captured_run_replays_under_a_new_step():
    need_gpu()
    m = Mlp(128, 256, 384, fa.MXFP4)
    m.run()  # first launches outside the capture
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        v = m.run()
    for step in (5, 6):
        m.step.fill_(step)
        graph.replay()
        torch.cuda.synchronize()
        check(m, v, step)
        eager = m.run()
        assert all(torch.equal(v[k], eager[k]) for k in v)
