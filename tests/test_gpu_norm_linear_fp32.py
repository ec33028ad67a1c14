"""GPU: the norm and product of an fp32 stream, whose gradient stays in fp32 between the two."""
import pytest
import torch

from tests import _ops_oracle as R
from tests._gpu import dev, lib, note

pytestmark = pytest.mark.gpu


def test_gradient_of_an_fp32_stream():
    dg, d = lib(), dev()
    note("fp8 norm linear, fp32 stream")
    g = torch.Generator().manual_seed(1)
    randn = lambda *s: torch.randn(*s, generator=g)
    layer = dg.FP8NormLinear.from_weight((randn(320, 256) * 0.05).to(d), eps=1e-5, out_dtype=torch.float32,
                                         norm_dtype=torch.float32)
    x, r = randn(70, 256).to(d).requires_grad_(), randn(70, 256).to(d).requires_grad_()
    y, h = layer(x, r)
    gy, gh = randn(70, 320), randn(70, 256)
    torch.autograd.backward([y, h], [gy.to(d), gh.to(d)])
    torch.cuda.synchronize()
    q, s = R.quantize(gy, 1, "e4m3")
    gv = R.values(q, s, 1, 320)
    wv = R.values(layer.qweight.data.cpu(), layer.qweight.scale.cpu(), 128, 256)
    hc = h.detach().cpu()
    rstd = 1 / torch.sqrt((hc.double() ** 2).mean(1) + 1e-5)
    dx, dw, mx, mw = R.rmsnorm_grad(gv @ wv, hc, torch.ones(256), rstd, gh)
    # the product's fp32 sums (three blocks) are relative to the magnitudes they add, and reach dx through
    # the norm's weight and rstd, and through the mean; the norm's own sums follow
    off = (128 * 2 + 6) * R.EPS32 * (gv.abs() @ wv.abs())
    through = rstd[:, None] * (off + hc.double().abs() * rstd[:, None] ** 2 * (off * hc.double().abs()).mean(1, keepdim=True))
    assert ((x.grad.cpu().double() - dx).abs() <= through + 130 * R.EPS32 * mx).all()
    assert torch.equal(x.grad, r.grad)
    werr = (off * hc.double().abs() * rstd[:, None]).sum(0) + 130 * R.EPS32 * mw
    assert ((layer.weight.grad.cpu().double() - dw).abs() <= werr).all()
