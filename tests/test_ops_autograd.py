"""CPU: the layers' autograd functions, with plain formulas in the place of the native calls."""
import pytest
import torch

from dequant_gemm_amd import nn_fp8
from dequant_gemm_amd._ops import FP8Tensor


def _norm(x, weight, residual=None, eps=1e-6, out_dtype=None):
    h = x if residual is None else x + residual
    rstd = ((h.double() ** 2).mean(1) + eps).rsqrt()
    return (h * rstd[:, None] * weight).to(out_dtype or x.dtype), h, rstd


def _norm_grad(dy, h, weight, rstd, dh=None):
    with torch.no_grad():
        r = rstd[:, None]
        g = dy * weight
        dx = r * (g - h * r * r * (g * h).mean(1, keepdim=True))
        return (dx if dh is None else dx + dh).to(h.dtype), (dy * h * r).sum(0).to(weight.dtype)


@pytest.fixture
def plain(monkeypatch):
    """The native calls replaced; `seen` lists the product's output types."""
    seen = []

    def matmul(x, w, out_dtype=torch.float32, out=None):
        seen.append(out_dtype)
        with torch.no_grad():
            return (x.dequantize() @ w.dequantize().t()).to(out_dtype)

    def quantize(x, block_rows=1, fmt="e4m3", out=None):
        data = x.detach().clamp(-448, 448).to(torch.float8_e4m3fn)
        return FP8Tensor.from_parts(data, torch.ones(-(-x.shape[0] // block_rows), -(-x.shape[1] // 128)), block_rows)

    def norm_fp8(x, weight, residual=None, eps=1e-6):
        y, h, rstd = _norm(x.detach(), weight.detach(), residual, eps)
        return quantize(y), h, rstd

    monkeypatch.setattr(nn_fp8, "nf4_rmsnorm_fwd", lambda *a: tuple(t.detach() for t in _norm(*a)))
    monkeypatch.setattr(nn_fp8, "nf4_rmsnorm_bwd", _norm_grad)
    monkeypatch.setattr(nn_fp8, "nf4_rmsnorm_fwd_fp8", norm_fp8)
    monkeypatch.setattr(nn_fp8, "nf4_fp8_matmul", matmul)
    monkeypatch.setattr(nn_fp8, "nf4_fp8_quantize", quantize)
    return seen


def _layers():
    g = torch.Generator().manual_seed(0)
    w = torch.randn(5, 7, generator=g).clamp(-2, 2)
    q = FP8Tensor.from_parts(w.to(torch.float8_e4m3fn), torch.ones(1, 1), 128)
    weight = (1 + 0.1 * torch.randn(7, generator=g)).requires_grad_()
    norm = nn_fp8.FP8NormLinear(q, norm_dtype=torch.float32, out_dtype=torch.float32)
    return [("rms_norm", lambda x: nn_fp8.rms_norm(x, weight)), ("residual", lambda x: nn_fp8.rms_norm(x, weight, x)[0]),
            ("fp8_linear", lambda x: nn_fp8.fp8_linear(x, q, q.t(), torch.float32)), ("norm_linear", norm),
            ("norm_linear_residual", lambda x: norm(x, x)[0])]


@pytest.mark.parametrize("i", range(5))
def test_second_derivatives_are_refused(plain, i):
    """The gradients are computed outside the graph: a derivative of them raises, it is not silently dropped."""
    name, f = _layers()[i]
    x = torch.randn(3, 7, generator=torch.Generator().manual_seed(1)).requires_grad_()
    first, = torch.autograd.grad(f(x).square().sum(), x)
    again, = torch.autograd.grad(f(x).square().sum(), x, create_graph=True)
    assert torch.equal(first, again), name
    with pytest.raises(RuntimeError, match="once_differentiable"):
        again.square().sum().backward()


def test_first_derivatives_of_the_norm(plain):
    x = torch.randn(4, 6, generator=torch.Generator().manual_seed(2), dtype=torch.float64).float().requires_grad_()
    w = torch.linspace(0.5, 1.5, 6).requires_grad_()
    y = nn_fp8.rms_norm(x, w, eps=1e-3)
    y.backward(torch.ones_like(y) * 0.3)
    xr, wr = x.detach().double().requires_grad_(), w.detach().double().requires_grad_()
    (xr * ((xr ** 2).mean(1, keepdim=True) + 1e-3).rsqrt() * wr).backward(torch.full((4, 6), 0.3).double())
    assert torch.allclose(x.grad.double(), xr.grad, atol=1e-6) and torch.allclose(w.grad.double(), wr.grad, atol=1e-6)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_the_norms_gradient_keeps_the_streams_type(plain, dt):
    """The gradient between the product and the norm is formed in x's type, as the two layers apart form it."""
    q = FP8Tensor.from_parts(torch.ones(5, 7).to(torch.float8_e4m3fn), torch.ones(1, 1), 128)
    layer = nn_fp8.FP8NormLinear(q, norm_dtype=torch.float32, out_dtype=torch.float32)
    x = torch.randn(3, 7).to(dt).requires_grad_()
    y = layer(x)
    del plain[:]
    y.sum().backward()
    assert plain == [dt] and x.grad.dtype == dt
