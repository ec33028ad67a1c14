"""GPU: the 8-bit product in every pair of activation format and output type."""
import pytest
import torch

from tests import _ops_oracle as R
from tests import test_gpu_fp8 as base
from tests._gpu import dev, lib, note

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
_randn = base._randn


def _blocks(t, rows):
    """|values| [R, K] -> the largest of each 1 x 128 block, [R, blocks]."""
    K = t.shape[1]
    return torch.nn.functional.pad(t.abs(), (0, R.up(K, 128) - K)).reshape(rows, -1, 128).amax(2)


def _check_bf16(y, xv, wv, where):
    """An element, and the mean square of all, against float64.

    The fp8 matrix cores keep 13 bits below the largest of the products they add at once, so that each of a
    block's 128 products is off by at most 2^-13 of max|x| max|w|; fp32 sums and one bf16 rounding follow."""
    M, N, K = xv.shape[0], wv.shape[0], xv.shape[1]
    ref, mag = xv @ wv.t(), xv.abs() @ wv.abs().t()
    cores = 128 * 2.0 ** -13 * (_blocks(xv, M) @ _blocks(wv, N).t())
    tol = cores + (-(-K // 128) + 3) * R.EPS32 * mag + R.half_step(BF) * 1.01 * (ref.abs() + cores) + 1e-300
    err = (y.cpu().double() - ref).abs()
    assert (err <= tol).all(), f"{where}: worst {float((err / tol).max()):.2f} of the bound"
    # the roundings alone: a uniform half step of each element, then 2^-13 of a block's largest product, 128
    # independent ones to a block (a product left out of every sum would be far above this)
    step = torch.exp2(torch.floor(torch.log2(ref.abs().clamp(min=1e-300))) - 7)
    rms = (step ** 2 / 12 + (cores / 128) ** 2 * 128).mean().sqrt()
    assert float((err ** 2).mean().sqrt()) <= 1.5 * float(rms) + 1e-300, f"{where}: mean square"


def _product(M, N, K, fmt, out):
    dg, d = lib(), dev()
    note(f"fp8 matmul {M}x{N}x{K} {fmt} -> {out}")
    x = _randn(M, K, seed=M + K, dtype=BF)
    w = _randn(N, K, seed=N, std=0.02)
    xq, wq = dg.nf4_fp8_quantize(x.to(d), 1, fmt), dg.nf4_fp8_quantize(w.to(d), 128)
    y = dg.nf4_fp8_matmul(xq, wq, out)
    torch.cuda.synchronize()
    return y, R.values(xq.data.cpu(), xq.scale.cpu(), 1, K), R.values(wq.data.cpu(), wq.scale.cpu(), 128, K)


@pytest.mark.parametrize("M,N,K", base.SHAPES + base.GROUPS)
def test_e4m3_to_bf16(M, N, K):
    """What the layers run by default."""
    _check_bf16(*_product(M, N, K, "e4m3", BF), f"{M}x{N}x{K}")


@pytest.mark.parametrize("M,N,K", base.SHAPES + base.GROUPS)
def test_e5m2_to_fp32(M, N, K):
    y, xv, wv = _product(M, N, K, "e5m2", F32)
    base._check(y, xv, wv, K, f"{M}x{N}x{K}")


@pytest.mark.parametrize("M,N,K", [(1999, 8003, 330), (2048, 7936, 128)])
def test_large_tiles_against_float64(M, N, K):
    """Sizes that take the 256 x 256 tiles: rows at the tiles' edges."""
    dg, d = lib(), dev()
    y, xv, wv = _product(M, N, K, "e4m3", BF)
    rows = torch.tensor([0, 1, 15, 16, 127, 128, 255, 256, 257, 1023, 1024, M - 2, M - 1])
    _check_bf16(y.cpu()[rows], xv[rows], wv, f"{M}x{N}x{K}")


@pytest.mark.parametrize("M,N,K", [(5, 96, 256), (40, 200, 384), (200, 384, 512), (600, 700, 384), (2048, 7936, 256)])
@pytest.mark.parametrize("fmt,out", [("e4m3", BF), ("e5m2", F32), ("e5m2", BF)])
def test_every_code(M, N, K, fmt, out):
    dg, d = lib(), dev()
    note(f"fp8 matmul, all codes {M}x{N}x{K} {fmt} -> {out}")
    g = torch.Generator().manual_seed(M)

    def pick(r, f):
        c = torch.arange(256, dtype=torch.uint8)
        c = c[c.view(R.TYPE[f]).float().isfinite()]
        return c[torch.randint(0, c.numel(), (r, K), generator=g)].view(R.TYPE[f])

    xd, wd = pick(M, fmt), pick(N, "e4m3")
    xs = torch.exp2(torch.randint(-20, 20, (M, K // 128), generator=g).float()) * 1.37
    ws = torch.exp2(torch.randint(-20, 20, (-(-N // 128), K // 128), generator=g).float()) * 0.73
    x, w = dg.FP8Tensor.from_parts(xd.to(d), xs.to(d), 1), dg.FP8Tensor.from_parts(wd.to(d), ws.to(d), 128)
    y = dg.nf4_fp8_matmul(x, w, out)
    torch.cuda.synchronize()
    rows = torch.arange(0, M, max(1, M // 400))
    xv, wv = R.values(xd[rows], xs[rows], 1, K), R.values(wd, ws, 128, K)
    if out == F32:
        base._check(y.cpu()[rows], xv, wv, K, "all codes")
    else:
        _check_bf16(y.cpu()[rows], xv, wv, "all codes")


def test_gradient_format_e5m2():
    dg, d = lib(), dev()
    note("fp8 linear, e5m2 gradients")
    layer = dg.FP8Linear.from_weight(_randn(200, 384, seed=1, std=0.05).to(d), grad_fmt="e5m2")
    x = _randn(40, 384, seed=2, dtype=BF).to(d).requires_grad_()
    gy = _randn(40, 200, seed=3, dtype=BF).to(d)
    layer(x).backward(gy)
    torch.cuda.synchronize()
    q, s = R.quantize(gy.cpu(), 1, "e5m2")
    wv = R.values(layer.qweight.data.cpu(), layer.qweight.scale.cpu(), 128, 384)
    _check_bf16(x.grad, R.values(q, s, 1, 200), wv.t().contiguous(), "dx")
