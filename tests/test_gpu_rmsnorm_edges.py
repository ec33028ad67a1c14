"""GPU: the RMS norm where its roundings, its padding and its gradient's sums can go wrong."""
import pytest
import torch

from tests import _ops_oracle as R
from tests._gpu import dev, lib, note

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _randn(*shape, seed, std=1.0, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype)


@pytest.mark.parametrize("H", [64, 512, 1000, 4096, 8192, 16384, 20000])
@pytest.mark.parametrize("dt", [BF, F32])
def test_rstd_is_rounded_about_once(H, dt):
    """A correctly rounded rstd is off by a uniform half step, 0.29 of a step in the mean square; the fp32
    additions of a thread's own squares (24 at most, averaged over the threads) leave it under 0.4."""
    dg, d = lib(), dev()
    note(f"rmsnorm: rstd of 2000 x {H} {dt}")
    x = _randn(2000, H, seed=H, std=2.0) * torch.linspace(0.5, 4.0, 2000)[:, None]
    x = x.to(dt)
    _, _, rstd = dg.nf4_rmsnorm_fwd(x.to(d), torch.ones(H, device=d), eps=2.0 ** -20)
    torch.cuda.synchronize()
    ref = 1.0 / torch.sqrt((x.double() ** 2).mean(1) + 2.0 ** -20)
    step = torch.exp2(torch.floor(torch.log2(ref)) - 23)
    off = float((((rstd.cpu().double() - ref) / step) ** 2).mean().sqrt())
    assert off < 0.4, off


@pytest.mark.parametrize("eps", [0.0, 2.0 ** -149, 1e-30, 1e30])
def test_rstd_of_extreme_rows(eps):
    dg, d = lib(), dev()
    note(f"rmsnorm: extreme rows, eps {eps}")
    x = torch.zeros(5, 24)
    x[1], x[2], x[3], x[4] = 1e-18, 1e18, 2.0 ** -75, 3e38
    _, _, rstd = dg.nf4_rmsnorm_fwd(x.to(d), torch.ones(24, device=d), eps=eps)
    torch.cuda.synchronize()
    s = (x * x).sum(1).double() / 24 + torch.tensor(eps, dtype=F32).double()     # the squares are fp32's
    ref = (1.0 / torch.sqrt(s)).float()
    got = rstd.cpu()
    assert torch.equal(got.isinf(), ref.isinf()) and not got.isnan().any()
    ok = ref.isfinite()
    # a thread's seven additions of equal squares, halved by the root, and one rounding
    assert ((got - ref).abs()[ok] <= ref[ok] * 5 * R.EPS32).all()


@pytest.mark.parametrize("H", [1, 100, 260, 300, 1100, 5001, 20100])
@pytest.mark.parametrize("dt,res", [(BF, False), (F32, True)])
def test_padding_of_rows_without_a_norm(H, dt, res):
    """Codes and scales past the row's end are zeros, also where rstd is NaN, infinite or zero."""
    dg, d = lib(), dev()
    note(f"rmsnorm fp8: padding of {H} {dt} res={res}")
    x = _randn(5, H, seed=H, dtype=dt)
    x[0, H // 2] = float("nan")
    x[1] = 0
    x[2, 0] = float("inf")
    r = torch.zeros_like(x) if res else None
    w = torch.ones(H)
    q, _, _ = dg.nf4_rmsnorm_fwd_fp8(x.to(d), w.to(d), None if r is None else r.to(d), eps=0.0)
    good, _, _ = dg.nf4_rmsnorm_fwd_fp8(x[3:].to(d), w.to(d), None if r is None else r[3:].to(d), eps=0.0)
    torch.cuda.synchronize()
    codes = q.data.cpu().view(torch.uint8)
    assert (codes[:, H:] == 0).all()
    assert (q.scale.cpu()[:, -(-H // 128):] == 0).all()
    v = q.dequantize().cpu()
    assert v[:2].isnan().all() and bool(v[2, 0].isnan())
    assert torch.equal(codes[3:], good.data.cpu().view(torch.uint8)) and torch.equal(q.scale[3:], good.scale)


# dense rows: several to a workgroup of one wave and of many, the kernel for rows wider than the registers
# with more than one row a workgroup, and the doubled workgroups of odd widths
@pytest.mark.parametrize("T,H", [(600, 16392), (600, 16401), (1111, 5001), (2100, 1000), (9000, 1123), (9000, 333),
                                 (700, 12000), (1200, 6001), (5000, 64)])
@pytest.mark.parametrize("xt,dt,wt,res", [(BF, BF, BF, True), (F32, BF, F32, False)])
def test_gradient_of_many_dense_rows(T, H, xt, dt, wt, res):
    dg, d = lib(), dev()
    note(f"rmsnorm bwd {T}x{H} h {xt} dy {dt} dh={res}")
    h, dy = _randn(T, H, seed=1, std=2.0, dtype=xt), _randn(T, H, seed=2, std=0.1, dtype=dt)
    w = (1 + _randn(H, seed=3, std=0.2)).to(wt)
    dh = _randn(T, H, seed=4, dtype=xt) if res else None
    rstd = (1 / torch.sqrt((h.double() ** 2).mean(1) + 1e-5)).float()
    dx, dw = dg.nf4_rmsnorm_bwd(dy.to(d), h.to(d), w.to(d), rstd.to(d), None if dh is None else dh.to(d))
    torch.cuda.synchronize()
    rx, rw, mx, mw = R.rmsnorm_grad(dy, h, w, rstd, dh)
    # dx: under 64 additions of a thread, the lanes and the waves, and a few products;
    # dw: at most 36 rows of a workgroup, 4096 / 64 of a lane, 63 lanes and two products
    for name, got, ref, mag, n in (("dx", dx, rx, mx, 128), ("dw", dw, rw, mw, 192)):
        err = (got.cpu().double() - ref).abs()
        tol = n * R.EPS32 * mag + R.half_step(got.dtype) * 1.01 * ref.abs() + 1e-300
        assert (err <= tol).all(), f"{name}: worst {float((err / tol).max()):.3f} of the bound"
