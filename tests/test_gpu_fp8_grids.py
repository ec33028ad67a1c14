"""GPU: more tiles of the 8-bit product than a launch holds workgroups along one axis."""
import pytest
import torch

from tests._gpu import dev, lib, note

pytestmark = pytest.mark.gpu


def test_more_tiles_than_a_row_of_the_grid():
    """536 871 012 x 16 x 128: four layers of 2^21 tiles of 64 rows and a part; rows at the layers' edges
    equal those of small calls, rows between are zeros."""
    dg, d = lib(), dev()
    M, N, K, layer = (1 << 29) + 100, 16, 128, 64 << 21
    note(f"fp8 matmul {M}x{N}x{K}, 95 GB")
    g = torch.Generator().manual_seed(1)
    w = dg.nf4_fp8_quantize(torch.randn(N, K, generator=g).to(d), 128)
    part = dg.nf4_fp8_quantize(torch.randn(200, K, generator=g).to(d))
    data = torch.zeros(M, K, dtype=torch.uint8, device=d)
    scale = torch.zeros(M, 4, device=d)
    starts = [0, layer - 100, 2 * layer - 100, 3 * layer - 100, M - 200]
    for at in starts:
        data[at:at + 200] = part.data.view(torch.uint8)
        scale[at:at + 200] = part.scale
    y = dg.nf4_fp8_matmul(dg.FP8Tensor(M, K, 1, data.view(torch.float8_e4m3fn), scale), w, torch.bfloat16)
    want = dg.nf4_fp8_matmul(part, w, torch.bfloat16)
    torch.cuda.synchronize()
    assert want.any()
    for at in starts:
        assert torch.equal(y[at:at + 200], want), at
        for lo in (at - 5000, at + 200):
            if 0 <= lo and lo + 5000 <= M:
                assert not y[lo:lo + 5000].any(), lo
    assert int(y.view(torch.int16).any(1).sum()) == sum(int(want.any(1).sum()) for _ in starts)
    del data, scale, y
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M,N", [(1, (1 << 25) + 40), (5, (1 << 24) + 7)])
def test_many_rows_of_the_weight(M, N):
    """Up to 16 rows of X by a weight of 2^25 rows: the ends and the middle against small calls."""
    dg, d = lib(), dev()
    note(f"fp8 matmul {M}x{N}x128")
    g = torch.Generator().manual_seed(2)
    x = dg.nf4_fp8_quantize(torch.randn(M, 128, generator=g).to(d))
    data = torch.randint(0, 120, (N, 128), dtype=torch.uint8, device=d).view(torch.float8_e4m3fn)
    w = dg.FP8Tensor.from_parts(data, torch.rand(-(-N // 128), 1, device=d) + 0.5)
    y = dg.nf4_fp8_matmul(x, w)
    for lo in (0, (N // 2) // 128 * 128, (N - 300) // 128 * 128):
        hi = min(lo + 256, N)
        own = dg.nf4_fp8_matmul(x, dg.FP8Tensor(hi - lo, 128, 128, w.data[lo:hi], w.scale[lo // 128:-(-hi // 128)]))
        torch.cuda.synchronize()
        assert torch.equal(y[:, lo:hi], own), lo
