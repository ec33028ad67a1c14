"""GPU: calls that write a caller's tensors count as in-place changes, which autograd then sees."""
import pytest
import torch

from tests import test_gpu_fp8 as base
from tests._gpu import dev, lib, note

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
_randn = base._randn


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_into_buffers(block_rows, fmt):
    """``out=`` gives what a call that allocates gives, and counts as a change of the buffers."""
    dg, d = lib(), dev()
    note(f"fp8 quantize into buffers, {block_rows} rows a scale, {fmt}")
    x = _randn(150, 300, seed=1, dtype=BF).to(d)
    want = dg.nf4_fp8_quantize(x, block_rows, fmt)
    out = dg.FP8Tensor.empty(150, 300, block_rows, fmt, d)
    before = out.data._version, out.scale._version
    assert dg.nf4_fp8_quantize(x, out=out) is out
    torch.cuda.synchronize()
    assert torch.equal(out.data.view(torch.uint8), want.data.view(torch.uint8)) and torch.equal(out.scale, want.scale)
    assert out.data._version > before[0] and out.scale._version > before[1]
    for bad in (dg.FP8Tensor.empty(150, 299, block_rows, fmt, d), dg.FP8Tensor.empty(150, 300, block_rows, fmt, "cpu")):
        with pytest.raises(ValueError):
            dg.nf4_fp8_quantize(x, out=bad)
    with pytest.raises(ValueError):
        dg.nf4_fp8_quantize(x.t(), out=dg.FP8Tensor.empty(300, 150, block_rows, fmt, d))


def test_product_into_a_buffer_is_a_change_of_it():
    dg, d = lib(), dev()
    note("fp8 matmul out=: the buffer's version")
    x, w = dg.nf4_fp8_quantize(_randn(8, 256, seed=1).to(d)), dg.nf4_fp8_quantize(_randn(64, 256, seed=2).to(d), 128)
    y = torch.zeros(8, 64, device=d)
    a = torch.ones(8, 64, device=d, requires_grad=True)
    z = (a * y).sum()
    assert dg.nf4_fp8_matmul(x, w, out=y) is y and y._version == 1
    with pytest.raises(RuntimeError, match="inplace"):
        z.backward()
    with torch.inference_mode():
        dg.nf4_fp8_matmul(x, w, out=torch.zeros(8, 64, device=d))     # keeps no version
    torch.cuda.synchronize()


@pytest.mark.parametrize("bits", [8, 32])
def test_an_optimizer_step_is_a_change_of_the_parameters(bits):
    """A backward pass through weights that have been stepped since raises, as with torch's optimizers."""
    dg, d = lib(), dev()
    note(f"adamw {bits}: parameters' versions")
    w = torch.nn.Parameter(_randn(16, 64, seed=1).to(d))
    other = torch.nn.Parameter(torch.ones(5, device=d))
    x = _randn(4, 64, seed=2).to(d).requires_grad_()
    y = (x @ w.t()).square().sum()
    opt = dg.AdamW([w, other], state_bits=bits)
    y.backward(retain_graph=True)
    opt.step()
    assert w._version == 1 and other._version == 0           # no gradient, not written
    with pytest.raises(RuntimeError, match="inplace"):
        y.backward()
    (x @ w.t()).square().sum().backward()                    # a new pass takes the new weights
    p = torch.zeros(8, device=d)
    with torch.inference_mode():
        q, g = torch.zeros(8, device=d), torch.ones(8, device=d)
        dg.nf4_adamw_step([q], [g], dg.AdamWState([8], bits, d), lr=1e-3)
    dg.nf4_adamw_step([p], [torch.ones(8, device=d)], dg.AdamWState([8], bits, d), lr=1e-3)
    torch.cuda.synchronize()
    assert torch.equal(p, q) and p._version == 1
