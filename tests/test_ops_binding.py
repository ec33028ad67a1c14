"""CPU: how the binding reaches the native module."""
import torch

import dequant_gemm_amd as dg
from dequant_gemm_amd import _ops


def test_quantize_into_buffers_goes_through_the_native_module(monkeypatch):
    """There the operands' device is made current before the launch, whichever was."""
    calls = []

    class Host:
        @staticmethod
        def fp8_quantize(*args):
            calls.append(args)
            return args[4], args[5]

    monkeypatch.setattr(_ops, "_host", lambda: Host)
    x = torch.zeros(5, 200)
    out = dg.FP8Tensor.empty(5, 200, 1, "e5m2", "cpu")
    assert dg.nf4_fp8_quantize(x, out=out) is out
    (args,) = calls
    assert args[0] is x and args[1] == 1 and args[4] is out.data and args[5] is out.scale
