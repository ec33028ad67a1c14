"""GPU: a copy of the optimizer and its parameters steps as the original does, and apart from it."""
import copy

import pytest
import torch

from tests._gpu import dev, lib, note

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [8, 32])
def test_a_copy_steps_alike_and_apart(bits):
    dg, d = lib(), dev()
    note(f"optimizer, {bits}-bit states: a deep copy")
    g = torch.Generator().manual_seed(1)
    model = torch.nn.ParameterList([torch.randn(300, generator=g).to(d, torch.bfloat16), torch.randn(40, 7, generator=g).to(d)])
    opt = dg.AdamW(list(model), lr=1e-2, state_bits=bits, seed=3)

    def step(ps, o, seed):
        h = torch.Generator().manual_seed(seed)
        for p in ps:
            p.grad = torch.randn(p.shape, generator=h).to(d, p.dtype)
        o.step()

    for i in range(3):
        step(model, opt, i)
    other, twin = copy.deepcopy((opt, model))
    kept = [p.detach().clone() for p in model]
    for i in range(3, 5):
        step(twin, other, i)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(model, kept))
    for i in range(3, 5):
        step(model, opt, i)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and not torch.equal(a, k) for a, b, k in zip(model, twin, kept))
