"""The 8-bit moments' definition on the CPU: updates stay bounded where a block's gradients differ widely."""
import pytest
import torch

from tests import _adam_oracle as A
from tests import _ops_oracle as R


def _worst(encode, outlier, rest, steps=250, n=256):
    g = torch.Generator().manual_seed(0)
    k = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "weight_decay": 0.0}
    size = torch.full((n,), rest, dtype=torch.float64)
    size[0] = outlier
    m, v, worst = torch.zeros(n).double(), torch.zeros(n).double(), 0.0
    for t in range(1, steps + 1):
        p, m, v = R.adamw(torch.zeros(n), torch.randn(n, generator=g).double() * size, m, v, {**k, "step": t})
        worst = max(worst, float(p.abs().max()) / k["lr"])
        h = R.random_bits(0, t, n)
        (qm, sm), (qv, sv) = R.encode_state(m, h & 0xFFFF), encode(v.sqrt(), h >> 16)
        m, v = qm * sm, (qv * sv) ** 2
    return worst


@pytest.mark.parametrize("outlier,rest", [(1.0, 1e-6), (0.1, 1e-7), (0.1, 1e-6), (1.0, 1e-5), (1.0, 1e-3), (1.0, 0.0)])
def test_updates_stay_bounded(outlier, rest):
    assert _worst(A.encode_root, outlier, rest) < A.BOUND


def test_a_root_rounded_to_zero_would_not():
    assert _worst(R.encode_state, 1.0, 1e-6) > 100


def test_only_roots_below_the_smallest_code_differ():
    x = torch.rand(4096, generator=torch.Generator().manual_seed(1)).double() ** 8
    x[100:200] = 0
    u = R.random_bits(0, 1, 4096) >> 16
    (a, sa), (b, sb) = R.encode_state(x, u), A.encode_root(x, u)
    n = x / sa.repeat_interleave(256)
    assert torch.equal(sa, sb) and torch.equal(a[n >= 2.0 ** -9], b[n >= 2.0 ** -9])
    assert (b[(n > 0) & (n < 2.0 ** -9)] == 2.0 ** -9).all() and (b[x == 0] == 0).all()
