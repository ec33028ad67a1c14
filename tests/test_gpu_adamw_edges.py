"""GPU: 8-bit moments of gradients that differ by many binades within a block, and of a very long tensor."""
import pytest
import torch

from tests import _adam_oracle as A
from tests import _ops_oracle as R
from tests._gpu import dev, lib, note

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _mixed(n, outlier, rest, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, generator=g) * torch.where(torch.arange(n) % 256 == 0, outlier, rest)


@pytest.mark.parametrize("outlier,rest", [(1.0, 1e-6), (0.1, 1e-7), (0.1, 1e-6), (1.0, 1e-5), (1.0, 1e-3), (1.0, 0.0)])
def test_updates_stay_bounded_beside_an_outlier(outlier, rest):
    """One large gradient a block: the small ones' steps stay of the learning rate's size (A.BOUND)."""
    dg, d = lib(), dev()
    note(f"adamw 8-bit: outliers of {outlier} among {rest}")
    n, lr = 1000, 1e-3
    st, worst = dg.AdamWState([n], 8, d), 0.0
    for t in range(1, 301):
        p = torch.zeros(n, device=d)
        dg.nf4_adamw_step([p], [_mixed(n, outlier, rest, t).to(d)], st, lr=lr, step=t, seed=t)
        worst = max(worst, float(p.abs().max()) / lr)
    assert worst < A.BOUND, worst


def test_codes_beside_an_outlier():
    """The codes of the definition: a root that is not zero takes no code of zero, a zero one does."""
    dg, d = lib(), dev()
    note("adamw 8-bit: codes beside an outlier")
    n, k = 700, {"lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "weight_decay": 0.0}
    g = _mixed(n, 1.0, 1e-5, 1)
    g[5:40] = 0.0
    st, p = dg.AdamWState([n], 8, d), torch.zeros(n, device=d)
    dg.nf4_adamw_step([p], [g.to(d)], st, step=1, seed=9, **k)
    torch.cuda.synchronize()
    _, m, v = R.adamw(torch.zeros(n), g, torch.zeros(n), torch.zeros(n), {**k, "step": 1})
    h = R.random_bits(0, 9, n)
    got = st.v.cpu().float().double()
    want, _ = A.encode_root(v.sqrt(), h >> 16)
    assert int((got != want).sum()) <= 1          # a value at the edge of its random rounding
    assert (got[5:40] == 0).all() and (got[:5] > 0).all() and (got[n:] == 0).all()
    want, _ = R.encode_state(m, h & 0xFFFF)
    assert int((st.m.cpu().float().double() != want).sum()) <= 1


def test_8bit_element_indexes_past_32_bits():
    """Past element 2^32 the random bits take the key that holds the index's high half."""
    dg, d = lib(), dev()
    note("adamw 8-bit: 2^32 + 1000 elements")
    n, tail = (1 << 32) + 1000, 1000
    k = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "weight_decay": 0.0}
    p, g = torch.zeros(n, dtype=BF, device=d), torch.zeros(n, dtype=BF, device=d)
    gt = (torch.randn(tail, generator=torch.Generator().manual_seed(3)) * 1e-2).to(BF)
    g[-tail:] = gt.to(d)
    st = dg.AdamWState([n], 8, d)
    dg.nf4_adamw_step([p], [g], st, step=1, seed=77, **k)
    torch.cuda.synchronize()
    _, m, v = R.adamw(torch.zeros(tail), gt, torch.zeros(tail), torch.zeros(tail), {**k, "step": 1})
    key = R.mix((R.mix(77) + 0x11D5D725) & 0xFFFFFFFF)
    h = R.mix((torch.arange(tail, dtype=torch.int64) + key) & 0xFFFFFFFF)
    lo = 1 << 32
    want, _ = R.encode_state(m, h & 0xFFFF)
    assert int((st.m[lo:].cpu().float().double() != want).sum()) <= 1
    want, _ = A.encode_root(v.sqrt(), h >> 16)
    assert int((st.v[lo:].cpu().float().double() != want).sum()) <= 1
    assert not st.m[:lo].view(torch.int64).any() and not st.v[:lo].view(torch.int64).any()
    del st, p, g
    torch.cuda.empty_cache()
