"""CPU: copies of the optimizer, and parameter groups it refuses (its step needs a GPU, its state does not)."""
import copy
import io

import pytest
import torch

import dequant_gemm_amd as dg


def _build(bits):
    ps = [torch.nn.Parameter(torch.randn(300, dtype=torch.bfloat16)), torch.nn.Parameter(torch.randn(7, 5))]
    opt = dg.AdamW([{"params": ps[:1], "lr": 1e-2}, {"params": ps[1:]}], state_bits=bits, seed=3)
    opt.calls = 4
    for g in range(2):
        for b in opt._buckets_of(g):
            for t in (b.state.m, b.state.v, b.state.m_scale, b.state.v_scale):
                if t is not None:
                    t.view(torch.uint8).random_(0, 100)
            for i, p in enumerate(b.params):
                b.steps[i] = opt.state[p]["step"] = 4
    return ps, opt


def _moments(opt):
    return [[m for b in opt._buckets_of(g) for i in range(len(b.params)) for m in b.state.moments(i)]
            for g in range(len(opt.param_groups))]


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("how", ["deepcopy", "saved"])
def test_a_copy_goes_on_by_itself(bits, how):
    ps, opt = _build(bits)
    if how == "deepcopy":
        other = copy.deepcopy(opt)
    else:
        f = io.BytesIO()
        torch.save(opt, f)
        f.seek(0)
        other = torch.load(f, weights_only=False)
    assert (other.state_bits, other.seed, other.calls) == (bits, 3, 4)
    a, b = _moments(opt), _moments(other)
    for x, y in zip(a, b):
        assert len(x) == len(y) and all(torch.equal(s, t) and s.data_ptr() != t.data_ptr() for s, t in zip(x, y))
    for g, (mine, its) in enumerate(zip(opt.param_groups, other.param_groups)):
        assert mine["lr"] == its["lr"]
        for bucket in other._buckets_of(g):
            assert bucket.steps == [4] * len(bucket.params)
            # the copy's own parameters, and views of the buffers that its steps write
            assert {id(p) for p in bucket.params} <= {id(p) for p in its["params"]}
            for i, p in enumerate(bucket.params):
                lo = bucket.state.starts[i]
                assert p is not mine["params"][i] and other.state[p]["step"] == 4
                assert other.state[p]["exp_avg"].data_ptr() == bucket.state.m[lo:].data_ptr()
    saved = other.state_dict()
    opt.load_state_dict(saved)
    assert all(torch.equal(s, t) for x, y in zip(_moments(opt), b) for s, t in zip(x, y))


def test_a_copy_made_before_the_first_step():
    p = torch.nn.Parameter(torch.zeros(3))
    other = copy.deepcopy(dg.AdamW([p], state_bits=8))
    assert all(not m.any() for x in _moments(other) for m in x)


def test_a_refused_group_is_not_added():
    p = torch.nn.Parameter(torch.zeros(3))
    opt = dg.AdamW([p])
    for bad, kind in ((torch.zeros(3, dtype=torch.float16), TypeError), (torch.zeros(4, 3).t(), ValueError)):
        with pytest.raises(kind):
            opt.add_param_group({"params": [torch.nn.Parameter(bad)]})
        assert len(opt.param_groups) == 1 and len(opt._buckets) == 1
    q = torch.nn.Parameter(torch.ones(2))
    opt.add_param_group({"params": q, "lr": 0.5})
    assert len(opt._buckets) == 2 and [list(b.params) for b in opt._buckets_of(1)] == [[q]]
