"""The second moment's 8-bit rounding in 64 bits (CPU), beside the definitions in _ops_oracle."""
import torch

from tests import _ops_oracle as R

# With exact moments |update| / lr stays near 1 for gradients of a steady size (1.1 at the most over some
# hundred steps).  Rounding leaves a root at least half its value (a step of the grid below 2 steps, and no
# root at zero) and a moment at most twice its value or its block's smallest code: a factor of 2 each.
BOUND = 4.5


def encode_root(x, u16):
    """As R.encode_state for a root: one that is not zero takes at least the smallest code."""
    q, scale = R.encode_state(x, u16)
    n = torch.zeros_like(q)
    n[:x.numel()] = x
    least = (n > 0) & (scale.repeat_interleave(256) > 0)
    return torch.where(least, q.clamp(min=2.0 ** -9), q), scale
