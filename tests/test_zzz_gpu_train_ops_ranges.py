"""The grouped products and the checkpoints at the far ends of their documented
ranges: long contractions, many weight rows, long segments, huge values, calls
without rows (bounds as in train_ops_ref, derived beside each test where they
are tighter)."""
import numpy as np
import pytest
import torch

import train_ops_ref as ref
from gpu_common import np64
from test_zzz_gpu_train_ops import _close, _dev, _offsets, _randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import sparse_mixture_experts_logits_b200 as m
    return m


def _positive(seed, shape):
    """bf16 values in [1, 2): every partial sum keeps its sign, so that truncated additions add up."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.rand(shape, device="cuda", generator=g) + 1).to(torch.bfloat16)


@pytest.mark.parametrize("long", [1 << 14, 1 << 22])
@pytest.mark.parametrize("direction", ["forward", "input_grad"])
def test_long_contractions_in_bf16(moe, direction, long):
    """A bf16 output is off by its rounding, and not by how long its sum is.

    At most 512 truncated steps of 16 products (3 * 2^-23 of the magnitudes
    each), one rounded addition for each 8192 terms, and the rounding to bf16."""
    x = _positive(1, (3, long))
    if direction == "forward":
        w = _positive(2, (1, 8, long))
        want = np64(x) @ np64(w[0]).T
        got = moe.GroupedLinear(w, 3).forward(x, _dev([0, 3]))
    else:
        w = _positive(2, (1, long, 8))
        want = np64(x) @ np64(w[0])
        got = moe.GroupedLinear(w, 3).input_grad(x, _dev([0, 3]))
    bound = (3 * 512 * 2.0 ** -23 + (long / 8192 + 1) * 2.0 ** -24 + 2.0 ** -8) * np.abs(want)
    _close(got, want, bound, direction)
