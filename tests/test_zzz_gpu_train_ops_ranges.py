"""The grouped products and the checkpoints at the far ends of their documented
ranges: long contractions and segments, calls without rows (bounds as in
train_ops_ref, derived beside each test where they are tighter)."""
import numpy as np
import pytest
import torch

import moe_synth as ms
from gpu_common import gpu_inputs, np64
from test_zzz_gpu_train_ops import DT, _close, _dev, _offsets, _randn

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


def _poison(nbytes):
    """Leaves blocks that are not zero for the allocator to give out again."""
    junk = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in (nbytes, nbytes + 256, 512, 1 << 20) for _ in range(8)]
    torch.cuda.synchronize()
    del junk


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_status_of_calls_without_rows(moe, dtype):
    """Nothing ran, so nothing was reported."""
    w = _randn(1, (3, 16, 24), DT[dtype])
    x, dy = torch.empty(0, 24, dtype=DT[dtype], device="cuda"), torch.empty(0, 16, dtype=DT[dtype], device="cuda")
    off, dt = _dev([0, 0, 0, 0]), moe.DTYPE_BF16 if dtype == "bf16" else moe.DTYPE_F32
    _poison(moe.moe_grouped_workspace_size(3, 16, 24, 0, dt))
    op = moe.GroupedLinear(w, 0)
    op.forward(x, off)
    assert op.device_status() == 0
    op = moe.GroupedLinear(w, 0)
    op.input_grad(dy, off)
    assert op.device_status() == 0
    _poison(moe.moe_grouped_wgrad_workspace_size(3, 16, 24, 0, dt))
    side = torch.cuda.Stream()
    for stream in (None, side):
        op = moe.GroupedLinear(w, 0)
        op.weight_grad(x, dy, off, stream=stream)
        assert op.device_status(stream=stream) == 0


@pytest.mark.parametrize("name", ["glm_small_bf16", "glam_tiny_f32"])
def test_status_of_a_layer_without_tokens(moe, name):
    cfg = ms.get_config(name)
    inp = gpu_inputs(cfg)
    layer = moe.MoELayer(cfg, inp, T=0)
    ck, x = moe.LayerCheckpoint(layer), inp["x"][:0]
    _poison(moe.moe_backward_saved_workspace_size(layer.desc))
    _poison(moe.moe_forward_save_workspace_size(layer.desc))
    layer.forward(x, checkpoint=ck)
    layer.backward(x, x, checkpoint=ck)
    assert layer.device_status() == 0 and layer.backward_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G", [1, 1024])
def test_bias_gradients_of_long_segments(moe, G, dtype):
    """One large row and 10^5 small ones whose last bits the large one's sum does
    not hold: at most 128 rounded additions in a row, and one for each 128 rows
    behind them (added up in one order for all the segment's shares), not one
    for each row.  1024 experts, all but one of them empty, are summed in one
    share."""
    rows, N, K = 100_000, 8, 8
    counts = np.zeros(G, np.int64)
    counts[G // 2] = rows
    dy = torch.full((rows, N), 1.0078125, dtype=DT[dtype], device="cuda")
    dy[0] = 2.0 ** 17
    x, w = torch.zeros((rows, K), dtype=DT[dtype], device="cuda"), torch.zeros((G, N, K), dtype=DT[dtype], device="cuda")
    db = moe.GroupedLinear(w, rows).weight_grad(x, dy, _dev(_offsets(counts)), db=True)[1]
    want = np.zeros((G, N))
    want[G // 2] = np64(dy).sum(0)
    _close(db, want, (128 + rows / 128) * 2.0 ** -24 * np.abs(want), "db")
