"""The grouped products and the checkpoints at the far ends of their documented
ranges: long contractions and segments, calls without rows (bounds as in
train_ops_ref, derived beside each test where they are tighter)."""
import numpy as np
import pytest
import torch

import moe_synth as ms
import train_ops_ref as ref
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


@pytest.mark.parametrize("dtype,out", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
def test_several_chunks_and_several_tiles(moe, dtype, out):
    """Accumulators taken out one to three times a tile, and several tiles for
    each pair of processors: what a tile leaves (the accumulator that is next,
    the store buffers, the prefetch a tile ahead) is carried to the next one."""
    counts = [600, 1100, 0, 64, 1, 513] if dtype == "bf16" else [600, 0, 65]
    offsets, N, K = _offsets(counts), 1032, 1544
    rows, G = int(offsets[-1]), len(counts)
    x, dy, w = _randn(1, (rows, K), DT[dtype]), _randn(2, (rows, N), DT[dtype]), _randn(3, (G, N, K), DT[dtype], K ** -0.5)
    off, op = _dev(offsets), moe.GroupedLinear(w, rows, out_dtype=DT[out])
    hx, hdy, hw = np64(x), np64(dy), np64(w)
    want, m = ref.grouped_gemm(hx, hw, None, offsets, np.zeros((rows, N)))
    _close(op.forward(x, off), want, ref.gamma(K, out) * m + ref.U[out] * np.abs(want), "y")
    want, m = ref.grouped_dgrad(hdy, hw, offsets, np.zeros((rows, K)))
    _close(op.input_grad(dy, off), want, ref.gamma(N, out) * m + ref.U[out] * np.abs(want), "dx")
    dw0, db0 = _randn(5, (G, N, K), torch.float32), _randn(6, (G, N), torch.float32)
    for add in (False, True):
        base = (np64(dw0), np64(db0)) if add else (None, None)
        ww, wb, mw, mb = ref.grouped_wgrad(hx, hdy, offsets, *base)
        dw, db = op.weight_grad(x, dy, off, dw=dw0.clone(), db=db0.clone(), accumulate=add)
        _close(dw, ww, (ref.gamma(max(counts), "f32") + 2.0 ** -24) * mw, "dw")
        _close(db, wb, (128 + max(counts) / 128 + 9) * 2.0 ** -24 * mb, "db")
    assert op.device_status() == 0


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_chunks_of_claimed_tiles(moe, out):
    """Many narrow experts and a long one: the pairs of processors claim their
    tiles from the counter, with two and three accumulators a tile."""
    counts = [1 + 13 * g % 40 for g in range(60)] + [700]
    offsets, N, K = _offsets(counts), 1288, 584   # 21 and 10 blocks of 64 terms
    rows, G = int(offsets[-1]), len(counts)
    x, dy, w = _randn(1, (rows, K), torch.bfloat16), _randn(2, (rows, N), torch.bfloat16), _randn(3, (G, N, K), torch.bfloat16, K ** -0.5)
    off, op = _dev(offsets), moe.GroupedLinear(w, rows, out_dtype=DT[out])
    for _ in range(3):
        want, m = ref.grouped_gemm(np64(x), np64(w), None, offsets, np.zeros((rows, N)))
        _close(op.forward(x, off), want, ref.gamma(K, out) * m + ref.U[out] * np.abs(want), "y")
        want, m = ref.grouped_dgrad(np64(dy), np64(w), offsets, np.zeros((rows, K)))
        _close(op.input_grad(dy, off), want, ref.gamma(N, out) * m + ref.U[out] * np.abs(want), "dx")
    assert op.device_status() == 0


@pytest.mark.parametrize("direction", ["forward", "input_grad"])
@pytest.mark.parametrize("counts", [[64 + g % 5 for g in range(40)], [1 + 13 * g % 40 for g in range(40)], [600]])
def test_long_contractions_over_several_tiles(moe, counts, direction):
    """bf16 outputs of three accumulators a tile and several tiles a pair of
    processors, in fixed rounds and claimed, the last block of the sum a partial one."""
    G, width, long = len(counts), 264, 2 * 8192 + 72
    offsets = _offsets(counts)
    rows = int(offsets[-1])
    forward = direction == "forward"
    x = _randn(1, (rows, long), torch.bfloat16)
    w = _randn(2, (G, width, long) if forward else (G, long, width), torch.bfloat16, long ** -0.5)
    bias = _randn(3, (G, width), torch.bfloat16) if forward else None
    op = moe.GroupedLinear(w, rows, bias=bias)
    for _ in range(2):
        got = op.forward(x, _dev(offsets)) if forward else op.input_grad(x, _dev(offsets))
        for g in range(G):
            r = slice(int(offsets[g]), int(offsets[g + 1]))
            a, b = x[r].double(), w[g].double().T if forward else w[g].double()
            want, m = a @ b, a.abs() @ b.abs()
            if forward:
                want, m = want + bias[g].double(), m + bias[g].double().abs()
            # as ref.gamma of 8192 terms, one rounded addition for each such part, and the rounding to bf16
            bound = (ref.gamma(8192, "bf16") + 4 * 2.0 ** -24) * m + ref.U["bf16"] * want.abs()
            assert bool(((got[r].double() - want).abs() <= bound).all()), g
    assert op.device_status() == 0


@pytest.mark.parametrize("rows", [1 << 31, (1 << 32) + 4])
def test_rows_that_32_bits_do_not_hold(moe, rows):
    with pytest.raises(ValueError, match="32-bit"):
        moe.GroupedLinear(_randn(1, (2, 16, 24), torch.bfloat16), rows)
