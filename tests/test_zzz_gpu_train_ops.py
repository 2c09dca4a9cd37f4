"""The grouped products and the 8-bit checkpoints on the GPU against 64-bit
references, element by element (bounds derived in train_ops_ref)."""
import numpy as np
import pytest
import torch

import train_ops_ref as ref
from gpu_common import np64

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def moe():
    import sparse_mixture_experts_logits_b200 as m
    return m


def _randn(seed, shape, dtype, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=g) * std).to(dtype)


def _offsets(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)


def _dev(offsets):
    return torch.tensor(np.asarray(offsets), dtype=torch.int32, device="cuda")


def _close(got, want, bound, what):
    got = np64(got)
    assert np.isfinite(got).all(), what
    over = np.abs(got - want) - bound
    i = np.unravel_index(np.argmax(over), over.shape)
    assert over[i] <= 0, f"{what}: at {i} {got[i]} against {want[i]}, off by {abs(got[i] - want[i])}, bound {bound[i]}"


# (counts of each expert, rows behind the last segment, N, K)
SHAPES = [
    ([1], 0, 8, 8),
    ([0, 1, 0, 2, 0], 3, 16, 24),
    ([63, 64, 65, 1, 0, 127], 1, 72, 136),
    ([255, 256, 257, 17], 0, 264, 520),
    ([5, 700, 0, 3], 9, 520, 1032),
    ([0, 0, 0], 4, 40, 64),
    ([1] * 40, 0, 256, 512),
    ([33], 0, 2056, 40),
    ([1111], 0, 24, 4104),
    ([3, 0, 90], 2, 7, 13),           # widths that TMA cannot address
    ([20, 64, 1], 0, 130, 65),
]


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_grouped_products(moe, shape, dtype, out):
    counts, extra, N, K = SHAPES[shape]
    offsets = _offsets(counts)
    rows, G = int(offsets[-1]) + extra, len(counts)
    x, dy = _randn(1, (rows, K), DT[dtype]), _randn(2, (rows, N), DT[dtype])
    w, bias = _randn(3, (G, N, K), DT[dtype], K ** -0.5), _randn(4, (G, N), DT[dtype])
    x[offsets[-1]:] = float("nan")    # rows of nobody: not read ...
    dy[offsets[-1]:] = float("nan")
    y = torch.full((rows, N), 7.0, dtype=DT[out], device="cuda")   # ... and not written
    dx = torch.full((rows, K), 7.0, dtype=DT[out], device="cuda")
    off = _dev(offsets)
    hx, hdy = np64(x), np64(dy)
    hx[offsets[-1]:] = 0
    hdy[offsets[-1]:] = 0
    for b in (None, bias):
        op = moe.GroupedLinear(w, rows, bias=b, out_dtype=DT[out])
        y.fill_(7.0)
        assert op.forward(x, off, y=y) is y
        want, m = ref.grouped_gemm(hx, np64(w), None if b is None else np64(b), offsets, np.full((rows, N), 7.0))
        _close(y, want, ref.gamma(K, out) * m + ref.U[out] * np.abs(want) * (m > 0), "y")
    assert op.input_grad(dy, off, dx=dx) is dx
    want, m = ref.grouped_dgrad(hdy, np64(w), offsets, np.full((rows, K), 7.0))
    _close(dx, want, ref.gamma(N, out) * m + ref.U[out] * np.abs(want) * (m > 0), "dx")
    longest = max(counts)
    dw, db = op.weight_grad(x, dy, off, db=True)
    ww, wb, mw, mb = ref.grouped_wgrad(hx, hdy, offsets)
    _close(dw, ww, ref.gamma(longest, "f32") * mw, "dw")
    _close(db, wb, (longest + 8) * 2.0 ** -24 * mb, "db")
    for g, c in enumerate(counts):    # an expert without rows gets zeros
        assert c > 0 or not dw[g].any()
    # added onto what is there
    dw0, db0 = _randn(5, (G, N, K), torch.float32), _randn(6, (G, N), torch.float32)
    ww, wb, mw, mb = ref.grouped_wgrad(hx, hdy, offsets, np64(dw0), np64(db0))
    dw, db = dw0.clone(), db0.clone()
    got = op.weight_grad(x, dy, off, dw=dw, db=db, accumulate=True)
    assert got[0] is dw and got[1] is db
    _close(dw, ww, (ref.gamma(longest, "f32") + 2.0 ** -24) * mw, "dw added")
    _close(db, wb, (longest + 9) * 2.0 ** -24 * mb, "db added")
    for g, c in enumerate(counts):
        assert c > 0 or torch.equal(dw[g], dw0[g])
    assert op.device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_bad_expert_stays_alone(moe, dtype):
    """NaN and infinity in one expert's rows reach no other expert's results,
    although the experts share 64-row blocks of the contraction."""
    counts = [5, 30, 70, 1, 64, 9]
    offsets = _offsets(counts)
    rows, N, K = int(offsets[-1]), 72, 80
    x, dy, w = _randn(1, (rows, K), DT[dtype]), _randn(2, (rows, N), DT[dtype]), _randn(3, (6, N, K), DT[dtype])
    off = _dev(offsets)
    op = moe.GroupedLinear(w, rows)
    clean = op.forward(x, off), op.input_grad(dy, off), *op.weight_grad(x, dy, off, db=True)
    for bad in (1, 3):
        b, e = offsets[bad], offsets[bad + 1]
        x2, dy2 = x.clone(), dy.clone()
        x2[b:e] = float("nan")
        dy2[b:e] = float("inf")
        y, dx, (dw, db) = op.forward(x2, off), op.input_grad(dy2, off), op.weight_grad(x2, dy2, off, db=True)
        keep = [g for g in range(6) if g != bad]
        rest = torch.cat([torch.arange(offsets[g], offsets[g + 1]) for g in keep])
        assert torch.equal(y[rest], clean[0][rest]) and torch.equal(dx[rest], clean[1][rest])
        assert torch.equal(dw[keep], clean[2][keep]) and torch.equal(db[keep], clean[3][keep])
        assert y[b:e].isnan().all() and dw[bad].isnan().all() and db[bad].isinf().all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,K", [(72, 80), (8, 136), (200, 264)])
def test_bad_weights_stay_alone(moe, N, K, dtype):
    """NaN and infinity in one expert's weights and bias reach no other expert's
    rows, although the contraction over N ends inside a block of 64."""
    counts = [5, 30, 70, 1, 64, 9]
    offsets = _offsets(counts)
    rows = int(offsets[-1])
    x, dy = _randn(1, (rows, K), DT[dtype]), _randn(2, (rows, N), DT[dtype])
    w, bias = _randn(3, (6, N, K), DT[dtype]), _randn(4, (6, N), DT[dtype])
    off = _dev(offsets)
    op = moe.GroupedLinear(w, rows, bias=bias)
    clean = op.forward(x, off), op.input_grad(dy, off)
    for bad, value in ((1, float("nan")), (3, float("inf")), (5, -float("inf"))):
        w2, bias2 = w.clone(), bias.clone()
        w2[bad], bias2[bad] = value, value
        op2 = moe.GroupedLinear(w2, rows, bias=bias2)
        y, dx = op2.forward(x, off), op2.input_grad(dy, off)
        b, e = offsets[bad], offsets[bad + 1]
        rest = torch.cat([torch.arange(0, b), torch.arange(e, rows)])
        assert torch.equal(y[rest], clean[0][rest]) and torch.equal(dx[rest], clean[1][rest])
        assert not y[b:e].isfinite().any() and not dx[b:e].isfinite().any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_that_are_no_dispatch_stay_inside(moe, dtype):
    """Bounds outside [0, rows] are clamped, a segment that ends before it starts is empty."""
    rows, N, K = 100, 40, 48
    offsets = [-5, 30, 20, 60, 1000]
    x, dy, w = _randn(1, (rows, K), DT[dtype]), _randn(2, (rows, N), DT[dtype]), _randn(3, (4, N, K), DT[dtype])
    op = moe.GroupedLinear(w, rows, out_dtype=torch.float32)
    off = _dev(offsets)
    # rows of two segments (20..30 of groups 0 and 2) get one of the two results: left out
    y = op.forward(x, off, y=torch.zeros(rows, N, device="cuda"))
    want, m = ref.grouped_gemm(np64(x), np64(w), None, offsets, np.zeros((rows, N)))
    ok = np.r_[0:20, 30:rows]
    _close(y[torch.from_numpy(ok)], want[ok], ref.gamma(K, "f32") * m[ok], "y")
    dw, db = op.weight_grad(x, dy, off, db=True)
    ww, wb, mw, mb = ref.grouped_wgrad(np64(x), np64(dy), offsets)
    _close(dw, ww, ref.gamma(rows, "f32") * mw, "dw")
    _close(db, wb, (rows + 8) * 2.0 ** -24 * mb, "db")


def test_as_many_experts_as_there_can_be(moe):
    """1024 experts of zero to three rows."""
    counts = np.arange(1024) * 7 % 4
    offsets, N, K = _offsets(counts), 24, 40
    rows = int(offsets[-1])
    x, dy, w = _randn(1, (rows, K), torch.bfloat16), _randn(2, (rows, N), torch.bfloat16), _randn(3, (1024, N, K), torch.bfloat16)
    op = moe.GroupedLinear(w, rows, out_dtype=torch.float32)
    off = _dev(offsets)
    want, m = ref.grouped_gemm(np64(x), np64(w), None, offsets, np.zeros((rows, N)))
    _close(op.forward(x, off), want, ref.gamma(K, "f32") * m, "y")
    dw, db = op.weight_grad(x, dy, off, db=True)
    ww, wb, mw, mb = ref.grouped_wgrad(np64(x), np64(dy), offsets)
    _close(dw, ww, ref.gamma(3, "f32") * mw, "dw")
    _close(db, wb, 11 * 2.0 ** -24 * mb, "db")
    with pytest.raises(moe.MoEError):
        moe.GroupedLinear(_randn(3, (1025, 8, 8), torch.bfloat16), rows)


def test_rows_behind_two_billion_elements(moe):
    """Element offsets past 32 bits, in the rows and in the segments."""
    K, N, rows = 8192, 16, 270_000
    x = torch.empty((rows, K), dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    w = _randn(3, (2, N, K), torch.bfloat16, K ** -0.5)
    offsets = [0, rows - 100, rows - 3]
    op = moe.GroupedLinear(w, rows, out_dtype=torch.float32)
    off = _dev(offsets)
    y = op.forward(x, off, y=torch.full((rows, N), 7.0, device="cuda"))
    for r in (0, 262_143, 262_145, rows - 101, rows - 100, rows - 4):
        want = np64(x[r]) @ np64(w[int(r >= offsets[1])]).T
        m = np.abs(np64(x[r])) @ np.abs(np64(w[int(r >= offsets[1])])).T
        _close(y[r], want, ref.gamma(K, "f32") * m, f"y[{r}]")
    assert y[rows - 3:].eq(7).all()
    dy = torch.zeros((rows, N), dtype=torch.bfloat16, device="cuda")
    dy[rows - 50, 3] = 1.0
    dw, _ = op.weight_grad(x, dy, off)
    assert not dw[0].any() and torch.equal(dw[1, 3], x[rows - 50].float())
    dy = _randn(4, (rows, N), torch.bfloat16)
    dx = moe.GroupedLinear(w, rows).input_grad(dy, off)
    want = np64(dy[rows - 4]) @ np64(w[1])
    m = np.abs(np64(dy[rows - 4])) @ np.abs(np64(w[1]))
    _close(dx[rows - 4], want, ref.gamma(N, "bf16") * m + ref.U["bf16"] * np.abs(want), "dx")
    c = moe.RowCheckpoint(rows, K, torch.bfloat16)
    c.save(x)
    idx = torch.tensor([rows - 1, 262_145], dtype=torch.int32, device="cuda")
    assert np.array_equal(np64(c.load(idx)), ref.keep(np64(x[idx.long()]))[2])
    ck = moe.ActivationCheckpoint("gelu_tanh", rows, K, torch.bfloat16)
    a = ck.save(x)
    last = np64(x[-1:])
    _close(a[-1:], ref.act(last, False)[0], ref.act(last, False)[1] + ref.U["bf16"] * np.abs(last) + 1e-36, "a")
    dh, _, _ = ck.backward(a)
    v = ref.keep(last)[2]
    d, bd = ref.act_grad(v, False)
    ga = np64(a[-1:])
    _close(dh[-1:], ga * d, np.abs(ga) * bd + ref.U["bf16"] * np.abs(ga * d) + 1e-36, "dh")


def test_what_the_handles_refuse(moe):
    w = _randn(1, (2, 16, 24), torch.bfloat16)
    op = moe.GroupedLinear(w, 4)
    x, off = _randn(2, (4, 24), torch.bfloat16), _dev([0, 1, 4])
    odd = torch.zeros(4 * 24 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(4, 24)   # contiguous, off its boundary
    for bad in (x.float(), x[:3], x.cpu(), _randn(2, (24, 4), torch.bfloat16).t()):
        with pytest.raises(ValueError, match="x must be"):
            op.forward(bad, off)
    with pytest.raises(ValueError, match="offsets"):
        op.forward(x, off.long())
    with pytest.raises(ValueError, match="y must be"):
        op.forward(x, off, y=torch.empty(4, 16, device="cuda"))
    with pytest.raises(moe.MoEError):
        op.forward(odd, off)
    with pytest.raises(ValueError, match="accumulate"):
        op.weight_grad(x, _randn(3, (4, 16), torch.bfloat16), off, accumulate=True)
    with pytest.raises(ValueError, match="bias"):
        moe.GroupedLinear(w, 4, bias=torch.zeros(2, 16, device="cuda"))
    with pytest.raises(ValueError, match="weight"):
        moe.GroupedLinear(w.transpose(1, 2), 4)
    with pytest.raises(ValueError, match="dtype"):
        moe.GroupedLinear(w.half(), 4)
    with pytest.raises(moe.MoEError):
        moe.GroupedLinear(w.float(), 4, out_dtype=torch.bfloat16).forward(x.float(), off)
    ck = moe.ActivationCheckpoint("swiglu", 4, 12, torch.bfloat16)
    with pytest.raises(ValueError, match="h must be"):
        ck.save(_randn(1, (4, 12), torch.bfloat16))
    with pytest.raises(ValueError, match="da must be"):
        ck.backward(_randn(1, (4, 24), torch.bfloat16))
    with pytest.raises(ValueError, match="q must be"):
        moe.ActivationCheckpoint("swiglu", 4, 12, torch.bfloat16, q=torch.zeros(4, 12, dtype=torch.int8, device="cuda"))
    c = moe.RowCheckpoint(4, 24, torch.bfloat16)
    with pytest.raises(ValueError, match="row_index"):
        c.load(torch.zeros(2, 2, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("cols", [40, 33])
def test_a_checkpoint_without_rows(moe, cols):
    """Every index lies outside it: zero rows and the status."""
    c = moe.RowCheckpoint(0, cols, torch.bfloat16)
    c.save(torch.empty(0, cols, dtype=torch.bfloat16, device="cuda"))
    assert c.load().shape == (0, cols)
    out = torch.full((3, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    c.load(_dev([0, -1, 5]), out=out)
    assert not out.any() and c.status.item() != 0


@pytest.mark.parametrize("act", ["swiglu", "gelu_tanh"])
def test_checkpoints_off_their_boundaries(moe, act):
    """Contiguous tensors that start anywhere: the same bits as on whole boundaries."""
    rows, I = 5, 64
    width = 2 * I if act == "swiglu" else I

    def off(t):
        b = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
        b.copy_(t)
        return b

    h, da = _randn(1, (rows, width), torch.bfloat16), _randn(2, (rows, I), torch.bfloat16)
    a1 = moe.ActivationCheckpoint(act, rows, I, torch.bfloat16)
    a2 = moe.ActivationCheckpoint(act, rows, I, torch.bfloat16, q=off(a1.q), e=off(a1.e))
    assert torch.equal(a1.save(h), a2.save(off(h), a=off(h[:, :I].contiguous())))
    assert torch.equal(a1.q, a2.q) and torch.equal(a1.e, a2.e)
    for x, y in zip(a1.backward(da, wa=True), a2.backward(off(da), dh=off(h), wa=off(da))):
        assert (x is None and y is None) or torch.equal(x, y)
    c1, c2 = moe.RowCheckpoint(rows, width, torch.bfloat16), moe.RowCheckpoint(rows, width, torch.bfloat16)
    c1.save(h)
    c2.save(off(h))
    assert torch.equal(c1.q, c2.q) and torch.equal(c1.load(), c2.load(out=off(h)))


def test_a_stream_of_its_own(moe):
    """Calls on a given stream while the current one is busy: nothing they allocate waits for, or is written by, the
    current stream."""
    counts = [40, 0, 7, 100]
    offsets, N, K = _offsets(counts), 48, 88
    rows = int(offsets[-1])
    off, x, w, dy = _dev(offsets), _randn(1, (rows, K), torch.bfloat16), _randn(2, (4, N, K), torch.bfloat16), _randn(3, (rows, N), torch.bfloat16)
    op = moe.GroupedLinear(w, rows)
    want = op.forward(x, off), op.input_grad(dy, off), *op.weight_grad(x, dy, off, db=True)
    ck = moe.ActivationCheckpoint("gelu_tanh", rows, K, torch.bfloat16)
    kept = ck.save(x), ck.load(), *ck.backward(x, wa=True, dw=True)
    torch.cuda.synchronize()
    side, busy = torch.cuda.Stream(), torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        junk = [torch.full((rows, N), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(8)]
        for _ in range(40):
            busy.fill_(1)
        del junk
        op = moe.GroupedLinear(w, rows)
        ck = moe.ActivationCheckpoint("gelu_tanh", rows, K, torch.bfloat16)
        got = op.forward(x, off, stream=side), op.input_grad(dy, off, stream=side), *op.weight_grad(x, dy, off, db=True, stream=side)
        again = ck.save(x, stream=side), ck.load(stream=side), *ck.backward(x, wa=True, dw=True, stream=side)
        torch.cuda.synchronize()
        for g, v in zip(got + again, want + kept):
            assert torch.equal(g, v)
        assert op.device_status(stream=side) == 0


def test_no_rows(moe):
    w = _randn(1, (3, 16, 24), torch.bfloat16)
    op = moe.GroupedLinear(w, 0)
    off = _dev([0, 0, 0, 0])
    x, dy = torch.empty(0, 24, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 16, dtype=torch.bfloat16, device="cuda")
    assert op.forward(x, off).shape == (0, 16) and op.input_grad(dy, off).shape == (0, 24)
    dw, db = op.weight_grad(x, dy, off, db=True)
    assert not dw.any() and not db.any()
    dw, db = torch.ones(3, 16, 24, device="cuda"), torch.ones(3, 16, device="cuda")
    op.weight_grad(x, dy, off, dw=dw, db=db, accumulate=True)
    assert dw.eq(1).all() and db.eq(1).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_against_differences(moe, dtype):
    """y is linear in x, w and b: <dy, y(x + d) - y(x)> = <dx, d>, and the same
    for the weights and biases, with d and dy on a grid that bf16 holds and
    the outputs in fp32 (so that only the sums' bounds enter)."""
    counts = [40, 0, 7, 100]
    offsets, N, K = _offsets(counts), 48, 88
    rows = int(offsets[-1])
    off = _dev(offsets)
    x, d = _randn(1, (rows, K), DT[dtype]), _randn(2, (rows, K), DT[dtype])
    w, dwt = _randn(3, (4, N, K), DT[dtype]), _randn(4, (4, N, K), DT[dtype])
    b, dy = _randn(5, (4, N), DT[dtype]), _randn(6, (rows, N), DT[dtype])
    f = lambda xx, ww: np64(moe.GroupedLinear(ww, rows, bias=b, out_dtype=torch.float32).forward(xx, off))  # noqa: E731
    op = moe.GroupedLinear(w, rows, bias=b, out_dtype=torch.float32)
    dx, (dw, db) = op.input_grad(dy, off), op.weight_grad(x, dy, off, db=True)
    hdy = np64(dy)
    # the step itself is exact: y(d) - y(0) through the same operator
    lhs = (hdy * (f(d, w) - f(torch.zeros_like(d), w))).sum()
    mag = (np.abs(hdy) * ref.grouped_gemm(np.abs(np64(d)), np.abs(np64(w)), np.abs(np64(b)), offsets, np.zeros((rows, N)))[0]).sum()
    assert abs(lhs - (np64(dx) * np64(d)).sum()) <= 4 * ref.gamma(K, "f32") * mag
    lhs = (hdy * (f(x, dwt) - f(x, torch.zeros_like(w)))).sum()
    mag = (np.abs(hdy) * ref.grouped_gemm(np.abs(np64(x)), np.abs(np64(dwt)), np.abs(np64(b)), offsets, np.zeros((rows, N)))[0]).sum()
    assert abs(lhs - (np64(dw) * np64(dwt)).sum()) <= 4 * ref.gamma(K, "f32") * mag
    assert np.allclose(np64(db), ref.grouped_wgrad(np64(x), hdy, offsets)[1], rtol=0, atol=1e-4)


# ------------------------------------------------------------------ 8 bits
WIDTHS = [1, 7, 8, 31, 32, 33, 40, 64, 199, 256, 257, 511, 545, 1000, 2056]


def _special(rows, cols, dtype):
    """Rows of every kind: normal, zero, one large value, tiny, subnormal, powers of two, values that round to 128."""
    x = _randn(11, (rows, cols), torch.float32)
    kinds = [lambda v: v, lambda v: v * 0, lambda v: v * 1e30, lambda v: v * 1e-30, lambda v: v * 2e-39,
             lambda v: torch.exp2(v.mul(4).round()), lambda v: v.sign() * 1.9999, lambda v: v * 1.5e-36,
             lambda v: v.abs() * 3e38 / v.abs().max()]
    for r in range(rows):
        x[r] = kinds[r % len(kinds)](x[r])
    x[rows // 2, :1] = 500.0
    return x.to(dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", WIDTHS)
def test_rows_are_kept_exactly_as_defined(moe, cols, dtype):
    rows = 27
    x = _special(rows, cols, DT[dtype])
    c = moe.RowCheckpoint(rows, cols, DT[dtype])
    c.save(x)
    q, e, v = ref.keep(np64(x))
    assert np.array_equal(c.q.cpu().numpy(), q) and np.array_equal(c.e.cpu().numpy(), e)
    back = c.load()
    # (the rows of the last kind hold infinities: they read back as NaN)
    assert np.array_equal(np64(back), np64(torch.from_numpy(v).to(DT[dtype])), equal_nan=True)
    ex = np.repeat(e, 32, 1)[:, :cols]
    fine = ex < 255
    off = np.abs(v - np64(x))[fine]
    assert (off <= (np.where(np.abs(q) == 127, 1.0, 0.5) * np.ldexp(1.0, ex - 133))[fine]).all()
    idx = torch.tensor([5, 0, 5, rows - 1, -1, rows, 7], dtype=torch.int32, device="cuda")
    got = c.load(idx)
    assert np.array_equal(np64(got[[0, 1, 2, 3, 6]]), np64(back[[5, 0, 5, rows - 1, 7]]), equal_nan=True)
    assert not got[[4, 5]].any()
    assert c.status.item() == moe.DEVERR_BAD_ROW_TOKEN


def test_the_largest_and_smallest_values(moe):
    top = torch.finfo(torch.float32).max
    x = torch.zeros(6, 40, device="cuda")
    x[0, 3], x[1, :], x[2, 39] = top, -top, top / 2
    x[3, 0], x[3, 1], x[4, 5] = 2.0 ** -126, 2.0 ** -133, 2.0 ** -149
    c = moe.RowCheckpoint(6, 40, torch.float32)
    c.save(x)
    q, e, v = ref.keep(np64(x))
    assert np.array_equal(c.q.cpu().numpy(), q) and np.array_equal(c.e.cpu().numpy(), e)
    assert np.array_equal(np64(c.load()), v) and v[0, 3] == 127 * 2.0 ** 121 and v[3, 0] == 2.0 ** -126


@pytest.mark.parametrize("cols", [5, 40, 96])
def test_what_is_not_finite_reads_back_as_nan(moe, cols):
    for bad in (float("nan"), float("inf"), -float("inf")):
        x = _randn(1, (6, cols), torch.bfloat16)
        x[2, cols - 1] = bad
        c = moe.RowCheckpoint(6, cols, torch.bfloat16)
        c.save(x)
        got = np64(c.load())
        want = ref.keep(np64(x))[2]
        assert np.array_equal(got, want, equal_nan=True) and np.isnan(got[2, cols - 1])
        a = moe.ActivationCheckpoint("gelu_tanh", 6, cols, torch.bfloat16)
        a.save(x)
        dh, wa, dw = a.backward(torch.ones_like(x), wa=True, dw=True)
        assert np.array_equal(np.isnan(np64(dh)), np.isnan(want)) and np.array_equal(np.isnan(np64(wa)), np.isnan(want))
        assert np.array_equal(np.isnan(np64(dw)), np.isnan(want).any(1))


@pytest.mark.parametrize("act", ["swiglu", "gelu_tanh"])
@pytest.mark.parametrize("dtype,src", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("I", WIDTHS)
def test_activation_saved_and_its_gradient(moe, I, dtype, src, act):
    rows, sw = 19, act == "swiglu"
    h = _randn(21, (rows, 2 * I if sw else I), torch.float32, 2.5).to(DT[src])
    h[0] = 0
    h[1] *= 20
    h[2] *= 1e-3
    ck = moe.ActivationCheckpoint(act, rows, I, DT[dtype], DT[src])
    a = ck.save(h)
    want, bound = ref.act(np64(h), sw)
    _close(a, want, bound + ref.U[dtype] * np.abs(want) + 1e-36, "a")
    q, e, v = ref.keep(np64(h), 2 if sw else 1)
    assert np.array_equal(ck.q.cpu().numpy(), q) and np.array_equal(ck.e.cpu().numpy(), e)
    assert np.array_equal(np64(ck.load()), v)
    da, rw = _randn(22, (rows, I), DT[src]), _randn(23, (rows,), torch.float32).abs()
    for row_w in (None, rw):
        dh, wa, dw = ck.backward(da, row_w=row_w, wa=True, dw=True)
        wt = np.ones((rows, 1)) if row_w is None else np64(rw)[:, None]
        hda = np64(da)
        d, bd = ref.act_grad(v, sw)
        full = np.concatenate([hda, hda], 1) if sw else hda
        want = wt * full * d
        _close(dh, want, wt * np.abs(full) * bd + ref.U[dtype] * np.abs(want) + 1e-36, "dh")
        av, ba = ref.act(v, sw)
        _close(wa, wt * av, wt * ba + ref.U[dtype] * np.abs(wt * av) + 1e-36, "wa")
        mag = (np.abs(hda) * np.abs(av)).sum(1)
        _close(dw, (hda * av).sum(1), (np.abs(hda) * ba).sum(1) + (I + 8) * 2.0 ** -24 * mag + 1e-36, "dw")
    only, none, nodw = ck.backward(da, row_w=rw)
    assert none is None and nodw is None and torch.equal(only, dh)


@pytest.mark.parametrize("act", ["swiglu", "gelu_tanh"])
def test_activation_gradient_against_differences(moe, act):
    """Central differences of act around the kept values, in 64 bits: with a step of 2^-12
    their own error is under 2^-24 of the third derivative, which is below 4 in magnitude."""
    sw, rows, I = act == "swiglu", 4, 48
    h = _randn(31, (rows, 2 * I if sw else I), torch.float32, 1.5)
    ck = moe.ActivationCheckpoint(act, rows, I, torch.float32)
    ck.save(h)
    v, da = np64(ck.load()), _randn(32, (rows, I), torch.float32)
    dh = np64(ck.backward(da)[0])
    t = 2.0 ** -12
    for c in range(v.shape[1]):
        up, dn = v.copy(), v.copy()
        up[:, c] += t
        dn[:, c] -= t
        diff = (np64(da) * (ref.act(up, sw)[0] - ref.act(dn, sw)[0])).sum(1) / (2 * t)
        scale = np.abs(np64(da)).max() * max(1.0, np.abs(v).max())
        assert (np.abs(diff - dh[:, c]) <= scale * (4 * 2.0 ** -24 + 2.0 ** -17)).all()


def test_only_the_first_rows(moe):
    """n_rows on the device: the other rows stay as they were."""
    n = torch.tensor([5], dtype=torch.int32, device="cuda")
    for I in (40, 33):
        x = _randn(1, (9, I), torch.bfloat16)
        c = moe.RowCheckpoint(9, I, torch.bfloat16)
        c.q.fill_(77)
        c.e.fill_(99)
        c.save(x, n_rows=n)
        assert c.q[5:].eq(77).all() and c.e[5:].eq(99).all() and not c.e[:5].eq(99).any()
        out = torch.full((9, I), 3.0, dtype=torch.bfloat16, device="cuda")
        c.load(n_rows=n, out=out)
        assert out[5:].eq(3).all() and np.array_equal(np64(out[:5]), ref.keep(np64(x))[2][:5])
        for act in ("swiglu", "gelu_tanh"):
            h = _randn(2, (9, 2 * I if act == "swiglu" else I), torch.bfloat16)
            ck = moe.ActivationCheckpoint(act, 9, I, torch.bfloat16)
            ck.q.fill_(77)
            a = ck.save(h, a=torch.full((9, I), 3.0, dtype=torch.bfloat16, device="cuda"), n_rows=n)
            assert a[5:].eq(3).all() and ck.q[5:].eq(77).all() and not a[:5].eq(3).all()
            dh = torch.full_like(h, 3.0)
            dw = torch.full((9,), 3.0, device="cuda")
            _, wa, _ = ck.backward(_randn(3, (9, I), torch.bfloat16), dh=dh, wa=torch.full_like(a, 3.0), dw=dw, n_rows=n)
            assert dh[5:].eq(3).all() and wa[5:].eq(3).all() and dw[5:].eq(3).all() and not dw[:5].eq(3).any()


# ------------------------------------------------------------------ together
def _experts_step(moe, cfg, dev="cuda"):
    """The tensors and handles of one training step of the routed experts."""
    T, D, M, I, k = cfg["T"], cfg["D"], cfg["M"], cfg["I"], cfg["k"]
    pairs, bf = T * k, torch.bfloat16
    s = dict(cfg)
    s["x"], s["dy"] = _randn(41, (T, D), bf), _randn(42, (T, D), bf)
    s["w1"], s["w2"] = _randn(43, (M, 2 * I, D), bf, D ** -0.5), _randn(44, (M, D, I), bf, I ** -0.5)
    idx = torch.rand(T, M, generator=torch.Generator().manual_seed(45)).argsort(1)[:, :k].to(torch.int32).cuda()
    s["idx"], s["tw"] = idx.contiguous(), _randn(46, (T, k), torch.float32).abs().contiguous()
    s["up"], s["down"] = moe.GroupedLinear(s["w1"], pairs), moe.GroupedLinear(s["w2"], pairs, out_dtype=torch.float32)
    s["da_op"] = moe.GroupedLinear(s["w2"], pairs, out_dtype=torch.float32)
    s["dx_op"] = moe.GroupedLinear(s["w1"], pairs, out_dtype=torch.float32)
    s["ck_x"], s["ck_h"] = moe.RowCheckpoint(T, D, bf), moe.ActivationCheckpoint("swiglu", pairs, I, bf)
    s["ck_b"] = moe.ActivationCheckpoint("swiglu", pairs, I, bf, torch.float32, q=s["ck_h"].q, e=s["ck_h"].e)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device=dev)  # noqa: E731
    s["counts"], s["off"], s["slot"], s["tok"] = i32(M), i32(M + 1), i32(pairs), i32(pairs)
    s["rw"] = torch.zeros(pairs, device=dev)
    n = moe.moe_permute_workspace_size(T, k, M)
    s["pws"] = torch.zeros(n + 256, dtype=torch.uint8, device=dev)
    s["pws_n"] = n
    s["desc"] = moe.desc_from_config(dict(dtype="bf16", T=T, D=D, M=M, k=k, I=16, gate="softmax", act="swiglu"))  # for moe_combine,
    # which reads T, D and k of it
    s["xp"], s["dyp"] = torch.zeros(pairs, D, dtype=bf, device=dev), torch.zeros(pairs, D, dtype=bf, device=dev)
    return s


def _run_step(moe, s):
    T, D, M, k = s["T"], s["D"], s["M"], s["k"]
    pairs = T * k
    st = torch.cuda.current_stream().cuda_stream
    ws = s["pws"].data_ptr() + (-s["pws"].data_ptr()) % 256
    moe.moe_permute(s["idx"].data_ptr(), s["tw"].data_ptr(), T, k, M, s["counts"].data_ptr(), s["off"].data_ptr(),
                    s["slot"].data_ptr(), s["tok"].data_ptr(), s["rw"].data_ptr(), ws, s["pws_n"], st)
    gather = lambda src, dst: moe.moe_gather_rows(src.data_ptr(), s["tok"].data_ptr(), s["off"][M:].data_ptr(),  # noqa: E731
                                                  dst.data_ptr(), pairs, T, D, moe.DTYPE_BF16, None, st)
    # forward: what the backward needs is kept in 8 bits
    s["ck_x"].save(s["x"])
    gather(s["x"], s["xp"])
    a = s["ck_h"].save(s["up"].forward(s["xp"], s["off"]))
    o = s["down"].forward(a, s["off"])
    o = o * s["rw"][:, None]
    y = torch.empty_like(s["x"])
    moe.moe_combine(s["desc"], o.data_ptr(), s["slot"].data_ptr(), None, None, y.data_ptr(), st)
    # backward, from the checkpoints
    xp = s["ck_x"].load(s["tok"])
    gather(s["dy"], s["dyp"])
    da = s["da_op"].input_grad(s["dyp"], s["off"])
    dh, wa, dw = s["ck_b"].backward(da, row_w=s["rw"], wa=True, dw=True)
    dw2, _ = s["down"].weight_grad(wa, s["dyp"], s["off"])
    dw1, _ = s["up"].weight_grad(xp, dh, s["off"])
    dxp = s["dx_op"].input_grad(dh, s["off"])
    dx = torch.empty_like(s["x"])
    moe.moe_combine(s["desc"], dxp.data_ptr(), s["slot"].data_ptr(), None, None, dx.data_ptr(), st)
    return dict(y=y, dx=dx, dw1=dw1, dw2=dw2, dtw=dw[s["slot"].long()].view(T, k))


def _step_ref(s):
    """The same step in 64 bits, with the kept values in the backward's places."""
    x, dy, w1, w2, tw = (np64(s[n]) for n in ("x", "dy", "w1", "w2", "tw"))
    idx = s["idx"].cpu().numpy()
    xk = ref.keep(x)[2]
    out = dict(y=np.zeros_like(x), dx=np.zeros_like(x), dw1=np.zeros_like(w1), dw2=np.zeros_like(w2), dtw=np.zeros_like(tw))
    for e in range(s["M"]):
        t, j = np.nonzero(idx == e)
        if not len(t):
            continue
        h = x[t] @ w1[e].T
        w = tw[t, j][:, None]
        np.add.at(out["y"], t, w * (ref.act(h, True)[0] @ w2[e].T))
        hb = torch.from_numpy(h).to(torch.bfloat16).double().numpy()
        hk = ref.keep(hb, 2)[2]
        a, d = ref.act(hk, True)[0], ref.act_grad(hk, True)[0]
        da = dy[t] @ w2[e]
        dh = w * np.concatenate([da, da], 1) * d
        out["dtw"][t, j] = (da * a).sum(1)
        out["dw2"][e] = dy[t].T @ (w * a)
        out["dw1"][e] = dh.T @ xk[t]
        np.add.at(out["dx"], t, dh @ w1[e])
    return out


STEP = dict(T=150, D=96, M=12, I=72, k=3)


def test_a_training_step_of_the_experts(moe):
    """Forward, checkpoints and backward one after another.  Each result carries
    the bf16 rounding of an operand (h, a, wa or dh: 2^-8 a term at most, with
    random signs) and of a checkpoint's value that falls on the other side of a
    rounding border: 2 % of the result's norm bounds several of them."""
    s = _experts_step(moe, STEP)
    got, want = _run_step(moe, s), _step_ref(s)
    for name, w in want.items():
        g = np64(got[name])
        assert np.linalg.norm(g - w) <= 0.02 * np.linalg.norm(w), name


def test_the_step_captured_and_replayed(moe):
    """Captured into a graph and replayed on other inputs and another routing:
    bit for bit the eager step on them."""
    s = _experts_step(moe, STEP)
    _run_step(moe, s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _run_step(moe, s)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = _run_step(moe, s)
    s["x"].copy_(_randn(51, s["x"].shape, torch.bfloat16))
    s["dy"].copy_(_randn(52, s["dy"].shape, torch.bfloat16))
    s["idx"].copy_(torch.where(s["idx"] < 5, s["idx"] * 2 % 7, s["idx"]))   # other, uneven segments
    g.replay()
    first = {k: v.clone() for k, v in out.items()}
    g.replay()
    t = _experts_step(moe, STEP)
    for n in ("x", "dy", "idx"):
        t[n].copy_(s[n])
    eager = _run_step(moe, t)
    for n in eager:
        assert torch.equal(first[n], eager[n]), n
        assert torch.equal(out[n], eager[n]), n


def test_two_streams_at_once(moe):
    """Two handles on two streams give what each gives alone."""
    a, b = _experts_step(moe, STEP), _experts_step(moe, dict(STEP, T=333))
    alone = _run_step(moe, a), _run_step(moe, b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            r1 = _run_step(moe, a)
        with torch.cuda.stream(s2):
            r2 = _run_step(moe, b)
        torch.cuda.synchronize()
        for n in r1:
            assert torch.equal(r1[n], alone[0][n]) and torch.equal(r2[n], alone[1][n]), n
