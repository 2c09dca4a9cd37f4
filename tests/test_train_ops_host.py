"""Refusals of the grouped products and the 8-bit checkpoints: every bad call
is answered on the host, before anything is launched (no GPU needed)."""
import pytest
import torch

P = 4096  # any aligned address: these calls never reach a kernel


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import sparse_mixture_experts_logits_b200 as m
    return m


def _status(moe, fn, *args):
    with pytest.raises(moe.MoEError) as e:
        fn(*args)
    return e.value.status


GOOD = dict(x=P, w=P, bias=None, offsets=P, G=4, N=64, K=32, rows=10, dtype=1, out=1, y=P, ws=P, n=1 << 20)


def _gemm(moe, **kw):
    a = dict(GOOD, **kw)
    return (moe.moe_grouped_gemm, a["x"], a["w"], a["bias"], a["offsets"], a["G"], a["N"], a["K"], a["rows"], a["dtype"],
            a["out"], a["y"], a["ws"], a["n"])


def _dgrad(moe, **kw):
    a = dict(GOOD, **kw)
    return (moe.moe_grouped_dgrad, a["x"], a["w"], a["offsets"], a["G"], a["N"], a["K"], a["rows"], a["dtype"], a["out"],
            a["y"], a["ws"], a["n"])


def _wgrad(moe, **kw):
    a = dict(GOOD, **{"dy": P, "acc": 0, "db": None, **kw})
    return (moe.moe_grouped_wgrad, a["x"], a["dy"], a["offsets"], a["G"], a["N"], a["K"], a["rows"], a["dtype"], a["acc"],
            a["y"], a["db"], a["ws"], a["n"])


BAD = [(dict(G=0), 1), (dict(N=0), 1), (dict(K=0), 1), (dict(rows=-1), 1), (dict(dtype=5), 2), (dict(G=1025), 2),
       (dict(N=1 << 20, K=1 << 20), 2), (dict(rows=1 << 30), 2), (dict(x=None), 1), (dict(offsets=None), 1),
       (dict(y=None), 1), (dict(ws=None), 1), (dict(ws=P + 8), 1), (dict(n=0), 1), (dict(x=P + 8), 1), (dict(y=P + 2), 1),
       (dict(K=1 << 24, N=8), 2)]


@pytest.mark.parametrize("kw,status", BAD)
def test_grouped_products_refuse(moe, kw, status):
    for call in (_gemm, _dgrad, _wgrad):
        assert _status(moe, *call(moe, **kw)) == status, call.__name__


def test_grouped_rows_products_refuse(moe):
    for call in (_gemm, _dgrad):
        assert _status(moe, *call(moe, w=None)) == 1
        assert _status(moe, *call(moe, out=7)) == 2
        assert _status(moe, *call(moe, dtype=0, out=1)) == 2      # fp32 in, bf16 out
        assert _status(moe, *call(moe, w=P + 4)) == 1
    for dy in (None, P + 4):
        assert _status(moe, *_wgrad(moe, dy=dy)) == 1


def test_workspace_queries(moe):
    for fn in (moe.moe_grouped_workspace_size, moe.moe_grouped_wgrad_workspace_size):
        assert fn(4, 64, 32, 10, 1) >= 256 and fn(4, 64, 32, 0, 0) >= 256
        for bad in ((0, 64, 32, 10, 1), (4, 0, 32, 10, 1), (4, 64, 32, -1, 1), (4, 64, 32, 10, 9), (2000, 64, 32, 10, 1)):
            assert fn(*bad) == 0
    assert [moe.moe_ckpt_blocks(c) for c in (-3, 0, 1, 32, 33, 64, 2 ** 31 - 1)] == [0, 0, 1, 1, 2, 2, 2 ** 26]


def test_zero_rows_launch_nothing(moe):
    moe.moe_grouped_gemm(None, None, None, None, 4, 64, 32, 0, 1, 1, None, None, 0)
    moe.moe_grouped_dgrad(None, None, None, 4, 64, 32, 0, 1, 1, None, None, 0)
    moe.moe_grouped_wgrad(None, None, None, 4, 64, 32, 0, 1, 1, P, None, None, 0)
    moe.moe_ckpt_quantize(None, None, 0, 8, 1, None, None)
    moe.moe_ckpt_dequantize(None, None, None, None, 0, 0, 8, 1, None)
    moe.moe_act_save(None, None, 0, 8, 1, 1, 1, None, None, None)
    moe.moe_act_backward(None, None, None, None, None, 0, 8, 1, 1, 1, None)


def test_checkpoints_refuse(moe):
    q, dq, sv, bw = moe.moe_ckpt_quantize, moe.moe_ckpt_dequantize, moe.moe_act_save, moe.moe_act_backward
    for args, st in [((P, None, -1, 8, 1, P, P), 1), ((P, None, 4, 0, 1, P, P), 1), ((P, None, 4, 8, 3, P, P), 2),
                     ((None, None, 4, 8, 1, P, P), 1), ((P, None, 4, 8, 1, None, P), 1), ((P, None, 4, 8, 1, P, None), 1),
                     ((P, None, 1 << 30, 8, 1, P, P), 2)]:
        assert _status(moe, q, *args) == st, args
    for args, st in [((P, P, None, None, 5, 4, 8, 1, P), 1),       # more rows than are kept
                     ((P, P, P, None, 5, -1, 8, 1, P), 1), ((P, P, P, None, 5, 4, 8, 2, P), 2),
                     ((None, P, P, None, 5, 4, 8, 1, P), 1), ((P, P, P, None, 5, 4, 8, 1, None), 1)]:
        assert _status(moe, dq, *args) == st, args
    for args, st in [((P, None, 4, 8, 2, 1, 1, P, P, P), 1), ((P, None, 4, 8, 1, 4, 1, P, P, P), 2),
                     ((P, None, 4, 8, 1, 1, 4, P, P, P), 2), ((P, None, 4, 0, 1, 1, 1, P, P, P), 1),
                     ((P, None, 4, 8, 1, 1, 1, None, P, P), 1), ((None, None, 4, 8, 1, 1, 1, P, P, P), 1)]:
        assert _status(moe, sv, *args) == st, args
    for args, st in [((None, P, P, None, None, 4, 8, 1, 1, 1, P), 1), ((P, None, P, None, None, 4, 8, 1, 1, 1, P), 1),
                     ((P, P, None, None, None, 4, 8, 1, 1, 1, P), 1), ((P, P, P, None, None, 4, 8, 1, 1, 1, None), 1),
                     ((P, P, P, None, None, 4, 8, 9, 1, 1, P), 1)]:
        assert _status(moe, bw, *args) == st, args


def test_handles_refuse_on_the_host(moe):
    with pytest.raises(ValueError, match="CUDA"):
        moe.GroupedLinear(torch.zeros(2, 8, 8), 4)
    with pytest.raises(ValueError, match=r"\[G, N, K\]"):
        moe.GroupedLinear(torch.zeros(8, 8), 4)
    with pytest.raises(ValueError, match="CUDA"):
        moe.RowCheckpoint(4, 8, torch.float32, device="cpu")
    with pytest.raises(ValueError, match="act"):
        moe.ActivationCheckpoint("relu", 4, 8, torch.float32)


def _layer(moe, **over):
    import moe_synth as ms
    d = moe.desc_from_config(ms.get_config("glm_small_bf16", **over))
    w = moe.Weights()
    w.w_r, w.w1, w.w2, w.sh_w1, w.sh_w2 = P, P, P, P, P
    return d, w, moe.Grads(dx=P, dw_r=P, dw1=P, dw2=P, dsh_w1=P, dsh_w2=P)


def test_layer_checkpoint_refuses(moe):
    d, w, g = _layer(moe)
    ck, fs, bs = moe.moe_checkpoint_size(d), moe.moe_forward_save_workspace_size(d), moe.moe_backward_saved_workspace_size(d)
    pairs, blocks = d.T * d.k, -(-d.I // 32)
    assert ck >= pairs * (2 * d.I + 2 * blocks + 8) + d.T * (4 * d.M + 2 * d.I_sh)
    assert fs >= moe.moe_workspace_size(d) and 0 < bs < moe.moe_backward_workspace_size(d)
    offs = moe.moe_checkpoint_offsets(d)
    assert offs == sorted(offs) and all(o % 256 == 0 for o in offs) and offs[-1] < ck
    for args in [(None, ck, P, fs), (P + 8, ck, P, fs), (P, ck - 1, P, fs), (P, ck, None, fs), (P, ck, P, fs - 1), (P, ck, P + 8, fs)]:
        assert _status(moe, moe.moe_forward_save, d, w, P, None, P, *args) == 1, args
    assert _status(moe, moe.moe_forward_save, d, w, None, None, P, P, ck, P, fs) == 1
    for args in [(None, ck, g, P, bs), (P + 8, ck, g, P, bs), (P, ck - 1, g, P, bs), (P, ck, g, None, bs),
                 (P, ck, g, P, bs - 1), (P, ck, moe.Grads(dx=P, dw_r=P, dw1=P), P, bs)]:
        assert _status(moe, moe.moe_backward_saved, d, w, P, P, *args) == 1, args
    bad, _, _ = _layer(moe)
    bad.k = 0
    for fn in (moe.moe_checkpoint_size, moe.moe_forward_save_workspace_size, moe.moe_backward_saved_workspace_size):
        assert fn(bad) == 0
    assert _status(moe, moe.moe_checkpoint_offsets, bad) == 1
    many, w, g = _layer(moe)   # 2^30 (token, expert) pairs: a SwiGLU row is kept as two, counted in 31 bits
    many.M, many.k, many.D, many.I, many.I_sh, many.n_group, many.T = 63, 32, 16, 16, 0, 0, (1 << 25) - 1
    assert moe.moe_checkpoint_size(many) > 0
    many.T += 1
    assert moe.moe_workspace_size(many) > 0
    for fn in (moe.moe_checkpoint_size, moe.moe_forward_save_workspace_size, moe.moe_backward_saved_workspace_size):
        assert fn(many) == 0
    assert _status(moe, moe.moe_forward_save, many, w, P, None, P, P, 1 << 60, P, 1 << 60) == 2
    assert _status(moe, moe.moe_backward_saved, many, w, P, P, P, 1 << 60, g, P, 1 << 60) == 2
    zero, w, _ = _layer(moe, T=0)
    moe.moe_forward_save(zero, w, None, None, None, None, 0, None, 0)
