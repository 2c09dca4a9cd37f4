"""The layer with a checkpoint at the far ends of its range: many tokens, huge
pre-activations."""
import pytest
import torch

import moe_synth as ms
from gpu_common import gpu_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    import sparse_mixture_experts_logits_b200 as B
    return B


def _uniform(seed, shape, lo, hi, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.rand(shape, device="cuda", generator=g) * (hi - lo) + lo).to(dtype)


def _kept(ck, name):
    """The kept values of SwiGLU pre-activations: (gate, up) in 64 bits (one block of at most 32 columns a half)."""
    q, e = ck.view(name + "q").double(), ck.view(name + "e").long()
    c = q.shape[1] // 2
    step = (e - 133 + 1023 << 52).view(torch.float64)
    return q[:, :c] * step[:, :1], q[:, c:] * step[:, 1:]


def _close(got, want, rel, what):
    off = float(((got.double() - want).abs() / want.abs()).max())
    assert off <= rel, f"{what}: {off:.3g} of the value, bound {rel:.3g}"


def test_gradients_over_many_tokens(B):
    """The weight gradients that sum over every token (the shared expert's and
    the router's) are off by the roundings of 512 terms at a time, and not by how
    many tokens there are.

    All terms are positive, so that a truncated addition's loss adds up.  Bound:
    32 truncated steps of 16 products (3 * 2^-23 each), one rounded addition for
    each 512 terms, and 2^-17 for the operands: they are rounded to bf16 from
    fp32 values a few 2^-21 off the reference's, which moves some of them to the
    neighbouring number, by 2^-21 of the sum on average."""
    T, I = 1 << 17, 16
    cfg = ms.get_config("glm_small_bf16", T=T, D=64, M=64, k=1, I=I, I_sh=I, norm_topk_prob=0, alpha=1.0)
    t = dict(gpu_inputs(dict(cfg, T=16)), x=_uniform(1, (T, 64), 0.5, 1.0), w_r=_uniform(2, (64, 64), 0.0, 0.02),
             w1=_uniform(3, (64, 2 * I, 64), 0.0, 0.05), w2=_uniform(4, (64, 64, I), 0.5, 1.0),
             sh_w1=_uniform(5, (2 * I, 64), 0.0, 0.05), sh_w2=_uniform(6, (64, I), 0.5, 1.0))
    t["e_bias"] = torch.zeros_like(t["e_bias"])
    t["e_bias"][0] = 100.0  # every token goes to expert 0, so that dispatch order is the tokens'
    x, dy = t["x"], _uniform(7, (T, 64), 1.0, 2.0)
    layer = B.MoELayer(cfg, t)
    ck = B.LayerCheckpoint(layer)
    layer.forward(x, checkpoint=ck)
    got = layer.backward(x, dy, checkpoint=ck)
    assert layer.backward_status() == 0 and not ck.view("topk_idx").any()
    bf = lambda v: v.to(torch.bfloat16).double()  # noqa: E731
    x, dy = x.double(), dy.double()
    g, u = _kept(ck, "shared_")
    s, G = torch.sigmoid(g), dy @ t["sh_w2"].double()
    dh = torch.cat([G * u * s * (1 + g * (1 - s)), G * g * s], 1)
    bound = 3 * 32 * 2.0 ** -23 + (T / 512 + 1) * 2.0 ** -24 + 2.0 ** -17
    _close(got["dsh_w2"], dy.T @ bf(g * s * u), bound, "dsh_w2")
    _close(got["dsh_w1"], bf(dh).T @ x, bound, "dsh_w1")
    g, u = _kept(ck, "")
    dw = (dy @ t["w2"][0].double() * g * torch.sigmoid(g) * u).sum(1)
    p = torch.sigmoid(ck.view("logits")[:, 0].double())
    _close(got["dw_r"][:, 0], x.T @ bf(dw * p * (1 - p)), bound, "dw_r")
    assert not got["dw_r"][:, 1:].any()


@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("name", ["glam_small_bf16", "glam_nonorm_f32"])
def test_huge_gelu_pre_activations(B, name, saved):
    """Scaling the up projection by 2^27 where every pre-activation is already far
    out on GELU's straight pieces scales some gradients by 2^27 and leaves the
    others, bit for bit; the squares of the larger ones are no fp32 numbers."""
    cfg = ms.get_config(name)
    inp = gpu_inputs(cfg)
    inp["b2"].zero_()
    dy = ms.upstream_grad(cfg, "cuda")
    got = []
    for p in (40, 67):
        t = dict(inp, w1=inp["w1"] * 2.0 ** p, b1=inp["b1"] * 2.0 ** p)
        layer = B.MoELayer(cfg, t)
        ck = B.LayerCheckpoint(layer) if saved else None
        y = layer.forward(t["x"], checkpoint=ck)
        got.append(dict(layer.backward(t["x"], dy, checkpoint=ck), y=y))
    for n, small in got[0].items():
        scale = 1.0 if n in ("dw1", "db1", "db2") else 2.0 ** 27
        assert got[1][n].isfinite().all(), n
        assert torch.equal(got[1][n], small * scale), n


@pytest.mark.parametrize("name,kept", [("glm_small_bf16", True), ("glm_small_bf16", False), ("glm_small_f32", True)])
def test_a_stream_of_its_own(B, name, kept):
    """A call on a given stream while the current one is busy: what it allocates
    is not written by work that is still to run on the current stream."""
    cfg = ms.get_config(name)
    inp = gpu_inputs(cfg)
    x, dy, h = inp["x"], ms.upstream_grad(cfg, "cuda"), inp["x"].clone()
    layer = B.MoELayer(cfg, inp)
    ck = B.LayerCheckpoint(layer) if kept else None
    y0 = layer.forward(x, addend=h, checkpoint=ck)
    want = layer.backward(x, dy, checkpoint=ck)
    layer = B.MoELayer(cfg, inp)
    ck = B.LayerCheckpoint(layer) if kept else None
    side, busy = torch.cuda.Stream(), torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for _ in range(100):
        busy.fill_(1)
    # blocks of the results' sizes that the current stream will still write, after a while
    sizes = [y0] + list(want.values())
    junk = [torch.full_like(t, float("nan")) for t in sizes for _ in range(2)]
    junk.append(torch.full((1 << 26,), 0x7F, dtype=torch.uint8, device="cuda"))
    del junk
    y = layer.forward(x, addend=h, checkpoint=ck, stream=side)
    got = layer.backward(x, dy, checkpoint=ck, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, y0)
    for n, v in want.items():
        assert torch.equal(got[n], v), n
    assert layer.device_status(stream=side) == 0 and layer.backward_status(stream=side) == 0


@pytest.mark.parametrize("name", ["glam_small_bf16", "glam_nonorm_f32"])
def test_bias_gradients_over_many_tokens(B, name):
    """One large gradient and 10^5 small ones whose last bits the large one's sum
    does not hold: at most 128 rounded additions in a row, and one for each 128
    rows behind them.  (One expert, whose gate weight is 1.)"""
    T = 100_000
    cfg = ms.get_config(name, T=T, D=16, M=1, k=1, I=16)
    inp = gpu_inputs(cfg)
    dy = torch.full_like(inp["x"], 1.0078125)
    dy[0] = 2.0 ** 17
    layer = B.MoELayer(cfg, inp)
    ck = B.LayerCheckpoint(layer)
    layer.forward(inp["x"], checkpoint=ck)
    got = layer.backward(inp["x"], dy, checkpoint=ck)
    assert ck.view("topk_w").eq(1).all()
    _close(got["db2"][0], dy.double().sum(0), (128 + T / 128 + 2) * 2.0 ** -24, "db2")
