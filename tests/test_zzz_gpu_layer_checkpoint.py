"""The layer's forward that keeps an 8-bit checkpoint, and its backward from
it, against the fp64 oracles.

The kept values are read back and checked against the oracle's
pre-activations (a value may be off by its rounding and by the fp32
accumulation of the pre-activation it rounds).  The gradients are those of
the kept values: the reference is the backward oracle with the GPU's kept
values in the place of its own pre-activations, and the bounds are those of
the plain backward's tests (the same operands are rounded to bf16)."""
import numpy as np
import pytest
import torch

import moe_synth as ms
import oracle
import train_ops_ref as ref
from gpu_common import check_routing, check_y, gpu_inputs, np64, oracle_route, oracle_y
from test_zzz_gpu_backward import check_all, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    import sparse_mixture_experts_logits_b200 as B
    return B


def kept_values(ck, halves, prefix=""):
    q, e = np64(ck.view(prefix + "q")), np64(ck.view(prefix + "e"))
    rows, width = q.shape
    c = width // halves
    ex = np.repeat(e.reshape(rows, halves, -1), 32, 2)[:, :, :c].reshape(rows, width)
    return np.ldexp(q, (ex - 133).astype(int)), ex, q


def check_kept(v, ex, q, h, mag, terms):
    """Half a step of rounding (a whole one at the clamp), plus the sums' own error; a block whose largest
    magnitude lies within that error of a power of two may have the neighbouring exponent (twice the step)."""
    err = ref.gamma(terms, "bf16") * mag
    step = np.ldexp(1.0, (ex - 133).astype(int))
    assert (np.abs(v - h) <= np.where(np.abs(q) == 127, 1.0, 0.5) * step + err).all()
    assert (np.abs(h) < 128.5 * step + err).all() and (ex <= 254).all()


def run(B, cfg, layer=None, inp=None, ck=None):
    inp = gpu_inputs(cfg) if inp is None else inp
    layer = B.MoELayer(cfg, inp) if layer is None else layer
    ck = B.LayerCheckpoint(layer) if ck is None else ck
    dy = ms.upstream_grad(cfg, "cuda")
    y = layer.forward(inp["x"], checkpoint=ck)
    g = layer.backward(inp["x"], dy, checkpoint=ck)
    torch.cuda.synchronize()
    assert layer.device_status() == 0 and layer.backward_status() == 0
    return inp, dy, layer, ck, y, g


def check(B, cfg):
    inp, dy, layer, ck, y, g = run(B, cfg)
    T, M, k = cfg["T"], cfg["M"], cfg["k"]
    idx, tw = ck.view("topk_idx").cpu().numpy(), ck.view("topk_w").cpu().numpy()
    w_ref, _ = check_routing(cfg, oracle_route(cfg, inp), idx, tw)
    check_y(dict(cfg, named=False), np64(y), oracle_y(cfg, inp, np.arange(T), idx, w_ref))
    halves = 2 if cfg["act"] == "swiglu" else 1
    v, ex, q = kept_values(ck, halves)
    hin = host(inp)
    slot = oracle.permute(idx, tw.astype(np.float64), M)["slot_of"]
    calls = []
    for e in range(M):
        tt, jj = np.nonzero(idx == e)
        if not len(tt):
            continue
        rows = slot[tt, jj]
        h, mag = hin["x"][tt] @ hin["w1"][e].T, np.abs(hin["x"][tt]) @ np.abs(hin["w1"][e]).T
        if hin.get("b1") is not None:
            h, mag = h + hin["b1"][e], mag + np.abs(hin["b1"][e])
        check_kept(v[rows], ex[rows], q[rows], h, mag, cfg["D"])
        calls.append(v[rows])
    if cfg.get("I_sh"):
        sv, sex, sq = kept_values(ck, 2, "shared_")
        check_kept(sv, sex, sq, hin["x"] @ hin["sh_w1"].T, np.abs(hin["x"]) @ np.abs(hin["sh_w1"]).T, cfg["D"])
        calls.append(sv)
    order = iter(calls)

    def ffn(xe, act, w1e, w2e, b1e, b2e, dout):
        pre = next(order)
        a, d = ref.act(pre, act == "swiglu")[0], ref.act_grad(pre, act == "swiglu")[0]
        da = dout @ w2e
        dpre = np.concatenate([da, da], 1) * d if act == "swiglu" else da * d
        out = a @ w2e.T + (0 if b2e is None else b2e)
        return {"out": out, "dx": dpre @ w1e, "dw1": dpre.T @ xe, "dw2": dout.T @ a,
                "db1": dpre.sum(0) if b1e is not None and act == "gelu_tanh" else None,
                "db2": dout.sum(0) if b2e is not None else None,
                "dw1_abs": np.abs(dpre).T @ np.abs(xe), "dw2_abs": np.abs(dout).T @ np.abs(a),
                "db1_abs": np.abs(dpre).sum(0)}

    real = oracle.moe_backward.expert_ffn_backward
    oracle.moe_backward.expert_ffn_backward = ffn
    try:
        want = oracle.moe_backward.moe_backward(cfg, hin, np64(dy), idx=idx)
    finally:
        oracle.moe_backward.expert_ffn_backward = real
    check_all(cfg, g, want)
    return inp, dy, layer, ck, y, g


@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("name", ["glam_small_bf16", "glm_small_bf16"])
def test_bad_weights_stay_alone(B, name, saved):
    """NaN in one expert's weights leaves the other experts' weight gradients
    as they were, at widths that end inside a block of 64."""
    cfg = dict(ms.get_config(name), D=272, I=144)
    inp = gpu_inputs(cfg)
    dy = ms.upstream_grad(cfg, "cuda")

    def grads(inp):
        layer = B.MoELayer(cfg, inp)
        ck = B.LayerCheckpoint(layer) if saved else None
        layer.forward(inp["x"], checkpoint=ck)
        return layer.backward(inp["x"], dy, checkpoint=ck)

    clean, bad = grads(inp), cfg["M"] // 2
    inp2 = dict(inp, w1=inp["w1"].clone(), w2=inp["w2"].clone())
    inp2["w1"][bad] = float("nan")
    inp2["w2"][bad] = float("nan")
    got = grads(inp2)
    rest = [g for g in range(cfg["M"]) if g != bad]
    for key in ("dw1", "dw2"):
        assert torch.equal(got[key][rest], clean[key][rest]), key


@pytest.mark.parametrize("name", ["glam_tiny_f32", "glam_small_bf16", "glm_small_bf16", "glm_small_f32",
                                  "glm_grouped_bf16", "glm_grouped_f32", "glam_nonorm_f32", "glm_medium_bf16"])
def test_layer_from_its_checkpoint(B, name):
    cfg = ms.get_config(name)
    inp, dy, layer, ck, y, g = check(B, cfg)
    # the same layer without a checkpoint: for bf16 the same forward, bit for bit (an fp32 layer's activation runs
    # in a kernel of its own here, and rounds apart from the one fused into the product: both were held to the oracle)
    plain = layer.forward(inp["x"])
    if cfg["dtype"] == "bf16" and cfg["T"] * cfg["k"] >= 4 * cfg["M"]:
        assert torch.equal(plain, y)
    assert torch.equal(layer.view("topk_idx"), ck.view("topk_idx"))


@pytest.mark.parametrize("name,over", [
    ("glm_small_bf16", dict(T=1)), ("glm_small_bf16", dict(T=65)), ("glm_small_bf16", dict(T=129, k=1)),
    ("glm_small_bf16", dict(k=16)), ("glam_small_bf16", dict(M=1, k=1)), ("glam_small_bf16", dict(T=700)),
    ("glm_small_bf16", dict(I_sh=0)), ("glm_medium_bf16", dict(e_bias=("zipf", 1.1, 1.0))),
    ("glm_medium_bf16", dict(M=160)), ("glm_small_bf16", dict(I=208, I_sh=144)), ("glam_small_bf16", dict(I=304)),
    ("glm_small_f32", dict(T=1)), ("glm_small_f32", dict(I=33, I_sh=47)), ("glam_nonorm_f32", dict(I=45))])
def test_layer_checkpoint_edge_shapes(B, name, over):
    """A single token, ragged tiles, k = 1 and k = M, one expert, experts without rows, no shared expert, and
    widths whose last block of 32 is a partial one."""
    check(B, ms.get_config(name, **over))


def test_addend_and_repeats(B):
    cfg = ms.get_config("glm_small_bf16")
    inp, dy, layer, ck, y, g = run(B, cfg)
    h = torch.randn(y.shape, generator=torch.Generator().manual_seed(3)).to(y).contiguous()
    assert torch.equal(layer.forward(inp["x"], addend=h, checkpoint=ck), layer.forward(inp["x"], addend=h))
    again = layer.backward(inp["x"], dy, checkpoint=ck)
    for n in g:
        assert torch.equal(g[n], again[n]), n


def test_two_checkpoints_of_one_layer(B):
    """Two micro-batches in flight: each backward reads its own checkpoint."""
    cfg = ms.get_config("glm_small_bf16")
    inp, dy, layer, c1, _, g1 = run(B, cfg)
    x2 = inp["x"].flip(0).contiguous()
    c2 = B.LayerCheckpoint(layer)
    layer.forward(x2, checkpoint=c2)
    g2 = layer.backward(x2, dy, checkpoint=c2)
    layer.forward(inp["x"], checkpoint=c1)
    layer.forward(x2, checkpoint=c2)
    h1, h2 = layer.backward(inp["x"], dy, checkpoint=c1), layer.backward(x2, dy, checkpoint=c2)
    for n in g1:
        assert torch.equal(g1[n], h1[n]) and torch.equal(g2[n], h2[n]), n
    assert not torch.equal(g1["dx"], g2["dx"])


@pytest.mark.parametrize("name", ["glm_small_bf16", "glm_small_f32"])
def test_views_and_status_follow_the_last_call(B, name):
    """The views and the status are those of the workspace that the last forward or backward used; what a
    checkpoint holds in their place is not read from an older pass."""
    cfg = ms.get_config(name)
    inp = gpu_inputs(cfg)
    layer = B.MoELayer(cfg, inp)
    with pytest.raises(RuntimeError, match="checkpoint"):
        layer.backward_view("topk_idx")
    _, dy, _, ck, _, _ = run(B, cfg, layer=layer, inp=inp)
    for view in (layer.view, layer.backward_view):
        with pytest.raises(RuntimeError, match="checkpoint"):
            view("topk_idx")
    kept = {n: layer.view(n).clone() for n in ("counts", "offsets", "slot_of", "row_token")}
    assert kept["counts"].sum() == cfg["T"] * cfg["k"]
    layer.view("status").fill_(3)
    assert layer.device_status() == 3 and layer.device_status() == 0
    layer.forward(inp["x"])
    assert torch.equal(layer.view("topk_idx"), ck.view("topk_idx"))
    assert all(torch.equal(layer.view(n), v) for n, v in kept.items())
    layer.backward(inp["x"], dy)
    assert torch.equal(layer.backward_view("topk_idx"), ck.view("topk_idx"))


def test_captured_and_replayed(B):
    """Forward and backward in one graph, replayed on another input: bit for bit the eager step."""
    cfg = ms.get_config("glm_small_bf16")
    inp, dy, layer, ck, _, _ = run(B, cfg)
    x, dy = inp["x"].clone(), dy.clone()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        layer.forward(x, checkpoint=ck)
        layer.backward(x, dy, checkpoint=ck)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.forward(x, checkpoint=ck)
        g = layer.backward(x, dy, checkpoint=ck)
    x.copy_(x.flip(0))
    dy.copy_(dy.flip(1))
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    other = B.MoELayer(cfg, inp)
    c2 = B.LayerCheckpoint(other)
    y2 = other.forward(x, checkpoint=c2)
    g2 = other.backward(x, dy, checkpoint=c2)
    assert torch.equal(y, y2)
    for n in g:
        assert torch.equal(g[n], g2[n]), n


def test_no_tokens(B):
    cfg = ms.get_config("glm_small_bf16")
    inp = gpu_inputs(cfg)
    layer = B.MoELayer(cfg, inp, T=0)
    ck = B.LayerCheckpoint(layer)
    x = inp["x"][:0]
    assert layer.forward(x, checkpoint=ck).shape == x.shape
    g = layer.backward(x, x, checkpoint=ck)
    assert all(not t.any() for t in g.values())


def test_decode_size(B):
    """The GLM-4.5 decode layer (32 tokens, 160 experts): the forward takes the larger sizes' path here, so y is
    compared within the bf16 bound; the gradients against the plain backward's, whose pre-activations differ by the
    kept values' rounding (under 1/64 of a block's largest value, 1.3 % of a typical one, random in sign): 3 % of the
    gradients' norm."""
    cfg = ms.get_config("glm45_decode_bf16")
    inp, dy, layer, ck, y, g = run(B, cfg)
    want = np64(layer.forward(inp["x"]))
    assert np.abs(np64(y) - want).max() <= 2e-2 * np.sqrt((want ** 2).mean())
    h = layer.backward(inp["x"], dy)
    for n in g:
        a, b = g[n].double(), h[n].double()
        assert float((a - b).norm()) <= 0.03 * float(b.norm()), n
