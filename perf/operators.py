"""Cases of the operators for training and serving the routed experts step by step.

Two families, which a training step of the experts uses together:

  grouped   matrix products grouped by expert over ragged row segments: the product
            y[r] = x[r] W_g^T + b_g, its input gradient dx[r] = dy[r] W_g, and its weight and bias
            gradients dW_g = sum_r dy[r]^T x[r], db_g = sum_r dy[r]
  8 bits    activation checkpoints in 8 bits: rows to 8 bits and back (gathered into dispatch
            order), the expert activation with the checkpoint of its input, and the activation's
            gradient from that checkpoint

The 8-bit form of a row: blocks of 32 consecutive columns (of each half, gate and up, for SwiGLU)
share the exponent byte E of their largest magnitude; an element is q = round(x 2^(133 - E)) clamped
to [-127, 127] and stands for q 2^(E - 133).

``own`` false runs plain torch forms in 32 bits, rounded once; true runs the framework's operators.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_ES = {"bf16": 2, "f32": 4}


def listed():
    return [
        # one token of a small layer through its experts: nothing but latency
        dict(name="gemm_one_token", kind="gemm", dtype="bf16", out="bf16", G=16, N=384, K=256, rows=4, skew=0.0, drop=0,
             bias=False),
        # down projection of a decode batch: 32 tokens x 8 experts over 160 experts, bound by the weights it touches
        dict(name="gemm_decode_down", kind="gemm", dtype="bf16", out="bf16", G=160, N=5120, K=1536, rows=256, skew=0.0,
             drop=0, bias=False),
        # up projection of a prompt or a training batch, biases, evenly loaded experts
        dict(name="gemm_prompt_up", kind="gemm", dtype="bf16", out="bf16", G=64, N=8192, K=2048, rows=16384, skew=0.0,
             drop=0, bias=True),
        # gradient reaching the activation, experts loaded unevenly (some empty), pairs dropped at the capacity behind
        # the last segment; kept in fp32 for the activation's gradient
        dict(name="dgrad_skewed", kind="dgrad", dtype="bf16", out="f32", G=64, N=6144, K=2048, rows=20001, skew=1.1,
             drop=333, bias=False),
        # weight and bias gradients of a micro-batch, added onto the earlier ones'
        dict(name="wgrad_accumulate", kind="wgrad", dtype="bf16", out="f32", G=32, N=2048, K=5120, rows=16383, skew=0.6,
             drop=0, bias=False),
        # a small layer's training step, all three products after one another
        dict(name="grouped_step_small", kind="step", dtype="bf16", out="bf16", G=16, N=384, K=256, rows=1199, skew=0.6,
             drop=5, bias=True),
        # the same in fp32 at sizes that fit no tile
        dict(name="grouped_step_f32_odd", kind="step", dtype="f32", out="f32", G=12, N=93, K=65, rows=231, skew=0.6, drop=0,
             bias=True),
        # layer input kept in 8 bits from the forward, read back into dispatch order by the backward
        dict(name="rows_8bit_gather", kind="rows", dtype="bf16", T=8192, cols=5120, k=4),
        # SwiGLU of the up projection's rows with the checkpoint, large batch, and its read-back
        dict(name="swiglu_save", kind="save", act="swiglu", dtype="bf16", src="bf16", rows=32768, I=2048),
        # GELU, fp32 pre-activations at an odd width
        dict(name="gelu_save_f32_odd", kind="save", act="gelu_tanh", dtype="f32", src="f32", rows=333, I=199),
        # gradient of SwiGLU from the checkpoint, with the gate weights and their gradients
        dict(name="swiglu_backward", kind="backward", act="swiglu", dtype="bf16", src="f32", rows=32768, I=2048),
        # the same for GELU experts, a ragged batch
        dict(name="gelu_backward", kind="backward", act="gelu_tanh", dtype="bf16", src="bf16", rows=4097, I=8192),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["gemm", "dgrad", "wgrad", "step", "rows", "save", "backward"])
    if kind in ("gemm", "dgrad", "wgrad", "step"):
        if rng.random() < 0.25:  # fp32: any width
            return dict(kind=kind, dtype="f32", out="f32", G=_log(rng, 1, 32), N=_log(rng, 1, 400), K=_log(rng, 1, 400),
                        rows=_log(rng, 1, 1500), skew=rng.choice([0.0, 0.6, 1.1]), drop=0, bias=rng.random() < 0.5)
        c = dict(kind=kind, dtype="bf16", out=rng.choice(["bf16", "f32"]) if kind != "wgrad" else "f32",
                 G=_log(rng, 1, 128), N=8 * _log(rng, 2, 1000), K=8 * _log(rng, 2, 750), rows=_log(rng, 1, 16384),
                 skew=rng.choice([0.0, 0.6, 1.1]), drop=0, bias=rng.random() < 0.5)
        while c["G"] * c["N"] * c["K"] > 4e8 or c["rows"] * c["N"] * c["K"] > 8e10:
            for s in ("G", "rows"):
                c[s] = max(1, c[s] * 3 // 4)
            for s in ("N", "K"):
                c[s] = max(16, c[s] * 7 // 8 // 8 * 8)
        c["drop"] = rng.choice([0, 0, c["rows"] // 7])
        return c
    if kind == "rows":
        return dict(kind="rows", dtype=rng.choice(["bf16", "f32"]), T=_log(rng, 1, 8192), cols=_log(rng, 8, 5120),
                    k=rng.choice([1, 2, 4]))
    src = rng.choice(["bf16", "f32"])
    return dict(kind=kind, act=rng.choice(["swiglu", "gelu_tanh"]), dtype="bf16" if src == "bf16" else rng.choice(["bf16", "f32"]),
                src=src, rows=_log(rng, 1, 16384), I=_log(rng, 8, 4096))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, shape, dtype, std=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def _activations(g, rows, cols, dtype):
    """N(0, 1) rows with a few channels an order of magnitude larger, as the inputs of trained layers have."""
    x = _randn(g, (rows, cols), dtype)
    big = torch.rand(cols, device="cuda", generator=g) < 0.005
    return torch.where(big, x * 12, x)


def _offsets(case, seed):
    """Segments of a random routing: expert e gets a row with probability ~ rank^-skew."""
    r = np.random.default_rng(int(seed))
    p = np.arange(1, case["G"] + 1, dtype=np.float64) ** -case["skew"]
    counts = r.multinomial(case["rows"] - case["drop"], r.permutation(p / p.sum()))
    return np.concatenate([[0], np.cumsum(counts)])


def _swiglu(case):
    return case["act"] == "swiglu"


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    kind = case["kind"]
    if kind in ("gemm", "dgrad", "wgrad", "step"):
        dt, G, N, K, rows = _DT[case["dtype"]], case["G"], case["N"], case["K"], case["rows"]
        host = _offsets(case, seed)
        s["longest"] = max(1, int(np.diff(host).max()))  # part of the host's plan of the batch
        s["offsets"] = torch.from_numpy(host.astype(np.int32)).cuda()
        s["w"] = _randn(g, (G, N, K), dt, K ** -0.5)
        s["bias"] = _randn(g, (G, N), dt, 0.1) if case["bias"] else None
        if kind != "dgrad":
            s["x"] = _activations(g, rows, K, dt)
        if kind != "gemm":
            s["dy"] = _randn(g, (rows, N), dt)
        out = _DT[case["out"]]
        s["y"] = torch.full((rows, N), 0.5, dtype=out, device="cuda") if kind in ("gemm", "step") else None
        s["dx"] = torch.full((rows, K), 0.5, dtype=out, device="cuda") if kind in ("dgrad", "step") else None
        if kind == "wgrad":  # the earlier micro-batches' sums
            s["dw"] = _randn(g, (G, N, K), torch.float32)
            s["db"] = _randn(g, (G, N), torch.float32)
    elif kind == "rows":
        s["x"] = _activations(g, case["T"], case["cols"], _DT[case["dtype"]])
        order = torch.rand(case["T"] * case["k"], device="cuda", generator=g).argsort()
        s["row_token"] = (order // case["k"]).to(torch.int32)
    elif kind == "save":
        n1 = 2 * case["I"] if _swiglu(case) else case["I"]
        s["h"] = _randn(g, (case["rows"], n1), _DT[case["src"]], 1.5)
    else:
        n1 = 2 * case["I"] if _swiglu(case) else case["I"]
        h = _randn(g, (case["rows"], n1), torch.float32, 1.5)
        s["q"], s["e"] = _to_8bit(h, 2 if _swiglu(case) else 1)  # what the forward left
        s["da"] = _randn(g, (case["rows"], case["I"]), _DT[case["src"]])
        s["row_w"] = torch.rand(case["rows"], device="cuda", generator=g) + 0.05
    return s


# ------------------------------------------------------------------ plain forms
def _blocks(x, halves):
    """[rows, halves * c] as [rows, halves * blocks, 32], the last block of a half filled up with zeros."""
    rows, c = x.shape[0], x.shape[1] // halves
    x = x.view(rows, halves, c)
    x = torch.nn.functional.pad(x, (0, -c % 32))
    return x.view(rows, halves * ((c + 31) // 32), 32)


def _to_8bit(x, halves):
    rows, cols = x.shape
    b = _blocks(x.float(), halves)
    e = b.abs().amax(2).view(torch.int32) >> 23
    scale = (254 - e << 23).view(torch.float32)  # 2^(127 - E), exactly
    q = torch.round(b * scale[..., None] * 64)
    q = q.clamp(-127, 127).to(torch.int8).view(rows, halves, -1)[:, :, :cols // halves].reshape(rows, cols)
    return q.contiguous(), e.to(torch.uint8)


def _from_8bit(q, e, halves):
    rows, cols = q.shape
    b = _blocks(q.float(), halves)
    scale = (e.to(torch.int32).clamp(min=7) - 6 << 23).view(torch.float32)  # 2^(E - 133); below 7 every q is 0 here
    v = b * scale[..., None]
    return v.view(rows, halves, -1)[:, :, :cols // halves].reshape(rows, cols)


def _padded(s, t):
    """Rows [rows, C] as fp32 [G, longest, C], each group's segment filled up with zeros."""
    off = s["offsets"].long()
    pos = torch.arange(s["longest"], device="cuda")
    idx = off[:-1, None] + pos
    live = idx < off[1:, None]
    return torch.where(live[..., None], t[idx.clamp(max=t.shape[0] - 1)].float(), 0.0)


def _unpadded(s, p, into):
    """The rows of [G, longest, C] back in one buffer; rows behind the last segment stay as they were."""
    off = s["offsets"].long()
    r = torch.arange(into.shape[0], device="cuda")
    grp = torch.searchsorted(off, r, right=True) - 1
    live = grp < off.numel() - 1
    grp = grp.clamp(max=off.numel() - 2)
    pos = (r - off[grp]).clamp(max=p.shape[1] - 1)
    return torch.where(live[:, None], p[grp, pos].to(into.dtype), into)


def _plain_gemm(s):
    y = _padded(s, s["x"]) @ s["w"].float().transpose(1, 2)
    if s["bias"] is not None:
        y = y + s["bias"].float()[:, None, :]
    return _unpadded(s, y, s["y"])


def _plain_dgrad(s):
    return _unpadded(s, _padded(s, s["dy"]) @ s["w"].float(), s["dx"])


def _plain_wgrad(s):
    dy = _padded(s, s["dy"])
    return dy.transpose(1, 2) @ _padded(s, s["x"]), dy.sum(1)


_C = math.sqrt(2.0 / math.pi)


def _act(h, swiglu):
    if swiglu:
        a, u = h.chunk(2, 1)
        return a * torch.sigmoid(a) * u
    return h * torch.sigmoid(2 * _C * (h + 0.044715 * h ** 3))


def _act_grad(h, da, swiglu):
    if swiglu:
        a, u = h.chunk(2, 1)
        sg = torch.sigmoid(a)
        return torch.cat([da * u * sg * (1 + a * torch.sigmoid(-a)), da * a * sg], 1)
    z = 2 * _C * (h + 0.044715 * h ** 3)
    sg = torch.sigmoid(z)
    return da * (sg + h * sg * torch.sigmoid(-z) * 2 * _C * (1 + 3 * 0.044715 * h * h))


def _plain(s):
    c = s["case"]
    kind = c["kind"]
    if kind == "gemm":
        return _plain_gemm(s)
    if kind == "dgrad":
        return _plain_dgrad(s)
    if kind == "wgrad":
        dw, db = _plain_wgrad(s)
        s["dw"] += dw
        s["db"] += db
        return {"dw": s["dw"], "db": s["db"]}
    if kind == "step":
        dw, db = _plain_wgrad(s)
        return {"y": _plain_gemm(s), "dx": _plain_dgrad(s), "dw": dw, "db": db}
    dt = _DT[c["dtype"]]
    if kind == "rows":
        q, e = _to_8bit(s["x"], 1)
        return _from_8bit(q, e, 1)[s["row_token"].long()].to(dt)
    sw = _swiglu(c)
    halves = 2 if sw else 1
    if kind == "save":
        h = s["h"].float()
        q, e = _to_8bit(h, halves)
        return {"a": _act(h, sw).to(dt), "kept": _from_8bit(q, e, halves).to(dt)}
    h, da, w = _from_8bit(s["q"], s["e"], halves), s["da"].float(), s["row_w"][:, None]
    a = _act(h, sw)
    return {"dh": (w * _act_grad(h, da, sw)).to(dt), "wa": (w * a).to(dt), "dw": (da * a).sum(1)}


# ------------------------------------------------------------------ the framework's operators
def _handle(s):
    """The object that a user's program keeps for its layer."""
    if "handle" not in s:
        import sparse_mixture_experts_logits_b200 as moe
        c = s["case"]
        if c["kind"] in ("gemm", "dgrad", "wgrad", "step"):
            s["handle"] = moe.GroupedLinear(s["w"], c["rows"], bias=s["bias"], out_dtype=_DT[c["out"]])
        elif c["kind"] == "rows":
            s["handle"] = moe.RowCheckpoint(c["T"], c["cols"], _DT[c["dtype"]], "cuda")
        else:
            s["handle"] = moe.ActivationCheckpoint(c["act"], c["rows"], c["I"], _DT[c["dtype"]], _DT[c["src"]], "cuda",
                                                   q=s.get("q"), e=s.get("e"))
    return s["handle"]


def _own(s):
    c = s["case"]
    kind = c["kind"]
    op = _handle(s)
    if kind == "gemm":
        return op.forward(s["x"], s["offsets"], y=s["y"])
    if kind == "dgrad":
        return op.input_grad(s["dy"], s["offsets"], dx=s["dx"])
    if kind == "wgrad":
        dw, db = op.weight_grad(s["x"], s["dy"], s["offsets"], dw=s["dw"], db=s["db"], accumulate=True)
        return {"dw": dw, "db": db}
    if kind == "step":
        y = op.forward(s["x"], s["offsets"], y=s["y"])
        dx = op.input_grad(s["dy"], s["offsets"], dx=s["dx"])
        dw, db = op.weight_grad(s["x"], s["dy"], s["offsets"], db=True)
        return {"y": y, "dx": dx, "dw": dw, "db": db}
    if kind == "rows":
        op.save(s["x"])
        return op.load(s["row_token"])
    if kind == "save":
        return {"a": op.save(s["h"]), "kept": op.load()}
    dh, wa, dw = op.backward(s["da"], row_w=s["row_w"], wa=True, dw=True)
    return {"dh": dh, "wa": wa, "dw": dw}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ work and the definition in 64 bits
def work(case):
    kind = case["kind"]
    if kind in ("gemm", "dgrad", "wgrad", "step"):
        es, eo, G, N, K = _ES[case["dtype"]], _ES[case["out"]], case["G"], case["N"], case["K"]
        rows = case["rows"] - case["drop"]
        # experts that an even routing reaches: only their weights are read
        reached = G * (1 - (1 - 1 / G) ** rows) if G > 1 else min(1, rows)
        product = 2.0 * rows * N * K
        gemm = es * (rows * K + reached * N * K) + eo * rows * N
        dgrad = es * (rows * N + reached * N * K) + eo * rows * K
        wgrad = es * rows * (N + K) + 4 * G * N * (K + 1) * (2 if kind == "wgrad" else 1)
        by = {"gemm": (gemm, 1), "dgrad": (dgrad, 1), "wgrad": (wgrad, 1), "step": (gemm + dgrad + wgrad, 3)}[kind]
        return {"bytes": float(by[0]), "flops": by[1] * product}
    es = _ES[case["dtype"]]
    if kind == "rows":
        T, c, k = case["T"], case["cols"], case["k"]
        kept = c + (c + 31) // 32
        return {"bytes": float(T * c * es + 2 * T * kept + T * k * (c * es + 4)), "flops": 4.0 * T * c}
    rows, I = case["rows"], case["I"]
    n1 = 2 * I if _swiglu(case) else I
    kept = n1 + (n1 + 31) // 32
    if kind == "save":
        return {"bytes": float(rows * (n1 * _ES[case["src"]] + I * es + 2 * kept + n1 * es)), "flops": 20.0 * rows * n1}
    return {"bytes": float(rows * (kept + I * _ES[case["src"]] + (n1 + I) * es + 8)), "flops": 30.0 * rows * n1}


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    d = torch.float64
    if kind in ("gemm", "dgrad", "wgrad", "step"):
        off = s["offsets"].tolist()
        y = s["y"].to(d) if s["y"] is not None else None
        dx = s["dx"].to(d) if s["dx"] is not None else None
        dw = db = None
        if kind == "wgrad":
            dw, db = s["dw"].to(d), s["db"].to(d)
        elif kind == "step":
            dw = torch.zeros(s["w"].shape, dtype=d, device="cuda")
            db = torch.zeros(s["w"].shape[:2], dtype=d, device="cuda")
        for g in range(case["G"]):
            r = slice(off[g], off[g + 1])
            if y is not None:
                y[r] = torch.einsum("rk,nk->rn", s["x"][r].to(d), s["w"][g].to(d))
                if s["bias"] is not None:
                    y[r] += s["bias"][g].to(d)
            if dx is not None:
                dx[r] = torch.einsum("rn,nk->rk", s["dy"][r].to(d), s["w"][g].to(d))
            if dw is not None:
                dw[g] += torch.einsum("rn,rk->nk", s["dy"][r].to(d), s["x"][r].to(d))
                db[g] += s["dy"][r].to(d).sum(0)
        if kind == "gemm":
            return y
        if kind == "dgrad":
            return dx
        return {"dw": dw, "db": db} if kind == "wgrad" else {"y": y, "dx": dx, "dw": dw, "db": db}

    def keep(x, parts):
        """The value that 8 bits stand for, from floor(log2) of each block's largest magnitude."""
        out = []
        for part in x.to(d).chunk(parts, 1):
            for lo in range(0, part.shape[1], 32):
                b = part[:, lo:lo + 32]
                top = torch.frexp(b.abs().amax(1, keepdim=True))[1] - 1  # 2^top <= max < 2^(top + 1); inputs are never subnormal
                step = (top.long() - 6 + 1023 << 52).view(d)  # 2^(top - 6), exactly
                out.append(torch.clamp(torch.round(b / step), -127, 127) * step)
        return torch.cat(out, 1)

    def slope(h):
        """act(h) and its derivatives by autograd, in 64 bits."""
        h = h.detach().requires_grad_(True)
        if _swiglu(case):
            a = torch.nn.functional.silu(h[:, :case["I"]]) * h[:, case["I"]:]
        else:
            a = torch.nn.functional.gelu(h, approximate="tanh")
        return h, a

    if kind == "rows":
        return keep(s["x"], 1)[s["row_token"].long()]
    parts = 2 if _swiglu(case) else 1
    if kind == "save":
        return {"a": slope(s["h"].to(d))[1].detach(), "kept": keep(s["h"], parts)}
    e = s["e"].to(d).repeat_interleave(32, 1).view(case["rows"], parts, -1)[:, :, :case["I"]].reshape(case["rows"], -1)
    h, a = slope(s["q"].to(d) * (e.long() - 133 + 1023 << 52).view(d))
    da = s["da"].to(d)
    (dh,) = torch.autograd.grad(a, h, da * s["row_w"].to(d)[:, None])
    a = a.detach()
    return {"dh": dh, "wa": a * s["row_w"].to(d)[:, None], "dw": (a * da).sum(1)}
