"""Torch-side convenience around the C ABI: descriptor and weight structs
from tensors, a workspace buffer, and views of the intermediates that
moe_forward leaves in it.  No computation happens here."""
from __future__ import annotations

import torch

from . import abi

_GATES = {"softmax": abi.GATE_SOFTMAX, "sigmoid_bias": abi.GATE_SIGMOID_BIAS}
_ACTS = {"gelu_tanh": abi.ACT_GELU_TANH, "swiglu": abi.ACT_SWIGLU}
_DTYPES = {"f32": abi.DTYPE_F32, "bf16": abi.DTYPE_BF16}


def desc_from_config(cfg: dict, T: int | None = None) -> abi.LayerDesc:
    d = abi.LayerDesc()
    d.dtype = _DTYPES[cfg["dtype"]]
    d.T = cfg["T"] if T is None else T
    d.D, d.M, d.k, d.I = cfg["D"], cfg["M"], cfg["k"], cfg["I"]
    d.gate = _GATES[cfg["gate"]]
    d.act = _ACTS[cfg["act"]]
    d.has_bias = int(bool(cfg.get("has_bias", 0)))
    d.norm_topk_prob = int(bool(cfg.get("norm_topk_prob", 1)))
    d.routed_scaling_factor = float(cfg.get("alpha", 1.0))
    d.eps = float(cfg.get("eps", 1e-20))
    d.I_sh = int(cfg.get("I_sh", 0) or 0)
    d.n_group = int(cfg.get("n_group", 1) or 1)
    d.topk_group = int(cfg.get("topk_group", 1) or 1)
    return d


def dense_desc_from_config(cfg: dict, T: int | None = None) -> abi.DenseDesc:
    d = abi.DenseDesc()
    d.dtype = _DTYPES[cfg["dtype"]]
    d.T = cfg["T"] if T is None else T
    d.D, d.I = cfg["D"], cfg["I"]
    d.act = _ACTS[cfg["act"]]
    d.has_bias = int(bool(cfg.get("has_bias", 0)))
    return d


def _ptr(t):
    return None if t is None else t.data_ptr()


def weights_from_tensors(t: dict) -> abi.Weights:
    w = abi.Weights()
    for name in ("w_r", "e_bias", "w1", "b1", "w2", "b2", "sh_w1", "sh_w2"):
        v = t.get(name)
        if v is not None and not v.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        setattr(w, name, _ptr(v))
    return w


def _stream_handle(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


class LayerCheckpoint:
    """What one forward of ``layer`` keeps for its backward: the routing, and
    the pre-activations in 8 bits.  Holds for one forward at a time; a step
    that keeps several (gradient accumulation over overlapping micro-batches)
    takes one each."""

    def __init__(self, layer: "MoELayer"):
        self.nbytes = abi.moe_checkpoint_size(layer.desc)
        if self.nbytes == 0 and layer.desc.T > 0:
            raise abi.MoEError("moe_checkpoint_size", abi.MOE_ERR_INVALID_ARG)
        self.buffer = torch.empty(self.nbytes + 256, dtype=torch.uint8, device=layer.device)
        self._off = (-self.buffer.data_ptr()) % 256
        self.ptr = self.buffer.data_ptr() + self._off
        self.desc = layer.desc

    def view(self, name: str) -> torch.Tensor:
        """A part of the checkpoint as a tensor: "topk_idx", "topk_w" [T, k],
        "logits" [T, M], "q", "e" (the routed experts' pre-activations, rows
        in dispatch order) or "shared_q", "shared_e"."""
        d = self.desc
        halves = 2 if d.act == abi.ACT_SWIGLU else 1
        shapes = {"topk_idx": ((d.T, d.k), torch.int32), "topk_w": ((d.T, d.k), torch.float32),
                  "logits": ((d.T, d.M), torch.float32), "q": ((d.T * d.k, halves * d.I), torch.int8),
                  "e": ((d.T * d.k, halves * abi.moe_ckpt_blocks(d.I)), torch.uint8),
                  "shared_q": ((d.T, 2 * d.I_sh), torch.int8),
                  "shared_e": ((d.T, 2 * abi.moe_ckpt_blocks(d.I_sh)), torch.uint8)}
        shape, dt = shapes[name]
        off = self._off + abi.moe_checkpoint_offsets(d)[list(shapes).index(name)]
        nbytes = shape[0] * shape[1] * torch.empty((), dtype=dt).element_size()
        return self.buffer[off:off + nbytes].view(dt).view(shape)


class MoELayer:
    """One MoE layer bound to device weight tensors (kept alive here)."""

    def __init__(self, cfg: dict, tensors: dict, T: int | None = None):
        self.cfg = cfg
        self.tensors = tensors
        self.desc = desc_from_config(cfg, T)
        self.weights = weights_from_tensors(tensors)
        self.device = tensors["w_r"].device
        self.ws_bytes = abi.moe_workspace_size(self.desc)
        if self.ws_bytes == 0:
            raise abi.MoEError("moe_workspace_size", abi.MOE_ERR_INVALID_ARG)
        self.ws = torch.zeros(self.ws_bytes + 256, dtype=torch.uint8, device=self.device)
        base = self.ws.data_ptr()
        self._ws_off = (-base) % 256
        self.layout = abi.moe_workspace_layout(self.desc)
        self._fwd = (self.ws, self._ws_off)  # the last forward's workspace
        self._fwd_kept = False
        self._bws = None
        self._save = None
        self._cws = None
        self._last_bws = None

    @property
    def ws_ptr(self) -> int:
        return self.ws.data_ptr() + self._ws_off

    def forward(self, x: torch.Tensor, y: torch.Tensor | None = None, stream=None,
                addend: torch.Tensor | None = None, checkpoint: LayerCheckpoint | None = None) -> torch.Tensor:
        """y = MoE-FFN(x), or addend + MoE-FFN(x) when ``addend`` is given.
        With ``checkpoint`` the pass also keeps there what
        ``backward(..., checkpoint=...)`` needs (moe_forward_save).  What a
        call allocates is allocated on the stream that it runs on."""
        if y is None:
            with torch.cuda.stream(stream):
                y = torch.empty_like(x)
        if checkpoint is not None:
            if self._save is None:
                nbytes = abi.moe_forward_save_workspace_size(self.desc)
                # a bf16 layer keeps them from its own workspace
                self._save = ((self.ws, self._ws_off, self.ws_bytes) if nbytes <= self.ws_bytes
                              else self._scratch(nbytes, stream))
            buf, off, nbytes = self._save
            abi.moe_forward_save(self.desc, self.weights, x.data_ptr(), _ptr(addend), y.data_ptr(), checkpoint.ptr,
                                 checkpoint.nbytes, buf.data_ptr() + off, nbytes, _stream_handle(stream))
            self._fwd, self._fwd_kept = (buf, off), True
            return y
        self._fwd, self._fwd_kept = (self.ws, self._ws_off), False
        if addend is None:
            abi.moe_forward(self.desc, self.weights, x.data_ptr(), y.data_ptr(), self.ws_ptr, self.ws_bytes,
                            _stream_handle(stream))
        else:
            abi.moe_forward_add(self.desc, self.weights, x.data_ptr(), addend.data_ptr(), y.data_ptr(),
                                self.ws_ptr, self.ws_bytes, _stream_handle(stream))
        return y

    def _scratch(self, nbytes: int, stream):
        """(buffer, offset of its first 256-byte boundary, bytes), allocated on the stream that will use it.  Its first
        word is the status, which every call with tokens clears and one without leaves as it is."""
        with torch.cuda.stream(stream):
            buf = torch.empty(nbytes + 256, dtype=torch.uint8, device=self.device)
            off = (-buf.data_ptr()) % 256
            if self.desc.T == 0:
                buf[off:off + 4].zero_()
        return buf, off, nbytes

    def device_status(self, stream=None) -> int:
        """The status of the last forward."""
        return abi.moe_device_status(self._fwd[0].data_ptr() + self._fwd[1], _stream_handle(stream))

    def grad_shapes(self) -> dict:
        """Shapes of the gradients moe_backward writes (None: not written)."""
        d = self.desc
        swiglu = d.act == abi.ACT_SWIGLU
        n1 = 2 * d.I if swiglu else d.I
        biases = (not swiglu) and bool(d.has_bias)
        return {
            "dx": (d.T, d.D), "dw_r": (d.D, d.M), "dw1": (d.M, n1, d.D), "dw2": (d.M, d.D, d.I),
            "db1": (d.M, d.I) if biases else None, "db2": (d.M, d.D) if biases else None,
            "dsh_w1": (2 * d.I_sh, d.D) if d.I_sh else None, "dsh_w2": (d.D, d.I_sh) if d.I_sh else None,
        }

    def backward(self, x: torch.Tensor, dy: torch.Tensor, grads: dict | None = None, stream=None,
                 checkpoint: LayerCheckpoint | None = None) -> dict:
        """Gradients of L = sum(dy * MoE-FFN(x)) (moe_backward): dx in the
        layer's dtype, every parameter gradient in fp32.  The backward has its
        own workspace (allocated on first use); ``backward_view`` reads the
        routing it recomputed.  With the ``checkpoint`` of a forward on the
        same x nothing of that forward is recomputed (moe_backward_saved)."""
        if checkpoint is not None and self._cws is None:
            self._cws = self._scratch(abi.moe_backward_saved_workspace_size(self.desc), stream)
        if checkpoint is None and self._bws is None:
            self.bws_bytes = abi.moe_backward_workspace_size(self.desc)
            if self.bws_bytes == 0:
                raise abi.MoEError("moe_backward_workspace_size", abi.MOE_ERR_INVALID_ARG)
            with torch.cuda.stream(stream):
                self._bws = torch.zeros(self.bws_bytes + 256, dtype=torch.uint8, device=self.device)
            self._bws_off = (-self._bws.data_ptr()) % 256
        if grads is None:
            grads = {}
            with torch.cuda.stream(stream):
                for name, shape in self.grad_shapes().items():
                    if shape is not None:
                        dt = x.dtype if name == "dx" else torch.float32
                        grads[name] = torch.empty(shape, dtype=dt, device=self.device)
        g = abi.Grads()
        for name in abi.Grads._fields_:
            setattr(g, name[0], _ptr(grads.get(name[0])))
        if checkpoint is not None:
            buf, off, nbytes = self._cws
            self._last_bws = buf.data_ptr() + off
            abi.moe_backward_saved(self.desc, self.weights, x.data_ptr(), dy.data_ptr(), checkpoint.ptr,
                                   checkpoint.nbytes, g, self._last_bws, nbytes, _stream_handle(stream))
            return grads
        self._last_bws = self._bws.data_ptr() + self._bws_off
        abi.moe_backward(self.desc, self.weights, x.data_ptr(), dy.data_ptr(), g, self._last_bws, self.bws_bytes,
                         _stream_handle(stream))
        return grads

    def backward_status(self, stream=None) -> int:
        """The status of the last backward."""
        return abi.moe_device_status(self._last_bws, _stream_handle(stream))

    def backward_view(self, name: str) -> torch.Tensor:
        """The routing intermediate ``name`` that the last backward recomputed."""
        if self._bws is None or self._last_bws != self._bws.data_ptr() + self._bws_off:
            raise RuntimeError("the last backward recomputed no routing: from a checkpoint it is the checkpoint's")
        return self.view(name, ws=(self._bws, self._bws_off))

    def view(self, name: str, dtype=None, ws=None) -> torch.Tensor:
        """The intermediate ``name`` of the last forward, as a tensor view."""
        d = self.desc
        pairs = d.T * d.k
        shapes = {
            "status": ((1,), torch.int32), "topk_idx": ((d.T, d.k), torch.int32),
            "topk_w": ((d.T, d.k), torch.float32), "counts": ((d.M,), torch.int32),
            "offsets": ((d.M + 1,), torch.int32), "slot_of": ((d.T, d.k), torch.int32),
            "row_token": ((pairs,), torch.int32), "row_w": ((pairs,), torch.float32),
            "out_perm": ((pairs, d.D), torch.float32),
        }
        shape, dt = shapes[name]
        if ws is None and self._fwd_kept and name in ("topk_idx", "topk_w"):
            raise RuntimeError(f"the last forward kept {name} in its checkpoint")
        buf, base = self._fwd if ws is None else ws
        off = base + getattr(self.layout, name)
        n = 1
        for s in shape:
            n *= s
        nbytes = n * torch.empty((), dtype=dt).element_size()
        return buf[off:off + nbytes].view(dt).view(*shape)


class DenseLayer:
    """One dense FFN layer (w1, b1, w2, b2 device tensors, kept alive here)."""

    def __init__(self, cfg: dict, tensors: dict, T: int | None = None):
        self.cfg = cfg
        self.tensors = tensors
        self.desc = dense_desc_from_config(cfg, T)
        for name in ("w1", "b1", "w2", "b2"):
            v = tensors.get(name)
            if v is not None and not v.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        self.ws_bytes = abi.moe_dense_ffn_workspace_size(self.desc)
        if self.ws_bytes == 0:
            raise abi.MoEError("moe_dense_ffn_workspace_size", abi.MOE_ERR_INVALID_ARG)
        self.ws = torch.zeros(self.ws_bytes + 256, dtype=torch.uint8, device=tensors["w1"].device)
        self._ws_off = (-self.ws.data_ptr()) % 256

    @property
    def ws_ptr(self) -> int:
        return self.ws.data_ptr() + self._ws_off

    def args(self):
        t = self.tensors
        return (_ptr(t["w1"]), _ptr(t.get("b1")), _ptr(t["w2"]), _ptr(t.get("b2")))

    def forward(self, x: torch.Tensor, addend: torch.Tensor | None = None, y: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
        """y = (addend +) FFN(x)."""
        if y is None:
            with torch.cuda.stream(stream):
                y = torch.empty_like(x)
        abi.moe_dense_ffn(self.desc, *self.args(), x.data_ptr(), _ptr(addend), y.data_ptr(), self.ws_ptr,
                          self.ws_bytes, _stream_handle(stream))
        return y

    def device_status(self, stream=None) -> int:
        return abi.moe_device_status(self.ws_ptr, _stream_handle(stream))
