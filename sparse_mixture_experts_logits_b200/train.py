"""Torch-side handles of the experts' step-by-step operators: the matrix
products grouped by expert (GroupedLinear) and the 8-bit activation
checkpoints (RowCheckpoint, ActivationCheckpoint).  Each checks its tensors,
holds its workspace or checkpoint and calls the C ABI; no computation happens
here.  Nothing is recorded for autograd: results are plain tensors, also for
parameters that require gradients.

Every call runs on ``stream``, or on the current stream of the handle's device
when none is given; what it allocates (outputs, and at the first call the
workspace) is allocated on that stream.  The caller keeps tensors made on
another stream alive and ordered, as for any torch extension.  Calls of one
handle share its workspace or checkpoint, so they must be ordered on one
stream; a step that is captured into a CUDA graph and replayed beside eager
calls takes a handle of its own.
"""
from __future__ import annotations

import torch

from . import abi

_ACTS = {"gelu_tanh": abi.ACT_GELU_TANH, "swiglu": abi.ACT_SWIGLU}
_DTYPES = {torch.float32: abi.DTYPE_F32, torch.bfloat16: abi.DTYPE_BF16}


def _dtype(dt):
    try:
        return _DTYPES[dt]
    except KeyError:
        raise ValueError(f"dtype must be torch.float32 or torch.bfloat16, not {dt}") from None


def _int32(name, v):
    """v, which the C interface takes in 32 bits."""
    if not -2 ** 31 <= int(v) < 2 ** 31:
        raise ValueError(f"{name} = {v} is no 32-bit number")
    return int(v)


def _device(device):
    d = torch.device(device)
    if d.type != "cuda":
        raise ValueError(f"the operators run on CUDA devices, not {d}")
    return torch.device("cuda", torch.cuda.current_device()) if d.index is None else d


class _Handle:
    """The device, and the checks of every tensor against it."""

    device: torch.device
    rows: int

    def _in(self, name, t, shape, dtype):
        """t's address; t must be a contiguous [shape] tensor of dtype on the handle's device."""
        if t.dtype is not dtype or t.shape != shape or t.device != self.device or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape} on {self.device}, got "
                             f"{t.dtype} {tuple(t.shape)} on {t.device}"
                             f"{'' if t.is_contiguous() else ', not contiguous'}")
        return t.data_ptr()

    def _opt(self, name, t, shape, dtype):
        return None if t is None else self._in(name, t, shape, dtype)

    def _new(self, shape, dtype, stream):
        if stream is not None:
            with torch.cuda.stream(stream):
                return self._new(shape, dtype, None)
        # from an empty tensor of the dtype: half a microsecond less than torch.empty with a dtype and a device
        protos = self.__dict__.setdefault("_protos", {})
        if dtype not in protos:
            protos[dtype] = torch.empty(0, dtype=dtype, device=self.device)
        return protos[dtype].new_empty(shape)

    def _out(self, name, t, shape, dtype, stream=None):
        if t is None:
            return self._new(shape, dtype, stream)
        self._in(name, t, shape, dtype)
        return t

    def _wanted(self, name, t, shape, dtype, stream):
        """An optional output: False or None (not written), True (allocated) or a tensor."""
        if t is None or t is False:
            return None
        return self._out(name, None if t is True else t, shape, dtype, stream)

    def _stream(self, stream):
        if stream is None:
            return torch._C._cuda_getCurrentRawStream(self.device.index)
        if stream.device != self.device:
            raise ValueError(f"the stream is on {stream.device}, the handle on {self.device}")
        return stream.cuda_stream

    def _call(self, fn, *args):
        if torch._C._cuda_getDevice() == self.device.index:
            fn(*args)
        else:
            with torch.cuda.device(self.device):
                fn(*args)

    def _workspace(self, nbytes, stream):
        """(256-byte aligned address, bytes, buffer).  Every call with rows clears the status word itself; without rows
        no call touches the workspace, so that the word has to start at 0."""
        buf = self._new((nbytes + 256,), torch.uint8, stream)
        off = (-buf.data_ptr()) % 256
        if self.rows == 0:
            with torch.cuda.stream(stream):
                buf[off:off + 4].zero_()
        return buf.data_ptr() + off, nbytes, buf


class GroupedLinear(_Handle):
    """One linear layer per expert over ragged row segments.

    weight  [G, N, K] (kept alive here, read at every call);
    rows    rows of x, y, dy and dx (an upper bound of offsets[G]: a batch of
            fewer rows uses the first ones);
    bias    [G, N] or None, in the weight's dtype;
    out_dtype  dtype of y and dx (default: the weight's).

    ``offsets`` is the int32 [G + 1] tensor that moe_permute writes: expert
    g's rows are offsets[g] .. offsets[g + 1].  Rows behind the last segment
    are not read and their outputs not written.
    """

    def __init__(self, weight: torch.Tensor, rows: int, bias: torch.Tensor | None = None,
                 out_dtype: torch.dtype | None = None):
        if weight.dim() != 3:
            raise ValueError("weight must be [G, N, K]")
        self.device = _device(weight.device)
        self.dtype, self.rows = weight.dtype, _int32("rows", rows)
        self.out_dtype = weight.dtype if out_dtype is None else out_dtype
        self.G, self.N, self.K = (_int32("a dimension of weight", d) for d in weight.shape)
        self._dt, self._odt = _dtype(self.dtype), _dtype(self.out_dtype)
        self._in("weight", weight, (self.G, self.N, self.K), self.dtype)
        self._opt("bias", bias, (self.G, self.N), self.dtype)
        self.weight, self.bias = weight, bias
        self._dims = (self.G, self.N, self.K, self.rows, self._dt)
        self._ws_bytes = abi.moe_grouped_workspace_size(*self._dims)
        if self._ws_bytes == 0:
            raise abi.MoEError("moe_grouped_workspace_size", abi.MOE_ERR_INVALID_ARG)
        self._ws = self._wg = None  # the row products' workspace, the weight gradient's

    def forward(self, x: torch.Tensor, offsets: torch.Tensor, y: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
        """y[r] = x[r] W_g^T (+ bias[g])."""
        px = self._in("x", x, (self.rows, self.K), self.dtype)
        po = self._in("offsets", offsets, (self.G + 1,), torch.int32)
        y = self._out("y", y, (self.rows, self.N), self.out_dtype, stream)
        if self._ws is None:
            self._ws = self._workspace(self._ws_bytes, stream)
        self._call(abi.moe_grouped_gemm, px, self.weight.data_ptr(),
                   None if self.bias is None else self.bias.data_ptr(), po, *self._dims, self._odt, y.data_ptr(),
                   self._ws[0], self._ws_bytes, self._stream(stream))
        return y

    def input_grad(self, dy: torch.Tensor, offsets: torch.Tensor, dx: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
        """dx[r] = dy[r] W_g."""
        pd = self._in("dy", dy, (self.rows, self.N), self.dtype)
        po = self._in("offsets", offsets, (self.G + 1,), torch.int32)
        dx = self._out("dx", dx, (self.rows, self.K), self.out_dtype, stream)
        if self._ws is None:
            self._ws = self._workspace(self._ws_bytes, stream)
        self._call(abi.moe_grouped_dgrad, pd, self.weight.data_ptr(), po, *self._dims, self._odt, dx.data_ptr(),
                   self._ws[0], self._ws_bytes, self._stream(stream))
        return dx

    def weight_grad(self, x: torch.Tensor, dy: torch.Tensor, offsets: torch.Tensor, dw: torch.Tensor | None = None,
                    db: torch.Tensor | bool | None = None, accumulate: bool = False, stream=None):
        """(dw, db): dw[g] = sum of dy[r]^T x[r] over g's rows (fp32 [G, N, K])
        and, when db is True or a tensor, db[g] = sum of dy[r] (fp32 [G, N]).
        accumulate adds onto dw and db, which the caller then gives."""
        if accumulate and (dw is None or db is True):
            raise ValueError("accumulate adds onto the dw and db that are given")
        px = self._in("x", x, (self.rows, self.K), self.dtype)
        pd = self._in("dy", dy, (self.rows, self.N), self.dtype)
        po = self._in("offsets", offsets, (self.G + 1,), torch.int32)
        dw = self._out("dw", dw, (self.G, self.N, self.K), torch.float32, stream)
        db = self._wanted("db", db, (self.G, self.N), torch.float32, stream)
        if self._wg is None:
            self._wg = self._workspace(abi.moe_grouped_wgrad_workspace_size(*self._dims), stream)
        self._call(abi.moe_grouped_wgrad, px, pd, po, *self._dims, int(bool(accumulate)), dw.data_ptr(),
                   None if db is None else db.data_ptr(), self._wg[0], self._wg[1], self._stream(stream))
        return dw, db

    def device_status(self, stream=None) -> int:
        """The first error that the last calls' kernels reported (0: none), and clears it.  Synchronises."""
        s = self._stream(stream)
        with torch.cuda.device(self.device):
            codes = [abi.moe_device_status(ws[0], s) for ws in (self._ws, self._wg) if ws is not None]
        return next((c for c in codes if c), 0)


class RowCheckpoint(_Handle):
    """Rows [rows, cols] kept in 8 bits: ``q`` int8 [rows, cols] and the blocks' exponents ``e``."""

    def __init__(self, rows: int, cols: int, dtype: torch.dtype, device="cuda"):
        self.device = _device(device)
        self.rows, self.cols, self.dtype = _int32("rows", rows), _int32("cols", cols), dtype
        self._dt = _dtype(dtype)
        self.blocks = abi.moe_ckpt_blocks(self.cols)
        if self.rows < 0 or self.blocks == 0:
            raise ValueError(f"a checkpoint of {rows} rows of {cols} columns")
        self.q = torch.empty((self.rows, self.cols), dtype=torch.int8, device=self.device)
        self.e = torch.empty((self.rows, self.blocks), dtype=torch.uint8, device=self.device)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)

    def save(self, x: torch.Tensor, n_rows: torch.Tensor | None = None, stream=None) -> None:
        """Keeps x [rows, cols] (its first n_rows[0] rows when the device int32 n_rows is given)."""
        self._call(abi.moe_ckpt_quantize, self._in("x", x, (self.rows, self.cols), self.dtype),
                   self._opt("n_rows", n_rows, (1,), torch.int32), self.rows, self.cols, self._dt, self.q.data_ptr(),
                   self.e.data_ptr(), self._stream(stream))

    def load(self, row_index: torch.Tensor | None = None, n_rows: torch.Tensor | None = None,
             out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """The kept rows, or rows row_index[r] of them (int32; an index out of
        range gives a zero row and sets ``status``)."""
        n = self.rows if row_index is None else _int32("rows of row_index", row_index.numel())
        pi = self._opt("row_index", row_index, (n,), torch.int32)
        out = self._out("out", out, (n, self.cols), self.dtype, stream)
        self._call(abi.moe_ckpt_dequantize, self.q.data_ptr(), self.e.data_ptr(), pi,
                   self._opt("n_rows", n_rows, (1,), torch.int32), n, self.rows, self.cols, self._dt, out.data_ptr(),
                   self.status.data_ptr(), self._stream(stream))
        return out


class ActivationCheckpoint(_Handle):
    """The experts' activation with its input kept in 8 bits for the backward.

    act "swiglu" (h [rows, 2I], gate columns first) or "gelu_tanh" (h [rows,
    I]); ``dtype`` is that of act(h), dh and wa, ``src_dtype`` (default: dtype)
    that of h and da.  q and e may be given (a checkpoint kept elsewhere).
    """

    def __init__(self, act: str, rows: int, I: int, dtype: torch.dtype, src_dtype: torch.dtype | None = None,
                 device="cuda", q: torch.Tensor | None = None, e: torch.Tensor | None = None):
        if act not in _ACTS:
            raise ValueError(f"act must be one of {sorted(_ACTS)}, not {act!r}")
        self.device = _device(device)
        self.act, self.rows, self.I, self.dtype = act, _int32("rows", rows), _int32("I", I), dtype
        self.src_dtype = dtype if src_dtype is None else src_dtype
        self._dts = (_ACTS[act], _dtype(dtype), _dtype(self.src_dtype))
        halves = 2 if act == "swiglu" else 1
        self.width = halves * self.I
        self.blocks = abi.moe_ckpt_blocks(self.I)
        if self.rows < 0 or self.blocks == 0:
            raise ValueError(f"a checkpoint of {rows} rows of width {I}")
        self._halves = halves
        self.q = self._out("q", q, (self.rows, self.width), torch.int8)
        self.e = self._out("e", e, (self.rows, halves * self.blocks), torch.uint8)

    def save(self, h: torch.Tensor, a: torch.Tensor | None = None, n_rows: torch.Tensor | None = None,
             stream=None) -> torch.Tensor:
        """a = act(h); h is kept."""
        ph = self._in("h", h, (self.rows, self.width), self.src_dtype)
        a = self._out("a", a, (self.rows, self.I), self.dtype, stream)
        self._call(abi.moe_act_save, ph, self._opt("n_rows", n_rows, (1,), torch.int32), self.rows, self.I, *self._dts,
                   a.data_ptr(), self.q.data_ptr(), self.e.data_ptr(), self._stream(stream))
        return a

    def load(self, stream=None) -> torch.Tensor:
        """The kept h [rows, width], in dtype."""
        out = self._new((self.rows, self.width), self.dtype, stream)
        n = _int32("rows", self.rows * self._halves)
        self._call(abi.moe_ckpt_dequantize, self.q.data_ptr(), self.e.data_ptr(), None, None, n, n, self.I,
                   self._dts[1], out.data_ptr(), None, self._stream(stream))
        return out

    def backward(self, da: torch.Tensor, row_w: torch.Tensor | None = None, dh: torch.Tensor | None = None,
                 wa: torch.Tensor | bool | None = None, dw: torch.Tensor | bool | None = None,
                 n_rows: torch.Tensor | None = None, stream=None):
        """(dh, wa, dw) from da [rows, I], the gradient reaching act(h) before
        the row's gate weight row_w (fp32 [rows], None: 1): dh = row_w da
        act'(h), wa = row_w act(h), dw[r] = <da[r], act(h)[r]>, all of the kept
        h.  wa and dw are written when True or a tensor is given."""
        pd = self._in("da", da, (self.rows, self.I), self.src_dtype)
        pw = self._opt("row_w", row_w, (self.rows,), torch.float32)
        dh = self._out("dh", dh, (self.rows, self.width), self.dtype, stream)
        wa = self._wanted("wa", wa, (self.rows, self.I), self.dtype, stream)
        dw = self._wanted("dw", dw, (self.rows,), torch.float32, stream)
        self._call(abi.moe_act_backward, self.q.data_ptr(), self.e.data_ptr(), pd, pw,
                   self._opt("n_rows", n_rows, (1,), torch.int32), self.rows, self.I, *self._dts, dh.data_ptr(),
                   None if wa is None else wa.data_ptr(), None if dw is None else dw.data_ptr(),
                   self._stream(stream))
        return dh, wa, dw
