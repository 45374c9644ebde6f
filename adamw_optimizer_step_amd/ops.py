"""Python binding of the operators around the optimizer step: embedding, norms,
8-bit activation checkpoints and the weight gradient that reads one, 4-bit
matrices and the product that reads them.

They fill the gradient buffers that ``adamw_step``, ``lion_step`` and
``muon_step`` read. As in ``api``, this is argument marshalling only: every
computation runs in the HIP kernels of ``libmuon_adamw.so``, on the current
stream of the tensors' device or on ``stream``. Tensors are contiguous; results
that are not passed in are allocated for that stream. Names follow the C ABI
(include/muon_adamw.h), which states each operator's rounding and limits.

As the steps, the operators stand outside autograd: inputs are read as data,
whether they require grad or not, results have no graph and no forward-mode
tangent, and the caller runs the backward calls. Between them and autograd
stands a ``torch.autograd.Function`` of the caller's.
"""
from __future__ import annotations

import ctypes as C
from typing import Optional, Tuple, Union

import torch

from . import _lib as L
from .api import _DT, _dt

_TOKENS = {torch.int32: 4, torch.int64: 8}
# (not the public calls: those build objects, 0.3 to 1.7 us each of a call's 6)
_current_device, _current_stream = (getattr(torch._C, n, None) for n in ("_cuda_getDevice", "_cuda_getCurrentRawStream"))
_STRIDED = torch.strided


def _check(what: str, t: torch.Tensor, dtypes, shape=None) -> torch.Tensor:
    """`t` is a dense, contiguous tensor of one of `dtypes` and of `shape`."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a tensor, got {type(t).__name__}")
    if t.dtype not in dtypes:
        raise TypeError(f"{what}: unsupported dtype {t.dtype} ({', '.join(str(d) for d in dtypes)})")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.layout is not _STRIDED or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous tensor")
    return t


def _rows(what: str, t: torch.Tensor) -> Tuple[int, int]:
    """(rows, cols) of a tensor normalised over its last dimension."""
    shape = t.shape
    if not shape or shape[-1] < 1:
        raise ValueError(f"{what}: expected at least one column, got {tuple(shape)}")
    return t.numel() // shape[-1], shape[-1]


def _device(*tensors: Optional[torch.Tensor]) -> int:
    """The one GPU that all tensors are on: the library takes raw device pointers."""
    index = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"every tensor must be on {tensors[0].device}, got one on {t.device}")
    if index < 0:
        raise ValueError(f"expected CUDA tensors, got a tensor on {tensors[0].device}")
    return index


def _here(dev: int, stream) -> bool:
    """Whether a call goes to the current stream of the current device."""
    return stream is None and _current_device() == dev


def _elsewhere(dev: int, stream, call):
    """``call()`` with the tensors' device current and, where a stream is given,
    that stream too, so that what it allocates belongs to it."""
    if stream is None:
        with torch.cuda.device(dev):
            return call()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=dev)
    if stream.device.index != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{dev}")
    with torch.cuda.stream(stream):   # makes its device current too
        return call()


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _workspace(given: Optional[torch.Tensor], need: int, beside: torch.Tensor) -> torch.Tensor:
    """The caller's workspace, or one allocated for this call."""
    return beside.new_empty(max(need, 1), dtype=torch.uint8) if given is None else given


def _check_workspace(given: Optional[torch.Tensor]) -> None:
    if given is not None:
        _check("workspace", given, (torch.uint8,))


# ---------------------------------------------------------------------------
# embedding
# ---------------------------------------------------------------------------
def embedding_forward(table: torch.Tensor, tokens: torch.Tensor, scale: float = 1.0, dtype: Optional[torch.dtype] = None,
                      out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """``scale * table[tokens]`` as ``[*tokens.shape, cols]`` in ``dtype`` (the
    table's by default). A token outside the table is ignored: zeros
    (``ma_embedding_forward``)."""
    _check("table", table, _DT)
    if table.dim() != 2:
        raise ValueError(f"table: expected [rows, cols], got {tuple(table.shape)}")
    _check("tokens", tokens, _TOKENS)
    rows, cols = table.shape
    shape = (*tokens.shape, cols)
    if out is not None:
        _check("out", out, (dtype,) if dtype is not None else _DT, shape)
    elif dtype is not None and dtype not in _DT:
        raise TypeError(f"unsupported dtype {dtype} (bf16 or fp32)")
    dev = _device(table, tokens, out)
    if not _here(dev, stream):
        return _elsewhere(dev, stream, lambda: embedding_forward(table, tokens, scale, dtype, out))
    if out is None:
        out = table.new_empty(shape) if dtype is None else table.new_empty(shape, dtype=dtype)
    L.check(L.lib().ma_embedding_forward(table.data_ptr(), _dt(table), rows, cols, tokens.data_ptr(), _TOKENS[tokens.dtype],
                                         tokens.numel(), scale, out.data_ptr(), _dt(out), _current_stream(dev)))
    return out


def embedding_workspace_size(rows: int, cols: int, n_tokens: int) -> int:
    """Bytes of workspace for at most ``n_tokens`` tokens."""
    n = L.lib().ma_embedding_workspace_size(rows, cols, n_tokens)
    if n == 0:
        L.check(L.MA_ERR_INVALID_ARG)
    return int(n)


def embedding_backward(dout: torch.Tensor, tokens: torch.Tensor, grad: torch.Tensor, scale: float = 1.0,
                       accumulate: bool = False, workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The table's gradient in ``grad`` (fp32 ``[rows, cols]``, what an AdamW
    segment reads), summed over equal tokens in a fixed order: written whole,
    or with ``accumulate`` added to the rows that occur
    (``ma_embedding_backward``). Returns ``grad``."""
    _check("dout", dout, _DT)
    _check("tokens", tokens, _TOKENS)
    _check("grad", grad, (torch.float32,))
    if grad.dim() != 2:
        raise ValueError(f"grad: expected [rows, cols], got {tuple(grad.shape)}")
    rows, cols = grad.shape
    if dout.shape != (*tokens.shape, cols):
        raise ValueError(f"dout: expected shape {(*tokens.shape, cols)}, got {tuple(dout.shape)}")
    _check_workspace(workspace)
    n = tokens.numel()
    dev = _device(dout, tokens, grad, workspace)
    if not _here(dev, stream):
        return _elsewhere(dev, stream, lambda: embedding_backward(dout, tokens, grad, scale, accumulate, workspace))
    ws = _workspace(workspace, embedding_workspace_size(rows, cols, n), grad)
    L.check(L.lib().ma_embedding_backward(dout.data_ptr(), _dt(dout), tokens.data_ptr(), _TOKENS[tokens.dtype], n, rows, cols,
                                          scale, int(bool(accumulate)), grad.data_ptr(), ws.data_ptr(), ws.numel(), _current_stream(dev)))
    return grad


# ---------------------------------------------------------------------------
# 8-bit activation checkpoints
# ---------------------------------------------------------------------------
class ActCheckpoint:
    """An activation matrix ``[rows, cols]`` held in 8 bits: ``q`` (uint8
    ``[rows, P]``, P = cols rounded up to a multiple of 128) and ``scale``
    (uint8 ``[rows, P / 128]``), as ``act_pack`` writes them. ``empty`` keeps
    both in one allocation."""

    __slots__ = ("rows", "cols", "_tensors", "_q", "_scale")

    def __init__(self, q: torch.Tensor, scale: torch.Tensor, cols: int):
        blocks = -(-int(cols) // L.MA_ACT_BLOCK)
        if cols < 1:
            raise ValueError("a checkpoint has at least one column")
        rows = q.shape[0] if isinstance(q, torch.Tensor) and q.dim() == 2 else -1
        self._q = _check("q", q, (torch.uint8,), (rows, blocks * L.MA_ACT_BLOCK))
        self._scale = _check("scale", scale, (torch.uint8,), (rows, blocks))
        self._tensors = (q, scale)
        self.rows, self.cols = rows, int(cols)

    @classmethod
    def empty(cls, rows: int, cols: int, device) -> "ActCheckpoint":
        """Room for the checkpoint of a ``[rows, cols]`` matrix."""
        if rows < 0 or cols < 1:
            raise ValueError(f"no checkpoint of {rows} rows and {cols} columns")
        self = cls.__new__(cls)
        self.rows, self.cols = rows, cols
        self._tensors = (torch.empty(rows * (-(-cols // L.MA_ACT_BLOCK)) * (L.MA_ACT_BLOCK + 1), dtype=torch.uint8, device=device),)
        self._q = self._scale = None
        return self

    def _views(self) -> None:
        blocks = -(-self.cols // L.MA_ACT_BLOCK)
        n = self.rows * blocks * L.MA_ACT_BLOCK
        self._q = self._tensors[0][:n].view(self.rows, blocks * L.MA_ACT_BLOCK)
        self._scale = self._tensors[0][n:].view(self.rows, blocks)

    @property
    def q(self) -> torch.Tensor:
        if self._q is None:
            self._views()
        return self._q

    @property
    def scale(self) -> torch.Tensor:
        if self._scale is None:
            self._views()
        return self._scale

    def nbytes(self) -> int:
        return self.rows * (-(-self.cols // L.MA_ACT_BLOCK)) * (L.MA_ACT_BLOCK + 1)

    def _pointers(self) -> Tuple[int, int]:
        t = self._tensors
        p = t[0].data_ptr()
        return p, t[1].data_ptr() if len(t) == 2 else p + self.rows * (-(-self.cols // L.MA_ACT_BLOCK)) * L.MA_ACT_BLOCK


def _check_checkpoint(what: str, c: "ActCheckpoint", rows: int, cols: int) -> "ActCheckpoint":
    if not isinstance(c, ActCheckpoint):
        raise TypeError(f"{what}: expected an ActCheckpoint, got {type(c).__name__}")
    if (c.rows, c.cols) != (rows, cols):
        raise ValueError(f"{what}: a checkpoint of {(c.rows, c.cols)}, expected {(rows, cols)}")
    return c


def act_pack(x: torch.Tensor, out: Optional[ActCheckpoint] = None, stream=None) -> ActCheckpoint:
    """The 8-bit checkpoint of ``x`` (its last dimension the columns, the
    others flattened to rows; ``ma_act_pack``)."""
    _check("x", x, _DT)
    rows, cols = _rows("x", x)
    if out is not None:
        _check_checkpoint("out", out, rows, cols)
    dev = _device(x, *out._tensors) if out is not None else _device(x)
    if not _here(dev, stream):
        return _elsewhere(dev, stream, lambda: act_pack(x, out))
    if out is None:
        out = ActCheckpoint.empty(rows, cols, x.device)
    L.check(L.lib().ma_act_pack(x.data_ptr(), _dt(x), rows, cols, *out._pointers(), _current_stream(dev)))
    return out


def act_unpack(checkpoint: ActCheckpoint, dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """The values a checkpoint holds as ``[rows, cols]`` in ``dtype`` (exact in
    bf16 and fp32 alike; ``ma_act_unpack``)."""
    if not isinstance(checkpoint, ActCheckpoint):
        raise TypeError(f"expected an ActCheckpoint, got {type(checkpoint).__name__}")
    rows, cols = checkpoint.rows, checkpoint.cols
    if out is not None:
        _check("out", out, _DT)
        if out.dim() < 1 or out.shape[-1] != cols or out.numel() != rows * cols:
            raise ValueError(f"out: expected {rows} rows of {cols} columns, got {tuple(out.shape)}")
    elif dtype not in _DT:
        raise TypeError(f"unsupported dtype {dtype} (bf16 or fp32)")
    dev = _device(*checkpoint._tensors, out)
    if not _here(dev, stream):
        return _elsewhere(dev, stream, lambda: act_unpack(checkpoint, dtype, out))
    if out is None:
        out = checkpoint._tensors[0].new_empty((rows, cols), dtype=dtype)
    L.check(L.lib().ma_act_unpack(*checkpoint._pointers(), rows, cols, out.data_ptr(), _dt(out), _current_stream(dev)))
    return out


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------
def _param(what: str, t: Optional[torch.Tensor], cols: int) -> Optional[torch.Tensor]:
    return None if t is None else _check(what, t, (torch.float32,), (cols,))


def layernorm_forward(x: torch.Tensor, gain: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, eps: float = 1e-5,
                      dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
                      stats: Optional[torch.Tensor] = None, checkpoint: Optional[ActCheckpoint] = None,
                      stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Layer norm over the last dimension of ``x``; ``gain`` and ``bias`` are
    fp32 ``[cols]``. Returns ``(y, stats)``: ``y`` in ``dtype`` (x's by default)
    and fp32 ``[rows, 2]`` mean and reciprocal deviation, which the backward
    pass reads. With ``checkpoint`` (``ActCheckpoint.empty(rows, cols, device)``)
    the same pass also packs ``x`` into it (``ma_layernorm_forward``)."""
    _check("x", x, _DT)
    rows, cols = _rows("x", x)
    _param("gain", gain, cols)
    _param("bias", bias, cols)
    if out is not None:
        _check("out", out, (dtype,) if dtype is not None else _DT, x.shape)
    elif dtype is not None and dtype not in _DT:
        raise TypeError(f"unsupported dtype {dtype} (bf16 or fp32)")
    if stats is not None:
        _check("stats", stats, (torch.float32,), (rows, 2))
    held = () if checkpoint is None else _check_checkpoint("checkpoint", checkpoint, rows, cols)._tensors
    dev = _device(x, gain, bias, out, stats, *held)
    if not _here(dev, stream):
        return _elsewhere(dev, stream, lambda: layernorm_forward(x, gain, bias, eps, dtype, out, stats, checkpoint))
    if out is None:
        out = torch.empty_like(x) if dtype is None or dtype == x.dtype else x.new_empty(x.shape, dtype=dtype)
    if stats is None:
        stats = x.new_empty((rows, 2), dtype=torch.float32)
    q, sc = checkpoint._pointers() if checkpoint is not None else (None, None)
    L.check(L.lib().ma_layernorm_forward(x.data_ptr(), _dt(x), rows, cols, _ptr(gain), _ptr(bias), eps, out.data_ptr(), _dt(out),
                                         stats.data_ptr(), q, sc, _current_stream(dev)))
    return out, stats


def layernorm_workspace_size(rows: int, cols: int) -> int:
    """Bytes of workspace (0: none needed) for at most ``rows`` rows."""
    n = L.lib().ma_layernorm_workspace_size(rows, cols)
    if n == 0 and not (0 <= rows <= 1 << 24 and 1 <= cols <= 16384 and rows * cols <= 1 << 36):
        L.check(L.MA_ERR_INVALID_ARG)
    return int(n)


def layernorm_backward(dy: torch.Tensor, x: Union[torch.Tensor, ActCheckpoint], stats: torch.Tensor,
                       gain: Optional[torch.Tensor] = None, dgain: Optional[torch.Tensor] = None,
                       dbias: Optional[torch.Tensor] = None, accumulate: bool = False, dx: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The backward pass of ``layernorm_forward`` from ``dy``, ``stats`` and its
    input ``x`` or that input's 8-bit checkpoint. Returns ``dx`` (x's type; dy's
    for a checkpoint). The gradients of gain and bias go to the fp32 ``[cols]``
    buffers ``dgain`` and ``dbias`` where given, written or, with
    ``accumulate``, added to (``ma_layernorm_backward``)."""
    _check("dy", dy, _DT)
    rows, cols = _rows("dy", dy)
    if isinstance(x, ActCheckpoint):
        _check_checkpoint("x", x, rows, cols)
        xt, held, dx_dtype, xd = None, x._tensors, dy.dtype, 0
    else:
        _check("x", x, _DT, dy.shape)
        xt, held, dx_dtype, xd = x, (), x.dtype, _dt(x)
    _check("stats", stats, (torch.float32,), (rows, 2))
    _param("gain", gain, cols)
    _param("dgain", dgain, cols)
    _param("dbias", dbias, cols)
    if dx is not None:
        _check("dx", dx, (dx_dtype,), dy.shape)
    _check_workspace(workspace)
    dev = _device(dy, xt, *held, stats, gain, dgain, dbias, dx, workspace)
    if not _here(dev, stream):
        return _elsewhere(dev, stream, lambda: layernorm_backward(dy, x, stats, gain, dgain, dbias, accumulate, dx, workspace))
    if dx is None:
        dx = torch.empty_like(dy if xt is None else xt)
    q, sc = x._pointers() if held else (None, None)
    need = layernorm_workspace_size(rows, cols) if dgain is not None or dbias is not None else 0
    ws = _workspace(workspace, need, dy) if need or workspace is not None else None
    L.check(L.lib().ma_layernorm_backward(dy.data_ptr(), _dt(dy), _ptr(xt), xd, q, sc, rows, cols, stats.data_ptr(),
                                          _ptr(gain), dx.data_ptr(), _dt(dx), _ptr(dgain), _ptr(dbias), int(bool(accumulate)),
                                          _ptr(ws), ws.numel() if ws is not None else 0, _current_stream(dev)))
    return dx


# ---------------------------------------------------------------------------
# root-mean-square norm
# ---------------------------------------------------------------------------
def rmsnorm_forward(x: torch.Tensor, gain: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None, eps: float = 1e-5,
                    dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None, total: Optional[torch.Tensor] = None,
                    rstd: Optional[torch.Tensor] = None, held: Optional[ActCheckpoint] = None,
                    stream=None) -> Tuple[Union[torch.Tensor, ActCheckpoint], torch.Tensor, torch.Tensor]:
    """Root-mean-square norm over the last dimension of ``x + residual``; ``gain``
    is fp32 ``[cols]``. Returns ``(y, total, rstd)``: ``y`` in ``dtype`` (x's by
    default), the sum in the residual's type (``x`` itself without a residual),
    which is what is normalised, and fp32 ``[rows]`` reciprocal roots; the
    backward pass reads the last two. With ``held``
    (``ActCheckpoint.empty(rows, cols, device)``) y goes there, in 8 bits, and is
    returned so; with ``out`` as well it goes to both and ``out`` is returned
    (``ma_rmsnorm_forward``)."""
    _check("x", x, _DT)
    rows, cols = _rows("x", x)
    _param("gain", gain, cols)
    if residual is not None:
        _check("residual", residual, _DT, x.shape)
    if out is not None:
        _check("out", out, (dtype,) if dtype is not None else _DT, x.shape)
    elif dtype is not None and held is not None:
        raise ValueError("dtype is that of out: with held alone y has none")
    elif dtype is not None and dtype not in _DT:
        raise TypeError(f"unsupported dtype {dtype} (bf16 or fp32)")
    if total is not None:
        if residual is None:
            raise ValueError("total: there is no residual to add")
        _check("total", total, (residual.dtype,), x.shape)
    if rstd is not None:
        _check("rstd", rstd, (torch.float32,), (rows,))
    kept = () if held is None else _check_checkpoint("held", held, rows, cols)._tensors
    dev = _device(x, gain, residual, out, total, rstd, *kept)
    if not _here(dev, stream):
        return _elsewhere(dev, stream, lambda: rmsnorm_forward(x, gain, residual, eps, dtype, out, total, rstd, held))
    if out is None and held is None:
        out = torch.empty_like(x) if dtype is None or dtype == x.dtype else x.new_empty(x.shape, dtype=dtype)
    if total is None and residual is not None:
        total = torch.empty_like(residual)
    if rstd is None:
        rstd = x.new_empty((rows,), dtype=torch.float32)
    q, sc = held._pointers() if held is not None else (None, None)
    L.check(L.lib().ma_rmsnorm_forward(x.data_ptr(), _dt(x), _ptr(residual), 0 if residual is None else _dt(residual), rows, cols,
                                       _ptr(gain), eps, _ptr(total), _ptr(out), 0 if out is None else _dt(out), rstd.data_ptr(), q, sc,
                                       _current_stream(dev)))
    return held if out is None else out, x if total is None else total, rstd


def rmsnorm_workspace_size(rows: int, cols: int) -> int:
    """Bytes of workspace (0: none needed) for at most ``rows`` rows."""
    n = L.lib().ma_rmsnorm_workspace_size(rows, cols)
    if n == 0 and not (0 <= rows <= 1 << 24 and 1 <= cols <= 16384 and rows * cols <= 1 << 36):
        L.check(L.MA_ERR_INVALID_ARG)
    return int(n)


def rmsnorm_backward(dy: torch.Tensor, total: Union[torch.Tensor, ActCheckpoint], rstd: torch.Tensor,
                     gain: Optional[torch.Tensor] = None, dtotal: Optional[torch.Tensor] = None,
                     dgain: Optional[torch.Tensor] = None, accumulate: bool = False, dx: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The backward pass of ``rmsnorm_forward`` from ``dy``, ``rstd`` and what it
    normalised, ``total`` or that as an 8-bit checkpoint. ``dtotal`` is the
    gradient that reaches ``total`` on other ways. Returns ``dx`` (total's type;
    dy's for a checkpoint; dtotal has the same), the gradient of ``x`` and of
    ``residual`` alike. The gain's gradient goes to the fp32 ``[cols]`` buffer
    ``dgain`` where given, written or, with ``accumulate``, added to
    (``ma_rmsnorm_backward``)."""
    _check("dy", dy, _DT)
    rows, cols = _rows("dy", dy)
    if isinstance(total, ActCheckpoint):
        _check_checkpoint("total", total, rows, cols)
        t, held, dx_dtype, td = None, total._tensors, dy.dtype, 0
    else:
        _check("total", total, _DT, dy.shape)
        t, held, dx_dtype, td = total, (), total.dtype, _dt(total)
    _check("rstd", rstd, (torch.float32,), (rows,))
    _param("gain", gain, cols)
    _param("dgain", dgain, cols)
    if dtotal is not None:
        _check("dtotal", dtotal, (dx_dtype,), dy.shape)
    if dx is not None:
        _check("dx", dx, (dx_dtype,), dy.shape)
    _check_workspace(workspace)
    dev = _device(dy, t, *held, rstd, gain, dtotal, dgain, dx, workspace)
    if not _here(dev, stream):
        return _elsewhere(dev, stream, lambda: rmsnorm_backward(dy, total, rstd, gain, dtotal, dgain, accumulate, dx, workspace))
    if dx is None:
        dx = torch.empty_like(dy if t is None else t)
    q, sc = total._pointers() if held else (None, None)
    need = rmsnorm_workspace_size(rows, cols) if dgain is not None else 0
    ws = _workspace(workspace, need, dy) if need or workspace is not None else None
    L.check(L.lib().ma_rmsnorm_backward(dy.data_ptr(), _dt(dy), _ptr(t), td, q, sc, rows, cols, rstd.data_ptr(), _ptr(gain),
                                        _ptr(dtotal), dx.data_ptr(), _dt(dx), _ptr(dgain), int(bool(accumulate)),
                                        _ptr(ws), ws.numel() if ws is not None else 0, _current_stream(dev)))
    return dx


# ---------------------------------------------------------------------------
# 4-bit matrices and their product
# ---------------------------------------------------------------------------
class Mx4Matrix:
    """A matrix ``[rows, cols]`` held in 4 bits: ``q`` (uint8 ``[rows, P / 2]``,
    P = cols rounded up to a multiple of 128; the even column in a byte's lower
    half) and ``scale`` (uint8 ``[P / 128, rows, 4]``: for each 128 columns and
    row the powers of two of its 4 blocks of 32), as ``mx4_pack`` writes them.
    ``empty`` keeps both in one allocation."""

    __slots__ = ("rows", "cols", "_tensors")

    def __init__(self, q: torch.Tensor, scale: torch.Tensor, cols: int):
        if cols < 1:
            raise ValueError("a 4-bit matrix has at least one column")
        tiles = -(-int(cols) // L.MA_MX4_TILE)
        rows = q.shape[0] if isinstance(q, torch.Tensor) and q.dim() == 2 else -1
        _check("q", q, (torch.uint8,), (rows, tiles * (L.MA_MX4_TILE // 2)))
        _check("scale", scale, (torch.uint8,), (tiles, rows, 4))
        self._tensors = (q, scale)
        self.rows, self.cols = rows, int(cols)

    @classmethod
    def empty(cls, rows: int, cols: int, device) -> "Mx4Matrix":
        """Room for a ``[rows, cols]`` matrix."""
        if rows < 0 or cols < 1:
            raise ValueError(f"no 4-bit matrix of {rows} rows and {cols} columns")
        self = cls.__new__(cls)
        self.rows, self.cols = rows, cols
        self._tensors = (torch.empty(self.nbytes(), dtype=torch.uint8, device=device),)
        return self

    def _q_bytes(self) -> int:
        return self.rows * (-(-self.cols // L.MA_MX4_TILE)) * (L.MA_MX4_TILE // 2)

    @property
    def q(self) -> torch.Tensor:
        t = self._tensors
        return t[0] if len(t) == 2 else t[0][:self._q_bytes()].view(self.rows, -(-self.cols // L.MA_MX4_TILE) * (L.MA_MX4_TILE // 2))

    @property
    def scale(self) -> torch.Tensor:
        t = self._tensors
        return t[1] if len(t) == 2 else t[0][self._q_bytes():].view(-(-self.cols // L.MA_MX4_TILE), self.rows, 4)

    def nbytes(self) -> int:
        return self.rows * (-(-self.cols // L.MA_MX4_TILE)) * (L.MA_MX4_TILE // 2 + L.MA_MX4_TILE // L.MA_MX4_BLOCK)

    def _pointers(self) -> Tuple[int, int]:
        t = self._tensors
        p = t[0].data_ptr()
        return p, t[1].data_ptr() if len(t) == 2 else p + self._q_bytes()


def mx4_pack(x: torch.Tensor, transpose: bool = False, out: Optional[Mx4Matrix] = None, stream=None) -> Mx4Matrix:
    """``x`` (its last dimension the columns, the others flattened to rows) in 4
    bits; with ``transpose`` its transpose, ``[cols, rows]``, whose blocks of 32
    go along x's rows (``ma_mx4_pack``)."""
    _check("x", x, _DT)
    rows, cols = _rows("x", x)
    if transpose and rows == 0:
        raise ValueError("x has no rows: its transpose would have no columns")
    shape = (cols, rows) if transpose else (rows, cols)
    if out is not None:
        if not isinstance(out, Mx4Matrix):
            raise TypeError(f"out: expected an Mx4Matrix, got {type(out).__name__}")
        if (out.rows, out.cols) != shape:
            raise ValueError(f"out: a 4-bit matrix of {(out.rows, out.cols)}, expected {shape}")
    dev = _device(x, *out._tensors) if out is not None else _device(x)
    if not _here(dev, stream):
        return _elsewhere(dev, stream, lambda: mx4_pack(x, transpose, out))
    if out is None:
        out = Mx4Matrix.empty(*shape, x.device)
    L.check(L.lib().ma_mx4_pack(x.data_ptr(), _dt(x), rows, cols, int(bool(transpose)), *out._pointers(), _current_stream(dev)))
    return out


def mx4_unpack(matrix: Mx4Matrix, dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """The values a 4-bit matrix holds as ``[rows, cols]`` in ``dtype`` (exact in
    bf16 and fp32 alike; ``ma_mx4_unpack``)."""
    if not isinstance(matrix, Mx4Matrix):
        raise TypeError(f"expected an Mx4Matrix, got {type(matrix).__name__}")
    rows, cols = matrix.rows, matrix.cols
    if out is not None:
        _check("out", out, _DT)
        if out.dim() < 1 or out.shape[-1] != cols or out.numel() != rows * cols:
            raise ValueError(f"out: expected {rows} rows of {cols} columns, got {tuple(out.shape)}")
    elif dtype not in _DT:
        raise TypeError(f"unsupported dtype {dtype} (bf16 or fp32)")
    dev = _device(*matrix._tensors, out)
    if not _here(dev, stream):
        return _elsewhere(dev, stream, lambda: mx4_unpack(matrix, dtype, out))
    if out is None:
        out = matrix._tensors[0].new_empty((rows, cols), dtype=dtype)
    L.check(L.lib().ma_mx4_unpack(*matrix._pointers(), rows, cols, out.data_ptr(), _dt(out), _current_stream(dev)))
    return out


def mx4_matmul_workspace_size(rows: int, outs: int, ins: int, x_bits: int = 4) -> int:
    """Bytes of workspace (0: none needed) for exactly these sizes, and rows held
    in ``x_bits`` (4 or 8) bits: fewer rows can need more."""
    n = L.lib().ma_mx4_matmul_workspace_size(rows, outs, ins, x_bits)
    if n == 0:
        pitch = -(-ins // L.MA_MX4_TILE) * L.MA_MX4_TILE
        if x_bits not in (4, 8):
            L.check(L.MA_ERR_UNSUPPORTED)
        if not (0 <= rows <= 1 << 24 and 1 <= outs <= 1 << 23 and 1 <= ins <= 1 << 23 and max(rows * outs, rows * pitch, outs * pitch) <= 1 << 36):
            L.check(L.MA_ERR_INVALID_ARG)
    return int(n)


def mx4_matmul(x: Union[Mx4Matrix, ActCheckpoint], w: Mx4Matrix, dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
               accumulate: bool = False, workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """A linear layer on held values: ``x w^T`` as ``[rows, outs]`` in ``dtype``
    (bf16 by default), of ``x`` ``[rows, ins]`` in 4 bits or as an 8-bit
    checkpoint and the 4-bit weights ``w`` ``[outs, ins]``. With ``accumulate`` the
    product is added to ``out`` (``ma_mx4_matmul``)."""
    if not isinstance(x, (Mx4Matrix, ActCheckpoint)):
        raise TypeError(f"x: expected an Mx4Matrix or an ActCheckpoint, got {type(x).__name__}")
    if not isinstance(w, Mx4Matrix):
        raise TypeError(f"w: expected an Mx4Matrix, got {type(w).__name__}")
    rows, outs, ins, bits = x.rows, w.rows, w.cols, 8 if isinstance(x, ActCheckpoint) else 4
    if x.cols != ins:
        raise ValueError(f"x has {x.cols} columns, w {ins}")
    if out is not None:
        _check("out", out, (dtype,) if dtype is not None else _DT)
        if out.dim() < 1 or out.shape[-1] != outs or out.numel() != rows * outs:
            raise ValueError(f"out: expected {rows} rows of {outs} columns, got {tuple(out.shape)}")
    elif accumulate:
        raise ValueError("accumulate: there is no out to add to")
    elif dtype is not None and dtype not in _DT:
        raise TypeError(f"unsupported dtype {dtype} (bf16 or fp32)")
    _check_workspace(workspace)
    dev = _device(*x._tensors, *w._tensors, out, workspace)
    if not _here(dev, stream):
        return _elsewhere(dev, stream, lambda: mx4_matmul(x, w, dtype, out, accumulate, workspace))
    if out is None:
        out = w._tensors[0].new_empty((rows, outs), dtype=dtype or torch.bfloat16)
    need = mx4_matmul_workspace_size(rows, outs, ins, bits)
    ws = _workspace(workspace, need, out) if need or workspace is not None else None
    L.check(L.lib().ma_mx4_matmul(*x._pointers(), bits, rows, *w._pointers(), outs, ins, out.data_ptr(), _dt(out), int(bool(accumulate)),
                                  _ptr(ws), ws.numel() if ws is not None else 0, _current_stream(dev)))
    return out


# ---------------------------------------------------------------------------
# weight gradient
# ---------------------------------------------------------------------------
def act_weight_grad_workspace_size(tokens: int, outs: int, ins: int, dtype: torch.dtype = torch.bfloat16) -> int:
    """Bytes of workspace (0: none needed) for dy of ``dtype`` and exactly these
    sizes: fewer tokens can need more, so a workspace for calls of several
    sizes takes the largest of theirs."""
    if dtype not in _DT:
        raise TypeError(f"unsupported dtype {dtype} (bf16 or fp32)")
    n = L.lib().ma_act_weight_grad_workspace_size(tokens, outs, ins, _DT[dtype])
    if n == 0 and not (0 <= tokens <= 1 << 25 and 1 <= outs <= 1 << 23 and 1 <= ins <= 1 << 23 and outs * ins <= 1 << 31
                       and tokens * max(outs, -(-ins // L.MA_ACT_BLOCK) * L.MA_ACT_BLOCK) <= 1 << 36):
        L.check(L.MA_ERR_INVALID_ARG)
    return int(n)


def act_weight_grad(dy: torch.Tensor, x: ActCheckpoint, grad: torch.Tensor, accumulate: bool = False,
                    workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The weight gradient of ``y = x W^T`` in ``grad`` (``[outs, ins]``, bf16
    or fp32: a matrix of a ``MuonGroup``'s gradients), out of the 8-bit
    checkpoint of ``x``: ``grad (+)= dy^T x`` (``ma_act_weight_grad``). ``dy``:
    ``[..., outs]`` with as many rows as the checkpoint. Returns ``grad``."""
    _check("dy", dy, _DT)
    tokens, outs = _rows("dy", dy)
    if not isinstance(x, ActCheckpoint):
        raise TypeError(f"x: expected an ActCheckpoint, got {type(x).__name__}")
    if x.rows != tokens:
        raise ValueError(f"dy has {tokens} rows, the checkpoint {x.rows}")
    _check("grad", grad, _DT, (outs, x.cols))
    _check_workspace(workspace)
    dev = _device(dy, *x._tensors, grad, workspace)
    if not _here(dev, stream):
        return _elsewhere(dev, stream, lambda: act_weight_grad(dy, x, grad, accumulate, workspace))
    need = act_weight_grad_workspace_size(tokens, outs, x.cols, dy.dtype)
    ws = _workspace(workspace, need, grad) if need or workspace is not None else None
    L.check(L.lib().ma_act_weight_grad(dy.data_ptr(), _dt(dy), *x._pointers(), tokens, outs, x.cols, grad.data_ptr(), _dt(grad),
                                       int(bool(accumulate)), _ptr(ws), ws.numel() if ws is not None else 0, _current_stream(dev)))
    return grad
