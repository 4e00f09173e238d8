"""Binding of the operators at a model's ends and of its dense layers (token
embedding, block-scaled E4M3 matrices, global gradient norm): argument
marshalling only, by the rules of ``_ops``."""
from __future__ import annotations

import ctypes
from ctypes import byref
from dataclasses import dataclass

import numpy as np

from . import _ops
from ._lib import F32, Fp8BlocksView, GradNormEntry, Tokens, _check, load
from ._ops import _float_code, _given_workspace, _matrix, _on, _refuse_device, _vec

FP8_BLOCK = 128      # SS1_FP8_BLOCK


def _elsewhere(stream, dev: int) -> bool:
    """Whether a call has to change the stream or the device first."""
    return stream is not None or dev < 0 or dev != _ops._current_device()


def _room(workspace, nbytes: int, like, dev: int):
    """(tensor to keep, address, bytes) of a call's workspace."""
    if workspace is not None:
        return workspace, *_given_workspace(workspace, dev)
    if nbytes == 0:
        return None, None, 0
    workspace = _ops._torch.empty((nbytes,), dtype=_ops._torch.uint8, device=like.device)
    return workspace, workspace.data_ptr(), nbytes


# ------------------------------------------------------------- gradient norm
@dataclass
class GradNormPlan:
    """The global gradient norm over many tensors, and clipping by it: the table
    of the gradients' addresses and the list of work items, made once on the
    host and copied to the GPU, and a workspace.  It holds for as long as the
    gradients stay where they are (it keeps them alive).  A deep copy or a
    loaded plan has gradients of its own, and a table of them."""
    entries: object      # uint8 device tensor: the ss1_gradnorm_entry table
    map: object          # int32 device tensor [chunks][2]
    count: int
    chunks: int
    grads: list

    def __reduce__(self):
        # not the table: a copy's tensors lie at other addresses
        return GradNormPlan.make, (self.grads,)

    @classmethod
    def make(cls, grads):
        """``grads``: GPU tensors (float32 or bfloat16, contiguous) that share
        no memory; the lists that :class:`AdamWPlan` takes serve."""
        torch = _ops._torch or _ops._setup()
        grads = list(grads)
        n = len(grads)
        table = (GradNormEntry * max(n, 1))()
        rows = np.frombuffer(table, dtype=np.dtype(GradNormEntry))[:n]
        dev = grads[0].get_device() if grads else 0
        if dev < 0:
            _refuse_device(dev)
        for g in grads:
            if g.get_device() != dev:
                _refuse_device(g.get_device())
            if not g.is_contiguous():
                raise ValueError("gradients must be contiguous")
        rows["grad"], rows["numel"] = [g.data_ptr() for g in grads], [g.numel() for g in grads]
        rows["dtype"] = [_float_code(g, "grad") for g in grads]
        used = np.flatnonzero(rows["numel"] > 0)
        at = rows["grad"][used]
        end = at + (rows["numel"][used] * np.where(rows["dtype"][used] == F32, 4, 2)).astype(np.uint64)
        order = np.argsort(at, kind="stable")
        if (end[order[:-1]] > at[order[1:]]).any():
            raise ValueError("gradients must not share memory")
        lib, chunks = load(), ctypes.c_int64(0)
        _check(lib.ss1_gradnorm_plan(table, n, byref(chunks), None), "ss1_gradnorm_plan")
        host_map = np.empty((max(chunks.value, 1), 2), dtype=np.int32)
        _check(lib.ss1_gradnorm_plan(table, n, byref(chunks), host_map.ctypes.data), "ss1_gradnorm_plan")
        device = grads[0].device if grads else "cuda"
        entries = torch.from_numpy(np.frombuffer(table, dtype=np.uint8).copy()).to(device)
        return cls(entries, torch.from_numpy(host_map).to(device), n, chunks.value, grads)

    def norm(self, max_norm: float = float("inf"), norm=None, coef=None, workspace=None, stream=None):
        """(norm, coef), float32 GPU tensors of one element (ss1_gradnorm): the
        2-norm over all the gradients, and max_norm / norm where the norm is
        above max_norm, 1 where it is not.  The host sees neither: ``coef`` is
        the ``grad_scale`` that :meth:`AdamWPlan.step` takes."""
        return self._call("ss1_gradnorm", max_norm, norm, coef, workspace, stream)

    def clip(self, max_norm: float, norm=None, coef=None, workspace=None, stream=None):
        """As :meth:`norm`, and the gradients are multiplied by ``coef`` in
        place (ss1_gradnorm_clip); where it is 1 nothing is written."""
        return self._call("ss1_gradnorm_clip", max_norm, norm, coef, workspace, stream)

    def _call(self, name, max_norm, norm, coef, workspace, stream):
        dev = self.entries.get_device()
        if _elsewhere(stream, dev):
            return _on(stream, self.entries, self._call, name, max_norm, norm, coef, workspace, None)
        torch, lib = _ops._torch, load()
        if norm is None:
            norm = torch.empty((1,), dtype=torch.float32, device=self.entries.device)
        if coef is None:
            coef = torch.empty_like(norm)
        n = ctypes.c_size_t(0)
        _check(lib.ss1_gradnorm_query(self.chunks, byref(n)), "ss1_gradnorm_query")
        workspace, wp, wb = _room(workspace, n.value, self.entries, dev)
        st = getattr(lib, name)(self.entries.data_ptr(), self.count, self.map.data_ptr(), self.chunks, max_norm,
                                _vec(norm, torch.float32, 1, "norm", dev), _vec(coef, torch.float32, 1, "coef", dev),
                                wp, wb, _ops._raw_stream(dev))
        if st:
            _check(st, name)
        return norm, coef


# ----------------------------------------------------------------- embedding
def _tokens(ids, dev: int) -> Tokens:
    if ids.get_device() != dev:
        _refuse_device(ids.get_device())
    torch = _ops._torch
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"ids must be int32 or int64, got {ids.dtype}")
    if ids.dim() != 1 or not ids.is_contiguous():
        raise ValueError("ids must be 1-D and contiguous")
    return Tokens(ids.data_ptr(), ids.shape[0], 4 if ids.dtype == torch.int32 else 8, 0)


def embedding_forward(ids, table, scale: float = 1.0, y=None, dtype=None, stream=None):
    """Rows of an embedding table, scaled (ss1_embedding_forward): y [M][K] with
    y[m] = scale * table[ids[m]], zero for an id outside the table (padding).
    ``ids`` is int32 or int64 [M], ``table`` bf16 or float32 [V][K]; ``dtype`` of
    y is the table's unless it is given."""
    torch = _ops._torch or _ops._setup()
    dev = table.get_device()
    if _elsewhere(stream, dev):
        return _on(stream, table, embedding_forward, ids, table, scale, y, dtype)
    te, tk = _matrix(table, dev), _tokens(ids, dev)
    if y is None:
        y = torch.empty((tk.count, te.cols), dtype=dtype or table.dtype, device=table.device)
    elif dtype is not None and dtype != y.dtype:
        raise TypeError(f"y is {y.dtype}, not {dtype}")
    st = load().ss1_embedding_forward(byref(tk), byref(te), scale, byref(_matrix(y, dev)), _ops._raw_stream(dev))
    if st:
        _check(st, "ss1_embedding_forward")
    return y


def embedding_backward(dy, ids, rows: int, scale: float = 1.0, dE=None, dtype=None, accumulate: bool = False,
                       workspace=None, stream=None):
    """Gradient of :func:`embedding_forward` for the table of ``rows`` rows
    (ss1_embedding_backward): dE [rows][K] with dE[v] = scale * the sum of dy[m]
    over the tokens of v, zero for rows without tokens; with ``accumulate`` the
    sums are added to the given ``dE`` (the gradient of a table that an output
    layer shares) and rows without tokens stay as they are.  ``dtype`` of a new
    dE is dy's unless it is given."""
    torch = _ops._torch or _ops._setup()
    dev = dy.get_device()
    if _elsewhere(stream, dev):
        return _on(stream, dy, embedding_backward, dy, ids, rows, scale, dE, dtype, accumulate, workspace)
    td, tk, lib = _matrix(dy, dev), _tokens(ids, dev), load()
    if dE is None:
        if accumulate:
            raise ValueError("accumulate needs the dE to add to")
        dE = torch.empty((rows, td.cols), dtype=dtype or dy.dtype, device=dy.device)
    elif dtype is not None and dtype != dE.dtype:
        raise TypeError(f"dE is {dE.dtype}, not {dtype}")
    elif dE.shape[0] != rows:
        raise ValueError(f"dE must have {rows} rows, got {dE.shape[0]}")
    te, n = _matrix(dE, dev), ctypes.c_size_t(0)
    st = lib.ss1_embedding_backward_query(byref(tk), byref(te), byref(n))
    if st:
        _check(st, "ss1_embedding_backward_query")
    workspace, wp, wb = _room(workspace, n.value, dy, dev)
    st = lib.ss1_embedding_backward(byref(td), byref(tk), scale, int(bool(accumulate)), byref(te), wp, wb,
                                    _ops._raw_stream(dev))
    if st:
        _check(st, "ss1_embedding_backward")
    return dE


# ---------------------------------------------- block-scaled E4M3 matrices
def _code_cols(cols: int) -> int:
    return -(-cols // FP8_BLOCK) * FP8_BLOCK


def _scale_cols(cols: int) -> int:
    return -(-cols // (4 * FP8_BLOCK)) * 4


@dataclass
class Fp8Blocks:
    """A matrix [rows][cols] in E4M3 with a power-of-two scale for each block:
    value[r][c] = codes[r][c] * 2^(scale[r // block][c // 128] - 127).
    ``codes`` is float8_e4m3fn (or uint8) [rows][cols up to a multiple of 128],
    zeros from ``cols`` on; ``scale`` is uint8 [ceil(rows / block)][...], a row as
    long as a multiple of 4; ``block`` is 1 (a scale for 128 elements of a row)
    or 128 (one for a tile of 128 x 128)."""
    codes: object
    scale: object
    block: int
    cols: int

    @classmethod
    def empty(cls, rows: int, cols: int, block: int = 1, device="cuda"):
        """Uninitialised memory of the right sizes, for an output."""
        torch = _ops._torch or _ops._setup()
        if block not in (1, FP8_BLOCK):
            raise ValueError(f"block must be 1 or {FP8_BLOCK}")
        codes = torch.empty((rows, _code_cols(cols)), dtype=torch.float8_e4m3fn, device=device)
        scale = torch.empty((-(-rows // block), _scale_cols(cols)), dtype=torch.uint8, device=device)
        return cls(codes, scale, block, cols)

    @property
    def rows(self) -> int:
        return self.codes.shape[0]

    def _struct(self, dev: int) -> Fp8BlocksView:
        torch, codes, scale, cols = _ops._torch, self.codes, self.scale, self.cols
        for t, what, dtypes in ((codes, "codes", (torch.float8_e4m3fn, torch.uint8)), (scale, "scale", (torch.uint8,))):
            if t.get_device() != dev:
                _refuse_device(t.get_device())
            if t.dtype not in dtypes:
                raise TypeError(f"{what} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
            if t.dim() != 2 or not t.is_contiguous():
                raise ValueError(f"{what} must be 2-D and contiguous")
        rows = codes.shape[0]
        if self.block not in (1, FP8_BLOCK):
            raise ValueError(f"block must be 1 or {FP8_BLOCK}")
        if codes.shape[1] != _code_cols(cols):
            raise ValueError(f"codes of {cols} columns must be {_code_cols(cols)} wide, got {codes.shape[1]}")
        if tuple(scale.shape) != (-(-rows // self.block), _scale_cols(cols)):
            raise ValueError(f"scale must be {(-(-rows // self.block), _scale_cols(cols))}, got {tuple(scale.shape)}")
        return Fp8BlocksView(codes.data_ptr(), scale.data_ptr(), rows, cols, self.block, 0)


def _blocks_out(t, rows: int, cols: int, block: int, like, dev: int):
    """An output in blocks and the reference to its view: t itself, a new one for
    True, or neither for None."""
    if t is None:
        return None, None
    if t is True:
        t = Fp8Blocks.empty(rows, cols, block, like.device)
    return t, byref(t._struct(dev))


def quantize_fp8_blocks(x, tile: bool = False, q=True, qt=None, stream=None):
    """x [R][C] (bf16 or float32) as block-scaled E4M3 (ss1_quantize_fp8_blocks):
    returns (q, qt), :class:`Fp8Blocks` of x along its rows and of its transpose
    [C][R]; pass None for one that is not wanted, True to allocate it.  A scale
    holds for 128 elements of a row, or with ``tile`` for a tile of 128 x 128
    (weights; then both hold the same codes).  Given outputs say themselves
    which."""
    _ops._torch or _ops._setup()
    dev = x.get_device()
    if _elsewhere(stream, dev):
        return _on(stream, x, quantize_fp8_blocks, x, tile, q, qt)
    tx, block = _matrix(x, dev), FP8_BLOCK if tile else 1
    q, rq = _blocks_out(q, tx.rows, tx.cols, block, x, dev)
    qt, rqt = _blocks_out(qt, tx.cols, tx.rows, block, x, dev)
    st = load().ss1_quantize_fp8_blocks(byref(tx), rq, rqt, _ops._raw_stream(dev))
    if st:
        _check(st, "ss1_quantize_fp8_blocks")
    return q, qt


def matmul_fp8_blocks(a: Fp8Blocks, b: Fp8Blocks, y=None, dtype=None, workspace=None, stream=None):
    """The product of two block-scaled matrices along their common columns
    (ss1_matmul_fp8_blocks): y [M][N] = a [M][K] times b [N][K] transposed.  A
    new y is bfloat16 unless ``dtype`` says float32."""
    torch = _ops._torch or _ops._setup()
    dev = a.codes.get_device()
    if _elsewhere(stream, dev):
        return _on(stream, a.codes, matmul_fp8_blocks, a, b, y, dtype, workspace)
    ta, tb, lib, n = a._struct(dev), b._struct(dev), load(), ctypes.c_size_t(0)
    if y is None:
        y = torch.empty((ta.rows, tb.rows), dtype=dtype or torch.bfloat16, device=a.codes.device)
    elif dtype is not None and dtype != y.dtype:
        raise TypeError(f"y is {y.dtype}, not {dtype}")
    st = lib.ss1_matmul_fp8_blocks_query(byref(ta), byref(tb), byref(n))
    if st:
        _check(st, "ss1_matmul_fp8_blocks_query")
    workspace, wp, wb = _room(workspace, n.value, y, dev)
    st = lib.ss1_matmul_fp8_blocks(byref(ta), byref(tb), byref(_matrix(y, dev)), wp, wb, _ops._raw_stream(dev))
    if st:
        _check(st, "ss1_matmul_fp8_blocks")
    return y


# -------------------------------------------------------------- dense layers
def dense_forward_fp8(x, w: Fp8Blocks, y=None, xt=None, save_xt: bool = False, workspace=None, stream=None):
    """A layer that stays dense, in block-scaled E4M3 (ss1_dense_forward_fp8):
    returns (y, xt) with y [M][N] = x W^T.  ``x`` [M][K] (bf16 or float32) is
    quantised in the call, ``w`` [N][K] by :func:`quantize_fp8_blocks`.  ``xt``, x
    quantised along its columns, is what :func:`dense_backward_fp8` takes: None
    unless given or ``save_xt``."""
    torch = _ops._torch or _ops._setup()
    dev = x.get_device()
    if _elsewhere(stream, dev):
        return _on(stream, x, dense_forward_fp8, x, w, y, xt, save_xt, workspace)
    tx, tw, lib, n = _matrix(x, dev), w._struct(dev), load(), ctypes.c_size_t(0)
    st = lib.ss1_dense_forward_fp8_query(byref(tx), byref(tw), byref(n))
    if st:
        _check(st, "ss1_dense_forward_fp8_query")
    if y is None:
        y = torch.empty((tx.rows, tw.rows), dtype=x.dtype, device=x.device)
    xt, rxt = _blocks_out(True if xt is None and save_xt else xt, tx.cols, tx.rows, 1, x, dev)
    workspace, wp, wb = _room(workspace, n.value, x, dev)
    st = lib.ss1_dense_forward_fp8(byref(tx), byref(tw), byref(_matrix(y, dev)), rxt, wp, wb, _ops._raw_stream(dev))
    if st:
        _check(st, "ss1_dense_forward_fp8")
    return y, xt


def dense_backward_fp8(dy, xt: Fp8Blocks, wt: Fp8Blocks, dx=True, dW=True, dW_dtype=None, workspace=None, stream=None):
    """Gradients of :func:`dense_forward_fp8` (ss1_dense_backward_fp8): returns
    (dx, dW); pass None for one that is not wanted, True to allocate it.  ``xt``
    [K][M] is what the forward returned with ``save_xt`` (needed for dW only),
    ``wt`` [K][N] the weight quantised along its columns (needed for dx only);
    dy [M][N] is quantised in the call.  dW is float32 unless ``dW_dtype`` says
    bfloat16."""
    torch = _ops._torch or _ops._setup()
    dev = dy.get_device()
    if _elsewhere(stream, dev):
        return _on(stream, dy, dense_backward_fp8, dy, xt, wt, dx, dW, dW_dtype, workspace)
    td, lib, n = _matrix(dy, dev), load(), ctypes.c_size_t(0)
    rx = rw = None
    if dx is not None:
        tw = wt._struct(dev)
        rw = byref(tw)
        if dx is True:
            dx = torch.empty((td.rows, tw.rows), dtype=dy.dtype, device=dy.device)
    if dW is not None:
        tx = xt._struct(dev)
        rx = byref(tx)
        if dW is True:
            dW = torch.empty((td.cols, tx.rows), dtype=dW_dtype or torch.float32, device=dy.device)
        elif dW_dtype is not None and dW_dtype != dW.dtype:
            raise TypeError(f"dW is {dW.dtype}, not {dW_dtype}")
    st = lib.ss1_dense_backward_fp8_query(byref(td), rx, rw, byref(n))
    if st:
        _check(st, "ss1_dense_backward_fp8_query")
    workspace, wp, wb = _room(workspace, n.value, dy, dev)
    st = lib.ss1_dense_backward_fp8(byref(td), rx, rw, None if dx is None else byref(_matrix(dx, dev)),
                                    None if dW is None else byref(_matrix(dW, dev)), wp, wb, _ops._raw_stream(dev))
    if st:
        _check(st, "ss1_dense_backward_fp8")
    return dx, dW
