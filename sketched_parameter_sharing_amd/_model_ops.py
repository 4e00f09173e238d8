"""Binding of the operators at a model's ends and of its dense layers (token
embedding, block-scaled E4M3 matrices, global gradient norm): argument
marshalling only, by the rules of ``_ops``."""
from __future__ import annotations

import ctypes
from ctypes import byref
from dataclasses import dataclass

import numpy as np

from . import _ops
from ._lib import F32, Fp8BlocksView, GradNormEntry, Tensor, Tokens, _check, load
from ._ops import _float_code, _given_workspace, _matrix, _on, _refuse_device, _vec

FP8_BLOCK = 128      # SS1_FP8_BLOCK


def _elsewhere(stream, dev: int) -> bool:
    """Whether a call has to change the stream or the device first."""
    return stream is not None or dev < 0 or dev != _ops._current_device()


def _new(rows: int, cols: int, dtype, device):
    """A new matrix (the strided form of empty costs a call 0.4 us less)."""
    return _ops._torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)


def _room(workspace, nbytes: int, like, dev: int):
    """(tensor to keep, address, bytes) of a call's workspace."""
    if workspace is not None:
        return workspace, *_given_workspace(workspace, dev)
    if nbytes == 0:
        return None, None, 0
    workspace = _ops._torch.empty_strided((nbytes,), (1,), dtype=_ops._torch.uint8, device=like.device)
    return workspace, workspace.data_ptr(), nbytes


def _view(t, code: int, rows: int, cols: int) -> Tensor:
    """The C ABI's view of a matrix that was made here."""
    return Tensor(t.data_ptr(), code, 0, rows, cols)


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
    workspace_bytes: int
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
        nbytes = ctypes.c_size_t(0)
        _check(lib.ss1_gradnorm_query(chunks.value, byref(nbytes)), "ss1_gradnorm_query")
        device = grads[0].device if grads else "cuda"
        entries = torch.from_numpy(np.frombuffer(table, dtype=np.uint8).copy()).to(device)
        return cls(entries, torch.from_numpy(host_map).to(device), n, chunks.value, nbytes.value, grads)

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
        torch, device = _ops._torch, self.entries.device
        if norm is None:
            norm = torch.empty_strided((1,), (1,), dtype=torch.float32, device=device)
            pn = norm.data_ptr()
        else:
            pn = _vec(norm, torch.float32, 1, "norm", dev)
        if coef is None:
            coef = torch.empty_strided((1,), (1,), dtype=torch.float32, device=device)
            pc = coef.data_ptr()
        else:
            pc = _vec(coef, torch.float32, 1, "coef", dev)
        workspace, wp, wb = _room(workspace, self.workspace_bytes, self.entries, dev)
        st = getattr(load(), name)(self.entries.data_ptr(), self.count, self.map.data_ptr(), self.chunks, max_norm, pn,
                                   pc, wp, wb, _ops._raw_stream(dev))
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
    _ops._torch or _ops._setup()
    dev = table.get_device()
    if _elsewhere(stream, dev):
        return _on(stream, table, embedding_forward, ids, table, scale, y, dtype)
    te, tk = _matrix(table, dev), _tokens(ids, dev)
    if y is None:
        y = _new(tk.count, te.cols, dtype or table.dtype, table.device)
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
    _ops._torch or _ops._setup()
    dev = dy.get_device()
    if _elsewhere(stream, dev):
        return _on(stream, dy, embedding_backward, dy, ids, rows, scale, dE, dtype, accumulate, workspace)
    td, tk, lib = _matrix(dy, dev), _tokens(ids, dev), load()
    if dE is None:
        if accumulate:
            raise ValueError("accumulate needs the dE to add to")
        dE = _new(rows, td.cols, dtype or dy.dtype, dy.device)
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
        return cls(_new(rows, _code_cols(cols), torch.float8_e4m3fn, device),
                   _new(-(-rows // block), _scale_cols(cols), torch.uint8, device), block, cols)

    @property
    def rows(self) -> int:
        return self.codes.shape[0]

    def _struct(self, dev: int) -> Fp8BlocksView:
        torch, codes, scale, block, cols = _ops._torch, self.codes, self.scale, self.block, self.cols
        if codes.get_device() != dev or scale.get_device() != dev:
            _refuse_device(min(codes.get_device(), scale.get_device()))
        if codes.dtype != torch.float8_e4m3fn and codes.dtype != torch.uint8:
            raise TypeError(f"codes must be torch.float8_e4m3fn or torch.uint8, got {codes.dtype}")
        if scale.dtype != torch.uint8:
            raise TypeError(f"scale must be torch.uint8, got {scale.dtype}")
        if codes.dim() != 2 or not codes.is_contiguous() or scale.dim() != 2 or not scale.is_contiguous():
            raise ValueError("codes and scale must be 2-D and contiguous")
        if block != 1 and block != FP8_BLOCK:
            raise ValueError(f"block must be 1 or {FP8_BLOCK}")
        rows, width = codes.shape
        if width != _code_cols(cols):
            raise ValueError(f"codes of {cols} columns must be {_code_cols(cols)} wide, got {width}")
        if tuple(scale.shape) != (-(-rows // block), _scale_cols(cols)):
            raise ValueError(f"scale must be {(-(-rows // block), _scale_cols(cols))}, got {tuple(scale.shape)}")
        return Fp8BlocksView(codes.data_ptr(), scale.data_ptr(), rows, cols, block, 0)


def _blocks_out(t, rows: int, cols: int, block: int, like, dev: int):
    """An output in blocks and the reference to its view: t itself, a new one for
    True, or neither for None."""
    if t is None:
        return None, None
    if t is True:
        t = Fp8Blocks.empty(rows, cols, block, like.device)
        return t, byref(Fp8BlocksView(t.codes.data_ptr(), t.scale.data_ptr(), rows, cols, block, 0))
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
    new y is bfloat16 unless ``dtype`` says float32.  A bfloat16 y comes from the
    8-bit matrix instructions, which keep 18 bits below the largest product of a
    block of 128; a float32 y has float32 sums of exact products, over values up
    to below 2^128 (a code times its scale beyond that counts as infinite)."""
    torch = _ops._torch or _ops._setup()
    dev = a.codes.get_device()
    if _elsewhere(stream, dev):
        return _on(stream, a.codes, matmul_fp8_blocks, a, b, y, dtype, workspace)
    ta, tb, lib, n = a._struct(dev), b._struct(dev), load(), ctypes.c_size_t(0)
    if y is None:
        y = _new(ta.rows, tb.rows, dtype or torch.bfloat16, a.codes.device)
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
    unless given or ``save_xt``.  y has x's dtype, and with it the arithmetic of
    :func:`matmul_fp8_blocks` for that dtype."""
    _ops._torch or _ops._setup()
    dev = x.get_device()
    if _elsewhere(stream, dev):
        return _on(stream, x, dense_forward_fp8, x, w, y, xt, save_xt, workspace)
    tx, tw, lib, n = _matrix(x, dev), w._struct(dev), load(), ctypes.c_size_t(0)
    st = lib.ss1_dense_forward_fp8_query(byref(tx), byref(tw), byref(n))
    if st:
        _check(st, "ss1_dense_forward_fp8_query")
    if y is None:
        y = _new(tx.rows, tw.rows, x.dtype, x.device)
        ty = _view(y, tx.dtype, tx.rows, tw.rows)
    else:
        ty = _matrix(y, dev)
    xt, rxt = _blocks_out(True if xt is None and save_xt else xt, tx.cols, tx.rows, 1, x, dev)
    workspace, wp, wb = _room(workspace, n.value, x, dev)
    st = lib.ss1_dense_forward_fp8(byref(tx), byref(tw), byref(ty), rxt, wp, wb, _ops._raw_stream(dev))
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
    if (dx is not None and wt is None) or (dW is not None and xt is None):
        raise ValueError("dx needs wt and dW needs xt")
    if dx is not None:
        tw = wt._struct(dev)
        rw = byref(tw)
        if dx is True:
            dx = _new(td.rows, tw.rows, dy.dtype, dy.device)
    if dW is not None:
        tx = xt._struct(dev)
        rx = byref(tx)
        if dW is True:
            dW = _new(td.cols, tx.rows, dW_dtype or torch.float32, dy.device)
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
