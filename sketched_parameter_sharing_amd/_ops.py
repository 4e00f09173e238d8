"""Binding of the operators around an SS1 layer (layer norm, the low-rank
adapters of many requests, AdamW over many tensors): argument marshalling only.

Like the layer calls, every function takes GPU tensors, enqueues on the given
or the current stream and returns without waiting; outputs and workspaces are
allocated here when they are not given, from the memory of the stream that the
call runs on (so that a block freed by another stream's work is not written
before that work is done, nor a workspace reused while the call runs).
"""
from __future__ import annotations

import ctypes
from ctypes import byref
from dataclasses import dataclass

import numpy as np

from . import _lib
from ._lib import BF16, F32, FP8_E4M3, AdamWEntry, AdamWHyper, Adapters, Segments, Tensor, _check, _check_vec, load

MAX_RANK = 128       # SS1_MAX_RANK
ADAMW_BLOCK = 256    # SS1_ADAMW_BLOCK

# Set by _setup at the first call (importing the package does not import torch).
_torch = None
_codes = {}
_raw_stream = None
_current_device = None


def _setup():
    global _torch, _raw_stream, _current_device
    import torch
    _codes.update({torch.float32: F32, torch.bfloat16: BF16})
    # the handle of a device's current stream, without a Stream object around it
    # (3 us of a small call); current_stream is the public way to the same handle,
    # as current_device is to the index
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: torch.cuda.current_stream(index).cuda_stream)
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _torch = torch
    return torch


def _refuse_device(index: int):
    """For a tensor on device ``index`` (-1: host memory) in a call on another."""
    if index < 0:
        raise ValueError("device entry points take GPU tensors")
    raise ValueError("the tensors of a call must be on one GPU")


def _matrix(t, dev: int) -> Tensor:
    """The C ABI's view of a 2-D, contiguous tensor on GPU ``dev``."""
    if t.get_device() != dev:
        _refuse_device(t.get_device())
    if t.dim() != 2 or not t.is_contiguous():
        raise ValueError("matrices must be 2-D and contiguous")
    code = _codes.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype} (bfloat16 or float32)")
    rows, cols = t.shape
    return Tensor(t.data_ptr(), code, 0, rows, cols)


def _row(t, dev: int) -> Tensor:
    """A vector as the [1][K] tensor of the C ABI."""
    if t.get_device() != dev:
        _refuse_device(t.get_device())
    if t.dim() != 1 or not t.is_contiguous():
        raise ValueError("gamma, beta and their gradients must be 1-D and contiguous")
    code = _codes.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype} (bfloat16 or float32)")
    return Tensor(t.data_ptr(), code, 0, 1, t.shape[0])


def _vec(t, dtype, numel: int, what: str, dev: int) -> int:
    """The address of a device array that the C ABI reads by pointer alone."""
    if t.get_device() != dev:
        _refuse_device(t.get_device())
    _check_vec(t, dtype, numel, what)
    return t.data_ptr()


def _fresh(t, d: Tensor):
    """A new tensor like t, whose view is d, and its own view."""
    o = _torch.empty_like(t)
    return o, Tensor(o.data_ptr(), d.dtype, 0, d.rows, d.cols)


def _ref(desc, t, dev: int):
    return None if t is None else byref(desc(t, dev))


def _out(t, desc, like, d: Tensor, dev: int):
    """An output and the reference to its view: t itself, a new tensor like
    ``like`` (whose view is d) for True, or neither for None."""
    if t is None:
        return None, None
    if t is True:
        t, v = _fresh(like, d)
        return t, byref(v)
    return t, byref(desc(t, dev))


def _given_workspace(workspace, dev: int):
    """Address and bytes of a caller's workspace."""
    if workspace.get_device() != dev:
        _refuse_device(workspace.get_device())
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _on(stream, t, call, *args):
    """The call with the GPU of its tensor t as the current device and, when it
    is given, ``stream`` as the current one, its allocations too."""
    torch = _torch or _setup()
    dev = t.get_device()
    if dev < 0:
        _refuse_device(dev)
    if stream is None:
        with torch.cuda.device(dev):
            return call(*args)
    if stream.device_index != dev:
        raise ValueError("the stream and the tensors of a call must be on one GPU")
    with torch.cuda.stream(stream):
        return call(*args)


# ---------------------------------------------------------------- layer norm
def layernorm_forward(x, gamma, beta=None, eps: float = 1e-5, y=None, mean=None, rstd=None, stream=None):
    """Layer norm of every row of x (ss1_layernorm_forward): returns
    (y, mean, rstd).  ``x`` is [M][K] bf16 or float32, ``gamma`` and ``beta``
    (may be None) are [K] of x's dtype or float32; mean and rstd, float32 [M],
    are what :func:`layernorm_backward` takes."""
    torch = _torch or _setup()
    dev = x.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _on(stream, x, layernorm_forward, x, gamma, beta, eps, y, mean, rstd)
    tx = _matrix(x, dev)
    M = tx.rows
    y, ry = _out(True if y is None else y, _matrix, x, tx, dev)
    if mean is None:
        mean = torch.empty((M,), dtype=torch.float32, device=x.device)
        pm = mean.data_ptr()
    else:
        pm = _vec(mean, torch.float32, M, "mean", dev)
    if rstd is None:
        rstd = torch.empty_like(mean)
        pr = rstd.data_ptr()
    else:
        pr = _vec(rstd, torch.float32, M, "rstd", dev)
    st = load().ss1_layernorm_forward(byref(tx), byref(_row(gamma, dev)), _ref(_row, beta, dev), eps, ry, pm, pr,
                                      _raw_stream(dev))
    if st:
        _check(st, "ss1_layernorm_forward")
    return y, mean, rstd


def layernorm_backward(dy, x, gamma, mean, rstd, dx=True, dgamma=True, dbeta=True, workspace=None, stream=None):
    """Gradients of layer norm (ss1_layernorm_backward): returns (dx, dgamma,
    dbeta); pass None for one that is not wanted, True to allocate it.  mean
    and rstd are what the forward returned."""
    torch = _torch or _setup()
    dev = x.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _on(stream, x, layernorm_backward, dy, x, gamma, mean, rstd, dx, dgamma, dbeta, workspace)
    tx, tg = _matrix(x, dev), _row(gamma, dev)
    M = tx.rows
    dx, rdx = _out(dx, _matrix, x, tx, dev)
    dgamma, rdg = _out(dgamma, _row, gamma, tg, dev)
    dbeta, rdb = _out(dbeta, _row, gamma, tg, dev)
    lib = load()
    wp, wb = None, 0
    if dgamma is not None or dbeta is not None:
        if workspace is None:
            n = ctypes.c_size_t(0)
            _check(lib.ss1_layernorm_backward_query(byref(tx), byref(n)), "ss1_layernorm_backward_query")
            workspace = torch.empty((n.value,), dtype=torch.uint8, device=x.device)
            wp, wb = workspace.data_ptr(), n.value
        else:
            wp, wb = _given_workspace(workspace, dev)
    st = lib.ss1_layernorm_backward(byref(_matrix(dy, dev)), byref(tx), byref(tg),
                                    _vec(mean, torch.float32, M, "mean", dev),
                                    _vec(rstd, torch.float32, M, "rstd", dev), rdx, rdg, rdb, wp, wb, _raw_stream(dev))
    if st:
        _check(st, "ss1_layernorm_backward")
    return dx, dgamma, dbeta


# ------------------------------------------------------------------ adapters
@dataclass
class AdapterSet:
    """The low-rank adapters of one projection K -> N.  Both factors are
    stored rank-major, A [R][K] and B [R][N] (R the sum of the ranks): adapter
    e owns rows row[e] .. row[e+1]-1 of both and adds
    scale[e] * (x A_e^T) B_e."""
    A: object
    B: object
    row: object
    scale: object
    max_rank: int
    ranks: tuple

    @classmethod
    def make(cls, A, B, ranks, scale):
        """``ranks`` and ``scale`` are host sequences, one value an adapter."""
        torch = _torch or _setup()
        dev = A.get_device()
        if dev < 0 or B.get_device() != dev:
            _refuse_device(min(dev, B.get_device()))
        ranks = tuple(int(r) for r in ranks)
        if any(r < 0 or r > MAX_RANK for r in ranks):
            raise ValueError(f"ranks must be 0 to {MAX_RANK}")
        if A.dim() != 2 or B.dim() != 2 or sum(ranks) != A.shape[0] or A.shape[0] != B.shape[0]:
            raise ValueError("A and B must be [sum of ranks][K] and [sum of ranks][N]")
        if len(scale) != len(ranks):
            raise ValueError("one scale for each adapter")
        row = torch.from_numpy(np.concatenate([[0], np.cumsum(ranks)]).astype(np.int32)).to(A.device)
        sc = torch.tensor([float(s) for s in scale], dtype=torch.float32).to(A.device)
        return cls(A, B, row, sc, max(ranks, default=0), ranks)

    def __setattr__(self, name, value):
        self.__dict__[name] = value
        self.__dict__["_view"] = (None, None, -1)

    def __getstate__(self):
        # without the view: a copy has memory of its own
        return {**self.__dict__, "_view": (None, None, -1)}

    def _struct(self, dev: int) -> Adapters:
        """The C ABI's view of the set for a call on GPU ``dev``, made and checked
        again when an attribute, the memory of a tensor or the sizes, type or
        layout of a factor changed."""
        A, B, row, scale = self.A, self.B, self.row, self.scale
        now = (A.data_ptr(), A.shape, A.dtype, A.is_contiguous(), B.data_ptr(), B.shape, B.dtype, B.is_contiguous(),
               row.data_ptr(), scale.data_ptr())
        seen, ad, place = self._view
        if seen != now or place != dev:
            count, torch = len(self.ranks), _torch or _setup()
            ad = Adapters(_matrix(A, dev), _matrix(B, dev), _vec(row, torch.int32, count + 1, "row", dev),
                          _vec(scale, torch.float32, count, "scale", dev), count, self.max_rank)
            self.__dict__["_view"] = (now, ad, dev)
        return ad


def _segments(seg, seg_adapter, dev: int) -> Segments:
    S, i32 = seg_adapter.numel(), _torch.int32
    return Segments(_vec(seg, i32, S + 1, "seg", dev), _vec(seg_adapter, i32, S, "seg_adapter", dev), S, 0)


def _workspace(workspace, query, M: int, ad: Adapters, x, dev: int, where: str):
    if workspace is None:
        n = ctypes.c_size_t(0)
        st = query(M, byref(ad), byref(n))
        if st:
            _check(st, where)
        workspace = _torch.empty((n.value,), dtype=_torch.uint8, device=x.device)
        return workspace, workspace.data_ptr(), n.value
    return workspace, *_given_workspace(workspace, dev)


def adapter_forward(x, adapters: AdapterSet, seg, seg_adapter, base=None, y=None, v=None, save_v: bool = False,
                    workspace=None, stream=None):
    """The adapters of many requests beside their shared projection
    (ss1_adapter_forward): returns (y, v) with
    y = base + scale[e] * (x A_e^T) B_e for the tokens of each segment.
    ``seg`` (int32 [S+1], from 0 to M) and ``seg_adapter`` (int32 [S], -1 for
    none) are device tensors; ``base`` is the projection's output, or None for
    zero, and ``y`` may be base itself.  v = x A_e^T, float32 [M][max_rank], is
    what :func:`adapter_backward` takes: None unless given or ``save_v``."""
    torch = _torch or _setup()
    dev = x.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _on(stream, x, adapter_forward, x, adapters, seg, seg_adapter, base, y, v, save_v, workspace)
    tx, ad, lib = _matrix(x, dev), adapters._struct(dev), load()
    M = tx.rows
    rbase = None
    if base is not None:
        tb = _matrix(base, dev)
        rbase = byref(tb)
    if y is not None:
        ry = byref(_matrix(y, dev))
    elif base is not None:
        y, ty = _fresh(base, tb)
        ry = byref(ty)
    else:
        y = torch.empty((M, ad.B.cols), dtype=x.dtype, device=x.device)
        ry = byref(Tensor(y.data_ptr(), tx.dtype, 0, M, ad.B.cols))
    if v is None and save_v:
        v = torch.empty((M, adapters.max_rank), dtype=torch.float32, device=x.device)
    workspace, wp, wb = _workspace(workspace, lib.ss1_adapter_forward_query, M, ad, x, dev,
                                   "ss1_adapter_forward_query")
    st = lib.ss1_adapter_forward(byref(tx), byref(ad), byref(_segments(seg, seg_adapter, dev)), rbase, ry,
                                 _ref(_matrix, v, dev), wp, wb, _raw_stream(dev))
    if st:
        _check(st, "ss1_adapter_forward")
    return y, v


def adapter_backward(dy, x, v, adapters: AdapterSet, seg, seg_adapter, dx_base=None, dx=True, dA=True, dB=True,
                     workspace=None, stream=None):
    """Gradients of :func:`adapter_forward` (ss1_adapter_backward): returns
    (dx, dA, dB); pass None for one that is not wanted, True to allocate it.
    ``v`` is what the forward returned with ``save_v`` (needed for dB only);
    ``dx_base`` is the projection's own input gradient (ss1.backward's dx), to
    which the adapters' is added, and dx may be dx_base itself."""
    _torch or _setup()
    dev = x.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _on(stream, x, adapter_backward, dy, x, v, adapters, seg, seg_adapter, dx_base, dx, dA, dB, workspace)
    tx, ad, lib = _matrix(x, dev), adapters._struct(dev), load()
    M = tx.rows
    dx, rdx = _out(dx, _matrix, x, tx, dev)
    dA, rdA = _out(dA, _matrix, adapters.A, ad.A, dev)
    dB, rdB = _out(dB, _matrix, adapters.B, ad.B, dev)
    workspace, wp, wb = _workspace(workspace, lib.ss1_adapter_backward_query, M, ad, x, dev,
                                   "ss1_adapter_backward_query")
    st = lib.ss1_adapter_backward(byref(_matrix(dy, dev)), byref(tx), _ref(_matrix, v, dev), byref(ad),
                                  byref(_segments(seg, seg_adapter, dev)), _ref(_matrix, dx_base, dev), rdx, rdA, rdB,
                                  wp, wb, _raw_stream(dev))
    if st:
        _check(st, "ss1_adapter_backward")
    return dx, dA, dB


# --------------------------------------------------------------------- AdamW
def _float_code(t, what: str) -> int:
    code = _codes.get(t.dtype)
    if code is None:
        raise TypeError(f"{what} must be float32 or bfloat16, got {t.dtype}")
    return code


def _check_apart(rows, numel, blocks):
    """What a step writes lies in separate memory: it is one launch, in which two
    entries over the same bytes (a tied parameter listed twice, one tensor as both
    states) would race."""
    n, k = np.array(numel, dtype=np.int64), np.array(blocks, dtype=np.int64)
    state = np.where(rows["state_dtype"] == FP8_E4M3, 1, 4)
    spans = [(rows["param"], n * np.where(rows["param_dtype"] == F32, 4, 2)), (rows["m"], n * state),
             (rows["v"], n * state), (rows["master"], n * 4), (rows["m_scale"], k * 4), (rows["v_scale"], k * 4)]
    at = np.concatenate([a for a, _ in spans])
    end = at + np.concatenate([b for _, b in spans]).astype(np.uint64)
    used = np.flatnonzero((at != 0) & (end > at))
    order = used[np.argsort(at[used], kind="stable")]
    if (end[order[:-1]] > at[order[1:]]).any():
        raise ValueError("params, states, masters and scales must not share memory")


@dataclass
class AdamWPlan:
    """An AdamW step over many tensors: the table of their addresses and the
    list of work items, made once on the host and copied to the GPU.  It holds
    for as long as the tensors stay where they are (it keeps them alive).  A
    deep copy or a loaded plan (``torch.save``) has tensors of its own, and a
    table of them.

    8-bit states are ``torch.float8_e4m3fn`` (or uint8 codes) with one float32
    scale per 256 elements; ``v`` then stands for the square root of the
    second moment."""
    entries: object      # uint8 device tensor: the ss1_adamw_entry table
    map: object          # int32 device tensor [chunks][2]
    count: int
    chunks: int
    tensors: tuple
    m: list
    v: list
    m_scales: list | None
    v_scales: list | None
    masters: list | None
    weight_decay: list

    def __reduce__(self):
        # not the table: a copy's tensors lie at other addresses
        return _plan_of, (*self.tensors, self.weight_decay)

    @classmethod
    def make(cls, params, grads, m=None, v=None, masters=None, m_scales=None, v_scales=None, weight_decay=0.0,
             state: str = "f32"):
        """``params`` and ``grads`` are lists of GPU tensors (float32 or
        bfloat16, contiguous); ``m`` and ``v`` the states (zeros of kind
        ``state``, "f32" or "fp8", when None); ``masters`` float32 copies of
        bf16 params, or None; ``weight_decay`` one value or one a tensor."""
        torch = _torch or _setup()
        params, grads = list(params), list(grads)
        n = len(params)
        if state not in ("f32", "fp8"):
            raise ValueError('state must be "f32" or "fp8"')

        def fresh(p):
            return torch.zeros(p.shape, dtype=torch.float8_e4m3fn if state == "fp8" else torch.float32, device=p.device)

        def ones(p):
            return torch.ones((-(-p.numel() // ADAMW_BLOCK),), dtype=torch.float32, device=p.device)

        m = [fresh(p) for p in params] if m is None else list(m)
        v = [fresh(p) for p in params] if v is None else list(v)
        eight = bool(m) and m[0].dtype not in (torch.float32,)
        if eight and m_scales is None:
            m_scales = [ones(p) for p in params]
        if eight and v_scales is None:
            v_scales = [ones(p) for p in params]
        decay = [float(weight_decay)] * n if isinstance(weight_decay, (int, float)) else [float(w) for w in weight_decay]
        lists = [("grads", grads), ("m", m), ("v", v), ("masters", masters), ("m_scales", m_scales),
                 ("v_scales", v_scales), ("weight_decay", decay)]
        for what, t in lists:
            if t is not None and len(t) != n:
                raise ValueError(f"{what} must hold one for each of the {n} params")
        table = (AdamWEntry * max(n, 1))()
        rows = np.frombuffer(table, dtype=np.dtype(AdamWEntry))[:n]
        numel = [p.numel() for p in params]
        blocks = [-(-k // ADAMW_BLOCK) for k in numel]

        dev = params[0].get_device() if params else 0
        if dev < 0:
            _refuse_device(dev)

        def column(name, ts, what, dtype, sizes):
            """The tensors' addresses into one field of the table."""
            for t, k in zip(ts, sizes):
                if t.get_device() != dev or not t.is_contiguous() or t.numel() != k or (
                        dtype is not None and t.dtype != dtype):
                    _vec(t, dtype or t.dtype, k, what, dev)
            rows[name] = [t.data_ptr() for t in ts]

        if any(not p.is_contiguous() for p in params):
            raise ValueError("params must be contiguous")
        column("param", params, "param", None, numel)
        column("grad", grads, "grad", None, numel)
        kinds = {t.dtype for t in m} | {t.dtype for t in v}
        codes = {_lib._dtype_code(t) for t in m} | {_lib._dtype_code(t) for t in v} if len(kinds) > 1 else \
            {_lib._dtype_code(t) for t in m[:1]}
        if len(codes) > 1 or BF16 in codes or (FP8_E4M3 in codes) != eight:
            raise TypeError("states must all be float32 or all E4M3 codes")
        column("m", m, "m", None, numel)
        column("v", v, "v", None, numel)
        if masters is not None:
            has = [i for i, t in enumerate(masters) if t is not None]
            for i in has:
                rows["master"][i] = _vec(masters[i], torch.float32, numel[i], "master", dev)
        if eight:
            column("m_scale", m_scales, "m_scale", torch.float32, blocks)
            column("v_scale", v_scales, "v_scale", torch.float32, blocks)
        rows["numel"], rows["weight_decay"] = numel, decay
        rows["param_dtype"] = [_float_code(p, "param") for p in params]
        rows["grad_dtype"] = [_float_code(g, "grad") for g in grads]
        rows["state_dtype"] = FP8_E4M3 if eight else F32
        _check_apart(rows, numel, blocks)
        lib, chunks = load(), ctypes.c_int64(0)
        _check(lib.ss1_adamw_plan(table, n, byref(chunks), None), "ss1_adamw_plan")
        host_map = np.empty((max(chunks.value, 1), 2), dtype=np.int32)
        _check(lib.ss1_adamw_plan(table, n, byref(chunks), host_map.ctypes.data), "ss1_adamw_plan")
        device = params[0].device if params else "cuda"
        entries = torch.from_numpy(np.frombuffer(table, dtype=np.uint8).copy()).to(device)
        keep = (params, grads, m, v, masters, m_scales, v_scales)
        return cls(entries, torch.from_numpy(host_map).to(device), n, chunks.value, keep, m, v, m_scales, v_scales,
                   masters, decay)

    def step(self, step: int, lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
             grad_scale=1.0, seed: int | None = None, stream=None):
        """One step over every tensor, in place (ss1_adamw_step).  ``step``
        counts from 1; ``grad_scale`` multiplies the gradients: a number, or a
        float32 GPU tensor of one element (a clip coefficient that the host
        has not seen); ``seed``, another each step (``step`` itself when None),
        feeds the stochastic rounding of 8-bit states and of bf16 params without
        masters.  These are values of the call: a captured graph replays the
        step, the rate and the random bits that it was captured with."""
        dev = self.entries.get_device()
        if stream is not None or dev < 0 or dev != _current_device():
            return _on(stream, self.entries, self.step, step, lr, beta1, beta2, eps, grad_scale, seed)
        scale, on_device = grad_scale, None
        if not isinstance(grad_scale, (int, float)):
            scale, on_device = 1.0, _vec(grad_scale, _torch.float32, 1, "grad_scale", dev)
        h = AdamWHyper(lr, beta1, beta2, eps, scale, on_device, step, int(step if seed is None else seed) & (2**64 - 1))
        st = load().ss1_adamw_step(self.entries.data_ptr(), self.count, self.map.data_ptr(), self.chunks, byref(h),
                                   _raw_stream(dev))
        if st:
            _check(st, "ss1_adamw_step")


def _plan_of(params, grads, m, v, masters, m_scales, v_scales, weight_decay):
    """A plan over the tensors of a copied or unpickled one (AdamWPlan.tensors)."""
    return AdamWPlan.make(params, grads, m, v, masters, m_scales, v_scales, weight_decay)
