"""Binding of the operators around an SS1 layer (layer norm, the low-rank
adapters of many requests, AdamW over many tensors): argument marshalling only.

Like the layer calls, every function takes GPU tensors, enqueues on the given
or the current stream and returns without waiting; outputs and workspaces are
allocated here when they are not given.
"""
from __future__ import annotations

import ctypes
from ctypes import byref
from dataclasses import dataclass

import numpy as np

from . import _lib
from ._lib import (BF16, F32, FP8_E4M3, OK, AdamWEntry, AdamWHyper, Adapters, Segments, Tensor, _check,
                   _check_device, _check_vec, _desc, _stream, load)

MAX_RANK = 128       # SS1_MAX_RANK
ADAMW_BLOCK = 256    # SS1_ADAMW_BLOCK


def _row(t) -> Tensor:
    """A vector as the [1][K] tensor of the C ABI."""
    if t.dim() != 1:
        raise ValueError("gamma, beta and their gradients must be 1-D")
    return _desc(t.view(1, -1))


# ---------------------------------------------------------------- layer norm
def layernorm_forward(x, gamma, beta=None, eps: float = 1e-5, y=None, mean=None, rstd=None, stream=None):
    """Layer norm of every row of x (ss1_layernorm_forward): returns
    (y, mean, rstd).  ``x`` is [M][K] bf16 or float32, ``gamma`` and ``beta``
    (may be None) are [K] of x's dtype or float32; mean and rstd, float32 [M],
    are what :func:`layernorm_backward` takes."""
    import torch
    _check_device(x, gamma)
    M = x.shape[0]
    if y is None:
        y = torch.empty_like(x)
    if mean is None:
        mean = torch.empty((M,), dtype=torch.float32, device=x.device)
    if rstd is None:
        rstd = torch.empty((M,), dtype=torch.float32, device=x.device)
    _check_device(y, mean, rstd)
    _check_vec(mean, torch.float32, M, "mean")
    _check_vec(rstd, torch.float32, M, "rstd")
    b = None
    if beta is not None:
        _check_device(beta)
        b = byref(_row(beta))
    st = load().ss1_layernorm_forward(byref(_desc(x)), byref(_row(gamma)), b, eps, byref(_desc(y)),
                                      mean.data_ptr(), rstd.data_ptr(), _stream(stream))
    _check(st, "ss1_layernorm_forward")
    return y, mean, rstd


def layernorm_backward(dy, x, gamma, mean, rstd, dx=True, dgamma=True, dbeta=True, workspace=None, stream=None):
    """Gradients of layer norm (ss1_layernorm_backward): returns (dx, dgamma,
    dbeta); pass None for one that is not wanted, True to allocate it.  mean
    and rstd are what the forward returned."""
    import torch
    _check_device(dy, x, gamma, mean, rstd)
    M = x.shape[0]
    _check_vec(mean, torch.float32, M, "mean")
    _check_vec(rstd, torch.float32, M, "rstd")
    if dx is True:
        dx = torch.empty_like(x)
    if dgamma is True:
        dgamma = torch.empty_like(gamma)
    if dbeta is True:
        dbeta = torch.empty_like(gamma)
    _check_device(*(t for t in (dx, dgamma, dbeta, workspace) if t is not None))
    lib, tx = load(), _desc(x)
    wp, wb = None, 0
    if dgamma is not None or dbeta is not None:
        if workspace is None:
            n = ctypes.c_size_t(0)
            _check(lib.ss1_layernorm_backward_query(byref(tx), byref(n)), "ss1_layernorm_backward_query")
            workspace = torch.empty((n.value,), dtype=torch.uint8, device=x.device)
        wp, wb = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    st = lib.ss1_layernorm_backward(byref(_desc(dy)), byref(tx), byref(_row(gamma)), mean.data_ptr(),
                                    rstd.data_ptr(), None if dx is None else byref(_desc(dx)),
                                    None if dgamma is None else byref(_row(dgamma)),
                                    None if dbeta is None else byref(_row(dbeta)), wp, wb, _stream(stream))
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
        import torch
        _check_device(A, B)
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

    def _struct(self) -> Adapters:
        return Adapters(_desc(self.A), _desc(self.B), self.row.data_ptr(), self.scale.data_ptr(), len(self.ranks),
                        self.max_rank)


def _segments(seg, seg_adapter) -> Segments:
    import torch
    _check_device(seg, seg_adapter)
    S = seg_adapter.numel()
    _check_vec(seg, torch.int32, S + 1, "seg")
    _check_vec(seg_adapter, torch.int32, S, "seg_adapter")
    return Segments(seg.data_ptr(), seg_adapter.data_ptr(), S, 0)


def _workspace(workspace, query, M: int, ad: Adapters, device, where: str):
    import torch
    if workspace is None:
        n = ctypes.c_size_t(0)
        _check(query(M, byref(ad), byref(n)), where)
        workspace = torch.empty((n.value,), dtype=torch.uint8, device=device)
    _check_device(workspace)
    return workspace, workspace.data_ptr() or None, workspace.numel() * workspace.element_size()


def adapter_forward(x, adapters: AdapterSet, seg, seg_adapter, base=None, y=None, v=None, save_v: bool = False,
                    workspace=None, stream=None):
    """The adapters of many requests beside their shared projection
    (ss1_adapter_forward): returns (y, v) with
    y = base + scale[e] * (x A_e^T) B_e for the tokens of each segment.
    ``seg`` (int32 [S+1], from 0 to M) and ``seg_adapter`` (int32 [S], -1 for
    none) are device tensors; ``base`` is the projection's output, or None for
    zero, and ``y`` may be base itself.  v = x A_e^T, float32 [M][max_rank], is
    what :func:`adapter_backward` takes: None unless given or ``save_v``."""
    import torch
    _check_device(x)
    M, N = x.shape[0], adapters.B.shape[1]
    if y is None:
        y = torch.empty((M, N), dtype=x.dtype, device=x.device)
    if v is None and save_v:
        v = torch.empty((M, adapters.max_rank), dtype=torch.float32, device=x.device)
    _check_device(*(t for t in (y, base, v) if t is not None))
    lib, ad = load(), adapters._struct()
    workspace, wp, wb = _workspace(workspace, lib.ss1_adapter_forward_query, M, ad, x.device,
                                   "ss1_adapter_forward_query")
    st = lib.ss1_adapter_forward(byref(_desc(x)), byref(ad), byref(_segments(seg, seg_adapter)),
                                 None if base is None else byref(_desc(base)), byref(_desc(y)),
                                 None if v is None else byref(_desc(v)), wp, wb, _stream(stream))
    _check(st, "ss1_adapter_forward")
    return y, v


def adapter_backward(dy, x, v, adapters: AdapterSet, seg, seg_adapter, dx_base=None, dx=True, dA=True, dB=True,
                     workspace=None, stream=None):
    """Gradients of :func:`adapter_forward` (ss1_adapter_backward): returns
    (dx, dA, dB); pass None for one that is not wanted, True to allocate it.
    ``v`` is what the forward returned with ``save_v`` (needed for dB only);
    ``dx_base`` is the projection's own input gradient (ss1.backward's dx), to
    which the adapters' is added, and dx may be dx_base itself."""
    import torch
    _check_device(dy, x)
    M = x.shape[0]
    if dx is True:
        dx = torch.empty_like(x)
    if dA is True:
        dA = torch.empty_like(adapters.A)
    if dB is True:
        dB = torch.empty_like(adapters.B)
    _check_device(*(t for t in (v, dx_base, dx, dA, dB) if t is not None))
    lib, ad = load(), adapters._struct()
    workspace, wp, wb = _workspace(workspace, lib.ss1_adapter_backward_query, M, ad, x.device,
                                   "ss1_adapter_backward_query")
    opt = lambda t: None if t is None else byref(_desc(t))  # noqa: E731
    st = lib.ss1_adapter_backward(byref(_desc(dy)), byref(_desc(x)), opt(v), byref(ad),
                                  byref(_segments(seg, seg_adapter)), opt(dx_base), opt(dx), opt(dA), opt(dB), wp, wb,
                                  _stream(stream))
    _check(st, "ss1_adapter_backward")
    return dx, dA, dB


# --------------------------------------------------------------------- AdamW
def _float_code(t, what: str) -> int:
    import torch
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"{what} must be float32 or bfloat16, got {t.dtype}")


@dataclass
class AdamWPlan:
    """An AdamW step over many tensors: the table of their addresses and the
    list of work items, made once on the host and copied to the GPU.  It holds
    for as long as the tensors stay where they are (it keeps them alive).

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

    @classmethod
    def make(cls, params, grads, m=None, v=None, masters=None, m_scales=None, v_scales=None, weight_decay=0.0,
             state: str = "f32"):
        """``params`` and ``grads`` are lists of GPU tensors (float32 or
        bfloat16, contiguous); ``m`` and ``v`` the states (zeros of kind
        ``state``, "f32" or "fp8", when None); ``masters`` float32 copies of
        bf16 params, or None; ``weight_decay`` one value or one a tensor."""
        import torch
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
        for i, p in enumerate(params):
            _check_device(p, grads[i], m[i], v[i])
            numel = p.numel()
            if not p.is_contiguous():
                raise ValueError("params must be contiguous")
            _check_vec(grads[i], grads[i].dtype, numel, "grad")
            code = _lib._dtype_code(m[i])
            if code == BF16 or _lib._dtype_code(v[i]) != code or (code == FP8_E4M3) != eight:
                raise TypeError("states must all be float32 or all E4M3 codes")
            _check_vec(m[i], m[i].dtype, numel, "m")
            _check_vec(v[i], v[i].dtype, numel, "v")
            e = table[i]
            e.param, e.grad, e.m, e.v = (t.data_ptr() or None for t in (p, grads[i], m[i], v[i]))
            if masters is not None and masters[i] is not None:
                _check_device(masters[i])
                _check_vec(masters[i], torch.float32, numel, "master")
                e.master = masters[i].data_ptr() or None
            if eight:
                _check_device(m_scales[i], v_scales[i])
                _check_vec(m_scales[i], torch.float32, -(-numel // ADAMW_BLOCK), "m_scale")
                _check_vec(v_scales[i], torch.float32, -(-numel // ADAMW_BLOCK), "v_scale")
                e.m_scale, e.v_scale = m_scales[i].data_ptr() or None, v_scales[i].data_ptr() or None
            e.numel, e.weight_decay = numel, decay[i]
            e.param_dtype, e.grad_dtype, e.state_dtype = _float_code(p, "param"), _float_code(grads[i], "grad"), code
        lib, chunks = load(), ctypes.c_int64(0)
        _check(lib.ss1_adamw_plan(table, n, byref(chunks), None), "ss1_adamw_plan")
        host_map = np.empty((max(chunks.value, 1), 2), dtype=np.int32)
        _check(lib.ss1_adamw_plan(table, n, byref(chunks), host_map.ctypes.data), "ss1_adamw_plan")
        device = params[0].device if params else "cuda"
        entries = torch.from_numpy(np.frombuffer(table, dtype=np.uint8).copy()).to(device)
        keep = (params, grads, m, v, masters, m_scales, v_scales)
        return cls(entries, torch.from_numpy(host_map).to(device), n, chunks.value, keep, m, v, m_scales, v_scales,
                   masters)

    def step(self, step: int, lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
             grad_scale=1.0, seed: int = 0, stream=None):
        """One step over every tensor, in place (ss1_adamw_step).  ``step``
        counts from 1; ``grad_scale`` multiplies the gradients: a number, or a
        float32 GPU tensor of one element (a clip coefficient that the host
        has not seen); ``seed``, another each step, feeds the stochastic
        rounding of 8-bit states and of bf16 params without masters."""
        scale, dev = grad_scale, None
        if not isinstance(grad_scale, (int, float)):
            import torch
            _check_device(grad_scale)
            _check_vec(grad_scale, torch.float32, 1, "grad_scale")
            scale, dev = 1.0, grad_scale.data_ptr()
        h = AdamWHyper(lr, beta1, beta2, eps, scale, dev, step, int(seed) & (2**64 - 1))
        st = load().ss1_adamw_step(self.entries.data_ptr(), self.count, self.map.data_ptr(), self.chunks, byref(h),
                                   _stream(stream))
        _check(st, "ss1_adamw_step")
