"""Host-side tests of the operators around an SS1 layer (no GPU): every
argument check returns its status before any HIP call, the work list of the
AdamW plan, and the binding's structures and constants."""
import ctypes
import os
import re

import numpy as np
import pytest

import sketched_parameter_sharing_amd as ss1
from sketched_parameter_sharing_amd import _lib, _ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x10000  # fake device address: the checks below fail before it is used
NULL, SHAPE, DTYPE, ALIGN, OK = (_lib.ERR_NULL, _lib.ERR_SHAPE, _lib.ERR_DTYPE, _lib.ERR_ALIGN, _lib.OK)
F32, BF16, FP8 = _lib.F32, _lib.BF16, _lib.FP8_E4M3
byref = ctypes.byref


def T(rows, cols, dtype=BF16, data=A, reserved=0):
    return _lib.Tensor(data, dtype, reserved, rows, cols)


def opt(t):
    return None if t is None else byref(t)


# ---------------------------------------------------------------- layer norm
def lnf(x=T(4, 64), gamma=T(1, 64, F32), beta=T(1, 64, F32), eps=1e-5, y=T(4, 64), mean=A, rstd=A):
    return _lib.load().ss1_layernorm_forward(opt(x), opt(gamma), opt(beta), eps, opt(y), mean, rstd, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), NULL), (dict(gamma=None), NULL), (dict(y=None), NULL),
    (dict(x=T(4, 64, data=None)), NULL), (dict(y=T(4, 64, data=None)), NULL),
    (dict(gamma=T(1, 64, F32, data=None)), NULL),
    (dict(x=T(4, 64, 7)), DTYPE), (dict(x=T(4, 64, FP8)), DTYPE), (dict(y=T(4, 64, F32)), DTYPE),
    (dict(x=T(4, 64, F32), y=T(4, 64, F32), gamma=T(1, 64, BF16), beta=None), DTYPE),
    (dict(beta=T(1, 64, BF16)), DTYPE),
    (dict(x=T(-1, 64)), SHAPE), (dict(x=T(4, 0)), SHAPE), (dict(x=T(4, 1 << 24)), SHAPE),
    (dict(x=T(1 << 31, 64)), SHAPE), (dict(x=T((1 << 31) - 1, 1 << 20)), SHAPE),
    (dict(gamma=T(1, 63, F32)), SHAPE), (dict(gamma=T(2, 64, F32)), SHAPE), (dict(beta=T(1, 65, F32)), SHAPE),
    (dict(y=T(5, 64)), SHAPE), (dict(y=T(4, 64, reserved=1)), SHAPE), (dict(x=T(4, 64, reserved=1)), SHAPE),
    (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(eps=float("inf")), SHAPE),
    (dict(x=T(4, 64, data=A + 2)), ALIGN), (dict(y=T(4, 64, data=A + 8)), ALIGN),
    (dict(gamma=T(1, 64, F32, data=A + 4)), ALIGN), (dict(mean=A + 2), ALIGN), (dict(rstd=A + 1), ALIGN),
    (dict(x=T(0, 64, data=None), y=T(0, 64, data=None)), OK),
])
def test_layernorm_forward_checks(kw, status):
    assert lnf(**kw) == status


def lnb(dy=T(4, 64), x=T(4, 64), gamma=T(1, 64, F32), mean=A, rstd=A, dx=T(4, 64), dgamma=T(1, 64, F32),
        dbeta=T(1, 64, F32), ws=A, nbytes=1 << 30):
    return _lib.load().ss1_layernorm_backward(opt(dy), opt(x), opt(gamma), mean, rstd, opt(dx), opt(dgamma),
                                              opt(dbeta), ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), NULL), (dict(x=None), NULL), (dict(gamma=None), NULL), (dict(mean=None), NULL),
    (dict(rstd=None), NULL), (dict(ws=None), NULL), (dict(dx=T(4, 64, data=None)), NULL),
    (dict(dy=T(4, 64, F32)), DTYPE), (dict(dx=T(4, 64, F32)), DTYPE), (dict(dgamma=T(1, 64, BF16)), DTYPE),
    (dict(dbeta=T(1, 64, BF16)), DTYPE), (dict(dy=T(3, 64)), SHAPE), (dict(dx=T(4, 63)), SHAPE),
    (dict(dgamma=T(1, 63, F32)), SHAPE), (dict(dbeta=T(2, 64, F32)), SHAPE), (dict(nbytes=16), SHAPE),
    (dict(ws=A + 4), ALIGN), (dict(mean=A + 2), ALIGN), (dict(dx=T(4, 64, data=A + 2)), ALIGN),
    (dict(dx=None, dgamma=None, dbeta=None), OK),
    (dict(dy=T(0, 64), x=T(0, 64), dx=T(0, 64), dgamma=None, dbeta=None, mean=None, rstd=None), OK),
])
def test_layernorm_backward_checks(kw, status):
    assert lnb(**kw) == status


def test_layernorm_query():
    lib, n = _lib.load(), ctypes.c_size_t(7)
    assert lib.ss1_layernorm_backward_query(byref(T(0, 64)), byref(n)) == OK and n.value == 0
    assert lib.ss1_layernorm_backward_query(byref(T(4, 64)), byref(n)) == OK and n.value >= 2 * 64 * 4
    assert lib.ss1_layernorm_backward_query(byref(T(4, 0)), byref(n)) == SHAPE
    assert lib.ss1_layernorm_backward_query(None, byref(n)) == NULL
    assert lib.ss1_layernorm_backward_query(byref(T(4, 64)), None) == NULL


# ------------------------------------------------------------------ adapters
def AD(a=T(16, 64), b=T(16, 40), row=A, scale=A, count=2, max_rank=8):
    return _lib.Adapters(a, b, row, scale, count, max_rank)


def SG(offset=A, adapter=A, count=3, reserved=0):
    return _lib.Segments(offset, adapter, count, reserved)


def adf(x=T(5, 64), ad=AD(), sg=SG(), base=T(5, 40), y=T(5, 40), v=T(5, 8, F32), ws=A, nbytes=1 << 30):
    return _lib.load().ss1_adapter_forward(opt(x), opt(ad), opt(sg), opt(base), opt(y), opt(v), ws, nbytes, None)


SET_ERRORS = [
    (dict(ad=AD(a=T(16, 64, FP8))), DTYPE), (dict(ad=AD(b=T(16, 40, F32))), DTYPE),
    (dict(ad=AD(b=T(15, 40))), SHAPE), (dict(ad=AD(a=T(16, 60))), SHAPE), (dict(ad=AD(b=T(16, 44))), SHAPE),
    (dict(ad=AD(a=T(16, 0))), SHAPE), (dict(ad=AD(a=T(16, 1 << 24))), SHAPE), (dict(ad=AD(count=-1)), SHAPE),
    (dict(ad=AD(max_rank=129)), SHAPE), (dict(ad=AD(max_rank=-1)), SHAPE), (dict(ad=AD(a=T(16, 64, reserved=2))), SHAPE),
    (dict(ad=AD(row=None)), NULL), (dict(ad=AD(scale=None)), NULL), (dict(ad=AD(a=T(16, 64, data=None))), NULL),
    (dict(ad=AD(row=A + 2)), ALIGN), (dict(ad=AD(scale=A + 1)), ALIGN), (dict(ad=AD(a=T(16, 64, data=A + 8))), ALIGN),
    (dict(sg=None), NULL), (dict(sg=SG(offset=None)), NULL), (dict(sg=SG(adapter=None)), NULL),
    (dict(sg=SG(count=-1)), SHAPE), (dict(sg=SG(reserved=1)), SHAPE), (dict(sg=SG(offset=A + 2)), ALIGN),
    (dict(ws=None), NULL), (dict(ws=A + 8), ALIGN), (dict(nbytes=4), SHAPE), (dict(x=None), NULL),
    (dict(ad=None), NULL), (dict(x=T(5, 72)), SHAPE), (dict(x=T(5, 64, F32)), DTYPE),
    (dict(x=T(5, 64, data=None)), NULL), (dict(x=T(5, 64, data=A + 2)), ALIGN), (dict(v=T(5, 7, F32)), SHAPE),
    (dict(v=T(5, 8, BF16)), DTYPE),
]


@pytest.mark.parametrize("kw,status", SET_ERRORS + [
    (dict(y=None), NULL), (dict(y=T(5, 48)), SHAPE), (dict(y=T(4, 40)), SHAPE), (dict(base=T(5, 48)), SHAPE),
    (dict(base=T(5, 40, F32)), DTYPE), (dict(y=T(5, 40, data=A + 4)), ALIGN), (dict(x=T(-1, 64)), SHAPE),
    (dict(x=T(1 << 31, 64)), SHAPE),
    (dict(x=T(0, 64, data=None), base=None, y=T(0, 40, data=None), v=T(0, 8, F32, data=None)), OK),
])
def test_adapter_forward_checks(kw, status):
    assert adf(**kw) == status


def adb(dy=T(5, 40), x=T(5, 64), v=T(5, 8, F32), ad=AD(), sg=SG(), dxb=T(5, 64), dx=T(5, 64), dA=T(16, 64),
        dB=T(16, 40), ws=A, nbytes=1 << 30):
    return _lib.load().ss1_adapter_backward(opt(dy), opt(x), opt(v), opt(ad), opt(sg), opt(dxb), opt(dx), opt(dA),
                                            opt(dB), ws, nbytes, None)


@pytest.mark.parametrize("kw,status", SET_ERRORS + [
    (dict(dy=None), NULL), (dict(v=None), NULL), (dict(dy=T(5, 48)), SHAPE), (dict(dy=T(5, 40, F32)), DTYPE),
    (dict(dxb=T(5, 72)), SHAPE), (dict(dx=T(4, 64)), SHAPE), (dict(dA=T(15, 64)), SHAPE), (dict(dA=T(16, 64, F32)), DTYPE),
    (dict(dB=T(16, 48)), SHAPE), (dict(dB=T(16, 40, data=A + 2)), ALIGN), (dict(dA=T(16, 64, data=None)), NULL),
    (dict(dx=None, dA=None, dB=None), OK),
])
def test_adapter_backward_checks(kw, status):
    assert adb(**kw) == status


def test_adapter_queries():
    lib, n = _lib.load(), ctypes.c_size_t(0)
    for f in (lib.ss1_adapter_forward_query, lib.ss1_adapter_backward_query):
        assert f(5, byref(AD(a=T(16, 64, data=None), b=T(16, 40, data=None), row=None, scale=None)), byref(n)) == OK
        assert n.value >= 5 * 8 * 4
        assert f(-1, byref(AD()), byref(n)) == SHAPE and f(1 << 31, byref(AD()), byref(n)) == SHAPE
        assert f(5, byref(AD()), None) == NULL and f(5, None, byref(n)) == NULL
        assert f(5, byref(AD(max_rank=200)), byref(n)) == SHAPE


# --------------------------------------------------------------------- AdamW
def E(param=A, grad=A, m=A, v=A, master=None, m_scale=None, v_scale=None, numel=100, decay=0.0, pd=F32, gd=F32, sd=F32):
    return _lib.AdamWEntry(param, grad, m, v, master, m_scale, v_scale, numel, decay, pd, gd, sd)


def plan(*entries, count=None, chunks=True, want_map=False):
    lib, n = _lib.load(), ctypes.c_int64(-1)
    table = (_lib.AdamWEntry * max(1, len(entries)))(*entries)
    m = np.full((1 << 12, 2), -1, dtype=np.int32)
    st = lib.ss1_adamw_plan(table, len(entries) if count is None else count, byref(n) if chunks else None,
                            m.ctypes.data if want_map else None)
    return (st, n.value, m[:max(0, n.value)]) if want_map else st


@pytest.mark.parametrize("kw,status", [
    (dict(param=None), NULL), (dict(grad=None), NULL), (dict(m=None), NULL), (dict(v=None), NULL),
    (dict(sd=FP8, m_scale=A), NULL), (dict(sd=FP8, v_scale=A), NULL), (dict(numel=-1), SHAPE),
    (dict(numel=1 << 39), SHAPE), (dict(decay=-0.1), SHAPE), (dict(decay=float("nan")), SHAPE),
    (dict(master=A), SHAPE), (dict(pd=FP8), DTYPE), (dict(gd=FP8), DTYPE), (dict(sd=BF16), DTYPE), (dict(pd=9), DTYPE),
    (dict(param=A + 4), ALIGN), (dict(grad=A + 2), ALIGN), (dict(m=A + 8), ALIGN), (dict(v=A + 1), ALIGN),
    (dict(pd=BF16, master=A + 4), ALIGN), (dict(sd=FP8, m_scale=A + 2, v_scale=A), ALIGN),
    (dict(), OK), (dict(pd=BF16, master=A), OK), (dict(sd=FP8, m_scale=A, v_scale=A), OK),
    (dict(param=None, grad=None, m=None, v=None, numel=0), OK),
])
def test_adamw_plan_checks(kw, status):
    assert plan(E(), E(**kw)) == status


def test_adamw_plan_covers_every_element_once():
    assert plan(count=-1) == SHAPE and plan(count=1 << 23) == SHAPE and plan(chunks=False) == NULL
    assert _lib.load().ss1_adamw_plan(None, 1, byref(ctypes.c_int64()), None) == NULL
    st, n, m = plan(want_map=True)
    assert (st, n) == (OK, 0)
    sizes = [1, 0, 5000, 256, 1 << 20, 3]
    st, n, m = plan(*[E(numel=s) for s in sizes], want_map=True)
    assert st == OK
    for i, s in enumerate(sizes):
        parts = m[m[:, 0] == i, 1]
        assert list(parts) == list(range(len(parts)))
        assert len(parts) == 0 if s == 0 else len(parts) >= 1


@pytest.mark.parametrize("kw,status", [
    (dict(step=0), SHAPE), (dict(beta1=1.0), SHAPE), (dict(beta1=-0.1), SHAPE), (dict(beta2=float("nan")), SHAPE),
    (dict(lr=-1.0), SHAPE), (dict(lr=float("inf")), SHAPE), (dict(eps=-1e-8), SHAPE), (dict(grad_scale=-1.0), SHAPE),
    (dict(chunks=-1), SHAPE), (dict(count=-1), SHAPE), (dict(entries=None), NULL), (dict(map=None), NULL),
    (dict(hyper=None), NULL), (dict(entries=A + 4), ALIGN), (dict(map=A + 2), ALIGN), (dict(dev=A + 2), ALIGN),
    (dict(chunks=0, entries=None, map=None), OK),
])
def test_adamw_step_checks(kw, status):
    d = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, grad_scale=1.0, dev=None, step=1, seed=0, entries=A, count=1,
             map=A, chunks=1, hyper=True)
    d.update(kw)
    h = _lib.AdamWHyper(d["lr"], d["beta1"], d["beta2"], d["eps"], d["grad_scale"], d["dev"], d["step"], d["seed"])
    assert _lib.load().ss1_adamw_step(d["entries"], d["count"], d["map"], d["chunks"],
                                      byref(h) if d["hyper"] else None, None) == status


# ------------------------------------------------------------------- binding
def test_structures_and_constants_match_the_header():
    text = open(os.path.join(ROOT, "include", "ss1.h")).read()
    assert int(re.search(r"SS1_MAX_RANK (\d+)", text).group(1)) == _ops.MAX_RANK
    assert int(re.search(r"SS1_ADAMW_BLOCK (\d+)", text).group(1)) == _ops.ADAMW_BLOCK
    plain = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    for name, cls in (("ss1_adapters", _lib.Adapters), ("ss1_segments", _lib.Segments),
                      ("ss1_adamw_entry", _lib.AdamWEntry), ("ss1_adamw_hyper", _lib.AdamWHyper)):
        body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", plain).group(1)
        names = [w for line in body.split(";") if line.strip() for w in
                 [p.strip().split()[-1].lstrip("*") for p in line.split(",")]]
        assert names == [f[0] for f in cls._fields_], name


def test_binding_refuses_host_tensors_and_wrong_vectors():
    torch = pytest.importorskip("torch")
    x, g = torch.zeros(2, 8), torch.zeros(8)
    with pytest.raises(ValueError, match="GPU tensors"):
        ss1.layernorm_forward(x, g)
    with pytest.raises(ValueError, match="GPU tensors"):
        ss1.layernorm_backward(x, x, g, g[:2], g[:2])
    with pytest.raises(ValueError, match="GPU tensors"):
        ss1.AdapterSet.make(x, x, [2], [1.0])
    with pytest.raises(ValueError, match="GPU tensors"):
        ss1.AdamWPlan.make([g], [g])
    with pytest.raises(ValueError, match="state must be"):
        ss1.AdamWPlan.make([g], [g], state="int8")
    with pytest.raises(ValueError, match="grads must hold"):
        ss1.AdamWPlan.make([g], [])
