"""Host-side tests of the embedding, the block-scaled matrices, the dense layer
and the gradient norm (no GPU): every argument check returns its status before
any HIP call, the work list of the gradient norm, the workspace queries, and the
binding's structures, constants and refusals."""
import copy
import ctypes
import os
import re

import numpy as np
import pytest

import sketched_parameter_sharing_amd as ss1
from sketched_parameter_sharing_amd import _lib, _model_ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x10000  # fake device address: the checks below fail before it is used
NULL, SHAPE, DTYPE, ALIGN, OK = (_lib.ERR_NULL, _lib.ERR_SHAPE, _lib.ERR_DTYPE, _lib.ERR_ALIGN, _lib.OK)
F32, BF16, FP8 = _lib.F32, _lib.BF16, _lib.FP8_E4M3
byref = ctypes.byref
INF, NAN = float("inf"), float("nan")


def T(rows, cols, dtype=BF16, data=A, reserved=0):
    return _lib.Tensor(data, dtype, reserved, rows, cols)


def Q(rows, cols, block=1, codes=A, scale=A, reserved=0):
    return _lib.Fp8BlocksView(codes, scale, rows, cols, block, reserved)


def K(count=8, nbytes=8, data=A, reserved=0):
    return _lib.Tokens(data, count, nbytes, reserved)


def opt(t):
    return None if t is None else byref(t)


# ------------------------------------------------------------- gradient norm
def entries(*rows):
    return (_lib.GradNormEntry * max(len(rows), 1))(*[_lib.GradNormEntry(*r) for r in rows])


@pytest.mark.parametrize("rows,status", [
    ([(A, 100, F32, 0)], OK), ([], OK), ([(None, 0, BF16, 0)], OK),
    ([(None, 5, F32, 0)], NULL), ([(A, 5, FP8, 0)], DTYPE), ([(A, 5, 9, 0)], DTYPE), ([(A, 5, F32, 1)], SHAPE),
    ([(A, -1, F32, 0)], SHAPE), ([(A, 1 << 39, F32, 0)], SHAPE), ([(A + 8, 5, F32, 0)], ALIGN),
])
def test_gradnorm_plan_checks(rows, status):
    n = ctypes.c_int64(0)
    assert _lib.load().ss1_gradnorm_plan(entries(*rows), len(rows), byref(n), None) == status


def test_gradnorm_plan_lists_every_element_once():
    sizes = [1, 0, 4096, 4097, 12288, 5]
    lib, n = _lib.load(), ctypes.c_int64(0)
    e = entries(*[(A, s, F32, 0) for s in sizes])
    assert lib.ss1_gradnorm_plan(e, len(sizes), byref(n), None) == OK
    m = np.full((n.value, 2), -7, dtype=np.int32)
    assert lib.ss1_gradnorm_plan(e, len(sizes), byref(n), m.ctypes.data) == OK
    for i, s in enumerate(sizes):
        assert m[m[:, 0] == i, 1].tolist() == list(range(-(-s // 4096)))
    assert lib.ss1_gradnorm_plan(None, 1, byref(n), None) == NULL
    assert lib.ss1_gradnorm_plan(e, 1, None, None) == NULL
    assert lib.ss1_gradnorm_plan(e, -1, byref(n), None) == SHAPE
    assert lib.ss1_gradnorm_plan(e, 1 << 23, byref(n), None) == SHAPE


@pytest.mark.parametrize("name", ["ss1_gradnorm", "ss1_gradnorm_clip"])
@pytest.mark.parametrize("kw,status", [
    (dict(entries=None), NULL), (dict(map=None), NULL), (dict(ws=None), NULL), (dict(count=-1), SHAPE),
    (dict(chunks=-1), SHAPE), (dict(chunks=1 << 31), SHAPE), (dict(max_norm=-1.0), SHAPE), (dict(max_norm=NAN), SHAPE),
    (dict(nbytes=8), SHAPE), (dict(entries=A + 4), ALIGN), (dict(map=A + 2), ALIGN), (dict(norm=A + 2), ALIGN),
    (dict(coef=A + 1), ALIGN), (dict(ws=A + 8), ALIGN),
])
def test_gradnorm_checks(name, kw, status):
    d = dict(entries=A, count=3, map=A, chunks=5, max_norm=1.0, norm=A, coef=A, ws=A, nbytes=1 << 20)
    d.update(kw)
    assert getattr(_lib.load(), name)(d["entries"], d["count"], d["map"], d["chunks"], d["max_norm"], d["norm"],
                                      d["coef"], d["ws"], d["nbytes"], None) == status


def test_gradnorm_query_and_a_call_without_results():
    lib, n = _lib.load(), ctypes.c_size_t(7)
    assert lib.ss1_gradnorm_query(0, byref(n)) == OK and n.value == 0
    assert lib.ss1_gradnorm_query(5, byref(n)) == OK and n.value >= 40
    assert lib.ss1_gradnorm_query(-1, byref(n)) == SHAPE
    assert lib.ss1_gradnorm_query(5, None) == NULL
    # neither result wanted, nothing to clip: nothing is enqueued
    assert lib.ss1_gradnorm(A, 3, A, 5, 1.0, None, None, A, 1 << 20, None) == OK
    assert lib.ss1_gradnorm_clip(A, 3, A, 0, 1.0, None, None, None, 0, None) == OK


# ----------------------------------------------------------------- embedding
@pytest.mark.parametrize("kw,status", [
    (dict(tokens=None), NULL), (dict(E=None), NULL), (dict(y=None), NULL), (dict(tokens=K(data=None)), NULL),
    (dict(E=T(50, 64, data=None)), NULL), (dict(y=T(8, 64, data=None)), NULL),
    (dict(tokens=K(nbytes=2)), DTYPE), (dict(E=T(50, 64, FP8)), DTYPE), (dict(y=T(8, 64, 5)), DTYPE),
    (dict(tokens=K(count=-1)), SHAPE), (dict(tokens=K(count=1 << 31)), SHAPE), (dict(tokens=K(reserved=1)), SHAPE),
    (dict(E=T(1 << 29, 64)), SHAPE), (dict(E=T(-1, 64)), SHAPE), (dict(E=T(50, 0), y=T(8, 0)), SHAPE),
    (dict(E=T(50, 65537), y=T(8, 65537)), SHAPE), (dict(y=T(7, 64)), SHAPE), (dict(y=T(8, 63)), SHAPE),
    (dict(y=T(8, 64, reserved=2)), SHAPE), (dict(scale=INF), SHAPE), (dict(scale=NAN), SHAPE),
    (dict(E=T(50, 64, data=A + 8)), ALIGN), (dict(y=T(8, 64, data=A + 2)), ALIGN), (dict(tokens=K(data=A + 4)), ALIGN),
    (dict(tokens=K(0, data=None), y=T(0, 64, data=None)), OK),
])
def test_embedding_forward_checks(kw, status):
    d = dict(tokens=K(), E=T(50, 64), scale=1.0, y=T(8, 64))
    d.update(kw)
    assert _lib.load().ss1_embedding_forward(opt(d["tokens"]), opt(d["E"]), d["scale"], opt(d["y"]), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), NULL), (dict(tokens=None), NULL), (dict(dE=None), NULL), (dict(ws=None), NULL),
    (dict(dy=T(5000, 64, data=None)), NULL), (dict(dE=T(50, 64, data=None)), NULL),
    (dict(tokens=K(5000, data=None)), NULL),
    (dict(dy=T(5000, 64, FP8)), DTYPE), (dict(dE=T(50, 64, 4)), DTYPE), (dict(tokens=K(5000, 1)), DTYPE),
    (dict(dy=T(5001, 64)), SHAPE), (dict(dE=T(50, 63)), SHAPE), (dict(accumulate=2), SHAPE), (dict(accumulate=-1), SHAPE),
    (dict(scale=NAN), SHAPE), (dict(nbytes=64), SHAPE), (dict(dE=T(1 << 29, 64)), SHAPE),
    (dict(dy=T(1 << 30, 64), tokens=K(1 << 30), nbytes=1 << 40), SHAPE),
    (dict(ws=A + 4), ALIGN), (dict(dy=T(5000, 64, data=A + 4)), ALIGN), (dict(dE=T(50, 64, data=A + 4)), ALIGN),
    (dict(tokens=K(0, data=None), dy=T(0, 64, data=None), accumulate=1), OK),
    (dict(dE=T(0, 64, data=None)), OK),
])
def test_embedding_backward_checks(kw, status):
    d = dict(dy=T(5000, 64), tokens=K(5000), scale=1.0, accumulate=0, dE=T(50, 64), ws=A, nbytes=1 << 30)
    d.update(kw)
    assert _lib.load().ss1_embedding_backward(opt(d["dy"]), opt(d["tokens"]), d["scale"], d["accumulate"],
                                              opt(d["dE"]), d["ws"], d["nbytes"], None) == status


def test_embedding_query():
    lib, n = _lib.load(), ctypes.c_size_t(0)
    q = lib.ss1_embedding_backward_query
    for M, V, k in ((0, 50, 64), (1, 1, 1), (8192, 50000, 1280), ((1 << 30) - 1, (1 << 29) - 1, 512)):
        assert q(byref(K(M, data=None)), byref(T(V, k, data=None)), byref(n)) == OK
        assert n.value >= (4 * (V + 1 + M) if M > 1024 else 0)
    assert q(byref(K(8)), byref(T(50, 65537)), byref(n)) == SHAPE
    assert q(byref(K((1 << 30) - 1)), byref(T(50, 1025)), byref(n)) == SHAPE
    assert q(byref(K(1 << 30)), byref(T(50, 1)), byref(n)) == SHAPE
    assert q(None, byref(T(50, 64)), byref(n)) == NULL
    assert q(byref(K(8)), None, byref(n)) == NULL
    assert q(byref(K(8)), byref(T(50, 64)), None) == NULL


# ---------------------------------------------- block-scaled E4M3 matrices
@pytest.mark.parametrize("kw,status", [
    (dict(x=None), NULL), (dict(x=T(40, 300, data=None)), NULL), (dict(q=Q(40, 300, codes=None)), NULL),
    (dict(q=Q(40, 300, scale=None)), NULL), (dict(qt=Q(300, 40, codes=None)), NULL), (dict(x=T(40, 300, FP8)), DTYPE),
    (dict(q=Q(40, 300, 2)), SHAPE), (dict(q=Q(40, 300, 0)), SHAPE), (dict(q=Q(41, 300)), SHAPE),
    (dict(q=Q(40, 299)), SHAPE), (dict(qt=Q(40, 300)), SHAPE), (dict(q=Q(40, 300, reserved=1)), SHAPE),
    (dict(x=T(-1, 300)), SHAPE), (dict(x=T(1 << 19, 1 << 19), q=Q(1 << 19, 1 << 19), qt=None), SHAPE),
    (dict(x=T(40, 300, data=A + 2)), ALIGN), (dict(q=Q(40, 300, codes=A + 8)), ALIGN),
    (dict(qt=Q(300, 40, scale=A + 2)), ALIGN),
    (dict(q=None, qt=None), OK),
    (dict(x=T(0, 300, data=None), q=Q(0, 300, codes=None, scale=None), qt=Q(300, 0, codes=None, scale=None)), OK),
])
def test_quantize_checks(kw, status):
    d = dict(x=T(40, 300), q=Q(40, 300), qt=Q(300, 40))
    d.update(kw)
    assert _lib.load().ss1_quantize_fp8_blocks(opt(d["x"]), opt(d["q"]), opt(d["qt"]), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(a=None), NULL), (dict(b=None), NULL), (dict(y=None), NULL), (dict(a=Q(40, 300, codes=None)), NULL),
    (dict(y=T(40, 90, data=None)), NULL), (dict(y=T(40, 90, FP8)), DTYPE), (dict(a=Q(40, 301)), SHAPE),
    (dict(a=Q(40, 300, 64)), SHAPE), (dict(y=T(41, 90)), SHAPE), (dict(y=T(40, 91)), SHAPE),
    (dict(a=Q(40, 1 << 23), b=Q(90, 1 << 23)), SHAPE),
    (dict(a=Q(1 << 18, 300), b=Q(1 << 18, 300), y=T(1 << 18, 1 << 18)), SHAPE),
    (dict(a=Q(40, 300, codes=A + 4)), ALIGN), (dict(b=Q(90, 300, scale=A + 1)), ALIGN),
    (dict(y=T(40, 90, data=A + 8)), ALIGN),
    (dict(a=Q(0, 300, codes=None, scale=None), y=T(0, 90, data=None)), OK),
])
def test_matmul_checks(kw, status):
    d = dict(a=Q(40, 300), b=Q(90, 300, 128), y=T(40, 90))
    d.update(kw)
    assert _lib.load().ss1_matmul_fp8_blocks(opt(d["a"]), opt(d["b"]), opt(d["y"]), A, 1 << 40, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), NULL), (dict(w=None), NULL), (dict(y=None), NULL), (dict(x=T(40, 300, data=None)), NULL),
    (dict(w=Q(90, 300, codes=None)), NULL), (dict(xt=Q(300, 40, codes=None)), NULL), (dict(ws=None), NULL),
    (dict(x=T(40, 300, FP8)), DTYPE), (dict(y=T(40, 90, F32)), DTYPE), (dict(w=Q(90, 301)), SHAPE),
    (dict(y=T(40, 91)), SHAPE), (dict(y=T(39, 90)), SHAPE), (dict(xt=Q(300, 41)), SHAPE),
    (dict(xt=Q(300, 40, 128)), SHAPE), (dict(nbytes=16), SHAPE), (dict(ws=A + 4), ALIGN),
    (dict(y=T(40, 90, data=A + 2)), ALIGN),
    (dict(x=T(0, 300, data=None), y=T(0, 90, data=None), xt=Q(300, 0, codes=None, scale=None)), OK),
])
def test_dense_forward_checks(kw, status):
    d = dict(x=T(40, 300), w=Q(90, 300), y=T(40, 90), xt=Q(300, 40), ws=A, nbytes=1 << 40)
    d.update(kw)
    assert _lib.load().ss1_dense_forward_fp8(opt(d["x"]), opt(d["w"]), opt(d["y"]), opt(d["xt"]), d["ws"],
                                             d["nbytes"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), NULL), (dict(xt=None), NULL), (dict(wt=None), NULL), (dict(ws=None), NULL),
    (dict(dy=T(40, 90, data=None)), NULL), (dict(dx=T(40, 300, data=None)), NULL), (dict(dW=T(90, 300, data=None)), NULL),
    (dict(dx=T(40, 300, F32)), DTYPE), (dict(dW=T(90, 300, FP8)), DTYPE), (dict(dy=T(40, 90, 9)), DTYPE),
    (dict(xt=Q(300, 41)), SHAPE), (dict(wt=Q(300, 91)), SHAPE), (dict(wt=Q(299, 90)), SHAPE),
    (dict(xt=Q(300, 40, 128)), SHAPE), (dict(dx=T(40, 299)), SHAPE), (dict(dW=T(91, 300)), SHAPE),
    (dict(nbytes=16), SHAPE), (dict(ws=A + 4), ALIGN), (dict(dx=T(40, 300, data=A + 2)), ALIGN),
    (dict(dx=None, dW=None), OK), (dict(dx=None, dW=None, xt=None, wt=None), OK),
])
def test_dense_backward_checks(kw, status):
    d = dict(dy=T(40, 90), xt=Q(300, 40), wt=Q(300, 90, 128), dx=T(40, 300), dW=T(90, 300, F32), ws=A, nbytes=1 << 40)
    d.update(kw)
    assert _lib.load().ss1_dense_backward_fp8(opt(d["dy"]), opt(d["xt"]), opt(d["wt"]), opt(d["dx"]), opt(d["dW"]),
                                              d["ws"], d["nbytes"], None) == status


def test_product_queries():
    lib, n = _lib.load(), ctypes.c_size_t(0)
    assert lib.ss1_matmul_fp8_blocks_query(byref(Q(4, 300)), byref(Q(9, 300)), byref(n)) == OK
    assert lib.ss1_matmul_fp8_blocks_query(byref(Q(4, 300)), byref(Q(9, 301)), byref(n)) == SHAPE
    assert lib.ss1_matmul_fp8_blocks_query(byref(Q(4, 300)), None, byref(n)) == NULL
    assert lib.ss1_matmul_fp8_blocks_query(byref(Q(4, 300)), byref(Q(9, 300)), None) == NULL
    for M in (0, 1, 17, 4096):
        assert lib.ss1_dense_forward_fp8_query(byref(T(M, 300, data=None)), byref(Q(9, 300, codes=None)), byref(n)) == OK
    assert n.value >= 4096 * 384
    assert lib.ss1_dense_forward_fp8_query(byref(T(4, 300)), byref(Q(9, 299)), byref(n)) == SHAPE
    assert lib.ss1_dense_forward_fp8_query(None, byref(Q(9, 299)), byref(n)) == NULL
    q = lib.ss1_dense_backward_fp8_query
    assert q(byref(T(40, 90)), byref(Q(300, 40)), byref(Q(300, 90)), byref(n)) == OK
    assert n.value >= 40 * 128 + 90 * 128
    assert q(byref(T(40, 90)), None, None, byref(n)) == OK and n.value == 0
    assert q(byref(T(40, 90)), byref(Q(300, 41)), None, byref(n)) == SHAPE
    assert q(byref(T(40, 90)), None, byref(Q(300, 91)), byref(n)) == SHAPE
    assert q(None, None, None, byref(n)) == NULL


# ------------------------------------------------------------------- binding
def test_structures_and_constants_match_the_header():
    text = open(os.path.join(ROOT, "include", "ss1.h")).read()
    assert int(re.search(r"SS1_FP8_BLOCK (\d+)", text).group(1)) == _model_ops.FP8_BLOCK
    plain = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    for name, cls in (("ss1_gradnorm_entry", _lib.GradNormEntry), ("ss1_tokens", _lib.Tokens),
                      ("ss1_fp8_blocks", _lib.Fp8BlocksView)):
        body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", plain).group(1)
        names = [line.strip().split()[-1].lstrip("*") for line in body.split(";") if line.strip()]
        assert names == [f[0] for f in cls._fields_], name


class On:
    """A host tensor that says it lies on GPU ``index``."""

    def __init__(self, t, index):
        self.t, self.index = t, index

    def get_device(self):
        return self.index

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_binding_refuses_wrong_tensors(monkeypatch):
    torch = pytest.importorskip("torch")
    from sketched_parameter_sharing_amd import _ops
    x, ids = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int64)
    b = ss1.Fp8Blocks(torch.zeros(2, 128, dtype=torch.uint8), torch.zeros(2, 4, dtype=torch.uint8), 1, 8)
    for call in (lambda: ss1.embedding_forward(ids, x), lambda: ss1.embedding_backward(x, ids, 4),
                 lambda: ss1.quantize_fp8_blocks(x), lambda: ss1.matmul_fp8_blocks(b, b),
                 lambda: ss1.dense_forward_fp8(x, b), lambda: ss1.dense_backward_fp8(x, b, b),
                 lambda: ss1.GradNormPlan.make([x])):
        with pytest.raises(ValueError, match="GPU tensors"):
            call()
    # what is refused on the GPU, with tensors that say they lie on one
    _ops._setup()
    monkeypatch.setattr(_ops, "_current_device", lambda: 0)
    gx, gids = On(x, 0), On(ids, 0)
    with pytest.raises(TypeError, match="int32 or int64"):
        ss1.embedding_forward(On(ids.float(), 0), gx)
    with pytest.raises(ValueError, match="1-D"):
        ss1.embedding_forward(On(ids[None], 0), gx)
    with pytest.raises(ValueError, match="one GPU"):
        ss1.embedding_forward(On(ids, 1), gx)
    with pytest.raises(TypeError, match="y is"):
        ss1.embedding_forward(gids, gx, y=gx, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="accumulate"):
        ss1.embedding_backward(gx, gids, 4, accumulate=True)
    with pytest.raises(ValueError, match="5 rows"):
        ss1.embedding_backward(gx, gids, 5, dE=gx)
    with pytest.raises(TypeError, match="dE is"):
        ss1.embedding_backward(gx, gids, 2, dE=gx, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="share memory"):
        ss1.GradNormPlan.make([gx, On(x[1:], 0)])
    with pytest.raises(ValueError, match="contiguous"):
        ss1.GradNormPlan.make([On(x.t(), 0)])
    with pytest.raises(ValueError, match="one GPU"):
        ss1.GradNormPlan.make([gx, On(x.clone(), 1)])
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        ss1.GradNormPlan.make([On(x.double(), 0)])

    def blocks(codes=b.codes, scale=b.scale, block=1, cols=8, at=0):
        return ss1.Fp8Blocks(On(codes, at), On(scale, at), block, cols)

    for bad, match in ((blocks(block=2), "block must be"), (blocks(cols=129), "256 wide"),
                       (blocks(codes=b.codes[:, :64]), "contiguous"), (blocks(scale=b.scale[:1]), "scale must be"),
                       (blocks(block=128), "scale must be"), (blocks(at=1), "one GPU")):
        with pytest.raises(ValueError, match=match):
            ss1.dense_forward_fp8(gx, bad)
    with pytest.raises(TypeError, match="codes must be"):
        ss1.dense_forward_fp8(gx, blocks(codes=b.codes.float()))
    with pytest.raises(TypeError, match="scale must be"):
        ss1.dense_forward_fp8(gx, blocks(scale=b.scale.float()))
    with pytest.raises(ValueError, match="block must be"):
        ss1.Fp8Blocks.empty(4, 4, 64, "cpu")
    e = ss1.Fp8Blocks.empty(130, 513, 128, "cpu")
    assert e.codes.shape == (130, 640) and e.scale.shape == (2, 8) and e.rows == 130
    assert copy.copy(e).cols == 513
