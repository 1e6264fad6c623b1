"""Argument checks of process_logits, top_logits and distill that need no GPU: every call
carries an invalid argument, so it returns before its first CUDA call."""

import ctypes

import pytest

import verify_spec_draft_gb300 as vsd
from verify_spec_draft_gb300 import build

A = 0x10000          # a 16-byte aligned fake device address
MIS = 0x10008        # misaligned
OK, INVALID, SHAPE, DTYPE, ALIGN, WORKSPACE = 0, 1, 2, 3, 4, 9


@pytest.fixture(scope="module")
def lib():
    if build.needs_build():
        build.build()
    return vsd.load()


def test_workspace_bytes(lib):
    wb = lib.spec_workspace_bytes
    assert wb(vsd.OP_PROCESS_LOGITS, 32, 8, 248320, 0) > 0
    assert wb(vsd.OP_PROCESS_LOGITS, 32, 65, 248320, 0) > 0       # gamma + 1 rows
    assert wb(vsd.OP_PROCESS_LOGITS, 32, 66, 248320, 0) == 0
    assert wb(vsd.OP_PROCESS_LOGITS, 65536, 8, 248320, 0) == 0
    for op in (vsd.OP_TOP_LOGITS, vsd.OP_DISTILL):
        assert wb(op, 256, 64, 248320, 0) > 0
        assert wb(op, 256, 129, 248320, 0) == 0
        assert wb(op, 256, 0, 248320, 0) == 0
        assert wb(op, 0, 64, 248320, 0) == 0
        assert wb(op, (1 << 24) + 1, 64, 8, 0) == 0
        assert wb(op, 256, 64, (1 << 20) + 1, 0) == 0
        assert wb(op, 512, 64, 248320, 0) >= wb(op, 256, 64, 248320, 0)


def test_process_logits_argument_errors(lib):
    def call(logits=A, dt=vsd.BF16, B=2, R=4, V=100, ld=100, hist=A, Lmax=16, len_=A, pl=A, blk=A, rep=A, freq=A,
             pres=A, temp=A, bi=A, bv=A, nb=3, mask=A, mr=4, out=A, ws=A, wsb=1 << 20):
        return lib.spec_process_logits(logits, dt, B, R, V, ld, hist, Lmax, len_, pl, blk, rep, freq, pres, temp, bi,
                                       bv, nb, mask, mr, out, ws, wsb, None)
    assert call(dt=2) == DTYPE
    assert call(B=0) == SHAPE and call(B=65536) == SHAPE
    assert call(R=0) == SHAPE and call(R=66) == SHAPE
    assert call(V=0, ld=0) == SHAPE and call(V=(1 << 26) + 1, ld=1 << 27) == SHAPE
    assert call(ld=99) == SHAPE
    assert call(Lmax=-1) == SHAPE and call(Lmax=(1 << 19) + 1) == SHAPE
    assert call(nb=-1) == SHAPE and call(nb=2048) == SHAPE
    assert call(mr=2) == SHAPE and call(mr=0) == SHAPE
    assert call(logits=0) == INVALID and call(out=0) == INVALID
    assert call(hist=0) == INVALID
    assert call(bi=0) == INVALID and call(bv=0) == INVALID
    assert call(logits=MIS) == ALIGN and call(out=MIS) == ALIGN
    assert call(ws=0) == WORKSPACE and call(wsb=100) == WORKSPACE


def test_top_logits_argument_errors(lib):
    def call(logits=A, dt=vsd.BF16, rows=4, V=100, ld=100, K=8, t=1.0, val=A, ids=A, tail=A, lse=0, ws=A, wsb=1 << 24):
        return lib.spec_top_logits(logits, dt, rows, V, ld, K, t, val, ids, tail, lse, ws, wsb, None)
    assert call(dt=9) == DTYPE
    assert call(rows=0) == SHAPE and call(rows=(1 << 24) + 1) == SHAPE
    assert call(V=0, ld=0) == SHAPE and call(V=(1 << 20) + 1, ld=1 << 21) == SHAPE and call(ld=99) == SHAPE
    assert call(K=0) == SHAPE and call(K=129) == SHAPE
    for t in (0.0, -1.0, float("inf"), float("nan")):
        assert call(t=t) == INVALID
    assert call(logits=0) == INVALID and call(val=0) == INVALID and call(ids=0) == INVALID and call(tail=0) == INVALID
    assert call(logits=MIS) == ALIGN
    need = lib.spec_workspace_bytes(vsd.OP_TOP_LOGITS, 4, 8, 100, 0)
    assert call(ws=0) == WORKSPACE and call(wsb=need - 1) == WORKSPACE


def test_distill_argument_errors(lib):
    def call(s=A, dt=vsd.BF16, rows=4, V=100, ld=100, val=A, vdt=vsd.F32, ids=A, K=8, tail=0, w=0, t=1.0, loss=A,
             lse=0, grad=A, ws=A, wsb=1 << 24):
        return lib.spec_distill(s, dt, rows, V, ld, val, vdt, ids, K, tail, w, t, loss, lse, grad, ws, wsb, None)
    assert call(dt=9) == DTYPE and call(vdt=-1) == DTYPE
    assert call(rows=0) == SHAPE and call(rows=(1 << 24) + 1) == SHAPE
    assert call(V=0, ld=0) == SHAPE and call(V=(1 << 20) + 1, ld=1 << 21) == SHAPE and call(ld=99) == SHAPE
    assert call(K=0) == SHAPE and call(K=129) == SHAPE
    for t in (0.0, -1.0, float("inf"), float("nan")):
        assert call(t=t) == INVALID
    assert call(s=0) == INVALID and call(val=0) == INVALID and call(ids=0) == INVALID and call(loss=0) == INVALID
    assert call(s=MIS) == ALIGN and call(grad=MIS) == ALIGN
    need = lib.spec_workspace_bytes(vsd.OP_DISTILL, 4, 8, 100, 0)
    assert call(ws=0) == WORKSPACE and call(wsb=need - 1) == WORKSPACE


def test_binding_refuses_cpu_tensors(lib):
    torch = pytest.importorskip("torch")
    x = torch.zeros((2, 3, 8))
    with pytest.raises(ValueError, match="CUDA tensor"):
        vsd.process_logits(x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        vsd.top_logits(x, 2)
    with pytest.raises(ValueError, match="CUDA tensor"):
        vsd.distill(x, x, x)
    assert ctypes.sizeof(ctypes.c_float) == 4


class _Rows:
    """Stands in for a CUDA tensor of a given shape and strides."""
    is_cuda, device = True, "cuda:0"

    def __init__(self, shape, strides):
        self.shape, self._strides = shape, strides

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        return self._strides if i is None else self._strides[i]


@pytest.mark.parametrize("shape,strides,ld", [
    ((4, 100), (100, 1), 100), ((4, 100), (128, 1), 128), ((2, 3, 100), (384, 128, 1), 128),
    ((2, 1, 100), (128, 7, 1), 128), ((1, 1, 100), (5, 3, 1), 100), ((2, 3, 1), (3, 1, 9), 1)])
def test_row_strides(shape, strides, ld):
    assert vsd._need_rows(_Rows(shape, strides), "x") == ld


@pytest.mark.parametrize("shape,strides", [
    ((4, 100), (100, 2)), ((4, 100), (99, 1)), ((4, 100), (0, 1)), ((2, 3, 100), (400, 128, 1)), ((100,), (1,)),
    ((2, 3, 100), (100, 200, 1))])
def test_row_strides_refused(shape, strides):
    with pytest.raises(ValueError):
        vsd._need_rows(_Rows(shape, strides), "x")
