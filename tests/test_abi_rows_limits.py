"""Arguments of process_logits, top_logits and distill at and beyond their limits, without a GPU: every
call here is refused before its first CUDA call."""

import types

import pytest

import verify_spec_draft_gb300 as vsd
from verify_spec_draft_gb300 import build

A = 0x10000          # a 16-byte aligned fake device address
INVALID, SHAPE, ALIGN = 1, 2, 4
TINY = 2.0 ** -126   # the smallest normal float32


@pytest.fixture(scope="module")
def lib():
    if build.needs_build():
        build.build()
    return vsd.load()


def top(lib, t=1.0, ws=A, logits=A):
    return lib.spec_top_logits(logits, vsd.BF16, 4, 100, 100, 8, t, A, A, A, 0, ws, 1 << 24, None)


def distill(lib, t=1.0, ws=A, student=A):
    return lib.spec_distill(student, vsd.BF16, 4, 100, 100, A, vsd.F32, A, 8, 0, 0, t, A, 0, A, ws, 1 << 24, None)


def process(lib, ws=A, logits=A):
    return lib.spec_process_logits(logits, vsd.BF16, 2, 4, 100, 100, A, 16, A, A, A, A, A, A, A, A, A, 3, A, 4, A, ws,
                                   1 << 20, None)


@pytest.mark.parametrize("call", [top, distill])
def test_subnormal_temperature(lib, call):
    """Its reciprocal has no float32."""
    assert call(lib, t=TINY / 2) == INVALID and call(lib, t=1e-45) == INVALID
    assert call(lib, t=TINY, ws=0) != INVALID


@pytest.mark.parametrize("call", [top, distill, process])
@pytest.mark.parametrize("off", [1, 4, 8])
def test_workspace_alignment(lib, call, off):
    """Its records are read and written as 8-byte words."""
    assert call(lib, ws=A + off) == ALIGN


class _Rows:
    """Stands in for a bf16 CUDA tensor: all that a call looks at before it allocates."""
    is_cuda, device = True, types.SimpleNamespace(type="cuda", index=0)

    def __init__(self, shape, strides):
        self.shape, self._strides = shape, strides

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for x in self.shape:
            n *= x
        return n

    def stride(self):
        return self._strides


@pytest.mark.parametrize("shape,strides", [
    ((2, 100), ((1 << 32) + 100, 1)),         # a row stride that is 100 modulo 2^32
    (((1 << 32) + 4, 100), (100, 1)),         # four rows modulo 2^32
    ((2, (1 << 32) + 100), ((1 << 32) + 100, 1))])
def test_sizes_past_32_bits(lib, monkeypatch, shape, strides):
    monkeypatch.setattr(vsd, "_current_device", lambda: 0, raising=False)
    x = _Rows(shape, strides)
    with pytest.raises(vsd.SpecError):
        vsd.top_logits(x, 3)
    with pytest.raises(vsd.SpecError):
        vsd.distill(x, x, x)
    x = _Rows((shape[0], 1, shape[1]), (strides[0], strides[0], 1))
    with pytest.raises(vsd.SpecError):
        vsd.process_logits(x)


def test_rows_on_another_device(lib, monkeypatch):
    """A call is made under the rows' device, whichever is current, and on its streams only."""
    torch = pytest.importorskip("torch")
    here, seen = [3], []

    class under:
        def __init__(self, device):
            seen.append(device)

        def __enter__(self):
            self.was, here[0] = here[0], seen[-1].index

        def __exit__(self, *a):
            here[0] = self.was

    monkeypatch.setattr(vsd, "_current_device", lambda: here[0])
    monkeypatch.setattr(torch.cuda, "device", under)
    x = _Rows(((1 << 32) + 4, 100), (100, 1))          # refused, but not before
    y = _Rows(((1 << 32) + 4, 1, 100), (100, 100, 1))
    for call in (lambda **kw: vsd.top_logits(x, 3, **kw), lambda **kw: vsd.distill(x, x, x, **kw),
                 lambda **kw: vsd.process_logits(y, **kw)):
        with pytest.raises(vsd.SpecError):
            call()
        assert seen.pop() is _Rows.device and not seen and here == [3]
        with pytest.raises(ValueError):
            call(stream=types.SimpleNamespace(device="another", cuda_stream=0))
        with pytest.raises(vsd.SpecError):
            call(stream=types.SimpleNamespace(device=_Rows.device, cuda_stream=0))
        assert seen.pop() is _Rows.device
