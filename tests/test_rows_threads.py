"""Host threads that call the library at the same time, each with its own stream and workspace."""

import threading

import pytest
import torch

import verify_spec_draft_gb300 as vsd

pytestmark = pytest.mark.gpu


def test_top_logits_of_different_sizes(spec):
    """Rows whose picks need different amounts of shared memory: a call's setting must not cut another's.
    The C calls by themselves, so that the threads are inside them most of the time."""
    lib = vsd.load()
    sizes, errors = [(1 << 20, 128), (500000, 100), (700001, 1)], []
    rows = [torch.randn((1, V), generator=torch.Generator().manual_seed(V)).cuda() for V, _ in sizes]
    want = [vsd.top_logits(z, K) for z, (_, K) in zip(rows, sizes)]
    out = [{k: torch.empty_like(w[k]) for k in ("values", "ids", "tail", "lse")} for w in want]
    streams = [torch.cuda.Stream() for _ in sizes]
    ws = [vsd.workspace(vsd.OP_TOP_LOGITS, 1, K, V, stream=s) for s, (V, K) in zip(streams, sizes)]
    torch.cuda.synchronize()

    def run(i):
        V, K = sizes[i]
        args = (rows[i].data_ptr(), vsd.F32, 1, V, V, K, 1.0, *(out[i][k].data_ptr() for k in out[i]),
                ws[i].data_ptr(), ws[i].numel(), streams[i].cuda_stream)
        for _ in range(20):
            for _ in range(300):
                code = lib.spec_top_logits(*args)
                if code != vsd.OK:
                    errors.append((i, code))
            streams[i].synchronize()

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(sizes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, (len(errors), errors[:3])
    for w, o in zip(want, out):
        for k in o:
            assert torch.equal(w[k], o[k])
