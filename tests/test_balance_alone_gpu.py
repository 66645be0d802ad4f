"""A balance loss whose rows one block covers: it needs no memory of its stream, so a stream that has none can be captured
at once."""
from __future__ import annotations

import pytest
import torch

from test_balance_gpu import F32, check_loss, ids_of, loss_of, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp8_gemm_nt_gb300 as L
    L.load_library()
    L.dg_get_device_status()
    return L


@pytest.mark.parametrize("T, E, scoring", [(0, 16, "softmax"), (1, 64, "softmax"), (40, 60, "sigmoid"), (128, 100, "softmax"), (8, 1000, "sigmoid")])
def test_no_workspace(lib, T, E, scoring):
    x = make(T, E, F32, 1)
    ids = ids_of(x, 3, 1)
    want = loss_of(lib, x, ids, scoring, 1.0)
    s = torch.cuda.Stream()
    lib.dg_release_workspace(s)          # (streams come from a pool: an earlier user of this one may have left some)
    assert lib.dg_get_workspace_size(s) == 0
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = loss_of(lib, x, ids, scoring, 1.0)
        assert lib.dg_get_workspace_size(s) == 0
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            lib.dg_moe_balance_loss(x, ids, *out, scoring=scoring)
        for t in out:
            t.zero_()
        g.replay()
        s.synchronize()
    assert lib.dg_get_workspace_size(s) == 0
    assert all(torch.equal(a, b) for a, b in zip(want, out))
    check_loss(x, ids, out, scoring, 1.0)


def test_more_blocks_take_the_workspace(lib):
    x = make(4000, 60, F32, 2)
    ids = ids_of(x, 3, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = loss_of(lib, x, ids, "softmax", 1.0)
        s.synchronize()
    assert lib.dg_get_workspace_size(s) > 0
    check_loss(x, ids, out, "softmax", 1.0)
    assert lib.dg_get_device_status() == 0
