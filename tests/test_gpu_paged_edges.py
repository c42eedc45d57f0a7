"""The paged cache at its edges: calls from several threads, bad pages beside the state arrays, queries
far from every position, values that a vanishing weight could hide.

Tolerances as in test_gpu_paged.
"""
import sys
import threading

import pytest
import torch

from streaming_flow_matching_b200 import _lib as L
from tests import _paged_ref as R
from tests.test_gpu_paged import BF, F32, Cache, ints, ladder, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d,h", [(BF, 128, 8), (BF, 128, 16), (F32, 64, 4)])
def test_two_host_threads(cuda_device, dtype, d, h):
    # calls of one kernel with different needs of shared memory (weights or none), from two threads at once
    lens = [100, 70]
    c = Cache(lens, 16, 1, d, dtype, seed=3)
    q = torch.randn(2, h, d, device="cuda").to(dtype)
    code = L.SFM_DTYPE_BF16 if dtype == BF else L.SFM_DTYPE_FP32
    n_pages, page = c.k.shape[:2]
    width, dev_lens = c.table.shape[1], ints(lens)
    for weights in (0, 1):
        assert L.lib.sfm_paged_attention_workspace_bytes(2, width * page, h, 1, d, code, weights) == 0
    w = torch.zeros(2, 1, 100, device="cuda")
    outs = [torch.zeros_like(q) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    want = run(c, q, lens)
    torch.cuda.synchronize()
    codes, start = [set(), set()], threading.Barrier(2)

    def caller(i):
        args = (q.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), c.table.data_ptr(), dev_lens.data_ptr(),
                outs[i].data_ptr(), 2, n_pages, page, width, h, 1, d, code, 0.0, None, None, None,
                w.data_ptr() if i else None, 100 if i else 0, None, 0, streams[i].cuda_stream)
        start.wait()
        for _ in range(20000):
            codes[i].add(L.lib.sfm_paged_attention(*args))

    every, threads = sys.getswitchinterval(), [threading.Thread(target=caller, args=(i,)) for i in range(2)]
    sys.setswitchinterval(1e-5)
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(every)
    torch.cuda.synchronize()
    assert codes == [{L.SFM_OK}, {L.SFM_OK}]
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    assert L.check_call_error() == 0
