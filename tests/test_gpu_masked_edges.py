"""Masked attention under a distance bias whose keys all lie far away.

Tolerances as in test_gpu_masked.
"""
import pytest
import torch

from streaming_flow_matching_b200 import _lib as L
from tests import _paged_ref as R
from tests.test_gpu_masked import F32, check, ints, ladder, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d", [(F32, 32), (F32, 64), (F32, 96), (F32, 128)])
@pytest.mark.parametrize("n_q,h,hk", [(40, 2, 1), (3, 3, 3)])
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_fp32_far_keys_keep_their_differences(cuda_device, dtype, d, n_q, h, hk, cap):
    from streaming_flow_matching_b200 import attention_masked
    n_kv = 60000
    q, k, v = make(n_q, n_kv, h, hk, d, dtype, seed=d, scale=1.0)
    for sl, lo, hi in ((ladder(h), 0, 3000), (ladder(h), 100, 300), (-ladder(h), 0, n_kv), (-ladder(h), 50000, 59000),
                       (torch.ones(h, device="cuda"), 20000, 50000)):
        los, his = ints([lo + 3 * i for i in range(n_q)]), ints([hi - i for i in range(n_q)])
        out = attention_masked(q, k, v, los, his, softcap=cap, slopes=sl)
        ref, mag, _ = R.attend(q, k, v, los, his, cap=cap, slopes=sl)
        check(out, ref, mag, dtype)
    assert L.check_call_error() == 0
