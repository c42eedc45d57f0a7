"""Masked attention under a distance bias whose keys all lie far away.

Tolerances as in test_gpu_masked.
"""
import math

import pytest
import torch

from streaming_flow_matching_b200 import _lib as L
from tests import _paged_ref as R
from tests.test_gpu_masked import BF, F32, check, ints, ladder, make

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


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 32)])
@pytest.mark.parametrize("n_q,h,hk", [(8, 2, 1), (1, 1, 1)])
@pytest.mark.parametrize("slope", [4.0, -4.0])
def test_splits_of_far_keys_join(cuda_device, dtype, d, n_q, h, hk, slope):
    # keys a million positions away in several splits, whose scores make up for the distances
    from streaming_flow_matching_b200 import attention_masked
    n_kv, seen = 1100000, 2048
    code = L.SFM_DTYPE_BF16 if dtype == BF else L.SFM_DTYPE_FP32
    assert L.lib.sfm_attention_masked_workspace_bytes(n_q, n_kv, h, hk, d, code) > 0
    q, k, v = make(n_q, n_kv, h, hk, d, dtype, seed=7, scale=1.0)
    q[:, :, 0] = 64.0
    tile = torch.arange(seen, device="cuda") // 128           # each tile's best key scores about the same
    up = slope * 128 * (seen // 128 - 1 - tile) if slope > 0 else -slope * 128 * tile
    k[:seen, :, 0] = (up * math.sqrt(d) / 64.0).to(dtype)[:, None]
    los, his = ints([0] * n_q), ints([seen] * n_q)
    sl = torch.full((h,), slope, device="cuda")
    out = attention_masked(q, k, v, los, his, slopes=sl)
    q_pos = n_kv - n_q + torch.arange(n_q, device="cuda")
    ref, mag, _ = R.attend(q, k[:seen], v[:seen], los, his, slopes=sl, q_pos=q_pos)
    if dtype == BF:
        check(out, ref, mag, dtype, far=True)
    else:
        # The tolerance of test_gpu_masked takes sum |q_d k_d| / sqrt(D) to be 11 at most.  Here one
        # product alone is up to slope x 128 x 15 = 7,680.  The score's D additions, its product with
        # the scale and its sum with the bias round by 2^-24 of at most that each: D + 2 roundings of
        # 4.6e-4, 0.016 at D 32, in numerator and denominator of the softmax.
        score = (d + 2) * 2.0 ** -24 * (abs(slope) * 128 * 15 + 11)
        assert bool(((out.double() - ref).abs() <= (2 * score + 2e-4) * mag).all())
    assert L.check_call_error() == 0
