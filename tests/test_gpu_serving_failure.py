"""A bounded wait that runs out in the latent projections (above 16 tokens), without faulting or hanging the GPU.

With the give-up limit at a few nanoseconds (valid inputs, nothing else changed) the waits for the first copies give
up; the CTAs drain their copies and MMAs in flight (that drain keeps its normal limit), free their tensor memory and
return. The calls complete, the device error word carries a timeout bit and no other, and a call with the normal limit
gives what it gave before.
"""
import pytest
import torch

import paged_kv_gqa_split_gb300 as pkg
from paged_kv_gqa_split_gb300 import _lib
from paged_kv_gqa_split_gb300.build import build

pytestmark = pytest.mark.gpu
ERR_TIMEOUT_FULL, ERR_TIMEOUT_EMPTY = 1, 2


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    build()
    _lib.load()
    yield
    _lib.gqa_paged_decode_test_wait_limit_ns(0)


@pytest.mark.parametrize("n,h", [(17, 1), (300, 64)])
@pytest.mark.parametrize("absorb", [True, False])
def test_projection_gives_up_and_the_next_call_is_right(n, h, absorb):
    g = torch.Generator().manual_seed(n)
    w = (torch.randn(h, 256, 512, generator=g) / 22).to(torch.bfloat16).cuda()
    x = torch.randn(n, h, 192 if absorb else 512, generator=g).to(torch.bfloat16).cuda()
    pos, freq = torch.arange(n, dtype=torch.int32).cuda(), pkg.rope_inv_freq(64)[0]
    run = (lambda: pkg.mla_absorb_q(x, w, pos, freq)) if absorb else (lambda: pkg.mla_expand_out(x, w))
    want = run()
    assert _lib.gqa_paged_decode_device_error() == 0
    try:
        assert _lib.gqa_paged_decode_test_wait_limit_ns(5) == 0
        for _ in range(3):
            run()
        torch.cuda.synchronize()
        flags = _lib.gqa_paged_decode_device_error()
        assert flags & (ERR_TIMEOUT_FULL | ERR_TIMEOUT_EMPTY), flags
        assert flags & ~(ERR_TIMEOUT_FULL | ERR_TIMEOUT_EMPTY) == 0, flags
    finally:
        _lib.gqa_paged_decode_test_wait_limit_ns(0)
    for _ in range(3):
        assert torch.equal(run(), want)
    assert _lib.gqa_paged_decode_device_error() == 0
