"""A bounded wait of the paged or packed attention that gives up leaves a usable context.

The test hook arms, for the next launch, a wait on a barrier that nothing arrives at, with a limit of 2 ms, in every CTA
that has work.  The kernel unwinds (copies and products in flight end, tensor memory is freed), the device status
says so once, and the next calls on the same pool and scratch give the bits they gave before.
"""

import ctypes

import pytest
import torch

from paged_util import TYPES, inputs, make_pool, starts

pytestmark = pytest.mark.gpu

LIMIT_NS = 2_000_000


@pytest.fixture(scope="module")
def kvc(cuda_device):
    import decode_attention_kv_cache_gb300 as m
    return m


def status(kvc):
    s = ctypes.c_int32(0)
    return kvc.lib.kvc_device_status(ctypes.byref(s)), s.value


def gives_up_and_goes_on(kvc, which, call):
    before = call()
    assert status(kvc) == (kvc.KVC_OK, 0)
    kvc.arm_test_wait_timeout(which, LIMIT_NS)
    call()
    rc, word = status(kvc)
    assert rc == kvc.KVC_EDEVICE and word != 0, (rc, word)
    assert status(kvc) == (kvc.KVC_OK, 0)          # read and cleared
    for _ in range(2):                             # the arm is used up
        after = call()
        assert all(torch.equal(a, b) for a, b in zip(before, after))
    assert status(kvc) == (kvc.KVC_OK, 0)


@pytest.mark.parametrize("held", [[20], [5000, 1, 700], [300] * 120])
@pytest.mark.parametrize("hq", [10, 24])
@pytest.mark.parametrize("cache_type,d", [("q8_0", 128), ("f16", 128), ("q8_0", 64)])
def test_decode_attn_paged(kvc, cache_type, d, hq, held):
    cache, pages, _ = make_pool(kvc, held, 16, 2, d, cache_type, "head_major", layers=1)
    q = inputs((len(held), hq, d), torch.bfloat16, 1)
    scratch = kvc.paged_scratch(cache, len(held), hq)

    def call():
        lse = torch.empty(len(held), hq, device="cuda")
        return kvc.decode_attn_paged(cache, 0, pages, q, lse=lse, scratch=scratch), lse

    gives_up_and_goes_on(kvc, kvc.TEST_PAGED, call)


@pytest.mark.parametrize("n", [[30], [3000, 1, 700], [100] * 200])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64)])
def test_attn_packed(kvc, dtype, d, n):
    q, k, v = (inputs((sum(n), h, d), TYPES[dtype], s) for h, s in ((10, 1), (2, 2), (2, 3)))
    at, scratch = starts(n), kvc.packed_scratch(sum(n), len(n), 10, 2, d)

    def call():
        lse = torch.empty(sum(n), 10, device="cuda")
        return kvc.attn_packed(q, k, v, at, lse=lse, scratch=scratch), lse

    gives_up_and_goes_on(kvc, kvc.TEST_PACKED, call)


def test_kinds_that_are_armed(kvc):
    for which in (-1, kvc.TEST_PACKED + 1):
        assert kvc.lib.kvc_test_arm_wait_timeout(which, LIMIT_NS) == kvc.KVC_EINVAL
    for which in (kvc.TEST_PAGED, kvc.TEST_PACKED):
        assert kvc.lib.kvc_test_arm_wait_timeout(which, 0) == kvc.KVC_OK
