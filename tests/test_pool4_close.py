"""The bound of long sums sees a lost tile (no GPU): mistakes are planted in attention computed here in 64 bits."""

import pytest
import torch

from pool4_close import attend_close, check_close


@pytest.fixture(scope="module")
def long():
    g = torch.Generator().manual_seed(1)
    n, hkv, d = 20000, 2, 64
    codes = lambda: torch.randint(-8, 8, (n, hkv, d), generator=g).double()
    scales = lambda: ((torch.rand(n, hkv, d // 32, generator=g) * 0.3 + 0.01) * (torch.randint(0, 2, (n, hkv, d // 32), generator=g) * 2 - 1)).half().double()
    q = torch.randn(3, 4, d, generator=g).half().double()
    return q, codes(), scales(), codes(), scales()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_what_is_right_passes_and_a_lost_or_doubled_tile_does_not(long, dtype):
    q, k, dk, v, dv = long
    want, dev, rest, _, _ = attend_close(q, k, dk, v, dv, roundings=1)
    check_close(want.to(dtype), want, dev, rest)
    for first in (0, 9984, 19968):
        keep = torch.ones(k.shape[0], dtype=torch.bool)
        keep[first:first + 32] = False
        lost = attend_close(q, *(t[keep] for t in (k, dk, v, dv)))[0]
        twice = attend_close(q, *(torch.cat([t, t[~keep]]) for t in (k, dk, v, dv)))[0]
        for wrong in (lost, twice):
            with pytest.raises(AssertionError):
                check_close(wrong.to(dtype), want, dev, rest)


def test_sums_of_unsigned_codes_are_too_coarse(long):
    # codes + 8 beside high nibbles summed in float32, 16 keys at a time, and the eights taken off at the end, where the
    # greatest value of a block has the same sign in all keys
    q, k, dk, v, dv = long
    dv = dv.abs()
    want, dev, rest, _, _ = attend_close(q, k, dk, v, dv)
    got = torch.empty_like(want)
    for h in range(4):
        s = q[:, h] @ (k[:, h // 2] * dk[:, h // 2].repeat_interleave(32, -1)).T / 8
        p = torch.exp(s - s.amax(-1, keepdim=True))
        for b in range(2):
            w = (p * dv[:, h // 2, b]).float()
            sums, eights = torch.zeros(3, 32), torch.zeros(3, 1)
            whole = (v[:, h // 2, 32 * b:32 * b + 32] + 8 + 16 * 8).float()   # beside a high nibble of 8
            for a in range(0, k.shape[0], 16):
                sums = sums + w[:, a:a + 16] @ whole[a:a + 16]
                eights = eights + w[:, a:a + 16].sum(-1, keepdim=True)
            got[:, h, 32 * b:32 * b + 32] = (sums - 136 * eights).double() / p.sum(-1, keepdim=True)
    with pytest.raises(AssertionError):
        check_close(got.float(), want, dev, rest)
