"""attn_packed with starts that no caller means: every value has a meaning, and none takes long."""

import pytest
import torch

from paged_util import attend64, check, check_lse, half_step, i32, inputs

pytestmark = pytest.mark.gpu

LOW, HIGH = -(1 << 31), (1 << 31) - 1


@pytest.fixture(scope="module")
def kvc(cuda_device):
    import decode_attention_kv_cache_gb300 as m
    return m


def run(kvc, qs, ks, d=64):
    q, k, v = (inputs((60, h, d), torch.float16, s) for h, s in ((4, 1), (2, 2), (2, 3)))
    out, lse = torch.full_like(q, 7.0), torch.full((60, 4), 5.0, device="cuda")
    kvc.attn_packed(q, k, v, i32(qs), i32(ks), out=out, lse=lse)
    assert kvc.kvc_device_status() == 0
    return q, k, v, out, lse


def nothing(out, lse, a, b):
    assert (out[a:b] == 0).all() and (lse[a:b] == -float("inf")).all()


def attends(q, k, v, out, lse, a, b, k0, k1, past=0):
    n = b - a + past
    o, l, bd, lb = attend64(q[a:b], k[k0:k1], v[k0:k1], torch.arange(b - a, device="cuda") + k1 - k0 - n,
                            p_step=half_step(q.dtype))
    check(out[a:b], o, bd)
    check_lse(lse[a:b], l, lb)


@pytest.mark.parametrize("end", [LOW, LOW + 5, -1, 0, 4, 5])
@pytest.mark.parametrize("d", [64, 128])
def test_key_starts_that_decrease(kvc, end, d):
    q, k, v, out, lse = run(kvc, [0, 20, 40], [5, end, 60], d)
    nothing(out, lse, 0, 20)
    attends(q, k, v, out, lse, 20, 40, max(end, 0), 60)
    assert (out[40:] == 7).all() and (lse[40:] == 5).all()


def test_key_starts_past_the_tensor(kvc):
    _, _, _, out, lse = run(kvc, [0, 20, 40, 60], [60, HIGH, HIGH, HIGH])
    nothing(out, lse, 0, 60)


@pytest.mark.parametrize("end", [HIGH, HIGH - 100, 1 << 30])
def test_a_sequence_of_more_rows_than_the_tensor_has(kvc, end):
    # its rows are the first of `end`, of which the keys belong to the last 60
    _, _, _, out, lse = run(kvc, [0, end], [0, 60])
    nothing(out, lse, 0, 60)


def test_rows_that_are_cut_still_count(kvc):
    q, k, v, out, lse = run(kvc, [0, 20, 70], [0, 20, 60])
    attends(q, k, v, out, lse, 0, 20, 0, 20)
    attends(q, k, v, out, lse, 20, 60, 20, 60, past=10)


def test_row_starts_that_decrease(kvc):
    q, k, v, out, lse = run(kvc, [30, 10, 25], [0, 20, 50])
    attends(q, k, v, out, lse, 10, 25, 20, 50)
    assert (out[:10] == 7).all() and (out[25:] == 7).all() and (lse[25:] == 5).all()
