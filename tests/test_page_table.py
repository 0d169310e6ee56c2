"""PageTable: a replaced table or length tensor is the one that the next call reads, and is checked like the first."""

import ctypes

import pytest
import torch


@pytest.fixture
def kvc(monkeypatch):
    import decode_attention_kv_cache_gb300 as m

    def need(t, what, dtype=None):     # the device check, without a device
        if not t.is_contiguous() or t.dtype != dtype:
            raise ValueError(what)

    monkeypatch.setattr(m, "_need", need)
    return m


def test_replaced_tensors_are_read(kvc):
    pages = kvc.PageTable(torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), 16)
    pages.lengths = pages.lengths + 1
    assert pages.c.len == pages.lengths.data_ptr() and pages.lengths.tolist() == [1, 1, 1]
    pages.lengths += 1                          # in place, and assigned back
    assert pages.c.len == pages.lengths.data_ptr() and pages.lengths.tolist() == [2, 2, 2]
    wider = torch.ones(3, 7, dtype=torch.int32)
    pages.table = wider
    assert pages.c.table == wider.data_ptr() and pages.c.max_pages == 7 and pages.table is wider
    assert pages.addr == ctypes.addressof(pages.c)


def test_replacements_are_checked(kvc):
    pages = kvc.PageTable(torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), 16)
    before = (pages.c.table, pages.c.len, pages.c.n_seq, pages.c.max_pages)
    for name, bad in (("lengths", torch.zeros(2, dtype=torch.int32)), ("lengths", torch.zeros(3, dtype=torch.int64)),
                      ("lengths", torch.zeros(6, dtype=torch.int32)[::2]), ("table", torch.zeros(2, 4, dtype=torch.int32)),
                      ("table", torch.zeros(4, 3, dtype=torch.int32).t()), ("table", torch.zeros(3, dtype=torch.int32))):
        with pytest.raises(ValueError):
            setattr(pages, name, bad)
    for name in ("n_seq", "page_size", "device"):
        with pytest.raises(AttributeError):
            setattr(pages, name, getattr(pages, name))
    assert before == (pages.c.table, pages.c.len, pages.c.n_seq, pages.c.max_pages)
