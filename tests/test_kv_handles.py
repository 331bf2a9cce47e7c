"""The handles of a key/value cache and of a batch follow their attributes
(CPU): what the library is given is what the attributes hold at the call."""
import copy

import pytest
import torch

from test_weight_quantization_ttq_b200 import ttq

i32 = torch.int32


def _batch(B=3, rows=5, cols=2):
    return ttq.KVBatch(torch.zeros((B, cols), dtype=i32), torch.zeros(B, dtype=i32), torch.zeros(B + 1, dtype=i32), rows, 2)


def _seen(batch):
    batch._arg(-1)          # the device number of CPU tensors
    s = batch._struct
    return s.page_table, s.table_stride, s.kv_len, s.cu_new, s.batch, s.rows, s.max_new


def _held(batch):
    return (batch.page_table.data_ptr(), batch.page_table.shape[1], batch.kv_len.data_ptr(), batch.cu_new.data_ptr(),
            batch.kv_len.shape[0], batch.rows, batch.max_new)


@pytest.mark.parametrize("name,value", [
    ("kv_len", torch.ones(3, dtype=i32)), ("cu_new", torch.ones(4, dtype=i32)), ("page_table", torch.ones((3, 9), dtype=i32)),
    ("rows", 7), ("max_new", 1)])
def test_a_batch_follows_its_attributes(name, value):
    batch = _batch()
    assert _seen(batch) == _held(batch)
    setattr(batch, name, value)
    assert _seen(batch) == _held(batch)
    assert batch._arg(-1) is batch._arg(-1)      # built once for as long as nothing is assigned


def test_every_attribute_at_once():
    batch, other = _batch(), _batch(6, 11, 4)
    _seen(batch)
    for name in ("page_table", "kv_len", "cu_new", "rows", "max_new"):
        setattr(batch, name, getattr(other, name))
    assert _seen(batch) == _held(batch) == _seen(other)


def test_a_copy_has_its_own():
    batch = _batch()
    before = _seen(batch)
    other = copy.copy(batch)
    other.rows = 9
    assert _seen(other)[5] == 9 and _seen(batch) == before


def test_what_is_assigned_is_checked():
    for name, value, error in [("kv_len", torch.zeros(3, dtype=torch.int64), TypeError), ("kv_len", torch.zeros(2, dtype=i32), ValueError),
                               ("cu_new", torch.zeros(3, dtype=i32), ValueError), ("page_table", torch.zeros((2, 2), dtype=i32), ValueError),
                               ("page_table", torch.zeros((3, 4), dtype=i32)[:, ::2], ValueError), ("rows", -1, ValueError),
                               ("max_new", -1, ValueError)]:
        batch = _batch()
        _seen(batch)
        setattr(batch, name, value)
        with pytest.raises(error):
            batch._arg(-1)
        with pytest.raises(error):               # and again: nothing of it is kept
            batch._arg(-1)


def test_a_cache_follows_its_attributes(monkeypatch):
    monkeypatch.setattr(ttq, "_dev", lambda t, name: None if t is None else t.data_ptr())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    cache = ttq.new_kv_cache(4, 32, 2, 128, 4, 64, device="cpu")

    def seen():
        cache._arg()
        s = cache._struct
        return s.pages, s.num_pages, s.D_k, s.D_k_rsqrt, s.scheme

    assert seen() == (cache.pages.data_ptr(), 4, None, None, ttq.TTQ_QSCHEME_ASYMMETRIC)
    cache.pages = torch.zeros((9, cache.pages.shape[1]), dtype=torch.uint8)
    assert seen()[:2] == (cache.pages.data_ptr(), 9)
    cache.D_k, cache.D_k_rsqrt = torch.ones(2, 128), torch.ones(2, 128)
    assert seen()[2:4] == (cache.D_k.data_ptr(), cache.D_k_rsqrt.data_ptr())
    cache.scheme = ttq.TTQ_QSCHEME_SYMMETRIC
    assert seen()[4] == ttq.TTQ_QSCHEME_SYMMETRIC
    for name, value in [("D_k", torch.ones(128)), ("D_k", None), ("pages", torch.zeros((9, 16), dtype=torch.uint8)),
                        ("group", 32)]:          # (another group: the pages' bytes are another format's)
        other = copy.copy(cache)
        setattr(other, name, value)
        with pytest.raises(ValueError):
            other._arg()
