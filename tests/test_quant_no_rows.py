"""A write or a read back of no rows is a no-op, also of tensors that hold none (their address is null).  CPU."""

import ctypes

import pytest

import lora_shared_kv_b200 as lrkv

FAKE = 0x10000  # never dereferenced


def _views():
    prob = lrkv.make_problem(2, 1, 2, 2, 128, 16)
    empty = lrkv.KVView(None, None, 2 * 128, 128, 128, None, 0, 0, 0, 0)
    codes = lrkv.QKVView(FAKE, FAKE, FAKE, FAKE, 2 * 8192 * 128, 8192 * 128, 128, 256, 128)
    return prob, empty, codes


@pytest.mark.parametrize("first", [None, FAKE])
def test_no_rows_of_an_empty_tensor(first):
    prob, empty, codes = _views()
    L = lrkv.lib()
    for T, status in ((0, 0), (1, 1)):
        assert L.lrkv_quantize_kv(ctypes.byref(prob), ctypes.byref(empty), T, ctypes.byref(codes), 8192, first, None,
                                  FAKE, 256, None) == status
        assert L.lrkv_dequantize_kv(ctypes.byref(prob), ctypes.byref(codes), 8192, T, ctypes.byref(empty), first,
                                    None, FAKE, 256, None) == status


def test_no_rows_still_need_a_cache_and_a_workspace():
    prob, empty, codes = _views()
    L = lrkv.lib()
    bad = lrkv.QKVView(None, FAKE, FAKE, FAKE, 2 * 8192 * 128, 8192 * 128, 128, 256, 128)
    assert L.lrkv_quantize_kv(ctypes.byref(prob), ctypes.byref(empty), 0, ctypes.byref(bad), 8192, None, None, FAKE,
                              256, None) == 1
    assert L.lrkv_quantize_kv(ctypes.byref(prob), ctypes.byref(empty), 0, ctypes.byref(codes), 8192, None, None, None,
                              256, None) == 1
    assert L.lrkv_quantize_kv(ctypes.byref(prob), ctypes.byref(empty), 0, ctypes.byref(codes), -1, None, None, FAKE,
                              256, None) == 1
