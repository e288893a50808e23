"""Refusals of the verification pass's entry points that need no GPU."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from model_free_suffix_gb300 import build as B
    B.build()
    from model_free_suffix_gb300 import _lib as L
    return L


def test_null_handles(lib):
    L = lib.load()
    assert L.sgd_verify(None, None, lib.F32, 1, 1, None, None, None, None, 1, None, None, None, 1, None, 0,
                        None, None, None, None) == lib.SGD_EINVAL
    assert L.sgd_kv_write(None, None, None, None, lib.F32, 1, 1, 1, 1, None, None, None, 1, 1, None) == lib.SGD_EINVAL
    assert L.sgd_kv_read(None, None, None, None, None, 1, 1, None, None, lib.F32, None) == lib.SGD_EINVAL
    assert L.sgd_kv_attend(None, None, None, lib.BF16, 1, 1, None, None, None, 1, 1, 1, 1.0, 0, 0, None,
                           None) == lib.SGD_EINVAL
    assert L.sgd_kv_destroy(None) == lib.SGD_EINVAL
    assert L.sgd_kv_get_error(None, None, 0) == lib.SGD_EINVAL
    assert L.sgd_kv_memory(None, None) == lib.SGD_EINVAL
    assert L.sgd_kv_launch_count(None, None) == lib.SGD_EINVAL


def test_geometry_is_checked_before_touching_the_gpu(lib):
    L = lib.load()
    good = dict(num_pages=8, page_size=32, kv_heads=2, q_heads=8, head_dim=64, max_batch=4, max_pages_per_row=4)
    bad = [("num_pages", 0), ("page_size", 8), ("page_size", 48), ("page_size", 256), ("kv_heads", 0),
           ("kv_heads", 3), ("q_heads", 1), ("q_heads", 7), ("q_heads", 256), ("head_dim", 96), ("head_dim", 256),
           ("max_batch", 0), ("max_pages_per_row", 0), ("max_pages_per_row", 1 << 26), ("num_pages", 1 << 26)]
    for field, value in bad:
        c = lib.SgdKvConfig(**dict(good, **{field: value}))
        h = ctypes.c_void_p()
        assert L.sgd_kv_create(ctypes.byref(c), 0, ctypes.byref(h)) == lib.SGD_EINVAL, field
        assert not h.value
    assert L.sgd_kv_create(None, 0, ctypes.byref(ctypes.c_void_p())) == lib.SGD_EINVAL
