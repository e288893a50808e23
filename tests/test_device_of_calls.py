"""A call runs on its handle's device, whichever is current, and leaves the caller's current."""
import ctypes

import pytest

import fake_runtime


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    so = fake_runtime.build(tmp_path_factory.mktemp("fake"))
    so.fake_seen.restype = ctypes.c_char_p
    from model_free_suffix_gb300 import _lib as L
    for name, (res, args) in ((n, (f.restype, f.argtypes)) for n, f in
                              ((n, getattr(L.load(), n)) for n in
                               ("sgd_create", "sgd_destroy", "sgd_verify", "sgd_kv_create", "sgd_kv_destroy",
                                "sgd_kv_write", "sgd_kv_read", "sgd_kv_attend", "sgd_kv_get_error",
                                "sgd_config_default"))):
        f = getattr(so, name)
        f.restype, f.argtypes = res, args
    return so


def _devices(lib, wanted):
    """Of the calls noted since the last time: where each of `wanted` ran."""
    calls = [c.rsplit("@", 1) for c in lib.fake_seen().decode().splitlines()]
    for w in wanted:
        assert any(w in name for name, _ in calls), (w, calls)
    return {int(d) for _, d in calls}


def _address(n=4096):
    block = ctypes.create_string_buffer(n + 16)
    return block, (ctypes.addressof(block) + 15) // 16 * 16


@pytest.mark.parametrize("device", [0, 1])
@pytest.mark.parametrize("current", [0, 1])
def test_cache_calls(lib, device, current):
    from model_free_suffix_gb300 import _lib as L
    keep, at = _address()
    cfg = L.SgdKvConfig(num_pages=2, page_size=16, kv_heads=1, q_heads=1, head_dim=64, max_batch=1,
                        max_pages_per_row=2)
    layer = L.SgdKvLayer(at, at, at, at)
    h = ctypes.c_void_p()
    lib.fake_set(current)
    lib.fake_seen()
    assert lib.sgd_kv_create(ctypes.byref(cfg), device, ctypes.byref(h)) == L.SGD_OK
    assert _devices(lib, ["cudaMalloc"]) == {device} and lib.fake_get() == current
    ref = ctypes.addressof(layer)
    flags = ctypes.c_uint32()
    for name, call in (
            ("launch_kv_write", lambda: lib.sgd_kv_write(h, ref, at, at, L.BF16, 64, 64, 64, 64, at, at, at, 1, 1, None)),
            ("launch_kv_read", lambda: lib.sgd_kv_read(h, ref, at, at, at, 1, 1, at, at, L.BF16, None)),
            ("launch_kv_attend", lambda: lib.sgd_kv_attend(h, ref, at, L.BF16, 64, 64, at, at, at, 1, 1, 1, 1.0, 0, 0,
                                                           at, None)),
            ("cudaMemcpy", lambda: lib.sgd_kv_get_error(h, ctypes.byref(flags), 1)),
            ("cudaFree", lambda: lib.sgd_kv_destroy(h))):
        assert call() == L.SGD_OK, name
        assert _devices(lib, [name]) == {device}, name
        assert lib.fake_get() == current, name


def test_create_on_a_device_that_is_not_there(lib):
    from model_free_suffix_gb300 import _lib as L
    cfg = L.SgdKvConfig(num_pages=2, page_size=16, kv_heads=1, q_heads=1, head_dim=64, max_batch=1,
                        max_pages_per_row=2)
    h = ctypes.c_void_p()
    lib.fake_set(0)
    lib.fake_seen()
    assert lib.sgd_kv_create(ctypes.byref(cfg), 7, ctypes.byref(h)) == L.SGD_ECUDA
    assert not h.value and lib.fake_get() == 0 and lib.fake_seen() == b""


def _drafter(lib, device):
    from model_free_suffix_gb300 import _lib as L
    cfg = L.SgdConfig()
    assert lib.sgd_config_default(ctypes.byref(cfg)) == L.SGD_OK
    cfg.max_batch, cfg.seq_capacity, cfg.vocab_size, cfg.k = 1, 64, 100, 4
    h = ctypes.c_void_p()
    assert lib.sgd_create(ctypes.byref(cfg), device, ctypes.byref(h)) == L.SGD_OK
    return h


@pytest.mark.parametrize("device", [0, 1])
@pytest.mark.parametrize("current", [0, 1])
def test_verification(lib, device, current):
    from model_free_suffix_gb300 import _lib as L
    keep, at = _address()
    h = _drafter(lib, device)
    lib.fake_set(current)
    lib.fake_seen()
    assert lib.sgd_verify(h, at, L.F32, 100, 5, None, at, at, None, 1, None, at, at, 100, None, 0, at, at, None,
                          None) == L.SGD_OK
    assert _devices(lib, ["launch_verify"]) == {device} and lib.fake_get() == current
    assert lib.sgd_destroy(h) == L.SGD_OK
