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
                                "sgd_config_default", "sgd_update_state", "sgd_propose", "sgd_propose_with_update",
                                "sgd_step", "sgd_step_host", "sgd_ingest", "sgd_build_sa", "sgd_poll",
                                "sgd_suffix_array", "sgd_get_error", "sgd_export_snapshot", "sgd_corpus_stats",
                                "sgd_save", "sgd_load", "sgd_reset_rows"))):
        f = getattr(so, name)
        f.restype, f.argtypes = res, args
    return so


def _devices(lib, wanted):
    """Of the calls noted since the last time: where each of `wanted` ran."""
    calls = [c.rsplit("@", 1) for c in lib.fake_seen().decode().splitlines()]
    for w in wanted:
        assert any(w in name for name, _ in calls), (w, calls)
    # (what only computes a size runs anywhere)
    return {int(d) for name, d in calls if name.startswith("cuda") or "launch" in name or "sa_build" in name}


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


def _drafter(lib, device, **over):
    from model_free_suffix_gb300 import _lib as L
    cfg = L.SgdConfig()
    assert lib.sgd_config_default(ctypes.byref(cfg)) == L.SGD_OK
    cfg.max_batch, cfg.seq_capacity, cfg.vocab_size, cfg.k = 1, 64, 100, 4
    for name, value in over.items():
        setattr(cfg, name, value)
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


@pytest.mark.parametrize("device", [0, 1])
@pytest.mark.parametrize("current", [0, 1])
@pytest.mark.parametrize("backoff", [1, 3])
def test_drafting_calls(lib, device, current, backoff, tmp_path):
    from model_free_suffix_gb300 import _lib as L
    keep, at = _address()
    h = _drafter(lib, device, corpus_capacity=256, max_docs=8, row_index=int(backoff == 1), num_backoff=backoff)
    lib.fake_set(current)
    lib.fake_seen()
    n, gen, flags = ctypes.c_int64(), ctypes.c_uint64(), ctypes.c_uint32()
    draft = "launch_backoff" if backoff > 1 else "launch_propose"
    path = str(tmp_path / "corpus").encode()
    for name, want, call in (
            ("launch_update", L.SGD_OK, lambda: lib.sgd_update_state(h, at, at, at, 1, 1, None)),
            (draft, L.SGD_OK, lambda: lib.sgd_propose(h, at, at, None, 1, at, at, None, None, None, None)),
            (draft, L.SGD_OK, lambda: lib.sgd_propose_with_update(h, at, at, at, 1, None, 1, at, at, None, None, None,
                                                                  None)),
            ("launch_ingest", L.SGD_OK, lambda: lib.sgd_step(h, at, at, at, 1, None, 1, at, at, None, None, None, at,
                                                             at, at, 1, None)),
            (draft, L.SGD_OK, lambda: lib.sgd_step(h, at, at, at, 1, None, 1, at, at, None, None, None, None, None,
                                                   None, 0, None)),
            ("cudaMemcpyAsync", L.SGD_OK, lambda: lib.sgd_step_host(h, at, at, at, 1, 1, None, None, None, 0, at, at,
                                                                    None, None, None, None)),
            ("launch_ingest", L.SGD_OK, lambda: lib.sgd_ingest(h, at, at, 1, at, at, at, 1, None)),
            ("launch_linearize", L.SGD_OK, lambda: lib.sgd_build_sa(h, None, None)),
            ("launch_swap", L.SGD_OK_SWAPPED, lambda: lib.sgd_poll(h, 1, -1, None, ctypes.byref(gen))),
            ("sa_build", L.SGD_OK, lambda: lib.sgd_suffix_array(h, at, 8, at, None)),
            ("launch_row_index_reset", L.SGD_OK, lambda: lib.sgd_reset_rows(h, at, at, at, 1, None)),
            ("cudaMemcpy", L.SGD_OK, lambda: lib.sgd_get_error(h, ctypes.byref(flags), 1)),
            ("cudaMemcpy", L.SGD_OK, lambda: lib.sgd_corpus_stats(h, ctypes.byref(n), None)),
            ("cudaDeviceSynchronize", L.SGD_OK,
             lambda: lib.sgd_export_snapshot(h, at, at, 256, ctypes.byref(n), ctypes.byref(gen))),
            ("cudaMemcpy", L.SGD_OK, lambda: lib.sgd_save(h, path, None)),
            ("launch_swap", L.SGD_OK, lambda: lib.sgd_load(h, path, None)),
            ("cudaFree", L.SGD_OK, lambda: lib.sgd_destroy(h))):
        assert call() == want, name
        if "row_index" in name and backoff > 1:   # (no such index then: nothing to do)
            continue
        assert _devices(lib, [name]) == {device}, name
        assert lib.fake_get() == current, name
