"""Refusals of the calls for prompts that need no GPU."""
import ctypes

import pytest
import torch

import fake_runtime


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    so = fake_runtime.build(tmp_path_factory.mktemp("fake"))
    so.fake_seen.restype = ctypes.c_char_p
    from model_free_suffix_gb300 import _lib as L
    for name in ("sgd_kv_create", "sgd_kv_destroy", "sgd_kv_attend_prompt", "sgd_kv_attend_chunk", "sgd_kv_assign",
                 "sgd_kv_launch_count"):
        f, g = getattr(so, name), getattr(L.load(), name)
        f.restype, f.argtypes = g.restype, g.argtypes
    return so


@pytest.fixture
def handle(lib):
    from model_free_suffix_gb300 import _lib as L
    cfg = L.SgdKvConfig(num_pages=4, page_size=16, kv_heads=2, q_heads=4, head_dim=64, max_batch=9000, max_pages_per_row=2)
    h = ctypes.c_void_p()
    assert lib.sgd_kv_create(ctypes.byref(cfg), 0, ctypes.byref(h)) == L.SGD_OK
    yield h
    assert lib.sgd_kv_destroy(h) == L.SGD_OK


BLOCK = ctypes.create_string_buffer(4096 + 16)
AT = (ctypes.addressof(BLOCK) + 15) // 16 * 16


def _prompt(lib, h, **over):
    a = dict(dict(q=AT, k=AT, v=AT, dtype=2, qt=256, qh=64, kt=128, kh=64, vt=128, vh=64, starts=AT, B=1, N=3, scale=1.0,
                  window=0, sinks=0, out=AT), **over)
    return lib.sgd_kv_attend_prompt(h, a["q"], a["k"], a["v"], a["dtype"], a["qt"], a["qh"], a["kt"], a["kh"], a["vt"],
                                    a["vh"], a["starts"], a["B"], a["N"], a["scale"], a["window"], a["sinks"], a["out"], None)


def _chunk(lib, h, **over):
    from model_free_suffix_gb300 import _lib as L
    layer = L.SgdKvLayer(AT, AT, AT, AT)
    a = dict(dict(layer=ctypes.addressof(layer), q=AT, k=AT, v=AT, dtype=1, qt=256, qh=64, kt=128, kh=64, vt=128, vh=64,
                  table=AT, lens=AT, starts=AT, B=1, N=3, scale=1.0, window=0, sinks=0, out=AT), **over)
    return lib.sgd_kv_attend_chunk(h, a["layer"], a["q"], a["k"], a["v"], a["dtype"], a["qt"], a["qh"], a["kt"], a["kh"],
                                   a["vt"], a["vh"], a["table"], a["lens"], a["starts"], a["B"], a["N"], a["scale"],
                                   a["window"], a["sinks"], a["out"], None)


def _assign(lib, h, **over):
    from model_free_suffix_gb300 import _lib as L
    a = dict(dict(table=AT, held=AT, free=AT, count=AT, keep=AT, new=AT, B=1, N=3, lens=AT, starts=AT, positions=AT, slots=AT,
                  rows=AT), **over)
    pages = L.SgdKvPages(a["table"], a["held"], a["free"], a["count"])
    return lib.sgd_kv_assign(h, ctypes.addressof(pages), a["keep"], a["new"], a["B"], a["N"], a["lens"], a["starts"],
                             a["positions"], a["slots"], a["rows"], None)


BOTH = [dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(starts=None), dict(dtype=0), dict(dtype=3), dict(qt=-1),
        dict(kh=-64), dict(vt=-1), dict(window=-1), dict(sinks=-1), dict(scale=float("nan")), dict(B=-1), dict(B=9001),
        dict(N=-1), dict(out=AT + 8), dict(q=AT + 1), dict(k=AT + 1), dict(v=AT + 1)]


@pytest.mark.parametrize("bad", BOTH, ids=str)
def test_attention_refuses(lib, handle, bad):
    from model_free_suffix_gb300 import _lib as L
    assert _prompt(lib, handle) == L.SGD_OK and _chunk(lib, handle) == L.SGD_OK
    lib.fake_seen()
    assert _prompt(lib, handle, **bad) == L.SGD_EINVAL and _chunk(lib, handle, **bad) == L.SGD_EINVAL
    assert b"launch" not in lib.fake_seen()


def test_chunk_refuses(lib, handle):
    from model_free_suffix_gb300 import _lib as L
    for bad in (dict(layer=None), dict(table=None), dict(lens=None)):
        assert _chunk(lib, handle, **bad) == L.SGD_EINVAL
    layer = L.SgdKvLayer(AT, AT + 8, AT, AT)
    assert _chunk(lib, handle, layer=ctypes.addressof(layer)) == L.SGD_EINVAL


def test_assign_refuses(lib, handle):
    from model_free_suffix_gb300 import _lib as L
    assert _assign(lib, handle) == L.SGD_OK
    assert b"launch_kv_assign" in lib.fake_seen()
    for bad in (dict(table=None), dict(held=None), dict(free=None), dict(count=None), dict(keep=None), dict(new=None),
                dict(lens=None), dict(starts=None), dict(B=-1), dict(B=9001), dict(N=-1)):
        assert _assign(lib, handle, **bad) == L.SGD_EINVAL, bad
    assert b"launch" not in lib.fake_seen()
    for less in (dict(positions=None), dict(slots=None), dict(rows=None), dict(N=0), dict(B=0, keep=None, new=None, lens=None)):
        assert _assign(lib, handle, **less) == L.SGD_OK, less


def test_more_rows_than_a_call_takes(lib, handle):
    from model_free_suffix_gb300 import _lib as L
    for call in (_prompt, _chunk, _assign):
        assert call(lib, handle, B=8193) == L.SGD_ETOOLARGE
        assert call(lib, handle, B=8192) == L.SGD_OK


def test_more_tokens_than_a_call_takes(lib, handle):
    from model_free_suffix_gb300 import _lib as L
    assert _assign(lib, handle, N=(1 << 30) + 1) == L.SGD_ETOOLARGE
    for call in (_prompt, _chunk):      # (two query heads a head: 2^30 rows)
        assert call(lib, handle, N=(1 << 29) + 1) == L.SGD_ETOOLARGE
        assert call(lib, handle, N=1 << 29) == L.SGD_OK


def test_nothing_to_do_launches_nothing(lib, handle):
    from model_free_suffix_gb300 import _lib as L
    lib.fake_seen()
    for call in (_prompt, _chunk):
        assert call(lib, handle, B=0) == L.SGD_OK and call(lib, handle, N=0) == L.SGD_OK
    assert b"launch" not in lib.fake_seen()


def test_null_handles():
    from model_free_suffix_gb300 import _lib as L
    lib = L.load()
    assert _prompt(lib, None) == L.SGD_EINVAL and _chunk(lib, None) == L.SGD_EINVAL and _assign(lib, None) == L.SGD_EINVAL


@pytest.mark.parametrize("device", [0, 1])
@pytest.mark.parametrize("current", [0, 1])
def test_calls_run_on_their_handles_device(lib, device, current):
    from model_free_suffix_gb300 import _lib as L
    cfg = L.SgdKvConfig(num_pages=4, page_size=16, kv_heads=2, q_heads=4, head_dim=64, max_batch=4, max_pages_per_row=2)
    h = ctypes.c_void_p()
    lib.fake_set(current)
    assert lib.sgd_kv_create(ctypes.byref(cfg), device, ctypes.byref(h)) == L.SGD_OK
    for call, name in ((_prompt, "launch_kv_new"), (_chunk, "launch_kv_new"), (_assign, "launch_kv_assign")):
        lib.fake_seen()
        assert call(lib, h) == L.SGD_OK
        seen = lib.fake_seen().decode().splitlines()
        assert {c.rsplit("@", 1)[1] for c in seen if name in c} == {str(device)}, name
        assert lib.fake_get() == current
    assert lib.sgd_kv_destroy(h) == L.SGD_OK
    lib.fake_set(0)


# ---- the Python methods, with a stand-in for the library -----------------------------------------------

class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append(name) or 0


@pytest.fixture
def cache():
    from model_free_suffix_gb300 import KVCache
    from model_free_suffix_gb300 import _lib as L
    c = KVCache.__new__(KVCache)
    c._lib, c._h = Library(), None
    c._index, c.device = -1, torch.device("cpu")
    c.cfg = L.SgdKvConfig(10, 16, 2, 4, 64, 3, 5)
    c.kv_heads, c.q_heads, c.head_dim, c.page_size, c.max_batch, c.max_pages = 2, 4, 64, 16, 3, 5
    c._layer_refs = [0]
    return c


I32 = dict(dtype=torch.int32)


def test_tensors_of_attention(cache):
    t = lambda n, h, d=64, dtype=torch.bfloat16: torch.zeros(n, h, d, dtype=dtype)  # noqa: E731
    q, k, starts, lens, table = t(6, 4), t(6, 2), torch.zeros(4, **I32), torch.zeros(3, **I32), torch.zeros(3, 5, **I32)
    half, wide = torch.float16, torch.float32
    bad = [(t(6, 3), k, k), (t(6, 4, 32), k, k), (q, t(6, 4), k), (q, k, t(5, 2)), (q, t(7, 2), t(7, 2)), (q, t(6, 2, dtype=half), k),
           (q, k, t(6, 2, dtype=half)), (t(6, 4, dtype=wide), t(6, 2, dtype=wide), t(6, 2, dtype=wide)),
           (q.transpose(0, 2)[:6, :, :64], k, k), (torch.zeros(6, 4, 128, dtype=torch.bfloat16)[..., ::2], k, k)]
    for args in bad:
        with pytest.raises(ValueError):
            cache.attend_prompt(*args, starts, stream=0)
        with pytest.raises(ValueError):
            cache.attend_chunk(*args, table, lens, starts, stream=0)
    for out in (t(5, 4), t(6, 4, dtype=half), t(6, 4).transpose(0, 1).contiguous().transpose(0, 1)):
        with pytest.raises(ValueError):
            cache.attend_prompt(q, k, k, starts, out=out, stream=0)
    for bad in ((table[:2], lens, starts), (table[:, :4], lens, starts), (table, lens, starts[:3]), (table.long(), lens, starts)):
        with pytest.raises(ValueError):
            cache.attend_chunk(q, k, k, *bad, stream=0)
    assert cache._lib.calls == []
    cache.attend_prompt(q, k, k, starts, stream=0)
    cache.attend_chunk(q, k, k, table, lens, starts, stream=0)
    assert cache._lib.calls == ["sgd_kv_attend_prompt", "sgd_kv_attend_chunk"]


def test_tensors_of_assign(cache):
    from model_free_suffix_gb300 import KVPages, PagePlan
    pages, keep = cache.new_pages(), torch.zeros(3, **I32)
    assert pages.free.tolist() == list(range(9, -1, -1)) and pages.free_count.tolist() == [10]
    z = lambda *n: torch.zeros(*n, **I32)  # noqa: E731
    with pytest.raises(ValueError):
        cache.assign(pages, keep, keep, stream=0)                          # room for how many tokens?
    for out in (PagePlan(z(2), z(4), z(6)), PagePlan(z(3), z(3), z(6)), PagePlan(z(3), z(4), z(6), z(5)),
                PagePlan(z(3), z(4)), PagePlan(z(3), z(4), z(6).long()), PagePlan(z(3), z(4), z(6, 1))):
        with pytest.raises(ValueError):
            cache.assign(pages, keep, keep, out=out, stream=0)
    for p in (KVPages(z(2, 5), z(3), z(10), z(1)), KVPages(z(3, 5), z(2), z(10), z(1)), KVPages(z(3, 5), z(3), z(9), z(1)),
              KVPages(z(3, 5), z(3), z(10), z(2)), KVPages(z(3, 5).long(), z(3), z(10), z(1))):
        with pytest.raises(ValueError):
            cache.assign(p, keep, keep, 6, stream=0)
    for k, n in ((z(3), z(2)), (z(3, 1), z(3, 1)), (z(3).long(), z(3))):
        with pytest.raises(ValueError):
            cache.assign(pages, k, n, 6, stream=0)
    assert cache._lib.calls == []
    cache.assign(pages, keep, keep, 6, stream=0)
    cache.assign(pages, keep, keep, 6, out=PagePlan(z(3), z(4)), stream=0)
    cache.assign(pages, keep[:1], keep[:1], out=cache.new_plan(1, 0), stream=0)
    assert cache._lib.calls == ["sgd_kv_assign"] * 3
