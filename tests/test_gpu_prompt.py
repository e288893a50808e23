"""Attention over whole prompts and over chunks, against its definition in 64 bits.

Bound per element, u the largest relative error of a rounding to the tensors' type
(2^-8 for bfloat16, 2^-11 for float16): u of the result for its own rounding, u of
sum_j p_j |v_j| for that of the probabilities to the type of the values, and 2^-12 of
that sum for what 32 bits lose: scores below 2^6 in units of log 2 with sums of up to
128 products (2^-24 each, relative to the largest partial sum: 2^-24 2^6 2^3), the
exponential (2^-22), and sums over up to 2^11 keys (2^-24 times the additions).  Where
float16 results are subnormal a rounding is 2^-25.
"""
import itertools
import math

import numpy as np
import pytest
import torch

import cache_reference as R

pytestmark = pytest.mark.gpu

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module")
def KV():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from model_free_suffix_gb300 import build
    build.build()
    from model_free_suffix_gb300 import KVCache
    return KVCache


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def _starts(counts):
    return _i32([0] + list(itertools.accumulate(counts)))


def _handle(KV, H, G, D, B, **over):
    return KV(**dict(dict(num_pages=1, page_size=64, kv_heads=H, head_dim=D, q_heads=H * G, max_batch=max(B, 1),
                          max_pages_per_row=1), **over))


def _qkv(N, H, G, D, dtype, seed=0, size=1.5):
    """Side by side in one row per token, as a projection leaves them."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(N, H * (G + 2), D, generator=g)
    x[:, :H * G] *= size
    x = x.to(DTYPES[dtype]).cuda()
    return x[:, :H * G], x[:, H * G:H * (G + 1)], x[:, H * (G + 1):]


def _check(got, want, mass, where):
    u = UNIT[got.dtype]
    off = (got.cpu().double() - want).abs()
    bound = u * want.abs() + (u + 2.0 ** -12) * mass + 2.0 ** -25
    assert bool((off <= bound).all()), (where, float((off / bound).nan_to_num(nan=math.inf).max()))


def _check_rows(out, q, k, v, counts, H, G, D, scale, window, sinks, old=None):
    """Rows of packed tokens; old: (keys, values) in 64 bits of each row's earlier positions."""
    at = 0
    q, k, v = (x.cpu().double() for x in (q, k, v))
    for b, c in enumerate(counts):
        if c:
            kb, vb, first = k[at:at + c], v[at:at + c], 0
            if old is not None:
                kb, vb, first = torch.cat([old[b][0], kb]), torch.cat([old[b][1], vb]), old[b][0].shape[0]
            want, mass = R.attend(q[at:at + c].view(c, H, G, D), kb, vb, first, scale, window, sinks)
            _check(out[at:at + c], want.reshape(c, H * G, D), mass.reshape(c, H * G, D), (b, c, first))
        at += c


# ---- whole prompts -----------------------------------------------------------------------------------

def _prompt(KV, counts, H, G, D, dtype, window=0, sinks=0, seed=0, scale=None):
    N = sum(counts)
    kv = _handle(KV, H, G, D, len(counts))
    q, k, v = _qkv(N, H, G, D, dtype, seed)
    out = kv.attend_prompt(q, k, v, _starts(counts), scale=scale, window=window, sinks=sinks)
    _check_rows(out, q, k, v, counts, H, G, D, scale if scale is not None else D ** -0.5, window, sinks)
    assert kv.get_error() == 0
    kv.close()


@pytest.mark.parametrize("counts", [[1], [2], [31], [64], [127], [128], [129], [200], [255], [256], [257], [700],
                                    [1, 1, 1], [0, 5, 0, 0, 130, 1, 0], [300, 17, 128, 64, 1, 511]])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 64)])
def test_lengths(KV, counts, dtype, D):
    _prompt(KV, counts, 2, 4, D, dtype)


@pytest.mark.parametrize("H,G", [(1, 1), (3, 1), (2, 2), (1, 3), (5, 3), (2, 5), (1, 6), (2, 7), (1, 8), (1, 16), (1, 64)])
@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("f16", 128)])
def test_heads(KV, H, G, dtype, D):
    _prompt(KV, [150, 1, 87, 300], H, G, D, dtype, seed=G)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 0), (64, 3), (128, 0), (130, 4), (300, 70), (100, 200),
                                          (2000, 5), (7, 1000), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("dtype,D,G", [("bf16", 128, 4), ("f16", 64, 1), ("bf16", 64, 3)])
def test_windows(KV, window, sinks, dtype, D, G):
    _prompt(KV, [700, 3, 129, 385], 1, G, D, dtype, window, sinks)


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3, 2.0 ** -10])
def test_scales(KV, scale):
    _prompt(KV, [140, 40], 2, 2, 64, "bf16", scale=scale)


@pytest.mark.parametrize("power", [-100, -60, 60, 100])
def test_values_of_any_size(KV, power):
    """bfloat16 has the range of 32 bits: values of 2^power give results of that size."""
    counts, H, G, D = [300, 70], 1, 2, 64
    q, k, v = _qkv(sum(counts), H, G, D, "bf16")
    kv = _handle(KV, H, G, D, len(counts))
    plain = kv.attend_prompt(q, k, v, _starts(counts))
    out = kv.attend_prompt(q, k, v * 2.0 ** power, _starts(counts))
    assert torch.equal(out.double(), plain.double() * 2.0 ** power)
    kv.close()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_scores_that_grow_along_a_row(KV, dtype):
    """Maxima far above those of the tiles before, in one half of a tile or the other, again and again."""
    counts, H, G, D = [900, 260], 1, 2, 64
    q, k, v = _qkv(sum(counts), H, G, D, dtype, size=1.0)
    step = torch.arange(sum(counts), device="cuda") // 50
    k = (k.float() * 0.25 + step[:, None, None] * 0.5).to(k.dtype)
    q = (q.float() * 0.25 + 0.5).to(q.dtype)
    kv = _handle(KV, H, G, D, len(counts))
    for window in (0, 333):
        out = kv.attend_prompt(q, k, v, _starts(counts), window=window)
        _check_rows(out, q, k, v, counts, H, G, D, D ** -0.5, window, 0)
    assert kv.get_error() == 0
    kv.close()


def test_long_rows(KV):
    """Several hundred tiles in one launch, cut in shares."""
    _prompt(KV, [3000, 2, 1501], 1, 2, 128, "bf16")
    _prompt(KV, [2500, 900], 2, 3, 64, "f16", window=700, sinks=9)


def test_layouts(KV):
    """Heads before tokens, starts off 16 bytes, heads that all groups share, odd strides."""
    counts, H, G, D = [150, 33, 1], 2, 2, 64
    N = sum(counts)
    q, k, v = (x.contiguous() for x in _qkv(N, H, G, D, "bf16"))
    kv = _handle(KV, H, G, D, len(counts))
    base = kv.attend_prompt(q, k, v, _starts(counts))
    _check_rows(base, q, k, v, counts, H, G, D, D ** -0.5, 0, 0)

    def heads_first(x):
        return x.transpose(0, 1).contiguous().transpose(0, 1)

    def shifted(x, by):
        flat = torch.empty(x.numel() + 8, dtype=x.dtype, device="cuda")
        flat[by:by + x.numel()] = x.reshape(-1)
        return flat[by:by + x.numel()].view(x.shape)

    def padded(x, to):
        y = torch.full((x.shape[0], x.shape[1], to), float("nan"), dtype=x.dtype, device="cuda")
        y[..., :D] = x
        return y[..., :D]

    for f in (heads_first, lambda x: shifted(x, 1), lambda x: shifted(x, 4), lambda x: padded(x, D + 1),
              lambda x: padded(x, D + 8)):
        for which in ((1, 1, 1), (1, 0, 0), (0, 1, 0), (0, 0, 1)):
            args = [f(x) if w else x for x, w in zip((q, k, v), which)]
            assert torch.equal(kv.attend_prompt(*args, _starts(counts)), base)
    one = k[:, :1]
    shared = kv.attend_prompt(q, one.expand(N, H, D), v, _starts(counts))
    assert torch.equal(shared, kv.attend_prompt(q, one.repeat(1, H, 1), v, _starts(counts)))
    assert kv.get_error() == 0
    kv.close()


def test_tokens_behind_the_last_row(KV):
    """They are not read (NaN here) and not written."""
    counts, H, G, D = [70, 130], 1, 2, 128
    q, k, v = _qkv(300, H, G, D, "bf16")
    for x in (q, k, v):
        x[200:] = float("nan")
    kv = _handle(KV, H, G, D, 2)
    out = torch.full((300, H * G, D), 7.0, dtype=torch.bfloat16, device="cuda")
    got = kv.attend_prompt(q, k, v, _starts(counts), out=out)
    assert got is out and bool((out[200:] == 7).all())
    _check_rows(out, q[:200], k[:200], v[:200], counts, H, G, D, D ** -0.5, 0, 0)
    assert kv.get_error() == 0
    kv.close()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("which", ["q", "k", "v"])
@pytest.mark.parametrize("dtype,D,G,window,sinks", [("bf16", 128, 4, 0, 0), ("f16", 64, 1, 40, 3), ("f16", 128, 3, 0, 0)])
def test_what_is_not_finite_stays_with_those_that_see_it(KV, bad, which, dtype, D, G, window, sinks):
    """One element in each of a few tokens: rows that do not see them are as without."""
    counts, H = [300, 140, 90], 2
    q, k, v = _qkv(sum(counts), H, G, D, dtype)
    kv = _handle(KV, H, G, D, len(counts))
    clean = kv.attend_prompt(q, k, v, _starts(counts), window=window, sinks=sinks)
    spots = [(1, 17), (129, 5), (260, 0), (299, 63), (300 + 130, 9), (440 + 2, 33)]
    x = dict(q=q, k=k, v=v)[which]
    for t, d in spots:
        x[t, 0, d] = bad
    out = kv.attend_prompt(q, k, v, _starts(counts), window=window, sinks=sinks)
    begin = [0, 300, 440, 530]
    touched = torch.zeros(out.shape, dtype=torch.bool)
    for t, d in spots:
        b = max(i for i in range(3) if begin[i] <= t)
        for i in range(begin[b], begin[b + 1]):
            p, j = i - begin[b], t - begin[b]
            if which == "q":
                if i == t:
                    touched[i, 0] = True
            elif j <= p and (window == 0 or j > p - window or j < sinks):
                if which == "k":
                    touched[i, :G] = True
                else:
                    touched[i, :G, d] = True
    assert torch.equal(out.cpu()[~touched], clean.cpu()[~touched])
    if which == "v":
        hit = out.cpu()[touched]
        assert bool((~hit.isfinite()).all())
        if not math.isnan(bad):  # (only infinities of one sign: never NaN)
            assert bool((hit == bad).all())
    elif math.isnan(bad):
        assert bool(out.cpu()[touched].isnan().all())
    elif which == "k" and (window == 0 or sinks > 1):
        # the first token's key: +inf or -inf times a query's element
        sign = (q[:300, :G, 17].float() * bad > 0).cpu()
        seen = touched[:300, :G, 0]
        assert bool(out.cpu()[:300, :G].isnan().all(-1)[sign & seen].all())
    kv.close()


@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 5)])
def test_values_that_are_not_finite_in_long_rows(KV, aligned, window, sinks):
    """In tiles that a unit's rows see in full, in part, or not at all; behind the row's last token; values
    whose start is off 16 bytes."""
    counts, H, G, D = [900, 3, 700], 1, 4, 64
    N = sum(counts)
    q, k, v = (x.contiguous() for x in _qkv(N, H, G, D, "bf16"))
    spots = [0, 3, 100, 127, 128, 400, 511, 640, 899, 900, 902, 903, 1500]
    kv = _handle(KV, H, G, D, len(counts))
    clean = kv.attend_prompt(q, k, v, _starts(counts), window=window, sinks=sinks).cpu()
    for i, t in enumerate(spots):
        v[t, 0, i] = math.nan if i % 2 else math.inf
    if not aligned:
        flat = torch.empty(v.numel() + 8, dtype=v.dtype, device="cuda")
        flat[1:1 + v.numel()] = v.reshape(-1)
        v = flat[1:1 + v.numel()].view(v.shape)
    out = kv.attend_prompt(q, k, v, _starts(counts), window=window, sinks=sinks).cpu()
    at = 0
    for c in counts:
        p, j = torch.arange(c)[:, None], torch.arange(c)[None]
        see = (j <= p) & ((j > p - window) | (j < sinks)) if window else j <= p
        hit = torch.zeros(c, D, dtype=torch.bool)
        for i, t in enumerate(spots):
            if at <= t < at + c:
                hit[:, i] |= see[:, t - at]
        got = out[at:at + c]
        assert bool((~got.isfinite()).eq(hit[:, None]).all())
        assert torch.equal(got[~hit[:, None].expand_as(got)], clean[at:at + c][~hit[:, None].expand_as(got)])
        at += c
    assert kv.get_error() == 0
    kv.close()


def test_bad_starts_are_reported(KV):
    from model_free_suffix_gb300 import _lib as L
    H, G, D = 1, 2, 64
    q, k, v = _qkv(200, H, G, D, "bf16")
    kv = _handle(KV, H, G, D, 3)
    # (what two rows claim, as tokens 60 to 80 of the first, is whichever's)
    for starts, fine in (([0, 80, 60, 200], [(0, 60)]), ([0, 80, 180, 250], [(0, 80), (80, 180)]),
                         ([-5, 80, 180, 200], [(80, 180), (180, 200)])):
        out = kv.attend_prompt(q, k, v, _i32(starts), out=torch.zeros(200, G, D, dtype=torch.bfloat16, device="cuda"))
        assert kv.get_error(clear=True) == L.KV_ERR_LENGTH, starts
        for lo, hi in fine:
            _check_rows(out[lo:hi], q[lo:hi], k[lo:hi], v[lo:hi], [hi - lo], H, G, D, D ** -0.5, 0, 0)
    # no tokens at all
    kv.attend_prompt(q, k, v, _i32([0, 0, 0, 0]))
    kv.attend_prompt(q[:0], k[:0], v[:0], _i32([0, 0, 0, 0]))
    kv.attend_prompt(q, k, v, _i32([0]))
    assert kv.get_error() == 0
    kv.close()


def test_many_rows(KV):
    counts = [1 + (7 * i) % 5 for i in range(1500)]
    _prompt(KV, counts, 1, 2, 64, "bf16")


@pytest.mark.parametrize("dtype,D,H,G,window", [("f16", 64, 3, 3, 0), ("bf16", 128, 2, 4, 150)])
def test_many_ragged_rows(KV, dtype, D, H, G, window):
    """Units of one and of two row tiles in turn, most of one or two tiles of keys: every role runs ahead of
    the others as far as it can."""
    counts = [1 + int(400 * ((i * 0.6180339887) % 1.0)) for i in range(110)]
    _prompt(KV, counts, H, G, D, dtype, window=window, sinks=2)


def test_graphs_streams_and_repetition(KV):
    """Captured calls replay with new lengths; another stream; the same bits each time."""
    H, G, D = 2, 4, 128
    q, k, v = _qkv(1200, H, G, D, "bf16")
    kv = _handle(KV, H, G, D, 3)
    starts = _starts([500, 400, 300])
    out = torch.zeros(1200, H * G, D, dtype=torch.bfloat16, device="cuda")
    first = kv.attend_prompt(q, k, v, starts).clone()
    for _ in range(3):
        assert torch.equal(kv.attend_prompt(q, k, v, starts), first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        kv.attend_prompt(q, k, v, starts, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    starts.copy_(_starts([100, 1000, 90]))
    graph.replay()
    with torch.cuda.stream(side):
        again = kv.attend_prompt(q, k, v, starts)
    other = kv.attend_prompt(q, k, v, starts, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out[:1190], again[:1190]) and torch.equal(other[:1190], again[:1190])
    assert torch.equal(out[1190:], first[1190:])
    _check_rows(out[:1190], q[:1190], k[:1190], v[:1190], [100, 1000, 90], H, G, D, D ** -0.5, 0, 0)
    assert kv.get_error() == 0
    kv.close()


def test_one_handle_on_several_streams_in_turn(KV):
    """Calls of one handle must not overlap: each stream waits for the one before it."""
    H, G, D = 2, 4, 128
    q, k, v = _qkv(1200, H, G, D, "bf16")
    kv = _handle(KV, H, G, D, 3)
    counts = [[500, 400, 300], [100, 1000, 90], [1200, 0, 0], [7, 600, 593]]
    want = [kv.attend_prompt(q, k, v, _starts(c)).clone() for c in counts]
    starts, out = _starts(counts[0]), torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.attend_prompt(q, k, v, starts, out=out)
    main, side = torch.cuda.current_stream(), torch.cuda.Stream()
    for _ in range(3):
        for c, w in zip(counts, want):
            n = sum(c)
            starts.copy_(_starts(c))
            graph.replay()
            side.wait_stream(main)
            with torch.cuda.stream(side):
                again = kv.attend_prompt(q, k, v, starts)
            other = torch.empty_like(q)
            side.wait_stream(main)
            kv.attend_prompt(q, k, v, starts, out=other, stream=side)
            main.wait_stream(side)
            assert all(torch.equal(x[:n], w[:n]) for x in (out, again, other))
    assert kv.get_error() == 0
    kv.close()


# ---- chunks over the cache ---------------------------------------------------------------------------

class Chunks:
    """A cache whose rows hold `olds` tokens, and its definition."""

    def __init__(self, KV, olds, counts, P=32, H=2, G=2, D=64, dtype="bf16", seed=0, spread=2.0, shift=0.0):
        rng = np.random.default_rng(seed)
        self.olds, self.counts, self.H, self.G, self.D, self.dtype = olds, counts, H, G, D, dtype
        need = [-(-(o + c) // P) for o, c in zip(olds, counts)]
        pages, width = sum(need) + 2, max(max(need), 1)
        order, at = rng.permutation(pages), 0
        self.table = np.full((len(olds), width), -1, np.int32)
        for b, m in enumerate(need):
            self.table[b, :m] = order[at:at + m]
            at += m
        self.dev_table = torch.from_numpy(self.table).cuda()
        self.kv = _handle(KV, H, G, D, len(olds), num_pages=pages, page_size=P, max_pages_per_row=width)
        # what no write has reached holds NaN bytes and NaN scales
        self.kv.k.view(torch.uint8).fill_(0x7f)
        self.kv.v.view(torch.uint8).fill_(0xff)
        self.kv.k_scale.fill_(float("nan"))
        self.kv.v_scale.fill_(float("nan"))
        self.ref = R.Cache(pages, H, P, D)
        N = sum(olds)
        if N:
            g = torch.Generator().manual_seed(seed + 1)
            size = torch.randn(N, 2, H, 1, generator=g) * torch.tensor([spread / 6, spread])[:, None, None]
            x = torch.randn(N, 2, H, D, generator=g) * torch.exp2(size + torch.tensor([0.0, shift])[:, None, None])
            x = x.to(torch.bfloat16)
            dev = x.cuda()
            self.kv.write(dev[:, 0], dev[:, 1], self.dev_table, _i32(olds), _starts(olds))
            self.ref.write({"k": x[:, 0], "v": x[:, 1]}, self.table, olds, olds)
        self.q, self.k, self.v = _qkv(sum(counts), H, G, D, dtype, seed + 2)
        self.lens = [o + c for o, c in zip(olds, counts)]

    def old(self):
        return [tuple(self.ref.rows(x, self.table[b], 0, o) for x in "kv") for b, o in enumerate(self.olds)]

    def run(self, window=0, sinks=0, **kw):
        return self.kv.attend_chunk(self.q, self.k, self.v, self.dev_table, _i32(self.lens), _starts(self.counts),
                                    window=window, sinks=sinks, **kw)

    def check(self, window=0, sinks=0):
        out = self.run(window, sinks)
        _check_rows(out, self.q, self.k, self.v, self.counts, self.H, self.G, self.D, self.D ** -0.5, window, sinks, self.old())
        assert self.kv.get_error() == 0
        return out


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype,D,H,G", [("bf16", 128, 2, 4), ("f16", 64, 1, 3), ("f16", 128, 1, 1), ("bf16", 64, 3, 2)])
def test_chunks(KV, P, dtype, D, H, G):
    Chunks(KV, [0, 1, 127, 128, 129, 300, 77, 513], [40, 129, 1, 130, 257, 3, 0, 200], P, H, G, D, dtype).check()


@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 2), (128, 0), (150, 4), (90, 200), (400, 1000)])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 64)])
def test_chunks_with_a_window(KV, window, sinks, dtype, D):
    Chunks(KV, [0, 5, 130, 700, 256], [300, 129, 1, 70, 257], 32, 1, 3, D, dtype).check(window, sinks)


@pytest.mark.parametrize("olds,counts", [([5000], [3]), ([4000], [300]), ([3000, 10], [1, 900])])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_long_caches(KV, olds, counts, dtype):
    """Few rows over many positions: the work is cut along them, and joined."""
    Chunks(KV, olds, counts, 64, 1, 2, 128, dtype).check()


@pytest.mark.parametrize("dtype,spread,shift", [("bf16", 6.0, 0.0), ("f16", 4.0, -7.0), ("f16", 2.0, 5.0)])
def test_scales_far_apart(KV, dtype, spread, shift):
    """Tokens' values from about 2^-20 to 2^20 times the usual size, and their blocks' scales with them."""
    c = Chunks(KV, [700, 300], [60, 200], 16, 2, 2, 64, dtype, spread=spread, shift=shift)
    out = c.run()
    at = 0
    for b, n in enumerate(c.counts):
        k, v = c.old()[b]
        want, mass = R.attend(c.q[at:at + n].cpu().double().view(n, c.H, c.G, c.D), torch.cat([k, c.k[at:at + n].cpu().double()]),
                              torch.cat([v, c.v[at:at + n].cpu().double()]), c.olds[b], c.D ** -0.5)
        if dtype == "f16":
            assert float(want.abs().max()) < 60000
        _check(out[at:at + n], want.reshape(n, -1, c.D), mass.reshape(n, -1, c.D), b)
        at += n


def test_a_chunk_without_a_past_is_a_prompt(KV):
    c = Chunks(KV, [0, 0, 0], [200, 1, 300], 32, 2, 4, 128, "bf16")
    assert torch.equal(c.run(), c.kv.attend_prompt(c.q, c.k, c.v, _starts(c.counts)))
    assert torch.equal(c.run(50, 3), c.kv.attend_prompt(c.q, c.k, c.v, _starts(c.counts), window=50, sinks=3))


def test_whether_the_chunk_is_written_makes_no_difference(KV):
    """(Pages of the past alone: one that the chunk shares may get another scale.)"""
    c = Chunks(KV, [96, 32], [50, 200])
    before = c.check()
    c.kv.write(c.k, c.v, c.dev_table, _i32(c.lens), _starts(c.counts))
    assert torch.equal(c.run(), before)


def test_pages_and_lengths_that_are_not_there(KV):
    from model_free_suffix_gb300 import _lib as L
    c = Chunks(KV, [200, 100, 64], [20, 150, 9], 32, 1, 2, 64)
    good = c.check()
    # a page that is not there: its positions are not seen, the other rows are as before
    for page in (-1, 10 ** 6, 2 ** 31 - 1, -2 ** 31):
        c.dev_table[0, 2] = page
        out = c.run()
        assert c.kv.get_error(clear=True) == L.KV_ERR_PAGE
        assert torch.equal(out[20:], good[20:])
        k, v = c.old()[0]
        keep = [j for j in range(200) if not 64 <= j < 96]
        _check_rows(out[:20], c.q[:20], c.k[:20], c.v[:20], [20], 1, 2, 64, 64 ** -0.5, 0, 0, [(k[keep], v[keep])])
    c.dev_table[0, 2] = int(c.table[0, 2])
    # entries of positions that are not in the cache yet are not looked at
    c.dev_table[1, 4:] = -1
    assert torch.equal(c.run(), good) and c.kv.get_error() == 0
    c.dev_table.copy_(torch.from_numpy(c.table))
    for n in (5, -3, 10 ** 6, 2 ** 31 - 1, -2 ** 31):
        lens = list(c.lens)
        lens[1] = n
        out = c.kv.attend_chunk(c.q, c.k, c.v, c.dev_table, torch.tensor(lens).int().cuda(), _starts(c.counts))
        assert c.kv.get_error(clear=True) == L.KV_ERR_LENGTH
        assert bool((out[20:170] == 0).all()) and torch.equal(out[:20], good[:20]) and torch.equal(out[170:], good[170:])


def test_captured_chunks_of_two_graphs_share_a_handle(KV):
    """Two captured calls of different sizes, replayed in turn."""
    c = Chunks(KV, [3000, 500], [40, 300], 64, 2, 2, 128)
    want = c.check()
    small = c.kv.attend_chunk(c.q[:40], c.k[:40], c.v[:40], c.dev_table, _i32([3040, 0]), _i32([0, 40, 40]))
    lens, starts, lens2, starts2 = _i32(c.lens), _starts(c.counts), _i32([3040, 0]), _i32([0, 40, 40])
    out, out2 = torch.zeros_like(want), torch.zeros_like(small)
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0]):
        c.kv.attend_chunk(c.q, c.k, c.v, c.dev_table, lens, starts, out=out)
    with torch.cuda.graph(graphs[1]):
        c.kv.attend_chunk(c.q[:40], c.k[:40], c.v[:40], c.dev_table, lens2, starts2, out=out2)
    for _ in range(4):
        for g, o, w in ((graphs[0], out, want), (graphs[1], out2, small)):
            o.zero_()
            g.replay()
            assert torch.equal(o, w)


def test_places_beyond_32_bits(KV):
    """Queries and results of more than 2^31 elements, and pages behind the first 4 GiB of a cache."""
    N, H, G, D, c = (1 << 18) + 300, 1, 64, 128, 300
    kv = _handle(KV, H, G, D, 1)
    q = torch.empty(N, H * G, D, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.empty(N, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x = _qkv(c, H, G, D, "bf16")
    for big, small in zip((q, k, v), x):
        big[N - c:] = small
    out = kv.attend_prompt(q, k, v, _i32([N - c, N]))
    want = kv.attend_prompt(*x, _starts([c]))
    assert torch.equal(out[N - c:], want)
    _check_rows(want[:40], *(y[:40] for y in x), [40], H, G, D, D ** -0.5, 0, 0)
    assert kv.get_error() == 0
    kv.close()
    del q, k, v, out
    pages = (1 << 32) // (8 * 128 * 128) + 40
    big = _handle(KV, 8, 1, 128, 1, num_pages=pages, page_size=128, max_pages_per_row=3)
    small = _handle(KV, 8, 1, 128, 1, num_pages=3, page_size=128, max_pages_per_row=3)
    q, k, v = _qkv(200, 8, 1, 128, "bf16", seed=3)
    tables = torch.tensor([[pages - 1, 5, pages - 17]]).int().cuda(), _i32([[0, 1, 2]])
    outs = []
    for kv, table in zip((big, small), tables):
        kv.write(k, v, table, _i32([200]), _i32([0, 200]))
        outs.append(kv.attend_chunk(q, k, v, table, _i32([384]), _i32([0, 184])))
        assert kv.get_error() == 0
        kv.close()
    assert torch.equal(outs[0][:184], outs[1][:184])


def test_two_handles_on_two_streams(KV):
    """Calls of different handles at the same time."""
    c = Chunks(KV, [700, 50, 3000], [300, 200, 100], 64, 2, 4, 128, "bf16")
    want_c = c.check(200, 4)
    H, G, D, counts = 3, 2, 64, [700, 33, 512]
    q, k, v = _qkv(sum(counts), H, G, D, "f16")
    kv, starts = _handle(KV, H, G, D, 3), _starts(counts)
    want_p = kv.attend_prompt(q, k, v, starts)
    lens, cstarts = _i32(c.lens), _starts(c.counts)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        got[0].append(c.kv.attend_chunk(c.q, c.k, c.v, c.dev_table, lens, cstarts, window=200, sinks=4,
                                        out=torch.empty_like(want_c), stream=streams[0]))
        got[1].append(kv.attend_prompt(q, k, v, starts, out=torch.empty_like(want_p), stream=streams[1]))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want_c) for x in got[0]) and all(torch.equal(x, want_p) for x in got[1])
    assert c.kv.get_error() == 0 and kv.get_error() == 0


# ---- a server's steps --------------------------------------------------------------------------------

@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 3)])
def test_prompts_in_chunks_through_pages_of_their_own(KV, window, sinks):
    """assign, write and attend_chunk together, then attend for single tokens: rows that come, grow by chunks,
    decode, reject and go, each step's result against the definition over what the cache holds."""
    H, G, D, P, B = 2, 2, 64, 16, 4
    kv = KV(num_pages=60, page_size=P, kv_heads=H, head_dim=D, q_heads=H * G, max_batch=B, max_pages_per_row=24)
    pages, plan = kv.new_pages(), kv.new_plan(B, 400)
    ref = R.Cache(60, H, P, D)
    have = [0] * B
    steps = [([0, 0, 0, 0], [100, 37, 0, 1]), ([100, 37, 0, 1], [129, 1, 64, 5]), ([229, 35, 64, 6], [1, 3, 65, 128]),
             ([0, 36, 129, 134], [0, 1, 1, 1]), ([0, 37, 130, 130], [150, 2, 1, 7])]
    for i, (keep, new) in enumerate(steps):
        kv.assign(pages, _i32(keep), _i32(new), out=plan)
        lens = [a + c for a, c in zip(keep, new)]
        assert plan.seq_lens.tolist() == lens and plan.q_start.tolist() == [0] + list(itertools.accumulate(new))
        N = sum(new)
        q, k, v = _qkv(400, H, G, D, "bf16", seed=i)     # (room for more tokens than the step has)
        out = kv.attend_chunk(q, k, v, pages.block_table, plan.seq_lens, plan.q_start, window=window, sinks=sinks)
        table = pages.block_table.cpu().numpy()
        old = [tuple(ref.rows(x, table[b], 0, a) for x in "kv") for b, a in enumerate(keep)]
        _check_rows(out[:N], q[:N], k[:N], v[:N], new, H, G, D, D ** -0.5, window, sinks, old)
        kv.write(k, v, pages.block_table, plan.seq_lens, plan.q_start)
        ref.write({"k": k.cpu(), "v": v.cpu()}, table, lens, new)
        # the slots are where write put the tokens
        slots = plan.slots[:N].long()
        bytes_ = kv.k[0].view(torch.uint8).transpose(1, 2).reshape(-1, H, D)[slots]
        scales = kv.k_scale[0][slots // P]
        got = (bytes_.view(torch.float8_e4m3fn).double() * scales.double()[..., None]).cpu()
        want = torch.cat([ref.rows("k", table[b], keep[b], lens[b]) for b in range(B)])
        assert torch.equal(got, want)
        assert bool((plan.slots[N:] == -1).all())
        have = lens
    assert kv.get_error() == 0
    kv.close()
