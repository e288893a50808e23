"""The paged 8-bit cache and the attention over it, against their definitions in 64 bits.

Writes and reads are exact: the reference rounds to the same e4m3 values, so
values and scales must be equal.  The attention's bound per element: the
result's rounding (half a unit in its last place: 2^-9 of it for bfloat16,
2^-12 for float16, with room for one unit), and 2^-10 of sum_j p_j |v_j| for
the probabilities, which the kernel may round to 11 bits (2^-12 each), and for
the exponential, the running sums and the division (each below 2^-13 of it at
these lengths and logits).
"""
import itertools

import numpy as np
import pytest
import torch

import cache_reference as R

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def KV():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from model_free_suffix_gb300 import build
    build.build()
    from model_free_suffix_gb300 import KVCache
    return KVCache


def _starts(counts):
    return torch.tensor([0] + list(itertools.accumulate(counts)), dtype=torch.int32).cuda()


class Pair:
    """A cache on the GPU and its definition, written alike."""

    def __init__(self, KV, lens, P=32, H=2, D=64, G=1, seed=0, extra=2, width=None):
        self.rng = np.random.default_rng(seed)
        self.g = torch.Generator().manual_seed(seed)
        self.P, self.H, self.D, self.G, self.B = P, H, D, G, len(lens)
        need = [-(-max(n, 1) // P) for n in lens]
        width = width or max(need)
        pages = sum(need) + extra
        order = self.rng.permutation(pages)
        self.table = np.full((self.B, width), -1, np.int32)
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = order[at:at + m]
            at += m
        self.dev_table = torch.from_numpy(self.table).cuda()
        self.kv = KV(num_pages=pages, page_size=P, kv_heads=H, head_dim=D, q_heads=H * G,
                     max_batch=self.B, max_pages_per_row=width)
        # what no write has reached holds NaN bytes and NaN scales
        self.kv.k.view(torch.uint8).fill_(0x7f)
        self.kv.v.view(torch.uint8).fill_(0xff)
        self.kv.k_scale.fill_(float("nan"))
        self.kv.v_scale.fill_(float("nan"))
        self.ref = R.Cache(pages, H, P, D)

    def write(self, lens, counts, dtype="bf16", spread=2.0, tensors=None):
        N = sum(counts)
        if tensors is None:
            x = torch.randn(N, 2, self.H, self.D, generator=self.g) * \
                torch.exp2(torch.randn(N, 1, self.H, 1, generator=self.g) * spread)
            x = x.to(DTYPES[dtype])
            tensors = x[:, 0], x[:, 1]           # (as a packed projection's output: apart in memory)
        k, v = tensors
        dev = torch.stack([k, v], 1).cuda()
        self.kv.write(dev[:, 0], dev[:, 1], self.dev_table, torch.tensor(lens, dtype=torch.int32).cuda(),
                      _starts(counts))
        self.ref.write({"k": k, "v": v}, self.table, lens, counts)

    def check(self, lens, dtype="f32"):
        counts = list(lens)
        k, v = self.kv.read(self.dev_table, torch.zeros(self.B, dtype=torch.int32).cuda(), _starts(counts),
                            total=sum(counts), dtype=DTYPES[dtype])
        for name, got in (("k", k), ("v", v)):
            want = torch.cat([self.ref.rows(name, self.table[b], 0, n) for b, n in enumerate(lens)]) \
                if sum(lens) else torch.zeros(0, self.H, self.D)
            assert torch.equal(got.cpu().double(), want.to(DTYPES[dtype]).double()), name
        used = [int(self.table[b, j]) for b, n in enumerate(lens) for j in range(-(-n // self.P))]
        for name, got in (("k", self.kv.k_scale), ("v", self.kv.v_scale)):
            assert torch.equal(got[0].cpu().double()[used], self.ref.s[name][used]), name

    def check_attend(self, lens, counts, dtype="bf16", window=0, sinks=0, scale=None, q=None, max_q=None):
        N, Hq = sum(counts), self.H * self.G
        if q is None:
            q = (torch.randn(N, Hq, self.D, generator=self.g) * 1.5).to(DTYPES[dtype])
        scale = scale if scale is not None else self.D ** -0.5
        out = self.kv.attend(q.cuda(), self.dev_table, torch.tensor(lens, dtype=torch.int32).cuda(),
                             _starts(counts), max_q or max(counts), scale=scale, window=window, sinks=sinks)
        got, at = out.cpu().double(), 0
        unit = 2.0 ** -8 if q.dtype == torch.bfloat16 else 2.0 ** -11
        for b, (n, c) in enumerate(zip(lens, counts)):
            if c:
                k, v = (self.ref.rows(x, self.table[b], 0, n) for x in "kv")
                want, mass = R.attend(q[at:at + c].view(c, self.H, self.G, self.D), k, v, n - c, scale, window, sinks)
                want, mass = want.reshape(c, Hq, self.D), mass.reshape(c, Hq, self.D)
                off = (got[at:at + c] - want).abs()
                bound = unit * want.abs() + 2.0 ** -10 * mass + 1e-7
                assert bool((off <= bound).all()), (b, n, c, float((off / bound).max()))
            at += c
        return out


# ---- write and read ----------------------------------------------------------------------------------

@pytest.mark.parametrize("P,H,D", [(16, 1, 64), (32, 3, 64), (64, 2, 128), (128, 1, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_write_in_steps_and_read_back(KV, P, H, D, dtype):
    """A prompt, then steps of 0..7 tokens: blocks filled over several writes,
    rows without new tokens, blocks that end inside a step."""
    rng = np.random.default_rng(P + D)
    lens = [1, P - 1, P, P + 1, 2 * P + 5, 3 * P]
    p = Pair(KV, [n + 40 for n in lens], P=P, H=H, D=D)
    p.write(lens, lens, dtype)
    p.check(lens)
    for _ in range(5):
        counts = [int(c) for c in rng.integers(0, 8, len(lens))]
        if not any(counts):
            counts[0] = 1
        lens = [n + c for n, c in zip(lens, counts)]
        p.write(lens, counts, dtype)
        p.check(lens)
    assert p.kv.get_error() == 0
    p.kv.close()


def test_rejected_drafts_leave_nothing_behind(KV):
    """Positions are written again with other values: scales follow the entries that count."""
    p = Pair(KV, [100, 70], P=32, H=2, D=64)
    p.write([50, 33], [50, 33])
    big = tuple(torch.full((10, 2, 64), 3e4, dtype=torch.bfloat16) for _ in range(2))
    p.write([55, 38], [5, 5], tensors=big)      # drafts of outlying size ...
    p.check([55, 38])
    p.write([52, 40], [2, 7])                   # ... none of which was accepted
    p.check([52, 40])
    p.kv.close()


@pytest.mark.parametrize("size", [1e-30, 1e-10, 1.0, 1e10, 1e30])
def test_scales_over_the_range(KV, size):
    p = Pair(KV, [40], P=16, H=1, D=64)
    x = torch.randn(40, 1, 64, generator=p.g, dtype=torch.float64)
    x[3] = 0.0
    x = (x * size).float()
    p.write([40], [40], tensors=(x, -x))
    p.check([40])
    p.kv.close()


def test_ties_limits_and_zeros(KV):
    """Halfway values, the largest, subnormals, an all-zero block."""
    vals = R.VALUES[:127].float()
    mid = (vals[1:] + vals[:-1]) / 2
    x = torch.cat([vals, mid, -mid, torch.tensor([448.0, 447.9, 464.0])])
    x = torch.cat([x, torch.zeros(-len(x) % 64)]).view(-1, 1, 64)
    p = Pair(KV, [16 + len(x)], P=16, H=1, D=64)
    x = torch.cat([torch.zeros(16, 1, 64), x])
    p.write([len(x)], [len(x)], tensors=(x, x))
    p.check([len(x)])
    assert p.kv.get_error() == 0
    p.kv.close()


def test_infinities_and_nan_are_reported_and_bounded(KV):
    from model_free_suffix_gb300 import _lib as L
    p = Pair(KV, [20], P=16, H=2, D=64)
    x = torch.randn(20, 2, 64, generator=p.g)
    x[1, 0, 5], x[2, 0, 6], x[17, 1, 7] = float("inf"), float("-inf"), float("nan")
    p.write([20], [20], tensors=(x, x.abs()))
    p.check([20])
    assert p.kv.get_error(clear=True) == L.KV_ERR_NONFINITE
    assert p.kv.get_error() == 0
    p.kv.close()


def test_strides_and_alignment(KV):
    """Tokens and heads apart in memory, and addresses that no vector load may use."""
    p = Pair(KV, [45], P=32, H=2, D=64)
    base = torch.randn(45 * 2 * 3 * 67 + 5, generator=p.g).to(torch.bfloat16)
    k = base[1:].as_strided((45, 2, 64), (6 * 67, 67, 1))
    v = base[3:].as_strided((45, 2, 64), (67, 45 * 67, 1))
    dev = base.cuda()
    lens = torch.tensor([45], dtype=torch.int32).cuda()
    p.kv.write(dev[1:].as_strided(k.shape, k.stride()), dev[3:].as_strided(v.shape, v.stride()), p.dev_table,
               lens, _starts([45]))
    p.ref.write({"k": k, "v": v}, p.table, [45], [45])
    p.check([45], "bf16")
    p.check([45], "f16")
    p.kv.close()


def test_bad_pages_and_lengths_are_skipped(KV):
    from model_free_suffix_gb300 import _lib as L
    p = Pair(KV, [40, 40, 40], P=16, H=1, D=64)
    before = p.kv.k.view(torch.uint8).clone()
    table = p.dev_table.clone()
    table[0, 0], table[1, 0] = -1, 10 ** 6
    x = torch.ones(9, 1, 64, dtype=torch.bfloat16).cuda()
    lens = torch.tensor([3, 3, 2], dtype=torch.int32).cuda()   # (the last row has 3 new tokens of 2)
    p.kv.write(x, x, table, lens, _starts([3, 3, 3]))
    assert p.kv.get_error(clear=True) == L.KV_ERR_PAGE | L.KV_ERR_LENGTH
    assert torch.equal(p.kv.k.view(torch.uint8), before)
    lens = torch.tensor([3, 16 * p.table.shape[1] + 1, 3], dtype=torch.int32).cuda()  # past the table
    p.kv.write(x[:1], x[:1], p.dev_table, lens, _starts([0, 1, 0]))
    assert p.kv.get_error(clear=True) & L.KV_ERR_PAGE
    assert torch.equal(p.kv.k.view(torch.uint8), before)
    k, _ = p.kv.read(table, torch.zeros(3, dtype=torch.int32).cuda(), _starts([3, 3, 0]), total=8)
    assert p.kv.get_error(clear=True) == L.KV_ERR_PAGE | L.KV_ERR_LENGTH
    assert not k.any()
    p.kv.close()


# ---- attention -----------------------------------------------------------------------------------------

LENS = [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 129, 300]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("P,H,D,G", [(16, 1, 64, 1), (16, 2, 128, 3), (32, 2, 64, 8), (64, 2, 128, 4),
                                     (128, 1, 128, 16), (32, 1, 64, 7)])
def test_attend_single_tokens(KV, P, H, D, G, dtype):
    p = Pair(KV, LENS, P=P, H=H, D=D, G=G)
    p.write(LENS, LENS, spread=1.0)
    p.check_attend(LENS, [1] * len(LENS), dtype)
    assert p.kv.get_error() == 0
    p.kv.close()


@pytest.mark.parametrize("P,H,D,G", [(16, 1, 64, 1), (64, 2, 128, 4), (32, 2, 64, 5), (128, 1, 128, 8)])
@pytest.mark.parametrize("most", [2, 5, 17, 33, 70])
def test_attend_drafted_tokens(KV, P, H, D, G, most):
    """0..most new tokens per row, among them whole short rows (a context that
    begins with this call); the cache beyond a row's length holds NaN."""
    rng = np.random.default_rng(most)
    lens = LENS + [500]
    counts = [int(min(n, c)) for n, c in zip(lens, rng.integers(0, most + 1, len(lens)))]
    counts[3], counts[-1] = min(lens[3], most), most
    p = Pair(KV, lens, P=P, H=H, D=D, G=G, seed=most)
    p.write(lens, lens, spread=1.0)
    p.check_attend(lens, counts)
    p.check_attend(lens, counts, "f16", max_q=most + 3)
    p.kv.close()


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 0), (16, 4), (33, 40), (64, 64), (100, 3), (1000, 5)])
@pytest.mark.parametrize("P,D", [(16, 64), (64, 128)])
def test_attend_window_and_sinks(KV, P, D, window, sinks):
    lens = LENS + [700]
    counts = [min(n, c) for n, c in zip(lens, itertools.cycle([1, 3, 9, 20]))]
    p = Pair(KV, lens, P=P, H=2, D=D, G=4, seed=window)
    p.write(lens, lens, spread=1.0)
    p.check_attend(lens, counts, window=window, sinks=sinks)
    p.kv.close()


MANY = [1, 2, 17, 63, 64, 65, 127, 128, 129, 191, 193, 300, 511, 640, 1000, 1500]


@pytest.mark.parametrize("P,H,D,G", [(64, 4, 128, 4), (128, 3, 64, 6), (64, 3, 64, 16), (128, 4, 128, 1)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 3), (64, 70), (1, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_attend_many_rows(KV, P, H, D, G, window, sinks, dtype):
    """Batches whose rows open 0..33 positions: units of up to 128 rows, several
    units a row, rows of every length around the tiles, cuts within a unit."""
    rng = np.random.default_rng(P + G + window)
    counts = [int(min(n, c)) for n, c in zip(MANY, rng.integers(0, 34, len(MANY)))]
    counts[-1], counts[4], counts[7] = 33, 20, 33
    p = Pair(KV, MANY, P=P, H=H, D=D, G=G, seed=P + window)
    p.write(MANY, MANY, spread=1.0)
    out = p.check_attend(MANY, counts, dtype, window=window, sinks=sinks)
    assert p.kv.get_error() == 0 and bool(out.isfinite().all())
    p.kv.close()


def test_attend_many_rows_of_unequal_blocks(KV):
    """Blocks of very unequal key and value scales, queries of unequal size, a
    negative scale and a scale of zero, a query that is not finite."""
    lens = [130 + 37 * i for i in range(20)]
    counts = [1 + i % 9 for i in range(20)]
    p = Pair(KV, lens, P=64, H=2, D=128, G=4, seed=5)
    N = sum(lens)
    g = p.g
    size = torch.exp2(torch.randint(-12, 13, (N // 16 + 1, 1, 1), generator=g).float()).repeat_interleave(16, 0)[:N]
    p.write(lens, lens, tensors=(torch.randn(N, 2, 128, generator=g), torch.randn(N, 2, 128, generator=g) * size))
    q = torch.randn(sum(counts), 8, 128, generator=g) * torch.exp2(torch.randn(sum(counts), 8, 1, generator=g) * 2)
    q = q.to(torch.bfloat16)
    p.check_attend(lens, counts, q=q)
    p.check_attend(lens, counts, q=q, scale=-0.2)
    p.check_attend(lens, counts, q=q, scale=0.0)
    p.check_attend(lens, counts, q=(q.float() * 1e-30).to(torch.bfloat16))
    clean = p.check_attend(lens, counts, q=q)
    bad = q.clone()
    bad[7, 3, 100] = float("inf")
    bad[20, 0, 0] = float("nan")
    out = p.kv.attend(bad.cuda(), p.dev_table, torch.tensor(lens, dtype=torch.int32).cuda(), _starts(counts), 9)
    assert bool(out[7, 3].isnan().all()) and bool(out[20, 0].isnan().all())
    out[7, 3], out[20, 0] = clean[7, 3], clean[20, 0]
    assert torch.equal(out, clean)
    p.kv.close()


def test_attend_many_rows_bad_pages_and_lengths(KV):
    from model_free_suffix_gb300 import _lib as L
    lens, counts = [200 + 10 * i for i in range(20)], [9] * 20
    p = Pair(KV, lens, P=64, H=2, D=64, G=4, seed=6)
    p.write(lens, lens, spread=1.0)
    q = torch.randn(180, 8, 64, generator=p.g).to(torch.bfloat16)
    clean = p.check_attend(lens, counts, q=q)
    table, n = p.dev_table.clone(), torch.tensor(lens, dtype=torch.int32).cuda()
    table[3] = 10 ** 6
    n[5], n[6] = 8, 64 * table.shape[1] + 1
    out = p.kv.attend(q.cuda(), table, n, _starts(counts), 9)
    assert p.kv.get_error(clear=True) == L.KV_ERR_LENGTH | L.KV_ERR_PAGE
    # (units of other rows may be cut elsewhere: two results within the bound of the same value)
    for b in range(20):
        now, before = out[9 * b:9 * b + 9].double(), clean[9 * b:9 * b + 9].double()
        if b in (3, 5, 6):
            assert not now.any()
        else:
            v = p.ref.rows("v", p.table[b], 0, lens[b]).abs().amax(0).cuda().repeat_interleave(4, 0)
            assert bool(((now - before).abs() <= 2.0 ** -7 * before.abs() + 2.0 ** -9 * v + 2e-7).all())
    p.kv.close()


@pytest.mark.parametrize("n,c", [(5000, 1), (5000, 9), (20000, 1), (3001, 3001)])
def test_attend_long_rows(KV, n, c):
    """One long row (split over many CTAs and joined), and a whole prompt at once."""
    G = 4 if c < 100 else 1
    p = Pair(KV, [n, 17], P=64, H=1, D=64, G=G)
    p.write([n, 17], [n, 17], spread=0.5)
    p.check_attend([n, 17], [c, 1])
    p.check_attend([n, 17], [c, 17], window=777, sinks=2)
    p.kv.close()


def test_attend_large_logits_and_scales(KV):
    """Logits of thousands (the largest takes all), keys and values of very
    unequal size from block to block, queries from tiny to huge."""
    n = 200
    p = Pair(KV, [n], P=16, H=1, D=64, G=4)
    g = p.g
    k = torch.randn(n, 1, 64, generator=g)
    v = torch.randn(n, 1, 64, generator=g) * torch.exp2(torch.arange(n) // 16 * 3.0 - 18)[:, None, None]
    p.write([n], [n], tensors=(k, v))
    q = torch.randn(3, 4, 64, generator=g)
    p.check_attend([n], [3], q=(q * 300).to(torch.bfloat16))
    p.check_attend([n], [3], q=(q * 1e-3).to(torch.float16))
    p.check_attend([n], [3], q=(q * 1e-30).to(torch.bfloat16))
    q[0] = 0.0
    p.check_attend([n], [3], q=q.to(torch.bfloat16), scale=-0.3)
    p.check_attend([n], [3], q=q.to(torch.bfloat16), scale=0.0)
    p.kv.close()


def test_attend_keeps_a_bad_query_to_its_row(KV):
    p = Pair(KV, [90, 50], P=32, H=1, D=64, G=2)
    p.write([90, 50], [90, 50], spread=1.0)
    q = torch.randn(8, 2, 64, generator=p.g).to(torch.bfloat16)
    clean = p.check_attend([90, 50], [5, 3], q=q)
    for bad in (float("nan"), float("inf")):
        dirty = q.clone()
        dirty[2, 1, 7] = bad
        out = p.kv.attend(dirty.cuda(), p.dev_table, torch.tensor([90, 50], dtype=torch.int32).cuda(),
                          _starts([5, 3]), 5)
        assert bool(out[2, 1].isnan().all())
        out[2, 1] = clean[2, 1]
        assert torch.equal(out, clean)
    p.kv.close()


def test_attend_bad_rows(KV):
    """Fewer cached than new tokens, a length past the table, pages outside the
    cache: reported; the row sees what is left, here nothing, and others are untouched."""
    from model_free_suffix_gb300 import _lib as L
    p = Pair(KV, [40, 40, 40], P=16, H=1, D=64, G=2)
    p.write([40, 40, 40], [40, 40, 40], spread=1.0)
    q = torch.randn(7, 2, 64, generator=p.g).to(torch.bfloat16)
    clean = p.check_attend([40, 40, 40], [3, 3, 1], q=q)
    for lens, table in (([2, 40, 40], p.dev_table), ([16 * p.table.shape[1] + 1, 40, 40], p.dev_table),
                        ([40, 40, 40], torch.where(torch.arange(3)[:, None].cuda() == 0, 10 ** 6, p.dev_table).int())):
        out = p.kv.attend(q.cuda(), table, torch.tensor(lens, dtype=torch.int32).cuda(), _starts([3, 3, 1]), 3)
        assert p.kv.get_error(clear=True) in (L.KV_ERR_LENGTH, L.KV_ERR_PAGE)
        assert not out[:3].any()
        assert torch.equal(out[3:], clean[3:])
    p.kv.close()


def test_attend_is_the_same_every_time_and_on_any_stream(KV):
    lens, counts = [4000, 900, 37], [5, 17, 1]
    p = Pair(KV, lens, P=64, H=2, D=128, G=4)
    p.write(lens, lens, spread=1.0)
    q = torch.randn(sum(counts), 8, 128, generator=p.g).to(torch.bfloat16).cuda()
    args = (p.dev_table, torch.tensor(lens, dtype=torch.int32).cuda(), _starts(counts), 17)
    first = p.kv.attend(q, *args).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (None, side, None):
        if s is not None:
            side.wait_stream(torch.cuda.current_stream())
        out = p.kv.attend(q, *args, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    p.kv.close()


def test_write_and_attend_in_a_graph(KV):
    """Captured once, replayed with other lengths and inputs in the same buffers."""
    lens = [300, 120, 65]
    p = Pair(KV, [n + 60 for n in lens], P=32, H=2, D=64, G=4)
    p.write(lens, lens, spread=1.0)
    counts = [3, 1, 5]
    N = sum(counts)
    x = torch.zeros(N, 2, 2, 64, dtype=torch.bfloat16).cuda()
    q = torch.zeros(N, 8, 64, dtype=torch.bfloat16).cuda()
    out = torch.zeros_like(q)
    n_dev = torch.tensor(lens, dtype=torch.int32).cuda()
    start = _starts(counts)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        p.kv.write(x[:, 0], x[:, 1], p.dev_table, n_dev, start)
        p.kv.attend(q, p.dev_table, n_dev, start, 8, out=out)
    for step in range(3):
        counts = [[3, 1, 5], [0, 8, 1], [1, 0, 8]][step]
        lens = [n + c for n, c in zip(lens, counts)]
        new = torch.randn(N, 2, 2, 64, generator=p.g).to(torch.bfloat16)
        qq = torch.randn(N, 8, 64, generator=p.g).to(torch.bfloat16)
        x.copy_(new)
        q.copy_(qq)
        n_dev.copy_(torch.tensor(lens, dtype=torch.int32))
        start.copy_(_starts(counts))
        graph.replay()
        torch.cuda.synchronize()
        p.ref.write({"k": new[:, 0], "v": new[:, 1]}, p.table, lens, counts)
        p.check(lens)
        got = out.clone()
        assert torch.equal(got, p.check_attend(lens, counts, q=qq, max_q=8))
    p.kv.close()


def test_empty_calls_and_refusals(KV):
    from model_free_suffix_gb300 import _lib as L
    p = Pair(KV, [40], P=16, H=2, D=64, G=2)
    lens, none = torch.tensor([40], dtype=torch.int32).cuda(), torch.zeros(2, dtype=torch.int32).cuda()
    x, q = torch.zeros(1, 2, 64, dtype=torch.bfloat16).cuda(), torch.zeros(1, 4, 64, dtype=torch.bfloat16).cuda()
    p.kv.write(x[:0], x[:0], p.dev_table, lens, none)
    assert p.kv.attend(q[:0], p.dev_table, lens, none, 1).shape[0] == 0
    assert p.kv.launch_count() == 0
    start = _starts([1])
    bad = [lambda: p.kv.write(x.double(), x.double(), p.dev_table, lens, start),
           lambda: p.kv.write(x, x.half(), p.dev_table, lens, start),
           lambda: p.kv.write(x.transpose(1, 2), x, p.dev_table, lens, start),
           lambda: p.kv.write(x.cpu(), x.cpu(), p.dev_table, lens, start),
           lambda: p.kv.write(x, x, p.dev_table[:, :1], lens, start),
           lambda: p.kv.write(x, x, p.dev_table, lens, lens),
           lambda: p.kv.write(x, x, p.dev_table, lens.long(), start),
           lambda: p.kv.attend(q.float(), p.dev_table, lens, start, 1),
           lambda: p.kv.attend(x, p.dev_table, lens, start, 1),
           lambda: p.kv.attend(q, p.dev_table, lens, start, 1, out=q[:, :2]),
           lambda: p.kv.read(p.dev_table, lens * 0, start)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for kw in (dict(max_q=0), dict(max_q=1, window=-1), dict(max_q=1, sinks=-1),
               dict(max_q=1, scale=float("nan"))):
        with pytest.raises(L.SgdError):
            p.kv.attend(q, p.dev_table, lens, start, **kw)
    assert p.kv.launch_count() == 0
    p.kv.close()


def test_offsets_past_32_bits(KV):
    """Blocks beyond 2^32 bytes of the cache are written, read and attended to in place."""
    P, H, D, pages = 128, 8, 128, 40000          # 5.2 GB each of keys and values
    if torch.cuda.mem_get_info()[0] < 30e9:
        pytest.skip("needs 30 GB")
    kv = KV(num_pages=pages, page_size=P, kv_heads=H, head_dim=D, q_heads=H, max_batch=1, max_pages_per_row=2)
    table = torch.tensor([[pages - 1, 33000]], dtype=torch.int32).cuda()
    g = torch.Generator().manual_seed(1)
    x = torch.randn(200, 2, H, D, generator=g).to(torch.bfloat16)
    dev = x.cuda()
    lens = torch.tensor([200], dtype=torch.int32).cuda()
    kv.write(dev[:, 0], dev[:, 1], table, lens, _starts([200]))
    ref = R.Cache(2, H, P, D)
    ref.write({"k": x[:, 0], "v": x[:, 1]}, [[0, 1]], [200], [200])
    k, v = kv.read(table, lens * 0, _starts([200]), total=200)
    q = torch.randn(3, H, D, generator=g).to(torch.bfloat16)
    want, mass = R.attend(q.view(3, H, 1, D), ref.rows("k", [0, 1], 0, 200), ref.rows("v", [0, 1], 0, 200), 197, D ** -0.5)
    assert torch.equal(k.cpu().double(), ref.rows("k", [0, 1], 0, 200))
    assert torch.equal(v.cpu().double(), ref.rows("v", [0, 1], 0, 200))
    out = kv.attend(q.cuda(), table, lens, _starts([3]), 3).cpu().double()
    want, mass = want[:, :, 0], mass[:, :, 0]
    assert bool(((out - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -10 * mass + 1e-7).all())
    kv.close()


@pytest.mark.parametrize("D,P,counts", [(128, 64, [8]), (64, 128, [1]), (64, 16, [20]), (128, 32, [1, 12])])
def test_attend_one_long_row(KV, D, P, counts):
    """A unit cut into as many parts as there are CTAs."""
    lens = [100_003, 5][:len(counts)]
    p = Pair(KV, lens, P=P, H=1, D=D, G=4, seed=9)
    p.write(lens, lens, spread=1.0)
    p.check_attend(lens, [min(c, n) for c, n in zip(counts, lens)])
    assert p.kv.get_error() == 0
    p.kv.close()


@pytest.mark.parametrize("counts,room", [([1, 1, 1], 4), ([3, 0, 9], 300)])
def test_room_for_more_tokens(KV, counts, room):
    """Tokens past q_start[B] are neither read nor written."""
    lens = [40, 7, 90]
    p = Pair(KV, lens, P=32, H=2, D=64, G=2)
    p.write(lens, lens, spread=1.0)
    N = sum(counts)
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    q = torch.full((N + room, 4, 64), float("nan"), dtype=torch.bfloat16)
    q[:N] = torch.randn(N, 4, 64, generator=p.g)
    out = torch.full((N + room, 4, 64), 7.0, dtype=torch.bfloat16).cuda()
    p.kv.attend(q.cuda(), p.dev_table, n, _starts(counts), max(counts), out=out)
    assert bool((out[N:] == 7).all())
    assert torch.equal(out[:N], p.check_attend(lens, counts, q=q[:N]))
    kv = torch.full((N + room, 2, 2, 64), float("nan"), dtype=torch.bfloat16)
    kv[:N] = torch.randn(N, 2, 2, 64, generator=p.g)
    dev = kv.cuda()
    p.kv.write(dev[:, 0], dev[:, 1], p.dev_table, n, _starts(counts))
    p.ref.write({"k": kv[:N, 0], "v": kv[:N, 1]}, p.table, lens, counts)
    p.check(lens)
    assert p.kv.get_error() == 0
    p.kv.close()
