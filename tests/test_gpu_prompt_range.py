"""Attention of prompts and chunks at the ends of its types' range (scores far from 0, values next to the largest)
and of what counts its work.

The scores here are exact in 32 bits (few products, few bits each), so nothing of the bound of
test_gpu_prompt.py grows with them: with results u |want| for their rounding, u sum_j p_j |v_j| for that of
the probabilities, 2^-12 of that sum for the exponentials and sums.
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
SCALE = 0.6875      # (exact; a step of 1 of a score is some 0.992 as a power of 2)


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


def _check(got, want, mass, where):
    u = UNIT[got.dtype]
    off = (got.cpu().double() - want).abs()
    bound = u * want.abs() + (u + 2.0 ** -12) * mass + 2.0 ** -25
    assert bool((off <= bound).all()), (where, float((off / bound).nan_to_num(nan=math.inf).max()))


def _rows(KV, counts, q, k, v, window=0, sinks=0, scale=SCALE):
    """attend_prompt of one head of keys, checked row by row."""
    kv = KV(num_pages=1, page_size=64, kv_heads=k.shape[1], head_dim=q.shape[2], q_heads=q.shape[1], max_batch=len(counts),
            max_pages_per_row=1)
    out = kv.attend_prompt(q.cuda(), k.cuda(), v.cuda(), _starts(counts), scale=scale, window=window, sinks=sinks)
    assert kv.get_error() == 0
    kv.close()
    at, H, G = 0, k.shape[1], q.shape[1] // k.shape[1]
    for c in counts:
        x = slice(at, at + c)
        want, mass = R.attend(q[x].double().view(c, H, G, -1), k[x].double(), v[x].double(), 0, scale, window, sinks)
        _check(out[x], want.reshape(c, H * G, -1), mass.reshape(c, H * G, -1), (at, c))
        at += c
    return out


def _scores(N, G, D, dtype, base, steps):
    """q, k whose scores are base + steps[j] (one head of keys), and values; base = x 2^(2 n), |x| = 1 or 0."""
    t = DTYPES[dtype]
    q, k = torch.zeros(N, G, D), torch.zeros(N, 1, D)
    root = 2.0 ** (math.log2(abs(base)) / 2) if base else 0.0
    q[..., 0], k[..., 0] = root, math.copysign(root, base)
    whole = torch.floor(torch.as_tensor(steps, dtype=torch.float64)).float()
    q[..., 1] = q[..., 2] = 1.0
    k[:, 0, 1], k[:, 0, 2] = whole, torch.as_tensor(steps).float() - whole
    for x in (q, k):
        assert torch.equal(x.to(t).float(), x)
    v = torch.randn(N, 1, D, generator=torch.Generator().manual_seed(1)).to(t)
    return q.to(t), k.to(t), v


@pytest.mark.parametrize("grow", [7.5, 7.75, 8.0, 8.125, 15.5])
@pytest.mark.parametrize("power", [10, 12, 16, 18, 20, 22])
@pytest.mark.parametrize("dtype,D", [("f16", 64), ("f16", 128), ("bf16", 128)])
def test_far_scores_that_grow(KV, dtype, D, power, grow):
    """By about as much as the reference may lag, from each half of a tile to the next, at scores of 2^power."""
    counts = [520, 70]
    j = np.concatenate([np.arange(c) for c in counts])
    steps = (j // 64) * grow + (j * 7 % 5) * 0.125
    steps = np.floor(steps * min(8.0, 2.0 ** (23 - power))) / min(8.0, 2.0 ** (23 - power))
    for sign in (1, -1):
        _rows(KV, counts, *_scores(sum(counts), 3, D, dtype, sign * 2.0 ** power, steps))


@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 2)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_far_scores_of_rows_that_are_cut(KV, dtype, window, sinks):
    """Parts whose references differ by less than 32 bits hold of them."""
    N = 2500
    j = np.arange(N)
    steps = (j * 37 % 101) / 4.0 + (j > 1200) * 2.0
    _rows(KV, [N], *_scores(N, 2, 128, dtype, 2.0 ** 20, steps), window=window, sinks=sinks)


@pytest.mark.parametrize("dtype,power", [("f16", 24), ("f16", 30), ("bf16", 24), ("bf16", 32), ("bf16", 60), ("bf16", 100)])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_far_apart(KV, dtype, power, sign):
    """All the weight is with the largest scores that a token sees, in equal shares."""
    counts, D = [700, 130, 1], 64
    N = sum(counts)
    rng = np.random.default_rng(power)
    q, k = torch.zeros(N, 2, D), torch.zeros(N, 1, D)
    q[..., 0] = 2.0 ** (power // 2)
    level = torch.from_numpy(rng.integers(0, 3, N) * (rng.random(N) < 0.05)).float()
    k[:, 0, 0] = sign * 2.0 ** (power // 2) * (1 + level / 8)
    v = torch.randn(N, 1, D, generator=torch.Generator().manual_seed(2))
    _rows(KV, counts, *(x.to(DTYPES[dtype]) for x in (q, k, v)), scale=1.0)


@pytest.mark.parametrize("grow", [0.0, 1.0, 8.0, 15.5])
@pytest.mark.parametrize("counts", [[520, 70], [2500]])
def test_values_next_to_the_largest(KV, counts, grow):
    """bfloat16 values of up to 2^127.6 give results of that size: as those of values 2^-126 times as large, bit by bit."""
    N = sum(counts)
    j = np.concatenate([np.arange(c) for c in counts])
    q, k, _ = _scores(N, 2, 64, "bf16", 0.0, (j // 64 % 12) * grow)
    v = (1 + torch.rand(N, 1, 64, generator=torch.Generator().manual_seed(3)) * 2).to(torch.bfloat16)
    plain = _rows(KV, counts, q, k, v)
    kv = KV(num_pages=1, page_size=64, kv_heads=1, head_dim=64, q_heads=2, max_batch=len(counts), max_pages_per_row=1)
    out = kv.attend_prompt(q.cuda(), k.cuda(), (v * 2.0 ** 126).cuda(), _starts(counts), scale=SCALE)
    assert bool(out.isfinite().all()) and torch.equal(out.double(), plain.double() * 2.0 ** 126)
    kv.close()


def test_many_equal_weights(KV):
    """Sums of p over tens of thousands of tokens, none of which has more than the first: 2^127 is still a result."""
    N, D = 66000, 64
    v = torch.full((N, 1, D), 2.0 ** 127, dtype=torch.bfloat16, device="cuda")
    kv = KV(num_pages=1, page_size=64, kv_heads=1, head_dim=D, q_heads=1, max_batch=1, max_pages_per_row=1)
    k = torch.zeros_like(v)
    out = kv.attend_prompt(torch.ones_like(v), k, v, _i32([0, N]))
    # (the weights are equal and add up to 1 but for 2^-24 an addition, joined or not)
    assert bool(((out.double() / 2.0 ** 127 - 1).abs() <= 2.0 ** -8).all())
    kv.close()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("top", [3, 20, 30])
def test_far_scores_over_a_cache(KV, dtype, top):
    """Cached keys of one dim, 1, 1.25 or 1.5 times powers of two up to 2^top, their pages' scales with them, then
    the chunk's own of up to 2^4."""
    olds, counts, P, D = [700, 40, 0], [60, 200, 5], 16, 64
    rng = np.random.default_rng(top)
    N, new = sum(olds), sum(counts)
    page = np.concatenate([np.arange(o) // P for o in olds if o])
    power = (page * 7 % (top + 1)).astype(np.float64)
    k_old = torch.zeros(N, 1, D)
    k_old[:, 0, 5] = torch.from_numpy(2.0 ** power * rng.choice([1.0, 1.25, 1.5], N)).float()
    v_old = torch.randn(N, 1, D, generator=torch.Generator().manual_seed(4))
    k, q = torch.zeros(new, 1, D), torch.zeros(new, 2, D)
    k[:, 0, 5] = torch.from_numpy(rng.integers(0, 64, new) / 4.0).float()
    q[..., 5] = torch.from_numpy(rng.choice([1.0, 0.5, 2.0], (new, 2))).float()
    v = torch.randn(new, 1, D, generator=torch.Generator().manual_seed(5))
    q, k, v = (x.to(DTYPES[dtype]) for x in (q, k, v))
    k_old, v_old = k_old.to(torch.bfloat16), v_old.to(torch.bfloat16)
    need = [-(-(o + c) // P) for o, c in zip(olds, counts)]
    table = np.full((3, max(need)), -1, np.int32)
    order, at = rng.permutation(sum(need)), 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    kv = KV(num_pages=sum(need), page_size=P, kv_heads=1, head_dim=D, q_heads=2, max_batch=3, max_pages_per_row=max(need))
    dev = torch.from_numpy(table).cuda()
    kv.write(k_old.cuda(), v_old.cuda(), dev, _i32(olds), _starts(olds))
    ref = R.Cache(sum(need), 1, P, D)
    ref.write({"k": k_old, "v": v_old}, table, olds, olds)
    lens = [o + c for o, c in zip(olds, counts)]
    out = kv.attend_chunk(q.cuda(), k.cuda(), v.cuda(), dev, _i32(lens), _starts(counts), scale=1.0)
    at = 0
    for b, c in enumerate(counts):
        x = slice(at, at + c)
        kb, vb = (torch.cat([ref.rows(n, table[b], 0, olds[b]), y[x].double()]) for n, y in (("k", k), ("v", v)))
        want, mass = R.attend(q[x].double().view(c, 1, 2, D), kb, vb, olds[b], 1.0)
        _check(out[x], want.reshape(c, 2, D), mass.reshape(c, 2, D), b)
        at += c
    assert kv.get_error() == 0
    kv.close()


@pytest.mark.parametrize("dtype,size", [("f16", 200.0), ("f16", 15000.0), ("bf16", 300.0), ("bf16", 2.0 ** 20)])
def test_large_queries_and_keys_give_finite_results(KV, dtype, size):
    """Random scores of about size^2 sqrt(D): beyond what 32 bits tell apart, but no infinities and no NaN, and
    nothing outside the values' range."""
    counts, D = [900, 33], 128
    g = torch.Generator().manual_seed(6)
    q, k, v = (torch.randn(sum(counts), h, D, generator=g) * s for h, s in ((4, size), (2, size), (2, 1.0)))
    q, k, v = (x.clamp(-6e4, 6e4).to(DTYPES[dtype]) if dtype == "f16" else x.to(DTYPES[dtype]) for x in (q, k, v))
    kv = KV(num_pages=1, page_size=64, kv_heads=2, head_dim=D, q_heads=4, max_batch=2, max_pages_per_row=1)
    for scale in (1.0, -0.125):
        out = kv.attend_prompt(q.cuda(), k.cuda(), v.cuda(), _starts(counts), scale=scale).cpu()
        assert bool(out.isfinite().all()) and float(out.abs().max()) <= float(v.abs().max()) * (1 + 2.0 ** -6)
    kv.close()


@pytest.mark.parametrize("chunk", [False, True])
def test_rows_that_claim_the_same_tokens_again_and_again(KV, chunk):
    """Starts that descend: far more work than the call's tokens are.  It is reported, and nothing is written."""
    from model_free_suffix_gb300 import _lib as L
    N, H, G, D, B = 2000, 1, 4, 64, 33
    kv = KV(num_pages=4, page_size=64, kv_heads=H, head_dim=D, q_heads=H * G, max_batch=B, max_pages_per_row=40)
    g = torch.Generator().manual_seed(7)
    q, k, v = (torch.randn(N, h, D, generator=g).bfloat16().cuda() for h in (H * G, H, H))
    out = torch.full_like(q, 7.0)

    def call(starts, lens):
        if not chunk:
            return kv.attend_prompt(q, k, v, _i32(starts), out=out)
        table = torch.full((B, 40), -1, dtype=torch.int32, device="cuda")
        return kv.attend_chunk(q, k, v, table, _i32(lens), _i32(starts), out=out)

    call([0, N] * 17, [N, 0] * 16 + [N])
    assert kv.get_error(clear=True) == L.KV_ERR_LENGTH and bool((out == 7).all())
    # (rows that follow one another may have many more units than their tokens fill)
    counts = [61] * 32 + [48]
    call([0] + list(itertools.accumulate(counts)), counts)
    assert kv.get_error() == 0
    at = 0
    for c in counts:
        x = slice(at, at + c)
        want, mass = R.attend(q[x].cpu().double().view(c, H, G, D), k[x].cpu().double(), v[x].cpu().double(), 0, D ** -0.5)
        _check(out[x], want.reshape(c, H * G, D), mass.reshape(c, H * G, D), at)
        at += c
    kv.close()
