"""sgd_verify against its definition in 64 bits.

Accepted counts and ids are whole numbers and must be equal: the random numbers
are inputs, and a decision closer than the arithmetic's error (relative 1e-6)
has a chance of about 1e-6 per row on these seeds.  Log probabilities: (l - m) / t and
log Z are each formed in 32 bits; with |l - m| / t < 2^7 their rounding is below
2^-17, and Z's relative error, from an exponential of 2^-21 and sums of at most
2^18 terms in a tree of partial sums (runs of at most 2^9), is below 2^-14: an
absolute bound of 1e-4 holds with room, and 2e-5 is asked for here.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def SD():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from model_free_suffix_gb300 import build
    build.build()
    from model_free_suffix_gb300 import SuffixDrafter
    return SuffixDrafter


def reference(logits, start, drafts, nv, u, noise, temp, q=None):
    """One row at a time, in 64 bits: (sampled, accepted, log probabilities)."""
    B, k = drafts.shape
    out, acc, logp = np.full((B, k + 1), -1, np.int64), np.zeros(B, np.int64), np.zeros((B, k + 1))

    def masses(x, t):
        x = np.where(np.isnan(x), -np.inf, x)
        m = x.max()
        if m == -np.inf:
            return None, None, -1
        if m == np.inf:
            w, lw = (x == np.inf).astype(float), np.where(x == np.inf, 0.0, -np.inf)
        else:
            lw = (x - m) / t
            w = np.exp(lw)
        return w / w.sum(), lw - math.log(w.sum()), int(np.argmax(x))

    for b in range(B):
        t = float(temp[b])
        greedy = not t >= 1e-5
        for i in range(nv[b] + 1):
            r = start[b] + i
            p, lp, top = masses(logits[r], 1.0 if greedy else t)
            if i < nv[b]:
                d = int(drafts[b, i])
                if p is not None and 0 <= d < len(p):
                    qd = 1.0 if q is None else float(q[r, d])
                    if d == top if greedy else float(u[b, i]) * qd < p[d]:
                        out[b, i], logp[b, i] = d, lp[d]
                        acc[b] = i + 1
                        continue
            if p is None:
                break
            token = top
            if not greedy:
                w = p.copy()
                if i < nv[b]:
                    if q is not None:
                        w = np.maximum(p - q[r], 0)
                    elif 0 <= d < len(p):
                        w[d] = 0
                if not (w > 0).any():
                    w = p
                token = int(np.argmax(w / np.maximum(noise[b], 2.0 ** -60)))
            out[b, i], logp[b, i] = token, lp[token]
            break
    return out, acc, logp


class Case:
    def __init__(self, B, k, V, dtype="f32", q=False, greedy=0.3, seed=0, spread=2.0, accept=0.7):
        g = self.g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.B, self.k, self.V = B, k, V
        self.nv = rng.integers(0, k + 1, B)
        self.nv[0] = k
        self.start = np.concatenate([[0], np.cumsum(self.nv + 1)])[:B]
        R = int((self.nv + 1).sum())
        x = torch.randn(R, V, generator=g) * spread
        self.drafts = np.full((B, k), -1, np.int64)
        qq = None
        if q:
            qq = torch.softmax(x * 0.8 + torch.randn(R, V, generator=g) * 0.5, -1)
        for b in range(B):
            for i in range(self.nv[b]):
                r = self.start[b] + i
                if q:
                    d = int((qq[r] / torch.empty(V).exponential_(generator=g)).argmax())
                else:
                    d = int(rng.integers(V))
                    if rng.random() < accept:
                        x[r, d] = float(torch.logsumexp(x[r], 0)) + 2.0
                self.drafts[b, i] = d
        self.logits = x.to(DTYPES[dtype])
        self.q = qq
        self.temp = torch.rand(B, generator=g) * 1.2 + 0.3
        self.temp[torch.rand(B, generator=g) < greedy] = 0.0
        self.u = torch.rand(B, k, generator=g)
        self.noise = torch.empty(B, V).exponential_(generator=g)

    def run(self, dr, rows=True, **over):
        c = lambda t: None if t is None else torch.as_tensor(t).cuda()  # noqa: E731
        kw = dict(row_start=c(self.start).int() if rows else None, temperature=c(self.temp), draft_probs=c(self.q))
        kw.update(over)
        r = dr.verify(c(self.logits), c(self.drafts).int(), c(self.nv).int(), c(self.u), c(self.noise), **kw)
        torch.cuda.synchronize()
        return r

    def check(self, r, rows=None):
        n = lambda t: None if t is None else t.double().numpy()  # noqa: E731
        out, acc, logp = reference(n(self.logits), self.start, self.drafts, self.nv, n(self.u), n(self.noise),
                                   n(self.temp), n(self.q))
        rows = np.arange(self.B) if rows is None else rows
        assert np.array_equal(r.num_accepted.cpu().numpy()[rows], acc[rows])
        assert np.array_equal(r.sampled.cpu().numpy()[rows], out[rows])
        got = r.logprobs.cpu().double().numpy()[rows]
        assert np.all(np.abs(got - logp[rows]) <= 2e-5 * np.maximum(1, np.abs(logp[rows])))
        return out, acc


def _drafter(SD, c, **kw):
    return SD(max_batch=c.B, seq_capacity=64, vocab_size=c.V, k=c.k, **kw)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 7, 255, 2048, 2049, 5003, 32000])
@pytest.mark.parametrize("q", [False, True])
def test_matches_the_definition(SD, V, dtype, q):
    c = Case(7, 5, V, dtype, q, seed=V)
    with _drafter(SD, c) as dr:
        c.check(c.run(dr))
        c.check(c.run(dr))   # (nothing of a call stays for the next)


@pytest.mark.parametrize("B,k", [(1, 1), (1, 64), (3, 16), (300, 4)])
def test_batches_and_draft_widths(SD, B, k):
    c = Case(B, k, 1009, "bf16", seed=B, accept=0.95)
    with _drafter(SD, c) as dr:
        out, acc = c.check(c.run(dr))
        assert acc.max() > k // 2 or B == 1


def test_large_vocabulary(SD):
    c = Case(3, 4, 151936, "bf16", seed=9, spread=2.5)
    with _drafter(SD, c) as dr:
        c.check(c.run(dr))


def test_rows_apart_and_unaligned(SD):
    c = Case(5, 4, 1001, "bf16", True, seed=3)
    R = c.logits.shape[0]
    wide = torch.zeros(R, 1003, dtype=torch.bfloat16).cuda()
    logits = wide[:, 1:1002]
    logits.copy_(c.logits)
    qw = torch.zeros(R, 1005).cuda()
    probs = qw[:, 3:1004]
    probs.copy_(c.q)
    nw = torch.zeros(5, 1002).cuda()
    noise = nw[:, 1:]
    noise.copy_(c.noise)
    with _drafter(SD, c) as dr:
        r = dr.verify(logits, torch.as_tensor(c.drafts).int().cuda(), torch.as_tensor(c.nv).int().cuda(),
                      c.u.cuda(), noise, row_start=torch.as_tensor(c.start).int().cuda(),
                      temperature=c.temp.cuda(), draft_probs=probs)
        c.check(r)


def test_default_rows_and_temperature(SD):
    c = Case(4, 3, 500, seed=4)
    c.nv[:] = 3
    c = _refill(c)
    c.temp = torch.ones(4)
    with _drafter(SD, c) as dr:
        c.check(c.run(dr, rows=False, temperature=None))


def _refill(c):
    """Drafts in every slot, logits at b (k + 1)."""
    rng = np.random.default_rng(1)
    c.start = np.arange(c.B) * (c.k + 1)
    c.logits = torch.randn(c.B * (c.k + 1), c.V, generator=c.g) * 2
    c.drafts = rng.integers(0, c.V, (c.B, c.k))
    for b in range(c.B):
        for i in range(c.k):
            c.logits[c.start[b] + i, c.drafts[b, i]] = 9.0
    return c


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_masks_infinities_and_nan(SD, dtype):
    c = _refill(Case(12, 3, 700, seed=5))
    c.nv[:] = 3
    x = c.logits.to(DTYPES[dtype])
    low = torch.finfo(DTYPES[dtype]).min
    S = c.k + 1
    x[0 * S:1 * S, 100:] = float("-inf")                      # a sampler's cut
    x[1 * S:2 * S, 100:] = low                                # the same with the lowest value
    x[2 * S:3 * S, 1:] = float("-inf")                        # one token left
    x[3 * S:4 * S] = low                                      # every token the lowest: uniform
    x[4 * S:5 * S, 30:40] = float("inf")                      # ten tokens share everything
    x[5 * S:6 * S, ::3] = float("nan")                        # as if -inf
    x[6 * S:7 * S] = float("-inf")                            # nothing left
    x[7 * S:8 * S] = float("nan")
    x[8 * S + 1] = float("-inf")                              # nothing left at the second position
    x[9 * S:10 * S] = torch.finfo(DTYPES[dtype]).max          # equal at the other end
    c.drafts[2], c.drafts[4] = 0, 33
    c.logits = x
    c.temp[:] = 0.7
    c.temp[10] = 1e30
    c.temp[11] = 1e-4
    from model_free_suffix_gb300 import _lib as L
    with _drafter(SD, c) as dr:
        out, acc = c.check(c.run(dr))
        assert dr.get_error(clear=True) == L.ERR_NO_TOKEN
        assert (out[6] == -1).all() and (out[7] == -1).all() and (out[2] == 0).all()
        c.temp[:] = 0.0
        c.check(c.run(dr))


def test_ties_go_to_the_lowest_index(SD):
    c = _refill(Case(6, 2, 4099, seed=6))
    c.nv[:] = 2
    c.logits = torch.randn(18, 4099, generator=c.g).round().to(torch.bfloat16)   # few values, many ties
    c.noise = torch.ones(6, 4099)
    c.temp = torch.tensor([0.0, 0.0, 0.0, 1.0, 1.0, 1.0])
    with _drafter(SD, c) as dr:
        c.check(c.run(dr))


def test_shared_logits_rows(SD):
    """Rows that verify against the same logits (several samples of one request)."""
    c = _refill(Case(4, 3, 900, seed=8))
    c.nv[:] = [3, 3, 2, 0]
    c.start[:] = 1
    with _drafter(SD, c) as dr:
        c.check(c.run(dr))


def test_extreme_random_numbers(SD):
    c = Case(6, 4, 800, "bf16", seed=11)
    c.temp[:] = 1.0
    c.u[0], c.u[1] = 0.0, 1 - 2.0 ** -24
    c.noise[2, ::2] = 0.0
    c.noise[3] = 1e-30
    c.noise[4] = 1e30
    with _drafter(SD, c) as dr:
        _, acc = c.check(c.run(dr))
        assert acc[0] == c.nv[0]


def test_draft_probabilities_equal_to_the_targets(SD):
    """q = p: every draft is accepted, whatever the random numbers below 1."""
    c = Case(8, 4, 300, "f32", True, greedy=0.0, seed=12)
    c.temp[:] = 1.0
    c.q = torch.softmax(c.logits.double(), -1).float()
    c.u[:] = c.u * 0.999
    with _drafter(SD, c) as dr:
        _, acc = c.check(c.run(dr))
        assert np.array_equal(acc, c.nv)


def test_inactive_and_bad_rows(SD):
    from model_free_suffix_gb300 import _lib as L
    c = _refill(Case(6, 3, 400, seed=13))
    c.nv[:] = [3, 2, 3, 3, 1, 0]
    c.temp = torch.tensor([1.0, 1.0, float("nan"), -1.0, 1.0, 1.0])
    active = torch.tensor([1, 0, 1, 1, 1, 1], dtype=torch.uint8).cuda()
    with _drafter(SD, c) as dr:
        r = c.run(dr, active=active)
        c.check(r, np.array([0, 2, 3, 4, 5]))
        assert (r.sampled[1] == -1).all() and r.num_accepted[1] == 0 and not r.logprobs[1].any()
        assert dr.get_error(clear=True) == L.ERR_TEMPERATURE
        c.temp[:] = 1.0
        good = c.nv.copy()
        c.drafts[0, 1], c.drafts[4, 0] = c.V, -7               # ids that no vocabulary has: not accepted
        c.check(c.run(dr))
        assert dr.get_error() == 0
        c.nv[:] = [3, 2, 9, -4, 1, 0]                          # clamped to [0, k], reported
        r = c.run(dr)
        c.nv[2], c.nv[3] = 3, 0
        c.check(r)
        assert dr.get_error(clear=True) == L.ERR_VERIFY_ROWS
        c.nv[:] = good
        start = c.start.copy()
        for bad in (-1, len(c.logits) - 3, 2 ** 31 - 1):
            c.start[0] = bad
            r = c.run(dr)
            assert (r.sampled[0] == -1).all() and r.num_accepted[0] == 0
            assert dr.get_error(clear=True) == L.ERR_VERIFY_ROWS
            c.start = start.copy()
            c.check(r, np.arange(1, 6))


def test_emitted_tokens_follow_the_target(SD):
    """The first emitted token of many rows against softmax(l / t), whatever
    was drafted: chi-square below its mean by 5 standard deviations (V = 40,
    and every expected count above 20)."""
    B, V = 8192, 40
    g = torch.Generator().manual_seed(3)
    x = torch.randn(1, V, generator=g).repeat(2, 1)
    for q in (None, torch.softmax(torch.randn(V, generator=g), -1)):
        with SD(max_batch=B, seq_capacity=64, vocab_size=V, k=1) as dr:
            d = torch.randint(0, 6, (B, 1), generator=g)
            probs = None
            if q is not None:
                d = torch.multinomial(q.expand(B, V), 1, generator=g)
                probs = q.expand(2, V).contiguous().cuda()
            r = dr.verify(x.cuda(), d.int().cuda(), torch.ones(B, dtype=torch.int32).cuda(),
                          torch.rand(B, 1, generator=g).cuda(), torch.empty(B, V).exponential_(generator=g).cuda(),
                          row_start=torch.zeros(B, dtype=torch.int32).cuda(),
                          temperature=torch.full((B,), 0.8).cuda(), draft_probs=probs)
            first = r.sampled[:, 0].cpu().long()
            want = torch.softmax(x[0].double() / 0.8, -1) * B
            chi = float(((torch.bincount(first, minlength=V) - want) ** 2 / want).sum())
            assert chi < (V - 1) + 5 * math.sqrt(2 * (V - 1)), chi


def test_output_feeds_the_drafter(SD):
    """sampled is what propose_with_update takes: rows grow by the accepted ids and the token."""
    c = Case(5, 4, 600, "bf16", seed=15)
    with _drafter(SD, c) as dr:
        r = c.run(dr)
        tok = torch.randint(0, 600, (5, 64)).int().cuda()
        n = torch.tensor([3, 10, 20, 30, 40], dtype=torch.int32).cuda()
        before = n.clone()
        dr.propose_with_update(tok, n, r.sampled)
        assert torch.equal(n - before, r.num_accepted + 1)
        for b in range(5):
            a = int(r.num_accepted[b]) + 1
            assert torch.equal(tok[b, int(before[b]):int(n[b])], r.sampled[b, :a])


def test_in_a_graph_and_on_a_stream(SD):
    c = Case(9, 5, 3001, "bf16", seed=16)
    dev = lambda t: torch.as_tensor(t).cuda()  # noqa: E731
    with _drafter(SD, c) as dr:
        args = [dev(c.logits), dev(c.drafts).int(), dev(c.nv).int(), dev(c.u), dev(c.noise)]
        start, temp = dev(c.start).int(), dev(c.temp)
        out = dr.new_verdict(9)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            dr.verify(*args, row_start=start, temperature=temp, out=out)
        for _ in range(3):
            out.sampled.fill_(-9)
            graph.replay()
            torch.cuda.synchronize()
            c.check(out)
            c.u = torch.rand(9, 5, generator=c.g)
            args[3].copy_(c.u)
        graph.replay()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        r = dr.verify(*args, row_start=start, temperature=temp, stream=side)
        torch.cuda.synchronize()
        c.check(r)
        assert dr.launch_count() > 0


def test_refusals(SD):
    from model_free_suffix_gb300 import _lib as L
    c = Case(3, 2, 100, seed=17)
    dev = lambda t: torch.as_tensor(t).cuda()  # noqa: E731
    x, d, nv, u, noise = dev(c.logits), dev(c.drafts).int(), dev(c.nv).int(), dev(c.u), dev(c.noise)
    with _drafter(SD, c) as dr:
        bad = [lambda: dr.verify(x.double(), d, nv, u, noise), lambda: dr.verify(x[:, :50], d, nv, u, noise),
               lambda: dr.verify(x, d[:, :1], nv, u, noise), lambda: dr.verify(x, d.long(), nv, u, noise),
               lambda: dr.verify(x, d, nv, u[:2], noise), lambda: dr.verify(x, d, nv, u, noise.half()),
               lambda: dr.verify(x.cpu(), d, nv, u, noise), lambda: dr.verify(x.t().contiguous().t(), d, nv, u, noise),
               lambda: dr.verify(x, d, nv, u, noise, draft_probs=x[:1]),
               lambda: dr.verify(x, d, nv, u, noise, row_start=nv[:2]),
               lambda: dr.verify(x, d, nv, u, noise, temperature=nv)]
        for f in bad:
            with pytest.raises(ValueError):
                f()
        with pytest.raises(L.SgdError):   # more rows than max_batch
            z = lambda t: torch.cat([t, t])  # noqa: E731
            dr.verify(x, z(d), z(nv), z(u), z(noise))
        r = dr.verify(x[:0], d[:0], nv[:0], u[:0], noise[:0])
        assert r.sampled.shape == (0, 3) and dr.launch_count() == 0
