"""What a rejected draft leaves in its block: the accepted entries against a cache that
never saw it.

While a draft is in the block, its entries are held at a scale s of the draft's
size: each moves by at most half a subnormal step, 2^-10 s, and is exact from
2^-6 s on (four significant bits, e4m3's own).  A value that is held once is held
exactly at any smaller scale that reaches it.  So two caches differ by at most
2^-10 of the scales that either held the block at, added up.
"""
import pytest
import torch

from test_gpu_kv_cache import KV, Pair, _starts  # noqa: F401 (KV: the fixture)

pytestmark = pytest.mark.gpu


class Run(Pair):
    """A cache of one row, its block's scales added up write by write."""

    def __init__(self, KV, accepted, **kw):
        super().__init__(KV, [64], P=64, H=2, D=64, extra=0, **kw)
        self.accepted, self.total, self.held = accepted, {"k": 0.0, "v": 0.0}, {}

    def put(self, n, x):
        self.write([n], [len(x)], tensors=(x, -x * 0.5))
        for name, s in (("k", self.kv.k_scale), ("v", self.kv.v_scale)):
            s = s[0, int(self.table[0, 0])].double().cpu()[None, :, None]
            self.total[name] = self.total[name] + s
            self.held[name] = torch.maximum(self.held.get(name, s), s)

    def values(self):
        k, v = self.kv.read(self.dev_table, torch.zeros(1, dtype=torch.int32).cuda(), _starts([self.accepted]),
                            total=self.accepted, dtype=torch.float32)
        return {"k": k.double().cpu(), "v": v.double().cpu()}


@pytest.mark.parametrize("size", [1.0, 60.0, 300.0, 3e4, 1e8])
@pytest.mark.parametrize("rounds", [1, 3])
def test_accepted_entries_after_rejected_drafts(KV, size, rounds):
    g = torch.Generator().manual_seed(31)
    n = 22
    x = torch.randn(n, 2, 64, generator=g)
    more = [torch.randn(1, 2, 64, generator=g) for _ in range(rounds)]
    saw, clean = Run(KV, n, seed=3), Run(KV, n, seed=3)
    for p in (saw, clean):
        p.put(n, x)
    for i in range(rounds):
        saw.put(n + i + 5, torch.full((5, 2, 64), size) * (-1) ** i)   # five drafts; none is accepted
        for p in (saw, clean):
            p.put(n + i + 1, more[i])
    got, want = saw.values(), clean.values()
    for name in "kv":
        off = (got[name] - want[name]).abs()
        assert bool((off <= 2.0 ** -10 * (saw.total[name] + clean.total[name])).all())
        exact = want[name].abs() >= 2.0 ** -6 * torch.maximum(saw.held[name], clean.held[name])
        assert bool((off[exact.expand_as(off)] == 0).all())
    if size >= 300:   # (so there is something to bound)
        assert bool((got["k"] != want["k"]).any())
    for p in (saw, clean):
        p.check([n + rounds])
        assert p.kv.get_error() == 0
        p.kv.close()
