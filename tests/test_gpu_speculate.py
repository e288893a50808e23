"""The example's loop: what it emits is what the target alone would choose."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(__file__), "..", "examples", "speculate.py")


@pytest.fixture(scope="module")
def speculate():
    spec = importlib.util.spec_from_file_location("speculate", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("window,sinks,page", [(0, 0, 64), (24, 2, 16)])
@pytest.mark.parametrize("group", [1, 4])
def test_greedy_rows_follow_the_target(speculate, window, sinks, page, group):
    """Along what was emitted, one token at a time and with no draft, each token's
    logit is the largest but for rounding.  The two passes round the same values
    to bf16 at five places a layer and at the end, 2^-9 of the values' size each:
    under 2^-4 of the largest logit together, twice over."""
    g = torch.Generator().manual_seed(group)
    prompts = [torch.randint(0, 512, (m,), generator=g).tolist() for m in (2, 17, 33, 80)]
    make = lambda: speculate.Target(group=group, batch=4, capacity=512, page=page, window=window, sinks=sinks)
    rows, rate = speculate.generate(make(), prompts, 40)
    assert rate > 1.2  # some drafts are accepted
    alone = make()
    n = [len(p) for p in prompts]
    longest = max(map(len, rows))
    for at in range(longest - 1):
        live = [b for b in range(4) if at + 1 < len(rows[b])]
        counts = torch.tensor([int(b in live) for b in range(4)], dtype=torch.int32)
        starts = torch.zeros(5, dtype=torch.int32)
        starts[1:] = counts.cumsum(0)
        lens = torch.tensor([min(at + 1, len(rows[b]) - 1) for b in range(4)], dtype=torch.int32)
        ids = torch.tensor([rows[b][at] for b in live], dtype=torch.int32)
        logits = alone(ids.cuda(), lens.cuda(), starts.cuda(), 1).float().cpu()
        for x, b in zip(logits, live):
            if at + 1 >= n[b]:
                assert x.max() - x[rows[b][at + 1]] <= 2.0 ** -4 * x.abs().max()
    assert alone.cache.get_error() == 0


def test_sampled_rows_stay_in_the_vocabulary(speculate):
    rows, rate = speculate.generate(speculate.Target(batch=3, capacity=512), [[5], [1, 2, 3], [7] * 40], 30,
                                    temperature=0.8)
    assert rate >= 1 and all(0 <= t < 512 for r in rows for t in r)
