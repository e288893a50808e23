"""The example of a server's steps runs, and gives its pages back."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(__file__), "..", "examples", "prompts.py")


@pytest.fixture(scope="module")
def prompts():
    spec = importlib.util.spec_from_file_location("prompts", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("rows,chunk,page", [(3, 64, 16), (5, 300, 64), (1, 7, 32)])
def test_requests_are_served_and_pages_come_back(prompts, rows, chunk, page):
    g = torch.Generator().manual_seed(rows)
    requests = [(torch.randint(0, 512, (int(n),), generator=g).tolist(), 1 + int(n) % 5)
                for n in torch.randint(1, 400, (7,), generator=g)]
    server = prompts.Server(rows, room=512, chunk=chunk, page=page)
    out, steps = server.serve(requests)
    assert sorted(map(len, out)) == sorted(r[1] for r in requests)
    assert all(0 <= t < 512 for row in out for t in row)
    assert server.pages.free_count.item() == server.cache.cfg.num_pages
    assert sorted(server.pages.free.tolist()) == list(range(server.cache.cfg.num_pages))
    assert bool((server.pages.block_table == -1).all()) and bool((server.pages.held == 0).all())


def test_a_prompt_in_one_chunk_is_the_prompt_s_attention(prompts):
    """Its first token is chosen from keys and values that no rounding to 8 bits has touched: the same with
    attend_prompt in attend_chunk's place."""
    prompt = torch.randint(0, 512, (333,), generator=torch.Generator().manual_seed(5)).tolist()
    first = prompts.Server(1, chunk=512).serve([(prompt, 1)])[0]
    other = prompts.Server(1, chunk=512)
    whole = other.cache.attend_prompt
    other.cache.attend_chunk = lambda q, k, v, table, lens, starts, layer: whole(q, k, v, starts)
    assert other.serve([(prompt, 1)])[0] == first
