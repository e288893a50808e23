"""What the cache's calls report, and what they give, for rows that ask for what is not there."""
import pytest
import torch

from test_gpu_kv_cache import KV, Pair  # noqa: F401 (KV: the fixture)

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


@pytest.mark.parametrize("max_q", [1, 20])     # (units of up to 16 rows, and of more)
@pytest.mark.parametrize("starts", [[0, 0, 25], [0, 0, -2], [-3, -3, 12], [12, 11, 11], [0, 50, 50]])
def test_attend_reports_starts_when_no_row_has_work(KV, starts, max_q):
    from model_free_suffix_gb300 import _lib as L
    p = Pair(KV, [40, 40], P=16, H=2, D=64, G=2)
    p.write([40, 40], [40, 40])
    q = torch.ones(20, 4, 64, dtype=torch.bfloat16).cuda()
    out = torch.full((20, 4, 64), 7.0, dtype=torch.bfloat16).cuda()
    p.kv.attend(q, p.dev_table, _i32([40, 40]), _i32(starts), max_q, out=out)
    assert p.kv.get_error(clear=True) == L.KV_ERR_LENGTH
    assert bool((out == 7).all())
    p.kv.attend(q, p.dev_table, _i32([40, 40]), _i32([0, 0, 0]), max_q, out=out)
    assert p.kv.get_error() == 0
    p.kv.close()


@pytest.mark.parametrize("B", [2, 40])         # (up to 32 rows are searched by one warp)
def test_read_before_the_first_position_gives_zeros(KV, B):
    from model_free_suffix_gb300 import _lib as L
    lens = [40] * B
    p = Pair(KV, lens, P=16, H=2, D=64)
    p.write(lens, lens)
    out = tuple(torch.full((3 * B, 2, 64), 7.0, dtype=torch.float32).cuda() for _ in range(2))
    first = [4] * B
    first[1] = -1
    p.kv.read(p.dev_table, _i32(first), _i32([3 * b for b in range(B + 1)]), out=out)
    assert p.kv.get_error(clear=True) & L.KV_ERR_LENGTH
    for name, got in zip("kv", out):
        for b in range(B):
            want = torch.zeros(3, 2, 64).double() if b == 1 else p.ref.rows(name, p.table[b], 4, 7)
            assert torch.equal(got[3 * b:3 * b + 3].cpu().double(), want)
    p.kv.close()
