"""dattn_summarize with a bound on the new tokens far above what a table holds: the grid follows the table."""
import pytest
import torch

from test_gpu_sparse import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dattn():
    import decode_attention_kv_dattn_gb300 as d
    return d


@pytest.mark.parametrize("P", [1, 16, 24])
def test_a_bound_without_end(dattn, P):
    lens = [40 * P, 7 * P + P // 2]
    c = Case(50 + P, 8, 2, 128, P, lens)
    h = c.handle(dattn, 1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    kd = c.k.cuda()
    cache = dattn.paged_cache(kd, kd, c.table.cuda(), i32(lens))
    want, got = (torch.full((kd.shape[0], 2, 128), -5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    start = i32([3 * P - 1 if P > 1 else 3, 0])
    count = i32([37 * P, 7 * P + P // 2])
    h.summarize(0, cache, want, start, count, max_tokens=40 * P)
    assert h.get_error() == dattn.OK
    h.summarize(0, cache, got, start, count, max_tokens=2 ** 31 - 1)
    assert h.get_error() == dattn.OK
    assert torch.equal(got, want)
    # pages behind the table are reported, those in it written
    got.fill_(-5.0)
    h.summarize(0, cache, got, start, i32([10 ** 9, 7 * P + P // 2]), max_tokens=2 ** 31 - 1)
    assert h.get_error() == dattn.EINDEX
    rows = c.table[1, :7].long().cuda()
    assert torch.equal(got[rows], want[rows])
    # the last tokens that an int32 counts
    h.summarize(0, cache, got, i32([2 ** 31 - 30 * P, 0]), i32([25 * P, 0]), max_tokens=2 ** 31 - 1)
    assert h.get_error() == dattn.EINDEX
    # nothing completed: nothing behind the table either
    h.summarize(0, cache, got, i32([60 * P, 0]), i32([P - 1, 0]), max_tokens=2 ** 31 - 1)
    assert h.get_error() == dattn.OK
