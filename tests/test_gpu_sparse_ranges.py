"""The selection over more candidates than shared memory holds at once (16,384), and with more pages chosen than its
lists hold (768, 1,024)."""
import pytest
import torch

from gpu_util import assert_close
from test_gpu_sparse import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dattn():
    import decode_attention_kv_dattn_gb300 as d
    return d


@pytest.fixture(scope="module")
def long():
    return Case(61, 4, 1, 128, 1, [40000, 20011, 3000], gate=False, r=32)


@pytest.mark.parametrize("num,first,last", [(40, 1, 2), (769, 0, 1), (900, 3, 5), (1027, 1, 2), (1500, 2, 1), (2900, 1, 1)])
def test_many_candidates_and_many_chosen(dattn, long, num, first, last):
    want = long.selection(num, first, last)
    out, sel = long.run(dattn, num, first, last, k=long.poison(want)[0], v=long.poison(want)[1])
    assert torch.equal(sel, want)
    assert_close(out.numpy(), long.attention(want).numpy())


@pytest.mark.parametrize("num", [50, 1200])
def test_many_equal_scores(dattn, num):
    """20,000 pages of three scores: the border lies among thousands of equal ones, and the lower pages win."""
    c = Case(62, 4, 1, 128, 1, [20000], gate=False, r=32)
    base = c.summary[0].clone()
    for i, f in enumerate((1.0, 0.5, 2.0)):
        rows = c.table[0, i::3][c.table[0, i::3] >= 0].long()
        c.summary[rows] = (base.float() * f).to(torch.bfloat16)
    assert torch.equal(c.run(dattn, num, 1, 2)[1], c.selection(num, 1, 2))


def test_scores_that_cancel_across_lanes(dattn):
    """Terms of 2^21 in dims 0 and 62, which cancel at the very end of a sum over lanes, and differences of 2^-12 in a dim
    that one of them is added to first: 24 bits lose those."""
    c = Case(63, 4, 2, 128, 16, [16 * 200], r=0)
    c.q[:] = 1.0
    c.q[..., 0] = 2.0
    s = torch.zeros_like(c.summary)
    s[..., 0], s[..., 62] = 2.0 ** 20, -(2.0 ** 21)
    order = torch.randperm(s.shape[0], generator=c.g)
    s[..., 2] = (order[:, None] - s.shape[0] // 2).float().to(torch.bfloat16) * 2.0 ** -12
    c.summary = s
    want = c.selection(16, 1, 1)
    assert want[0, 0].tolist() != list(range(16))
    assert torch.equal(c.run(dattn, 16, 1, 1)[1], want)
