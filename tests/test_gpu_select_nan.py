"""Key block selection where a NaN score is among the candidates, in the path that finds the list by histograms (more
than 32 candidates): a NaN score ranks last, behind minus infinity, and is listed when nothing else is left. The lists
lie in poisoned memory, so that an entry that is not written shows."""
import pytest
import torch

from gpu_helpers import require_gpu
from test_gpu_select_blocks import check, field

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("topk", [1, 20, 39, 40])
@pytest.mark.parametrize("bad", [{17: NAN}, {0: NAN, 39: NAN}, {3: -INF, 8: NAN, 30: INF}, {j: NAN for j in range(40)},
                                 {j: NAN for j in range(0, 40, 2)}])
def test_nan_key_blocks(topk, bad):
    require_gpu()
    q, k = field(1, 2, 300, 64, 1).abs(), field(1, 2, 64 * 40, 64, 2)
    for j, value in bad.items():
        k[:, :, 64 * j + 5, 7] = value
    blocks, counts = check(q, k, 64, topk)
    assert (counts == topk).all() and (blocks >= 0).all()


@pytest.mark.parametrize("topk", [5, 40])
@pytest.mark.parametrize("first,local", [(0, 0), (1, 1)])
def test_a_nan_query_row_lists_the_lowest_blocks(topk, first, local):
    """Every score of its block is NaN: all tie, behind the blocks that are always listed."""
    require_gpu()
    q, k = field(1, 2, 700, 128, 3), field(1, 1, 64 * 40, 128, 4)
    q[0, 1, 200] = NAN
    blocks, _ = check(q, k, 64, topk, first=first, local=local)
    if not local:
        assert (blocks[0, 1, 1] == torch.arange(topk, device="cuda")).all()


def test_opposite_infinities_in_a_block():
    """Their sum is NaN, as is that block's score."""
    require_gpu()
    q, k = field(1, 1, 128, 64, 5), field(1, 1, 64 * 50, 64, 6)
    k[0, 0, 64 * 20, 3], k[0, 0, 64 * 20 + 40, 3] = INF, -INF
    for topk in (49, 50):
        blocks, _ = check(q, k, 64, topk)
        assert (20 in blocks) == (topk == 50)


@pytest.mark.parametrize("topk", [33, 37, 60])
def test_clips_whose_candidates_are_all_listed(topk):
    """Clips with 60, 37 and 33 candidates, each with a NaN block."""
    require_gpu()
    kv_lens = [64 * 60, 64 * 37 - 5, 64 * 33]
    q, k = field(3, 2, 260, 64, 7), field(3, 2, 64 * 60, 64, 8)
    for b, n in enumerate(kv_lens):
        k[b, :, n - 1] = NAN
        k[b, :, n:] = INF
    _, counts = check(q, k, 64, topk, None, kv_lens)
    assert counts[:, 0, 0].tolist() == [min(topk, 60), min(topk, 37), min(topk, 33)]


def test_rows_of_scores_in_quarters():
    """More key blocks than sixteen rows of scores fit in shared memory."""
    require_gpu()
    q, k = field(1, 1, 600, 64, 9), field(1, 1, 64 * 1600, 64, 10)
    k[0, 0, 64 * 700] = NAN
    check(q, k, 64, 1600)
    check(q, k, 64, 1599)
