"""The sums behind the block means in 64 bits: lists that hang on what a sum in 32 bits loses. The rows' sums below are
exact in 64 bits, whatever the order of a block's rows, so that the lists are known exactly."""
import pytest
import torch

from gpu_helpers import require_gpu
from test_gpu_select_blocks import check, field, run

pytestmark = pytest.mark.gpu


def shuffled(rows, seed):
    """Each block's rows [blocks][rows][lanes] in an order of its own."""
    g = torch.Generator().manual_seed(seed)
    order = torch.rand(rows.shape[:2], generator=g).argsort(-1)
    return rows.gather(1, order[..., None].expand_as(rows)).reshape(1, 1, -1, rows.shape[-1]).to("cuda", torch.bfloat16)


@pytest.mark.parametrize("dh,block_k", [(64, 64), (128, 64), (64, 128), (128, 128)])
def test_blocks_of_the_same_rows_tie(dh, block_k):
    """The same rows in another order have the same mean: the lower blocks are listed. The rows are normal values on a
    grid of 2^-30, so that their sums have at most 41 bits."""
    require_gpu()
    g = torch.Generator().manual_seed(1)
    rows = torch.randn((block_k, dh), generator=g, dtype=torch.float64)
    rows[: block_k // 2] *= 2.0 ** -18
    rows = rows.to(torch.bfloat16).double()
    rows = (rows * 2.0 ** 30).round() / 2.0 ** 30
    rows = rows.to(torch.bfloat16).double()
    assert torch.equal((rows * 2.0 ** 30).round() / 2.0 ** 30, rows)
    for n in (20, 50):  # a key per lane, and the histograms
        k = shuffled(rows.expand(n, -1, -1).contiguous(), n)
        q = field(1, 4, 400, dh, 2)
        for topk in (3, n - 1):
            blocks, counts, _ = run(q, k, block_k, topk)
            assert (blocks == torch.arange(topk, dtype=torch.int32, device="cuda")).all() and (counts == topk).all()


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("big,small", [(1.0, 2.0 ** -30), (2.0 ** 10, 2.0 ** -24), (1.0, 2.0 ** -24)])
def test_small_rows_beside_large_ones_decide(dh, big, small):
    """Half of a block's rows hold `big`, half c_j * small: the order of the blocks is that of c_j."""
    require_gpu()
    n = 45
    c = torch.randperm(n, generator=torch.Generator().manual_seed(3)) + 1
    rows = torch.zeros((n, 64, dh), dtype=torch.float64)
    rows[:, :32, 0] = big
    rows[:, 32:, 0] = small * c[:, None]
    q = torch.zeros((1, 1, 128, dh), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    for topk in (1, 9, 44):
        blocks, _ = check(q, shuffled(rows, 4), 64, topk)
        assert blocks[0, 0, 0].tolist() == sorted(c.argsort(descending=True)[:topk].tolist())


@pytest.mark.parametrize("big", [2.0 ** 15, 2.0 ** 30, 2.0 ** 40])
def test_large_rows_that_cancel(big):
    """Rows of +big and -big leave the sum of the others: sums of at most 2^44 in units of 2^-7, 52 bits."""
    require_gpu()
    n, dh = 40, 128
    c = torch.randperm(n, generator=torch.Generator().manual_seed(5)) + 1
    rows = torch.zeros((n, 64, dh), dtype=torch.float64)
    rows[:, :16, 0], rows[:, 16:32, 0] = big, -big
    rows[:, 32:, 0] = c[:, None] / 128.0
    q = torch.zeros((1, 1, 128, dh), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    blocks, _ = check(q, shuffled(rows, 6), 64, 7)
    assert blocks[0, 0, 0].tolist() == sorted(c.argsort(descending=True)[:7].tolist())


def test_the_same_for_query_rows():
    """The queries' means: lane 0 cancels to what decides against lane 1."""
    require_gpu()
    dh, nqb = 64, 6
    rows = torch.zeros((nqb, 128, dh), dtype=torch.float64)
    rows[:, :32, 0], rows[:, 32:64, 0] = 2.0 ** 30, -2.0 ** 30
    rows[:, 64:, 0] = torch.arange(nqb, dtype=torch.float64)[:, None] / 4  # a mean of i / 8
    rows[..., 1] = -0.25
    k = torch.zeros((1, 1, 128, dh), dtype=torch.bfloat16, device="cuda")
    k[0, 0, 64:, 0] = 1.0
    k[0, 0, 64:, 1] = 1.0  # block 1 scores i / 8 - 1 / 4, block 0 scores 0: block 1 from i = 3 on, the tie goes to 0
    blocks, _ = check(shuffled(rows, 7), k, 64, 1)
    assert blocks.flatten().tolist() == [0, 0, 0, 1, 1, 1]


@pytest.mark.parametrize("dh", [64, 128])
def test_values_whose_sum_leaves_32_bits(dh):
    """Every row of a block near the largest value of the type: the sum of two is infinite in 32 bits."""
    require_gpu()
    n = 40
    c = torch.randperm(n, generator=torch.Generator().manual_seed(8))
    rows = torch.zeros((n, 64, dh), dtype=torch.float64)
    rows[..., 0] = 2.0 ** 127 * (1 + c[:, None] / 128.0)
    q = torch.zeros((1, 1, 128, dh), dtype=torch.bfloat16, device="cuda")
    for sign in (1.0, -1.0):
        q[..., 0] = sign * 2.0 ** 100
        blocks, _ = check(q, shuffled(rows, 9), 64, 5)
        assert blocks[0, 0, 0].tolist() == sorted(c.argsort(descending=sign > 0)[:5].tolist())


@pytest.mark.parametrize("dh", [64, 128])
def test_the_smallest_values(dh):
    """Subnormal values, whole multiples of 2^-133, beside zeros and minus zeros."""
    require_gpu()
    n = 40
    c = torch.randperm(n, generator=torch.Generator().manual_seed(10)) + 1
    rows = torch.zeros((n, 64, dh), dtype=torch.float64)
    rows[:, :60, 0], rows[:, 60:, 0] = (2.0 ** -133 * c)[:, None], -0.0
    q = torch.zeros((1, 1, 128, dh), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 2.0 ** -120
    blocks, _ = check(q, shuffled(rows, 11), 64, 6)
    assert blocks[0, 0, 0].tolist() == sorted(c.argsort(descending=True)[:6].tolist())
