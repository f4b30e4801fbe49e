"""The key block selection against scores formed in 64 bits: whole numbers, equal entry by entry.
Scores of these inputs differ by far more than 64-bit sums can be off; equal scores (repeated keys,
zero rows) are equal in both and go to the lower block."""
import pytest
import torch

import operator_refs as R
from gpu_helpers import no_device_error, require_gpu
from video_diffusion_transformer_adaln_b200 import h3b

pytestmark = pytest.mark.gpu


def field(B, H, L, dh, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    base = torch.randn((B, H, -(-L // 50), dh), generator=g, device="cuda")
    return (torch.randn((B, H, L, dh), generator=g, device="cuda")
            + base.repeat_interleave(50, dim=2)[:, :, :L]).to(torch.bfloat16)


def run(q, k, block_k, topk, q_lens=None, kv_lens=None, first=0, local=0, stream=None):
    B, H, Lq, dh = q.shape
    d = h3b.make_sparse(B, H, k.shape[1], dh, Lq, k.shape[2], block_k, topk, first, local)
    ws = torch.full((h3b.h3b_sparse_workspace_size(d),), 0xFF, dtype=torch.uint8, device="cuda")
    blocks = torch.full((B, H, d.nqb, topk), -7, dtype=torch.int32, device="cuda")
    counts = torch.full((B, H, d.nqb), -7, dtype=torch.int32, device="cuda")
    h3b.h3b_select_blocks(d, q, k, q_lens, kv_lens, blocks, counts, ws, stream=stream)
    return blocks, counts, ws


def check(q, k, block_k, topk, q_lens=None, kv_lens=None, first=0, local=0):
    lens = [None if t is None else torch.tensor(t, dtype=torch.int32, device="cuda") for t in (q_lens, kv_lens)]
    blocks, counts, _ = run(q, k, block_k, topk, *lens, first, local)
    rb, rc = R.select_blocks(q.cpu(), k.cpu(), block_k, topk, q_lens, kv_lens, first, local)
    assert torch.equal(counts.cpu(), rc)
    assert torch.equal(blocks.cpu(), rb)
    no_device_error()
    return blocks, counts


@pytest.mark.parametrize("B,H,KV,dh,Lq,Lk,block_k,topk", [
    (1, 1, 1, 64, 1, 1, 64, 1),            # one token
    (1, 4, 4, 64, 512, 512, 64, 4),
    (2, 4, 2, 128, 777, 777, 64, 5),       # ragged tails of both sides
    (1, 6, 2, 128, 300, 2000, 128, 3),     # more keys than queries
    (3, 2, 1, 64, 1000, 130, 64, 2),       # fewer keys than queries
    (1, 1, 1, 128, 129, 4097, 64, 64),     # one row behind a block, one key behind a block
    (1, 2, 2, 64, 64, 640, 128, 5),        # every key block is listed
    (1, 1, 1, 64, 130, 40000, 64, 50),     # 625 key blocks
])
def test_matches_the_scores(B, H, KV, dh, Lq, Lk, block_k, topk):
    require_gpu()
    check(field(B, H, Lq, dh, 1), field(B, KV, Lk, dh, 2), block_k, topk)


@pytest.mark.parametrize("block_k", [64, 128])
@pytest.mark.parametrize("first,local", [(2, 0), (0, 1), (1, 2), (3, 1)])
def test_kept_blocks(block_k, first, local):
    require_gpu()
    check(field(1, 3, 1100, 64, 3), field(1, 3, 1100, 64, 4), block_k, 7, first=first, local=local)


def test_padded_items_empty_items_and_lengths_out_of_range():
    require_gpu()
    q, k = field(5, 2, 700, 64, 5), field(5, 2, 900, 64, 6)
    q_lens, kv_lens = [700, 129, 0, 5000, 1], [900, 1, 640, 0, -3]
    for b in range(5):  # rows behind the valid ones hold anything
        q[b, :, min(q_lens[b], 700):] = float("nan")
        k[b, :, max(0, kv_lens[b]):] = float("inf")
    blocks, counts = check(q, k, 64, 6, q_lens, kv_lens, first=1)
    assert counts[2].sum() == 0 and counts[3].sum() == 0 and counts[4].sum() == 0
    assert (blocks[1, :, 0] == torch.tensor([0, -1, -1, -1, -1, -1], device="cuda")).all()


def test_equal_scores_go_to_the_lower_block():
    require_gpu()
    q = field(1, 1, 256, 64, 7)
    k = field(1, 1, 64, 64, 8).repeat(1, 1, 9, 1).contiguous()  # nine equal blocks
    blocks, _ = check(q, k, 64, 4)
    assert (blocks == torch.arange(4, device="cuda")).all()
    k[:, :, 64 * 5:64 * 6] = 0  # a score of zero, minus zeros among its terms
    check(q, k, 64, 4)
    check(torch.zeros_like(q), k, 64, 4)


def test_non_finite_scores():
    """An infinite score ranks where it belongs, a NaN one last, and only NaN ones are left out."""
    require_gpu()
    q, k = field(1, 1, 128, 64, 9).abs(), field(1, 1, 640, 64, 10)
    k[0, 0, 130] = float("inf")     # block 2: +inf
    k[0, 0, 200] = float("-inf")    # block 3: -inf
    k[0, 0, 300] = float("nan")     # block 4: NaN
    blocks, _ = check(q, k, 64, 8)
    assert 2 in blocks and 4 not in blocks
    check(q, k, 64, 1)
    blocks, _ = check(q, k, 64, 10)
    assert 4 in blocks


def test_values_of_every_size():
    """Rows whose values span 2^-60 to 2^60: sums of the means hold in 64 bits."""
    require_gpu()
    g = torch.Generator(device="cuda").manual_seed(11)
    e = torch.randint(-60, 61, (1, 2, 500, 1), generator=g, device="cuda").float()
    check((field(1, 2, 500, 64, 12) * 2.0 ** e).to(torch.bfloat16), field(1, 2, 500, 64, 13), 64, 3)
    check(field(1, 2, 500, 64, 12), (field(1, 2, 500, 64, 13) * 2.0 ** e).to(torch.bfloat16), 128, 2)


def test_two_calls_at_once_and_a_replayed_graph():
    require_gpu()
    q, k = field(2, 4, 1500, 128, 14), field(2, 4, 1500, 128, 15)
    d = h3b.make_sparse(2, 4, 4, 128, 1500, 1500, 64, 6)
    want, want_n, _ = run(q, k, 64, 6)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:  # each with a workspace of its own
        with torch.cuda.stream(s):
            got.append(run(q, k, 64, 6, stream=s))
    torch.cuda.synchronize()
    for b, n, _ in got:
        assert torch.equal(b, want) and torch.equal(n, want_n)
    b, n, ws = got[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h3b.h3b_select_blocks(d, q, k, None, None, b, n, ws)
    q.copy_(q.flip(2))
    want, want_n, _ = run(q, k, 64, 6)
    for _ in range(2):
        b.zero_(), n.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(b, want) and torch.equal(n, want_n)


def test_workspace_size_is_enough():
    require_gpu()
    q, k = field(2, 2, 300, 64, 16), field(2, 1, 700, 64, 17)
    d = h3b.make_sparse(2, 2, 1, 64, 300, 700, 64, 3)
    need = h3b.h3b_sparse_workspace_size(d)
    buf = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    blocks = torch.empty((2, 2, d.nqb, 3), dtype=torch.int32, device="cuda")
    counts = torch.empty((2, 2, d.nqb), dtype=torch.int32, device="cuda")
    h3b.h3b_select_blocks(d, q, k, None, None, blocks, counts, buf[:need])
    assert (buf[need:] == 0xA5).all()


def test_many_key_blocks():
    """More key blocks than 16 rows of scores fit in shared memory."""
    require_gpu()
    check(field(1, 1, 700, 64, 18), field(1, 1, 64 * 1537, 64, 19), 64, 100, local=1)
    check(field(1, 2, 130, 128, 20), field(1, 1, 64 * 1536, 128, 21), 64, 9)


@pytest.mark.parametrize("other", [0.5, 0.25, 2.0 ** -9, 2.0 ** -60, 0.0, -1.0])
@pytest.mark.parametrize("topk", [1, 7, 30, 59])
def test_scores_units_in_the_last_place_apart(other, topk):
    """Scores 1 + c 2^-52, exact in 64 bits, are told apart whatever the spread of all scores is."""
    require_gpu()
    nkb = 60
    q, k = (torch.zeros((1, 1, n, 64), dtype=torch.bfloat16, device="cuda") for n in (128, 64 * nkb))
    q[..., 0], q[..., 1] = 1.0, 2.0 ** -52
    c = torch.randperm(nkb, generator=torch.Generator().manual_seed(topk)) * 4
    k[..., 0] = 1.0
    k[..., 1] = c.repeat_interleave(64).to(device="cuda", dtype=torch.bfloat16)
    k[:, :, 64 * 31:64 * 32, 0] = other
    check(q, k, 64, topk)


@pytest.mark.parametrize("H,KV,Lq,Lk,q_lens,kv_lens", [
    (6, 2, 300, 1300, None, None), (4, 1, 1300, 300, None, None), (2, 2, 900, 900, [900, 200], [130, 900])])
def test_kept_blocks_of_shared_heads_and_unequal_lengths(H, KV, Lq, Lk, q_lens, kv_lens):
    require_gpu()
    check(field(2, H, Lq, 128, 22), field(2, KV, Lk, 128, 23), 64, 5, q_lens, kv_lens, first=1, local=2)
