"""Attention over listed key blocks against the softmax in 64 bits, element by element.

Tolerance of an element of o = sum_j p_j v_j / sum_j p_j, with A = sum_j p_j |v_j| / sum_j p_j:
  2^-8 A     each p_j is rounded to bf16 for the tensor core (the sum of the p_j is not)
  2^-11 A    the exponential (2^-13), its argument (a sum of 128 products in fp32 and the
             subtraction of the maximum: below 2^-13 for the scores here), the fp32 sums,
             each in numerator and denominator
  2^-8 |o|   the output's own rounding"""
import pytest
import torch

import operator_refs as R
from gpu_helpers import no_device_error, require_gpu
from video_diffusion_transformer_adaln_b200 import h3b

pytestmark = pytest.mark.gpu


def randn(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(torch.bfloat16)


def lists(B, H, nqb, nkb, topk, seed, counts=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    pick = torch.rand((B, H, nqb, nkb), generator=g, device="cuda").topk(topk, dim=-1).indices
    n = torch.randint(0, topk + 1, (B, H, nqb), generator=g, device="cuda").to(torch.int32) if counts else None
    return pick.sort(dim=-1).values.to(torch.int32), n


def run(q, k, v, blocks, counts, block_k, q_lens=None, kv_lens=None, absmax=True, stream=None):
    B, H, Lq, dh = q.shape
    d = h3b.make_sparse(B, H, k.shape[1], dh, Lq, k.shape[2], block_k, blocks.shape[-1])
    ws = torch.full((h3b.h3b_sparse_workspace_size(d),), 0xFF, dtype=torch.uint8, device="cuda")
    o = torch.full((B, Lq, H * dh), 9.0, dtype=torch.bfloat16, device="cuda")
    am = torch.zeros(B * Lq, device="cuda") if absmax else None
    h3b.h3b_attention_blocks(d, q, k, v, q_lens, kv_lens, blocks, counts, o, am, ws, stream=stream)
    return o, am, ws


def check(q, k, v, blocks, counts, block_k, q_lens=None, kv_lens=None):
    dev = [None if t is None else torch.tensor(t, dtype=torch.int32, device="cuda") for t in (q_lens, kv_lens)]
    o, am, _ = run(q, k, v, blocks, counts, block_k, *dev)
    ref, mag = R.attention_blocks(q, k, v, blocks, counts, block_k, q_lens, kv_lens)
    live = ~ref.isnan()
    assert (o[~live] == 9.0).all()  # rows behind q_lens are left as they were
    err = (o.double() - ref).abs()[live]
    tol = ((2.0 ** -8 + 2.0 ** -11) * mag + 2.0 ** -8 * ref.abs())[live]
    assert o[live].isfinite().all()
    assert (err <= tol).all(), ((err - tol).max().item(), int((err > tol).sum()))
    rows = live.all(-1).view(-1)
    want = torch.where(rows, o.view(rows.numel(), -1).abs().amax(-1).float(), 0.0)
    assert torch.equal(am, want)
    no_device_error()
    return o


@pytest.mark.parametrize("B,H,KV,dh,Lq,Lk,block_k,topk", [
    (1, 1, 1, 64, 1, 1, 64, 1),              # one query, one key
    (1, 4, 4, 64, 512, 512, 64, 4),          # the smallest workload's grid
    (1, 2, 2, 128, 512, 512, 64, 1),         # one block of 64 keys each
    (2, 4, 2, 128, 777, 777, 64, 5),         # an odd list, ragged tails
    (1, 6, 1, 64, 300, 2000, 128, 3),
    (3, 2, 1, 128, 1000, 130, 64, 2),
    (1, 3, 3, 64, 129, 4097, 64, 65),        # every block; one key in the last one
    (2, 8, 2, 128, 1, 5000, 64, 30),         # one new token: the list is split
    (1, 5, 5, 64, 100, 9000, 128, 70),
    (1, 1, 1, 128, 257, 20000, 64, 313),     # every key of a long latent
])
@pytest.mark.parametrize("counted", [False, True])
def test_matches_the_softmax(B, H, KV, dh, Lq, Lk, block_k, topk, counted):
    require_gpu()
    q, k, v = randn((B, H, Lq, dh), 1), randn((B, KV, Lk, dh), 2), randn((B, KV, Lk, dh), 3)
    nqb, nkb = -(-Lq // 128), -(-Lk // block_k)
    check(q, k, v, *lists(B, H, nqb, nkb, topk, 4, counted), block_k)


@pytest.mark.parametrize("dh,block_k", [(64, 64), (128, 64), (128, 128)])
def test_padded_items_and_garbage_behind_them(dh, block_k):
    require_gpu()
    B, H, KV, Lq, Lk = 6, 2, 1, 400, 500
    q, k, v = randn((B, H, Lq, dh), 5), randn((B, KV, Lk, dh), 6), randn((B, KV, Lk, dh), 7)
    q_lens, kv_lens = [400, 129, 0, 5000, 1, 128], [500, 1, 300, 0, -3, 65]
    for b in range(B):
        q[b, :, max(0, min(q_lens[b], Lq)):] = float("nan")
        k[b, :, max(0, kv_lens[b]):] = float("nan")
        v[b, :, max(0, kv_lens[b])::2] = float("inf")
        v[b, :, max(0, kv_lens[b]) + 1::2] = float("nan")
    nkb = -(-Lk // block_k)
    blocks, _ = lists(B, H, 4, nkb, nkb, 8)
    o = check(q, k, v, blocks, None, block_k, q_lens, kv_lens)
    assert (o[3] == 0).all() and (o[4, 0] == 0).all()
    blocks, counts = lists(B, H, 4, nkb, 3, 9)
    check(q, k, v, blocks, counts, block_k, q_lens, kv_lens)


@pytest.mark.parametrize("Lq", [300, 3, 2, 1])
def test_lists_that_hold_no_key_bad_entries_and_repeats(Lq):
    require_gpu()
    B, H, dh, Lk = 1, 2, 128, 1000
    nqb, nkb = -(-Lq // 128), 16
    q, k, v = randn((B, H, Lq, dh), 10), randn((B, H, Lk, dh), 11), randn((B, H, Lk, dh), 12)
    blocks = torch.full((B, H, nqb, 16), -1, dtype=torch.int32, device="cuda")
    blocks[0, 0, :, :5] = torch.tensor([nkb, -1, 2 ** 31 - 1, -2 ** 31, 3], device="cuda")  # one entry holds keys
    if nqb > 1:
        blocks[0, 0, 1, :6] = torch.tensor([5, 5, 5, 15, 15, 4], device="cuda")  # repeats, descending order
    o = check(q, k, v, blocks, None, 64)
    assert (o[:, :, dh:] == 0).all()  # head 1 lists nothing
    counts = torch.tensor([[99] * nqb, [-5] * nqb], dtype=torch.int32, device="cuda")[None]
    check(q, k, v, blocks, counts, 64)


@pytest.mark.parametrize("rise", [True, False])
def test_scores_that_jump_between_blocks(rise):
    """Each listed block's scores lie far above (below) those before it: the running maximum moves at
    every block (never)."""
    require_gpu()
    B, H, dh, L = 1, 1, 64, 640
    q, k, v = randn((B, H, L, dh), 13, 0.1), randn((B, H, L, dh), 14, 0.1), randn((B, H, L, dh), 15)
    step = torch.arange(L, device="cuda") // 64
    q[..., 0] = 4.0
    k[..., 0] = ((step if rise else 9 - step) * 16).to(torch.bfloat16)
    nqb, nkb = 5, 10
    blocks, _ = lists(B, H, nqb, nkb, nkb, 16)
    check(q, k, v, blocks, None, 64)


def test_large_scores():
    require_gpu()
    B, H, dh, L = 1, 2, 128, 512
    q, k, v = randn((B, H, L, dh), 17, 4.0), randn((B, H, L, dh), 18, 4.0), randn((B, H, L, dh), 19)
    # scores up to about 100 from products that sum to about 115 in magnitude: 115 * log2(e) * 2^-21 < 2^-13
    blocks, counts = lists(B, H, 4, 8, 6, 20)
    check(q, k, v, blocks, counts, 64)


def test_infinite_and_nan_inputs_stay_with_their_queries():
    require_gpu()
    B, H, dh, L = 1, 2, 64, 300
    q, k, v = randn((B, H, L, dh), 21), randn((B, H, L, dh), 22), randn((B, H, L, dh), 23)
    blocks, _ = lists(B, H, 3, 5, 3, 24)
    clean, _, _ = run(q, k, v, blocks, None, 64)
    q[0, 0, 5] = float("nan")
    got, _, _ = run(q, k, v, blocks, None, 64)
    same = torch.ones(L, dtype=torch.bool, device="cuda")
    same[5] = False
    assert got[0, 5, :dh].isnan().all()
    assert torch.equal(got[0, same], clean[0, same]) and torch.equal(got[0, 5, dh:], clean[0, 5, dh:])


def test_lists_of_the_selection():
    """All key blocks listed gives the library's dense attention within the two tolerances' sum."""
    require_gpu()
    B, H, dh, L = 2, 2, 128, 500
    q, k, v = randn((B, H, L, dh), 25), randn((B, H, L, dh), 26), randn((B, H, L, dh), 27)
    blocks = torch.arange(8, dtype=torch.int32, device="cuda").expand(B, H, 4, 8).contiguous()
    o = check(q, k, v, blocks, None, 64)
    dense = torch.empty_like(o)
    am = torch.zeros(B * L, device="cuda")
    dims = h3b.make_dims(B, 1, 1, L, H * dh, H, dh, 256, (0, 0, dh))
    h3b.h3b_attention(dims, torch.stack([q, k, v]), dense, am)
    _, mag = R.attention_blocks(q, k, v, blocks, None, 64)
    tol = 2 * (2.0 ** -8 + 2.0 ** -11) * mag + 2.0 ** -7 * dense.double().abs()
    assert ((o.double() - dense.double()).abs() <= tol).all()


@pytest.mark.parametrize("Lq,Lk,topk", [(700, 700, 5), (3, 6000, 60), (1, 6000, 60)])
def test_streams_graphs_and_repeats_are_bit_equal(Lq, Lk, topk):
    require_gpu()
    B, H, KV, dh = 2, 4, 2, 128
    q, k, v = randn((B, H, Lq, dh), 28), randn((B, KV, Lk, dh), 29), randn((B, KV, Lk, dh), 30)
    nqb, nkb = -(-Lq // 128), -(-Lk // 64)
    blocks, counts = lists(B, H, nqb, nkb, topk, 31)
    want, want_am, _ = run(q, k, v, blocks, counts, 64)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(run(q, k, v, blocks, counts, 64, stream=s))
    torch.cuda.synchronize()
    for o, am, _ in got:
        assert torch.equal(o, want) and torch.equal(am, want_am)
    o, am, ws = got[0]
    d = h3b.make_sparse(B, H, KV, dh, Lq, Lk, 64, topk)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        am.zero_()
        h3b.h3b_attention_blocks(d, q, k, v, None, None, blocks, counts, o, am, ws)
    v.copy_(v.flip(2))
    want, want_am, _ = run(q, k, v, blocks, counts, 64)
    for _ in range(2):
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(am, want_am)


def test_workspace_size_is_enough():
    require_gpu()
    B, H, KV, dh, Lq, Lk, topk = 2, 4, 1, 64, 3, 9000, 100
    q, k, v = randn((B, H, Lq, dh), 32), randn((B, KV, Lk, dh), 33), randn((B, KV, Lk, dh), 34)
    blocks, counts = lists(B, H, 1, 141, topk, 35)
    want, _, _ = run(q, k, v, blocks, counts, 64, absmax=False)
    d = h3b.make_sparse(B, H, KV, dh, Lq, Lk, 64, topk)
    need = h3b.h3b_sparse_workspace_size(d)
    buf = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    o = torch.full((B, Lq, H * dh), 9.0, dtype=torch.bfloat16, device="cuda")
    h3b.h3b_attention_blocks(d, q, k, v, None, None, blocks, counts, o, None, buf[:need])
    assert torch.equal(o, want) and (buf[need:] == 0xA5).all()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("Lq", [200, 5, 1])
def test_a_bad_key_reaches_every_query_that_lists_it(value, Lq):
    """A NaN or infinite score makes the formula's row NaN, wherever in its tile the key lies."""
    require_gpu()
    B, H, dh, Lk = 1, 1, 128, 3000
    nqb, nkb = -(-Lq // 128), 47
    q, v = randn((B, H, Lq, dh), 36).abs(), randn((B, H, Lk, dh), 37)
    blocks, _ = lists(B, H, nqb, nkb, 20, 38)
    blocks[0, 0, 0, 7] = int(blocks[0, 0, 0, 6])
    bad = int(blocks[0, 0, 0, 7])
    for lane in (0, 6, 7, 63):
        k = randn((B, H, Lk, dh), 39)
        k[0, 0, min(bad * 64 + lane, Lk - 1)] = value
        o, _, _ = run(q, k, v, blocks, None, 64)
        has = (blocks[0, 0] == bad).any(-1).repeat_interleave(128)[:Lq]
        assert o[0, has].isnan().all() and o[0, ~has].isfinite().all()


@pytest.mark.parametrize("dh,block_k,kv_lens", [(128, 64, None), (64, 64, [1900, 777, 64]), (128, 64, [1999, 130, 1]),
                                                (128, 128, [1500, 2000, 0])])
def test_more_pairs_of_query_blocks_than_processors(dh, block_k, kv_lens):
    """Lists of every length, empty ones among them, on CTAs that work on several pairs in turn."""
    require_gpu()
    B, H, KV, Lq, Lk = 3, 32, 8, 1024, 2000
    q, k, v = randn((B, H, Lq, dh), 40), randn((B, KV, Lk, dh), 41), randn((B, KV, Lk, dh), 42)
    nkb = -(-Lk // block_k)
    blocks, counts = lists(B, H, 8, nkb, nkb, 43)
    if kv_lens:
        for b in range(B):
            k[b, :, kv_lens[b]:] = float("nan")
            v[b, :, kv_lens[b]:] = float("nan")
    check(q, k, v, blocks, counts, block_k, None, kv_lens)
    check(q, k, v, blocks[..., :3].contiguous(), None, block_k, [1024, 1000, 1], kv_lens)


@pytest.mark.parametrize("Lq", [1, 2, 3, 9])
@pytest.mark.parametrize("B,H,KV,dh,Lk,block_k,topk", [
    (4, 40, 8, 128, 3000, 64, 20),
    (1, 2, 1, 64, 100, 64, 2),
    (3, 5, 5, 64, 9001, 128, 71),
    (1, 1, 1, 128, 64 * 600, 64, 600),
    (300, 1, 1, 128, 130, 64, 3),
])
def test_few_queries(Lq, B, H, KV, dh, Lk, block_k, topk):
    """A few new tokens of each stream over long and short latents, padded items among them."""
    require_gpu()
    q, k, v = randn((B, H, Lq, dh), 44), randn((B, KV, Lk, dh), 45), randn((B, KV, Lk, dh), 46)
    nkb = -(-Lk // block_k)
    blocks, counts = lists(B, H, 1, nkb, topk, 47)
    check(q, k, v, blocks, None, block_k)
    kv_lens = [(Lk - 37 * b) % (Lk + 1) for b in range(B)]
    q_lens = [Lq - b % 2 for b in range(B)]
    for b in range(B):
        k[b, :, kv_lens[b]:] = float("nan")
        v[b, :, kv_lens[b]:] = float("inf")
    check(q, k, v, blocks, counts, block_k, q_lens, kv_lens)


@pytest.mark.parametrize("Lq", [200, 5, 1])
@pytest.mark.parametrize("lane", [0, 63, 127])
def test_absmax_of_a_row_with_a_nan(Lq, lane):
    """One lane of a value is NaN: the rows that list it have a NaN there and as their largest magnitude."""
    require_gpu()
    B, H, dh, Lk = 2, 2, 128, 3000
    nqb, nkb = -(-Lq // 128), 47
    q, k, v = randn((B, H, Lq, dh), 48), randn((B, H, Lk, dh), 49), randn((B, H, Lk, dh), 50)
    blocks, _ = lists(B, H, nqb, nkb, 20, 51)
    v[0, 1, 64 * int(blocks[0, 1, 0, 9]) + 3, lane] = float("nan")
    o, am, _ = run(q, k, v, blocks, None, 64)
    rows = o.view(B * Lq, -1).isnan().any(-1)
    assert rows[0] and not rows[Lq:].any()
    assert torch.equal(am.isnan(), rows)
    assert torch.equal(am[~rows], o.view(B * Lq, -1)[~rows].abs().amax(-1).float())
