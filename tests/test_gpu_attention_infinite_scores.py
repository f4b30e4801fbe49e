"""Attention over listed key blocks: keys that score minus infinity have no weight, wherever in the list they lie, and a
query all of whose keys do gets zeros; values as large as the header allows."""
import pytest
import torch

import operator_refs as R
from gpu_helpers import require_gpu
from test_gpu_attention_blocks import check, lists, randn, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Lq", [200, 5, 1])
@pytest.mark.parametrize("dh", [64, 128])
def test_keys_that_score_minus_infinity(Lq, dh):
    require_gpu()
    B, H, Lk, topk = 1, 2, 3000, 20
    q, k, v = randn((B, H, Lq, dh), 1), randn((B, H, Lk, dh), 2), randn((B, H, Lk, dh), 3)
    q[..., 0] = q[..., 0].abs() + 1
    blocks, _ = lists(B, H, -(-Lq // 128), 47, topk, 4)
    g = torch.Generator(device="cuda").manual_seed(5)
    gone = torch.rand((B, H, Lk), generator=g, device="cuda") < 0.5
    for b in blocks[0, 0, 0, :3].tolist():  # whole blocks at the start of a list
        gone[0, 0, 64 * b:64 * b + 64] = True
    k[..., 0][gone] = float("-inf")
    check(q, k, v, blocks, None, 64)


@pytest.mark.parametrize("Lq", [200, 5, 1])
def test_only_such_keys(Lq):
    require_gpu()
    B, H, dh, Lk = 1, 2, 128, 3000
    q, k, v = randn((B, H, Lq, dh), 6), randn((B, H, Lk, dh), 7), randn((B, H, Lk, dh), 8)
    q[..., 0] = q[..., 0].abs() + 1
    k[:, 0, :, 0] = float("-inf")
    blocks, _ = lists(B, H, -(-Lq // 128), 47, 20, 9)
    o, am, _ = run(q, k, v, blocks, None, 64)
    assert (o[..., :dh] == 0).all()
    ref, mag = R.attention_blocks(q[:, 1:], k[:, 1:], v[:, 1:], blocks[:, 1:].contiguous(), None, 64)
    # the tolerance of the attention's own tests: P's rounding, the exponentials and sums, the output's rounding
    assert ((o[..., dh:].double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -11) * mag + 2.0 ** -8 * ref.abs()).all()
    assert torch.equal(am, o.view(B * Lq, -1).abs().amax(-1).float())


@pytest.mark.parametrize("Lq", [640, 9, 1])
@pytest.mark.parametrize("step", [0.0, 12.0])
def test_large_values(Lq, step):
    """Values of 2^90: finite where a running maximum lags behind the scores by as much as it may (`step` raises the
    scores of each listed block by log2(e) * step / 2 = 8.7 powers of two)."""
    require_gpu()
    B, H, dh, Lk = 1, 1, 64, 1280
    q, k, v = randn((B, H, Lq, dh), 10, 0.1), randn((B, H, Lk, dh), 11, 0.1), randn((B, H, Lk, dh), 12)
    q[..., 0] = 1.0
    k[..., 0] = (torch.arange(Lk, device="cuda") // 64 * 4 * step).to(torch.bfloat16)
    v = (v.sign() * 2.0 ** 90).to(torch.bfloat16)
    blocks, _ = lists(B, H, -(-Lq // 128), 20, 20, 13)
    check(q, k, v, blocks, None, 64)
