"""Lanes that no axis rotates pass as they are: beside an infinity, and minus zeros with their sign. Without weights
they are a copy, bit for bit, whatever else the head holds (a NaN stays a NaN)."""
import pytest
import torch

import operator_refs as R
from gpu_helpers import require_gpu
from video_diffusion_transformer_adaln_b200 import h3b

pytestmark = pytest.mark.gpu


def make(B, L, H, KV, dh, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn((B * L, (H + 2 * KV) * dh), generator=g, device="cuda").to(torch.bfloat16)
    pick = torch.randint(0, 12, qkv.shape, generator=g, device="cuda")
    for n, value in enumerate((float("inf"), float("-inf"), -0.0, 0.0)):
        qkv[pick == n] = value
    pos = 40 * torch.rand((B, L, 3), generator=g, device="cuda")
    return qkv, pos


def run(qkv, B, L, H, KV, dh, rope, wq, wk, pos):
    out = [torch.full((B, h, L, dh), 7.0, dtype=torch.bfloat16, device="cuda") for h in (H, KV, KV)]
    h3b.h3b_qk_norm_rope(h3b.make_qk(B, L, H, KV, dh, rope), qkv, wq, wk, pos, *out)
    return out


def bits(t):
    return t.contiguous().view(torch.int16)


@pytest.mark.parametrize("dh,rope", [(128, (16, 24, 24)), (64, (16, 24, 20)), (64, (2, 0, 0)), (128, (0, 0, 6)),
                                     (128, (0, 0, 0)), (64, (0, 0, 0))])
@pytest.mark.parametrize("with_pos", [True, False])
def test_unrotated_lanes_are_copied(dh, rope, with_pos):
    require_gpu()
    B, L, H, KV = 2, 37, 5, 2
    qkv, pos = make(B, L, H, KV, dh)
    got = run(qkv, B, L, H, KV, dh, rope, None, None, pos if with_pos else None)
    x = qkv.view(B, L, H + 2 * KV, dh).transpose(1, 2)
    first = sum(rope) if with_pos else 0
    for t, at, n in zip(got, (0, H, H + KV), (H, KV, KV)):
        cut = 0 if at == H + KV else first
        assert torch.equal(bits(t[..., cut:]), bits(x[:, at:at + n, :, cut:]))


@pytest.mark.parametrize("dh", [64, 128])
def test_normalised_but_unrotated(dh):
    """One rounding of the normalised value; a minus zero stays one."""
    require_gpu()
    B, L, H, KV = 1, 50, 3, 3
    g = torch.Generator(device="cuda").manual_seed(1)
    qkv = torch.randn((B * L, (H + 2 * KV) * dh), generator=g, device="cuda").to(torch.bfloat16)
    qkv[:, ::5] = -0.0
    w = 1 + 0.2 * torch.rand(dh, generator=g, device="cuda")
    got = run(qkv, B, L, H, KV, dh, (8, 8, 8), w, w, None)
    ref, _ = R.qk_norm_rope(qkv, B, L, H, KV, dh, (8, 8, 8), w, w, None)
    for t, r in zip(got[:2], ref[:2]):
        assert ((t.double() - r).abs() <= 2.0 ** -8 * r.abs()).all()
        assert torch.equal(t.signbit(), r.signbit())
