"""Per-head RMSNorm and per-token rotary positions against the formula in 64 bits.

Tolerance: each output is one bf16 rounding (2^-8 of the value) of an fp32 result. The fp32
error of a rotated lane a*cos - b*sin is a few 2^-24 of |a| + |b| for the norm (sum of 128
squares, a root and a division: below 2^-20), the two products, their difference, and a
(cos, sin) pair within 2^-22 of the angle's: together below 2^-19 (|a| + |b|)."""
import pytest
import torch

import operator_refs as R
from gpu_helpers import no_device_error, require_gpu
from video_diffusion_transformer_adaln_b200 import h3b

pytestmark = pytest.mark.gpu

ROUND, FP32 = 2.0 ** -8, 2.0 ** -19


def make(B, L, H, KV, dh, pad=0, seed=0, far=0.0, fractional=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    stride = (H + 2 * KV) * dh + pad
    qkv = torch.randn((B * L, stride), generator=g, device="cuda").to(torch.bfloat16)
    w = [1 + 0.2 * torch.randn(dh, generator=g, device="cuda") for _ in range(2)]
    pos = torch.randint(0, 60, (B, L, 3), generator=g, device="cuda").float() + far
    if fractional:
        pos = pos + torch.rand((B, L, 3), generator=g, device="cuda") - 30
    return qkv, w[0], w[1], pos


def outputs(B, L, H, KV, dh):
    return [torch.full((B, h, L, dh), 7.0, dtype=torch.bfloat16, device="cuda") for h in (H, KV, KV)]


def check(got, ref, mag):
    for name, a, r, m in zip("qkv", got, ref, mag):
        err = (a.double() - r).abs()
        bad = err > ROUND * r.abs() + FP32 * m
        assert not bad.any(), (name, err[bad].max().item())


@pytest.mark.parametrize("B,L,H,KV,dh,rope,pad", [
    (1, 1, 1, 1, 64, (16, 24, 24), 0),       # one token, one head
    (1, 512, 4, 4, 64, (16, 24, 24), 0),     # the smallest workload's grid
    (2, 77, 16, 16, 128, (32, 48, 48), 0),
    (3, 33, 10, 2, 128, (16, 24, 24), 64),   # shared key heads, half the lanes rotated, padded rows
    (2, 5, 3, 1, 64, (64, 0, 0), 8),         # one axis takes every lane
    (1, 9, 3, 3, 128, (0, 64, 64), 0),       # no time axis
    (1, 130, 40, 40, 128, (32, 48, 48), 0),  # more heads than a pass of the block covers
    (1, 3, 5, 1, 64, (2, 2, 2), 0),          # one pair per axis
])
def test_matches_the_formula(B, L, H, KV, dh, rope, pad):
    require_gpu()
    qkv, wq, wk, pos = make(B, L, H, KV, dh, pad, fractional=True)
    got = outputs(B, L, H, KV, dh)
    d = h3b.make_qk(B, L, H, KV, dh, rope, row_stride=qkv.shape[1])
    h3b.h3b_qk_norm_rope(d, qkv, wq, wk, pos, *got)
    ref, mag = R.qk_norm_rope(qkv, B, L, H, KV, dh, rope, wq, wk, pos)
    check(got, ref, mag)
    assert torch.equal(got[2].double(), ref[2])  # V is copied
    no_device_error()


@pytest.mark.parametrize("far", [1e5, -3e6, 2.0 ** 23])
def test_far_positions_lose_nothing(far):
    """An angle of 2^23 radians formed in 32 bits is off by whole radians; the tolerance stays the same."""
    require_gpu()
    B, L, H, KV, dh, rope = 1, 40, 2, 2, 128, (32, 48, 48)
    qkv, wq, wk, pos = make(B, L, H, KV, dh, far=far)
    got = outputs(B, L, H, KV, dh)
    h3b.h3b_qk_norm_rope(h3b.make_qk(B, L, H, KV, dh, rope), qkv, wq, wk, pos, *got)
    check(got, *R.qk_norm_rope(qkv, B, L, H, KV, dh, rope, wq, wk, pos))


@pytest.mark.parametrize("norm_q,norm_k,turn", [(False, False, True), (True, False, True), (False, True, False),
                                                (False, False, False)])
def test_optional_parts(norm_q, norm_k, turn):
    require_gpu()
    B, L, H, KV, dh, rope = 2, 19, 6, 3, 64, (16, 24, 24)
    qkv, wq, wk, pos = make(B, L, H, KV, dh)
    wq, wk, pos = wq if norm_q else None, wk if norm_k else None, pos if turn else None
    got = outputs(B, L, H, KV, dh)
    h3b.h3b_qk_norm_rope(h3b.make_qk(B, L, H, KV, dh, rope), qkv, wq, wk, pos, *got)
    ref, mag = R.qk_norm_rope(qkv, B, L, H, KV, dh, rope, wq, wk, pos)
    check(got, ref, mag)
    if not norm_q and not turn:
        assert torch.equal(got[0].double(), ref[0])


def test_the_grid_of_the_qkv_projection():
    """With the grid's integer positions and no norm, the rotation is that of the QKV projection: both
    round the same fp32 rotation once, so they agree to two roundings of the projected value."""
    require_gpu()
    T, Hh, W, dh, H = 2, 6, 5, 64, 4
    L, d = T * Hh * W, H * dh
    g = torch.Generator(device="cuda").manual_seed(3)
    a = torch.randint(-127, 128, (L, d), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-127, 128, (3 * d, d), generator=g, device="cuda", dtype=torch.int8)
    sa = torch.full((L,), 0.01, device="cuda")
    sw = torch.full((3 * d,), 0.001, device="cuda")
    dims = h3b.make_dims(1, T, Hh, W, d, H, dh, 256, (16, 24, 24))
    fused = torch.empty((3, 1, H, L, dh), dtype=torch.bfloat16, device="cuda")
    rope_ws = torch.empty(h3b.h3b_rope_table_bytes(dims), dtype=torch.uint8, device="cuda")
    h3b.h3b_qkv_projection(dims, a, sa, h3b.make_weights({"wqkv": w, "sqkv": sw}), fused, rope_ws)
    plain = torch.empty((L, 3 * d), dtype=torch.bfloat16, device="cuda")
    h3b.h3b_gemm_i8_dequant(a, sa, w, sw, None, plain)
    i = torch.arange(L, device="cuda")
    pos = torch.stack([i // (Hh * W), i // W % Hh, i % W], 1).float().view(1, L, 3).contiguous()
    got = outputs(1, L, H, H, dh)
    h3b.h3b_qk_norm_rope(h3b.make_qk(1, L, H, H, dh, (16, 24, 24)), plain, None, None, pos, *got)
    for n in range(2):
        size = fused[n].double().view(1, H, L, dh // 2, 2).square().sum(-1, keepdim=True).sqrt()
        size = size.expand(-1, -1, -1, -1, 2).reshape(1, H, L, dh)
        # the projection's rounding moves both lanes of a pair by 2^-8 of each (below 2^-7.5 of the
        # pair's length after the rotation), each output's own rounding by 2^-8 of it
        assert ((got[n].double() - fused[n].double()).abs() <= 2.0 ** -7.5 * size + 2 * ROUND * size).all()
    assert torch.equal(got[2], fused[2])


def test_columns_behind_the_projection_are_not_read_and_neighbours_not_written():
    require_gpu()
    B, L, H, KV, dh, rope = 1, 21, 2, 1, 64, (16, 24, 24)
    qkv, wq, wk, pos = make(B, L, H, KV, dh, pad=16)
    qkv[:, (H + 2 * KV) * dh:] = float("nan")
    bufs = [torch.full((h * L * dh + 128,), 5.0, dtype=torch.bfloat16, device="cuda") for h in (H, KV, KV)]
    got = [b[64:-64].view(B, h, L, dh) for b, h in zip(bufs, (H, KV, KV))]
    h3b.h3b_qk_norm_rope(h3b.make_qk(B, L, H, KV, dh, rope, row_stride=qkv.shape[1]), qkv, wq, wk, pos, *got)
    check(got, *R.qk_norm_rope(qkv, B, L, H, KV, dh, rope, wq, wk, pos))
    for b in bufs:
        assert (b[:64] == 5.0).all() and (b[-64:] == 5.0).all()


def test_non_finite_rows_stay_in_their_rows():
    require_gpu()
    B, L, H, KV, dh, rope = 1, 70, 3, 1, 128, (32, 48, 48)
    qkv, wq, wk, pos = make(B, L, H, KV, dh)
    clean = outputs(B, L, H, KV, dh)
    d = h3b.make_qk(B, L, H, KV, dh, rope)
    h3b.h3b_qk_norm_rope(d, qkv, wq, wk, pos, *clean)
    qkv[7, dh] = float("inf")       # token 7, query head 1
    qkv[50, H * dh] = float("nan")  # token 50, key head 0
    got = outputs(B, L, H, KV, dh)
    h3b.h3b_qk_norm_rope(d, qkv, wq, wk, pos, *got)
    same_q = torch.ones((B, H, L), dtype=torch.bool, device="cuda")
    same_q[0, 1, 7] = False
    assert torch.equal(got[0][same_q], clean[0][same_q]) and not got[0][0, 1, 7].isfinite().all()
    same_k = torch.ones((B, KV, L), dtype=torch.bool, device="cuda")
    same_k[0, 0, 50] = False
    assert torch.equal(got[1][same_k], clean[1][same_k]) and got[1][0, 0, 50].isnan().all()


def test_on_another_stream_and_in_a_graph():
    require_gpu()
    B, L, H, KV, dh, rope = 2, 200, 8, 4, 128, (32, 48, 48)
    qkv, wq, wk, pos = make(B, L, H, KV, dh)
    d = h3b.make_qk(B, L, H, KV, dh, rope)
    want = outputs(B, L, H, KV, dh)
    h3b.h3b_qk_norm_rope(d, qkv, wq, wk, pos, *want)
    got = outputs(B, L, H, KV, dh)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    h3b.h3b_qk_norm_rope(d, qkv, wq, wk, pos, *got, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h3b.h3b_qk_norm_rope(d, qkv, wq, wk, pos, *got)
    qkv.copy_(qkv.flip(0))
    for _ in range(2):
        [t.zero_() for t in got]
        graph.replay()
        torch.cuda.synchronize()
        h3b.h3b_qk_norm_rope(d, qkv, wq, wk, pos, *want)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("B,L,H,KV,dh,rope,pad", [
    (2, 4201, 18, 6, 128, (32, 48, 48), 8),   # many boxes per CTA; heads and tokens cut a box
    (3, 5003, 21, 7, 64, (16, 24, 24), 0),
])
def test_many_boxes(B, L, H, KV, dh, rope, pad):
    require_gpu()
    qkv, wq, wk, pos = make(B, L, H, KV, dh, pad, fractional=True)
    bufs = [torch.full((B * h * L * dh + 128,), 5.0, dtype=torch.bfloat16, device="cuda") for h in (H, KV, KV)]
    got = [b[64:-64].view(B, h, L, dh) for b, h in zip(bufs, (H, KV, KV))]
    h3b.h3b_qk_norm_rope(h3b.make_qk(B, L, H, KV, dh, rope, row_stride=qkv.shape[1]), qkv, wq, wk, pos, *got)
    ref, mag = R.qk_norm_rope(qkv, B, L, H, KV, dh, rope, wq, wk, pos)
    check(got, ref, mag)
    assert torch.equal(got[2].double(), ref[2])
    for b in bufs:
        assert (b[:64] == 5.0).all() and (b[-64:] == 5.0).all()
    no_device_error()
