"""The operators on tensors of more than 2^31 elements: what lies behind that offset is checked against
the plain 64-bit forms, with the tolerances of each operator's own tests."""
import pytest
import torch

import operator_refs as R
from gpu_helpers import no_device_error, require_gpu
from video_diffusion_transformer_adaln_b200 import h3b

pytestmark = pytest.mark.gpu


def randn(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


@pytest.mark.parametrize("Lq", [1, 130])
def test_a_long_cache(Lq):
    """Keys and values of 2.25e9 elements each; the last batch item's lists reach the last block."""
    require_gpu()
    B, H, dh, Lk, topk = 4, 40, 128, 110001, 12
    k, v, q = randn((B, H, Lk, dh), 1), randn((B, H, Lk, dh), 2), randn((B, H, Lq, dh), 3)
    d = h3b.make_sparse(B, H, H, dh, Lq, Lk, 64, topk, 1, 0)
    blocks = torch.empty((B, H, d.nqb, topk), dtype=torch.int32, device="cuda")
    counts = torch.empty((B, H, d.nqb), dtype=torch.int32, device="cuda")
    ws = torch.empty(h3b.h3b_sparse_workspace_size(d), dtype=torch.uint8, device="cuda")
    h3b.h3b_select_blocks(d, q, k, None, None, blocks, counts, ws)
    last = (slice(B - 1, B), slice(H - 1, H))
    rb, rc = R.select_blocks(q[last].cpu(), k[last].cpu(), 64, topk, first=1)
    assert torch.equal(blocks[last].cpu(), rb) and torch.equal(counts[last].cpu(), rc)
    blocks[..., -1] = d.nkb - 1
    o = torch.empty((B, Lq, H * dh), dtype=torch.bfloat16, device="cuda")
    h3b.h3b_attention_blocks(d, q, k, v, None, None, blocks, None, o, None, ws)
    ref, mag = R.attention_blocks(q[last], k[last], v[last], blocks[last], None, 64)
    err = (o[B - 1:, :, -dh:].double() - ref).abs()
    assert (err <= (2.0 ** -8 + 2.0 ** -11) * mag + 2.0 ** -8 * ref.abs()).all()
    no_device_error()


def test_many_rows_of_the_projection():
    require_gpu()
    B, L, H, KV, dh, rope = 2, 72001, 40, 40, 128, (32, 48, 48)
    qkv = randn((B * L, (H + 2 * KV) * dh), 4)
    pos = 100 * torch.rand((B, L, 3), device="cuda")
    w = 1 + 0.1 * torch.randn(dh, device="cuda")
    q, k, v = (torch.empty((B, n, L, dh), dtype=torch.bfloat16, device="cuda") for n in (H, KV, KV))
    h3b.h3b_qk_norm_rope(h3b.make_qk(B, L, H, KV, dh, rope), qkv, w, w, pos, q, k, v)
    tail = 200
    ref, mag = R.qk_norm_rope(qkv[-tail:], 1, tail, H, KV, dh, rope, w, w, pos[-1:, -tail:])
    for got, want, m in zip((q, k, v), ref, mag):
        err = (got[-1:, :, -tail:].double() - want).abs()
        assert (err <= 2.0 ** -8 * want.abs() + 2.0 ** -19 * m).all()
    no_device_error()


def test_many_rows_of_the_stream():
    require_gpu()
    rows, d, tail = 420001, 5120, 64
    y, x = randn((rows, d), 5), randn((rows, d), 6)
    w, mod = torch.rand(d, device="cuda"), torch.randn((2, 3, d), device="cuda")
    rpi = rows - 40  # the second item lies behind the offset
    dims = h3b.make_residual_norm(rows, d, rpi, 3 * d, "rms", "layer")
    ref, added = R.residual_out(y[-tail:-40], w, mod[:1, 0], x[-tail:-40], 1.0, "rms", 1e-6, tail)
    ref2, added2 = R.residual_out(y[-40:], w, mod[1:, 0], x[-40:], 1.0, "rms", 1e-6, tail)
    ref, added, x0 = torch.cat([ref, ref2]), torch.cat([added, added2]), x[-tail:].double()
    q, s = torch.empty((rows, d), dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    h = torch.empty_like(x)
    h3b.h3b_residual_norm(dims, y, w, mod[:, 0], x, x, mod[:, 1], mod[:, 2], h_out=h, q=q, s=s)
    assert ((x[-tail:].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -19 * (added.abs() + x0.abs())).all()
    qr, sr = R.quantized(h[-tail:])
    assert torch.equal(q[-tail:], qr) and torch.equal(s[-tail:], sr)
    no_device_error()
