"""A NaN in a row shows in the row's largest magnitude and quantizer scale, so that its products do not pass for finite
ones, and nothing of it reaches another row: the steps one by one, and the blocks that chain them."""
import pytest
import torch

from gpu_helpers import no_device_error, require_gpu
from test_gpu_sparse_block import setup
from video_diffusion_transformer_adaln_b200 import h3b, synth
from video_diffusion_transformer_adaln_b200.runtime import block_forward, sparse_block_forward, workspace

pytestmark = pytest.mark.gpu
NAN = float("nan")


def randn(*shape, seed=0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("d", [256, 512, 1024, 1280, 2048, 5120])
@pytest.mark.parametrize("lane", [0, 77, -1])
def test_layer_norm_quantizer(d, lane):
    require_gpu()
    rows = 37
    x, mod = randn(rows, d), randn(2, d, seed=1, dtype=torch.float32)

    def run():
        q, s = torch.empty((rows, d), dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
        h = torch.empty_like(x)
        h3b.h3b_ln_modulate_quantize(x, rows, d, 1e-6, mod[0], mod[1], rows, d, q, s, h_out=h)
        return q, s, h

    clean = run()
    x[5, lane], x[20, lane] = NAN, float("inf")
    q, s, h = run()
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[5] = keep[20] = False
    assert h[5].isnan().all() and s[5].isnan() and not s[20].isfinite()
    for a, b in zip((q, s, h), clean):
        assert torch.equal(a[keep], b[keep])


@pytest.mark.parametrize("cols", [16, 256, 5120, 20480])
@pytest.mark.parametrize("lane", [0, 9, -1])
def test_row_quantizers(cols, lane):
    require_gpu()
    rows = 6
    for dtype, call in ((torch.bfloat16, h3b.h3b_quantize_rows), (torch.float32, h3b.h3b_quantize_weights)):
        h = randn(rows, cols, seed=2, dtype=dtype)
        q, s = torch.empty((rows, cols), dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
        q2, s2 = torch.empty_like(q), torch.empty_like(s)
        call(h, q, s)
        h[3, lane] = NAN
        call(h, q2, s2)
        assert s2[3].isnan()
        keep = torch.arange(rows, device="cuda") != 3
        assert torch.equal(q[keep], q2[keep]) and torch.equal(s[keep], s2[keep])


@pytest.mark.parametrize("M,N,K", [(5, 272, 256), (300, 1040, 512)])
def test_gelu_product(M, N, K):
    require_gpu()
    g = torch.Generator(device="cuda").manual_seed(3)
    A, W = (torch.randint(-127, 128, (n, K), generator=g, device="cuda", dtype=torch.int8) for n in (M, N))
    sA, sW = (torch.full((n,), 0.01, device="cuda") for n in (M, N))
    sA[2] = NAN
    out, am = torch.empty((M, N), dtype=torch.bfloat16, device="cuda"), torch.zeros(M, device="cuda")
    h3b.h3b_gemm_i8_gelu(A, sA, W, sW, None, out, am)
    keep = torch.arange(M, device="cuda") != 2
    assert out[2].isnan().all() and am[2].isnan()
    assert torch.equal(am[keep], out[keep].abs().amax(-1).float())


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("lane", [0, 31, 63])
def test_dense_attention(dh, lane):
    require_gpu()
    B, H, L = 2, 2, 300
    qkv = randn(3, B, H, L, dh, seed=4)
    qkv[2, 0, 1, 150, lane] = NAN
    dims = h3b.make_dims(B, 1, 1, L, H * dh, H, dh, 256, (0, 0, dh))
    o, am = torch.empty((B, L, H * dh), dtype=torch.bfloat16, device="cuda"), torch.zeros(B * L, device="cuda")
    h3b.h3b_attention(dims, qkv, o, am)
    rows = o.view(B * L, -1).isnan().any(-1)
    assert rows[:L].all() and not rows[L:].any()
    assert torch.equal(am.isnan(), rows)
    assert torch.equal(am[L:], o[1].abs().amax(-1).float())


def test_block_over_selected_key_blocks():
    """The token's key block ranks last, so only its own query block lists it (keep_local): those rows are NaN."""
    require_gpu()
    wl = synth.WORKLOADS["d256_L512"].with_(B=2)
    dims, blk, norms, pos, c, x, state = setup(wl, topk=3, keep_local=1)
    clean = x.clone()
    sparse_block_forward(state, blk, norms, c, clean, pos)
    x[0, 200, 17] = NAN
    sparse_block_forward(state, blk, norms, c, x, pos)
    lists_it = (state.blocks == 200 // 64).any(-1).any(1).repeat_interleave(128, -1)  # [B][L]; B items of their own
    lists_it[1] = False
    rows = x.isnan().any(-1)
    assert lists_it[0, 128:256].all() and torch.equal(rows, lists_it)
    assert x[rows].isnan().all() and torch.equal(x[1], clean[1])
    no_device_error()


@pytest.mark.parametrize("qkv_int8", [True, False])
def test_dense_block(qkv_int8):
    """Every query attends the token: the whole item is NaN, the other item as it was."""
    require_gpu()
    from gpu_helpers import bf16_dev, to_dev
    from video_diffusion_transformer_adaln_b200.runtime import DeviceBlock, dims_of
    wl = synth.WORKLOADS["d256_L512"].with_(B=2, qkv_int8=qkv_int8)
    dims = dims_of(wl)
    blk, ws = DeviceBlock.from_host(synth.block_weights(wl), qkv_int8), workspace(dims)
    x, c = bf16_dev(synth.x_input(wl)).view(2, wl.L, wl.d), to_dev(synth.cond(wl))
    clean = x.clone()
    block_forward(dims, blk, c, clean, ws)
    x[0, 200, 17] = NAN
    block_forward(dims, blk, c, x, ws)
    assert x[0].isnan().all() and torch.equal(x[1], clean[1])
    no_device_error()
