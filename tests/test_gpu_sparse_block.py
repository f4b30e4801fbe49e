"""The block with attention over selected key blocks, as a user runs it (runtime.sparse_block_forward), against
the same chain in 64 bits with the formats' roundings at the same places.

Both sides round to bf16 and int8 at the same points, so they differ where a value lies next to a rounding
border. Were every one of the about ten bf16 roundings on the way of a branch independent on the two sides, each
would add 2^-9 / sqrt(3) * sqrt(2) of its value, together sqrt(10) * 1.6e-3 = 5e-3 of the branch's output; the
probabilities' rounding for the tensor core adds 2^-9 of the values' mean. The block's added part is held to 1e-2."""
import numpy as np
import pytest
import torch

import operator_refs as R
from gpu_helpers import bf16_dev, no_device_error, rel_l2, require_gpu, to_dev
from video_diffusion_transformer_adaln_b200 import synth
from video_diffusion_transformer_adaln_b200.runtime import (DeviceBlock, SparseBlockState, dims_of, grid_positions,
                                                            sparse_block_forward)

pytestmark = pytest.mark.gpu


def setup(wl, seed=0, **sparse):
    dims = dims_of(wl)
    blk = DeviceBlock.from_host(synth.block_weights(wl))
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = lambda n: 1 + 0.2 * torch.randn(n, generator=g, device="cuda")  # noqa: E731
    norms = {"q": w(wl.head_dim), "k": w(wl.head_dim), "post_attn": w(wl.d), "post_mlp": w(wl.d)}
    pos = grid_positions(dims, offset=(3.0, 0.5, 0.0), step=(0.5, 1.0, 1.0))
    x = bf16_dev(synth.x_input(wl)).view(wl.B, wl.L, wl.d)
    return dims, blk, norms, pos, to_dev(synth.cond(wl)), x, SparseBlockState(dims, **sparse)


def bf(t):
    return t.to(torch.bfloat16).double()


def quant(h):
    q, s = R.quantized(h.to(torch.bfloat16))
    return q.double() * s.double()[:, None]


def reference(wl, blk, norms, pos, c, x, state):
    """The chain in 64 bits, over the lists that the library selected. Returns x and the branches' added parts."""
    B, L, d, H, dh = wl.B, wl.L, wl.d, wl.n_heads, wl.head_dim
    t = blk.tensors
    w = {n: t[n].double() * t[s].double()[:, None] for n, s in (("wqkv", "sqkv"), ("wo", "so"), ("w1", "s1"), ("w2", "s2"))}
    mod = (c.double() @ t["w_ada"].double().T + t["b_ada"].double()).repeat_interleave(L, 0)
    sh_a, sc_a, g_a, sh_m, sc_m, g_m = mod.chunk(6, -1)
    x0 = x.view(B * L, d).double()
    qkv = bf(quant(R.normed(x0, "layer", wl.ln_eps) * (1 + sc_a) + sh_a) @ w["wqkv"].T)
    (q, k, v), _ = R.qk_norm_rope(qkv, B, L, H, H, dh, wl.rope, norms["q"], norms["k"], pos)
    o, _ = R.attention_blocks(bf(q), bf(k), bf(v), state.blocks, state.counts, state.sparse.block_k)
    y = bf(quant(bf(o.view(B * L, d))) @ w["wo"].T)
    a1 = g_a * R.normed(y, "rms", 1e-6) * norms["post_attn"].double()
    x1 = bf(x0 + a1)
    h = quant(R.normed(x1, "layer", wl.ln_eps) * (1 + sc_m) + sh_m) @ w["w1"].T
    h = 0.5 * h * (1 + torch.tanh(np.sqrt(2 / np.pi) * (h + 0.044715 * h ** 3)))
    y = bf(quant(bf(h)) @ w["w2"].T)
    x2 = x1 + g_m * R.normed(y, "rms", 1e-6) * norms["post_mlp"].double()
    return x2, x2 - x0


@pytest.mark.parametrize("kw,sparse", [
    (dict(), dict(block_k=64, topk=4, keep_local=1)),
    (dict(B=2, T=3, H=9, W=11), dict(block_k=64, topk=3, keep_first=1)),       # 297 tokens: cut blocks
    (dict(T=1, H=1, W=1), dict(block_k=64, topk=1)),                            # one token
    (dict(T=4, d=512, n_heads=4, head_dim=128, d_ff=512, rope=(32, 48, 48)), dict(block_k=128, topk=5)),
])
def test_block_matches_the_chain_in_64_bits(kw, sparse):
    require_gpu()
    wl = synth.WORKLOADS["d256_L512"].with_(**kw)
    dims, blk, norms, pos, c, x, state = setup(wl, **sparse)
    x0 = x.clone()
    sparse_block_forward(state, blk, norms, c, x, pos)
    ref, added = reference(wl, blk, norms, pos, c, x0, state)
    got = x.view(-1, wl.d).double() - x0.view(-1, wl.d).double()
    # x itself is held in bf16: its rounding, 2^-9 of the stream, is not the branches' error
    rounding = 2.0 ** -8 * ref.abs()
    off = ((got - added).abs() - 2 * rounding).clamp(min=0)
    assert off.norm() <= 1e-2 * added.norm(), (off.norm() / added.norm()).item()
    assert rel_l2(x.view(-1, wl.d).double().cpu().numpy(), ref.cpu().numpy()) <= 2.0 ** -7
    rb, rc = R.select_blocks(state.q.cpu(), state.k.cpu(), state.sparse.block_k, state.sparse.topk,
                             first=sparse.get("keep_first", 0), local=sparse.get("keep_local", 0))
    assert torch.equal(state.blocks.cpu(), rb) and torch.equal(state.counts.cpu(), rc)
    no_device_error()


def test_block_in_a_graph_and_two_states_at_once():
    require_gpu()
    wl = synth.WORKLOADS["d256_L512"].with_(B=2)
    dims, blk, norms, pos, c, x, state = setup(wl, topk=3, keep_local=1)
    other = SparseBlockState(dims, topk=3, keep_local=1)
    want = x.clone()
    sparse_block_forward(state, blk, norms, c, want, pos)
    torch.cuda.synchronize()
    xs, streams = [x.clone(), x.clone()], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for xx, st, s in zip(xs, (state, other), streams):
        with torch.cuda.stream(s):
            sparse_block_forward(st, blk, norms, c, xx, pos)
    torch.cuda.synchronize()
    assert torch.equal(xs[0], want) and torch.equal(xs[1], want)
    buf = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sparse_block_forward(state, blk, norms, c, buf, pos)
    for _ in range(2):
        buf.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf, want)


def test_state_refuses_other_projections():
    require_gpu()
    dims = dims_of(synth.WORKLOADS["d256_L512"].with_(qkv_int8=False))
    with pytest.raises(ValueError):
        SparseBlockState(dims)
