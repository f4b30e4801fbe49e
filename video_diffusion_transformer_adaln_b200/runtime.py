"""Device-side holders for the block's inputs, weights and workspace.

PyTorch is used only to allocate device memory and to move bytes; the weights'
per-output-channel quantization runs in the library (h3b_quantize_weights).
"""
from __future__ import annotations

from typing import Dict, List, Optional

import numpy as np
import torch

from . import h3b
from .synth import Workload


def dims_of(wl: Workload) -> h3b.Dims:
    return h3b.make_dims(wl.B, wl.T, wl.H, wl.W, wl.d, wl.n_heads, wl.head_dim, wl.d_ff, wl.rope,
                         wl.rope_theta, wl.ln_eps, wl.qkv_int8, wl.wo_bf16)


def bf16_from_bits(bits: np.ndarray, device="cuda") -> torch.Tensor:
    t = torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16)
    return t.to(device)


def bits_from_bf16(t: torch.Tensor) -> np.ndarray:
    return t.detach().contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def quantize_weight(w: torch.Tensor):
    """fp32 [rows][cols] device tensor -> (int8 codes, fp32 scales) via the library."""
    rows, cols = w.shape
    q = torch.empty((rows, cols), dtype=torch.int8, device=w.device)
    s = torch.empty(rows, dtype=torch.float32, device=w.device)
    h3b.h3b_quantize_weights(w, q, s)
    return q, s


class DeviceBlock:
    """One block's weights in device memory, in the layout the C ABI takes."""

    def __init__(self, tensors: Dict[str, torch.Tensor]):
        self.tensors = tensors
        self.struct = h3b.make_weights(tensors)

    @classmethod
    def from_host(cls, raw: dict, qkv_int8: bool = True, device="cuda") -> "DeviceBlock":
        """raw: host arrays from synth.block_weights (fp32 projections, bf16 AdaLN)."""
        t = {"w_ada": bf16_from_bits(raw["w_ada"], device),
             "b_ada": torch.from_numpy(raw["b_ada"]).to(device)}
        for name, sname in (("wqkv", "sqkv"), ("wo", "so"), ("w1", "s1"), ("w2", "s2")):
            if name == "wqkv" and not qkv_int8:
                continue
            w32 = torch.from_numpy(raw[name]).to(device)
            t[name], t[sname] = quantize_weight(w32)
            del w32
        if not qkv_int8:
            t["wqkv_bf16"] = bf16_from_bits(raw["wqkv_bf16"], device)
        if "wo_bf16" in raw:
            t["wo_bf16"] = bf16_from_bits(raw["wo_bf16"], device)
        return cls(t)

    @classmethod
    def random_on_device(cls, wl: Workload, generator: torch.Generator, device="cuda") -> "DeviceBlock":
        """Same distributions as synth.block_weights, drawn by a seeded device RNG
        (for workloads too large to generate on the host)."""
        d, F = wl.d, wl.d_ff
        w_ada = torch.zeros((6 * d, d), dtype=torch.bfloat16, device=device)
        for k in (0, 1, 3, 4):
            w_ada[k * d:(k + 1) * d] = (torch.randn((d, d), generator=generator, device=device) / d ** 0.5).to(
                torch.bfloat16)
        b_ada = torch.zeros(6 * d, dtype=torch.float32, device=device)
        b_ada[2 * d:3 * d] = torch.randn(d, generator=generator, device=device) * 0.5 ** 0.5
        b_ada[5 * d:] = torch.randn(d, generator=generator, device=device) * 0.5 ** 0.5
        t = {"w_ada": w_ada, "b_ada": b_ada}
        for name, sname, n_out, n_in in (("wqkv", "sqkv", 3 * d, d), ("wo", "so", d, d),
                                         ("w1", "s1", F, d), ("w2", "s2", d, F)):
            w32 = torch.randn((n_out, n_in), generator=generator, device=device) / n_in ** 0.5
            if name == "wqkv" and not wl.qkv_int8:
                t["wqkv_bf16"] = w32.to(torch.bfloat16)
            elif name == "wo" and wl.wo_bf16:
                t["wo_bf16"] = w32.to(torch.bfloat16)
            else:
                t[name], t[sname] = quantize_weight(w32)
            del w32
        return cls(t)


def workspace(dims: h3b.Dims, device="cuda") -> torch.Tensor:
    n = h3b.h3b_workspace_size(dims)
    return torch.empty(n, dtype=torch.uint8, device=device)


def block_forward(dims: h3b.Dims, blk: DeviceBlock, c: torch.Tensor, x: torch.Tensor, ws: torch.Tensor):
    h3b.h3b_block_forward(dims, blk.struct, c, x, ws)


def blocks_forward(dims: h3b.Dims, blocks: List[DeviceBlock], c: torch.Tensor, x: torch.Tensor,
                   ws: torch.Tensor):
    h3b.h3b_blocks_forward(dims, [b.struct for b in blocks], c, x, ws)


def paired_block_forward(full: h3b.Dims, merged: h3b.Dims, blk: DeviceBlock, c: torch.Tensor, x: torch.Tensor,
                         ws: torch.Tensor, ym: Optional[torch.Tensor] = None):
    """Token reduction around one block: pair -> block on the merged grid -> unpair (in place
    on x). The pairing writes the merged tokens once, into ym, where the block then runs; the
    unpairing recomputes the merged input from x. Returns ym (the block's merged output)."""
    shape = (full.B, full.T, full.H, full.W // 2, full.d)
    ym = ym if ym is not None else torch.empty(shape, dtype=torch.bfloat16, device=x.device)
    h3b.h3b_token_pair(full, x, ym)
    h3b.h3b_block_forward(merged, blk.struct, c, ym, ws)
    h3b.h3b_token_unpair(full, x, None, ym, x)
    return ym


def grid_positions(wl_or_dims, offset=(0.0, 0.0, 0.0), step=(1.0, 1.0, 1.0), device="cuda") -> torch.Tensor:
    """fp32 [B][L][3] (t, h, w) positions of a latent grid's tokens for h3b_qk_norm_rope: offset + step * index
    along each axis (a clip that starts late, a frame rate, the midpoints of merged tokens)."""
    d = wl_or_dims
    axes = [o + s * torch.arange(n, dtype=torch.float32, device=device)
            for n, o, s in zip((d.T, d.H, d.W), offset, step)]
    grid = torch.stack(torch.meshgrid(*axes, indexing="ij"), -1).reshape(1, d.T * d.H * d.W, 3)
    return grid.expand(d.B, -1, -1).contiguous()


class SparseBlockState:
    """Buffers and plans of sparse_block_forward for one grid, kept between calls. Calls that may run at the same
    time need a state each.

    topk of the key blocks of block_k tokens are attended by each block of 128 queries; keep_first and keep_local
    as in h3b_select_blocks."""

    def __init__(self, dims: h3b.Dims, block_k: int = 64, topk: int = 1, keep_first: int = 0, keep_local: int = 0,
                 norm_eps: float = 1e-6, device="cuda"):
        if not dims.qkv_int8 or dims.wo_bf16:
            raise ValueError("sparse_block_forward takes int8 projections (qkv_int8 = 1, wo_bf16 = 0)")
        B, L, d, F, H, dh = dims.B, dims.L, dims.d, dims.d_ff, dims.n_heads, dims.head_dim
        R = B * L
        e = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device=device)  # noqa: E731
        self.dims = dims
        self.qk = h3b.make_qk(B, L, H, H, dh, (dims.rope_t, dims.rope_h, dims.rope_w), dims.rope_theta, norm_eps)
        self.sparse = h3b.make_sparse(B, H, H, dh, L, L, block_k, topk, keep_first, keep_local)
        # after attention: the next branch's LayerNorm and quantizer; after the MLP: the residual alone
        self.after = h3b.make_residual_norm(R, d, L, 6 * d, "rms", "layer", norm_eps, dims.ln_eps)
        self.mod = e(B, 6 * d, dtype=torch.float32)
        self.codes, self.scales = e(R * max(d, F), dtype=torch.int8), e(R, dtype=torch.float32)
        self.absmax = e(R, dtype=torch.float32)
        self.proj = e(R, 3 * d)        # Q | K | V of the projection, then the branches' outputs
        self.hidden = e(R, F)
        self.q, self.k, self.v, self.o = e(B, H, L, dh), e(B, H, L, dh), e(B, H, L, dh), e(B, L, d)
        nqb = self.sparse.nqb
        self.blocks, self.counts = e(B, H, nqb, topk, dtype=torch.int32), e(B, H, nqb, dtype=torch.int32)
        self.ws = e(h3b.h3b_sparse_workspace_size(self.sparse), dtype=torch.uint8)
        self.device = self.ws.device  # with its index
        f32 = torch.float32
        # what each tensor of a call has to be: type, and shape or number of elements
        self.inputs = {"x": (torch.bfloat16, R * d), "pos": (f32, 3 * R), "c": (f32, B * d)}
        self.norms = {"q": (f32, dh), "k": (f32, dh), "post_attn": (f32, d), "post_mlp": (f32, d)}
        self.weights = {"w_ada": (torch.bfloat16, (6 * d, d)), "b_ada": (f32, 6 * d)}
        for w, sw, b, n, k in (("wqkv", "sqkv", "bqkv", 3 * d, d), ("wo", "so", "bo", d, d), ("w1", "s1", "b1", F, d),
                               ("w2", "s2", "b2", d, F)):
            self.weights.update({w: (torch.int8, (n, k)), sw: (f32, n), b: (f32, n)})
        self.needed = [name for name in self.weights if not name.startswith("b")]  # biases may be missing

    def check(self, tensors: Dict[str, Optional[torch.Tensor]], wanted: Dict[str, tuple], what: str = ""):
        """Refuses tensors that the kernels, which get their addresses alone, would read as something else."""
        device = self.device
        for name, got in tensors.items():
            if got is None:
                continue
            dtype, size = wanted[name]
            if ((got.numel() if type(size) is int else got.shape) != size or got.dtype is not dtype or not got.is_contiguous()
                    or got.device != device or got.data_ptr() & 15):
                raise ValueError(f"{what}{name}: {got.dtype} {tuple(got.shape)} on {got.device} is not contiguous from a "
                                 f"16-byte boundary, or does not fit the state's grid and device ({dtype}, {size}, {device})")


def sparse_block_forward(state: SparseBlockState, blk: DeviceBlock, norms: Dict[str, torch.Tensor], c: torch.Tensor,
                         x: torch.Tensor, pos: torch.Tensor):
    """One block in place on x (bf16 [B][L][d]) with attention over selected key blocks, per-head norms of Q and K
    at the tokens' positions `pos` (fp32 [B][L][3]), and an RMSNorm of each branch's output ahead of its gate:

      A1 = quant(LN(x)(1 + scale_attn) + shift_attn);  Q, K, V = A1 Wqkv^T, Q and K normalised and rotated
      O = softmax over the listed key blocks;          x += gate_attn * (RMS(quant(O) Wo^T) * post_attn)
      A3 = quant(LN(x)(1 + scale_mlp) + shift_mlp);    x += gate_mlp * (RMS(quant(GELU(A3 W1^T)) W2^T) * post_mlp)

    norms: fp32 vectors "q", "k" [head_dim] and "post_attn", "post_mlp" [d] (missing ones, or None: see h3b_qk_norm_rope
    and h3b_residual_norm). The listed blocks stay in state.blocks and state.counts. ValueError, before any launch, for
    tensors and weights that do not fit the state's grid, for unknown norms, and where the current device is not the
    state's."""
    s, dims, t = state, state.dims, blk.tensors
    d, F, R = dims.d, dims.d_ff, dims.B * dims.L
    if s.device.type == "cuda" and s.device.index != torch.cuda.current_device():
        raise ValueError(f"the state's device is {s.device}, the current one cuda:{torch.cuda.current_device()}")
    s.check({"x": x, "pos": pos, "c": c}, s.inputs)
    unknown = norms.keys() - s.norms.keys()
    if unknown:
        raise ValueError(f"norms: {sorted(unknown)}, known are {list(s.norms)}")
    s.check(norms, s.norms, "norms: ")
    weights = {name: t.get(name) for name in s.weights}
    for name in s.needed:
        if weights[name] is None:
            raise ValueError(f"{name} is missing")
    s.check(weights, s.weights)
    shift_a, scale_a, gate_a, shift_m, scale_m, gate_m = (s.mod[:, i * d:(i + 1) * d] for i in range(6))
    a_d, a_f = s.codes[:R * d].view(R, d), s.codes[:R * F].view(R, F)
    y = s.proj.view(-1)[:R * d].view(R, d)
    xf = x.view(R, d)
    h3b.h3b_adaln_modulation(dims, t["w_ada"], t.get("b_ada"), c, s.mod)
    h3b.h3b_ln_modulate_quantize(xf, R, d, dims.ln_eps, shift_a, scale_a, dims.L, 6 * d, a_d, s.scales,
                                 absmax_zero=s.absmax)
    h3b.h3b_gemm_i8_dequant(a_d, s.scales, t["wqkv"], t["sqkv"], t.get("bqkv"), s.proj)
    h3b.h3b_qk_norm_rope(s.qk, s.proj, norms.get("q"), norms.get("k"), pos, s.q, s.k, s.v)
    h3b.h3b_select_blocks(s.sparse, s.q, s.k, None, None, s.blocks, s.counts, s.ws)
    h3b.h3b_attention_blocks(s.sparse, s.q, s.k, s.v, None, None, s.blocks, s.counts, s.o, s.absmax, s.ws)
    h3b.h3b_quantize_rows(s.o.view(R, d), a_d, s.scales, absmax=s.absmax)
    h3b.h3b_gemm_i8_dequant(a_d, s.scales, t["wo"], t["so"], t.get("bo"), y)
    h3b.h3b_residual_norm(s.after, y, norms.get("post_attn"), gate_a, xf, xf, shift_m, scale_m, q=a_d, s=s.scales,
                          absmax_zero=s.absmax)
    h3b.h3b_gemm_i8_gelu(a_d, s.scales, t["w1"], t["s1"], t.get("b1"), s.hidden, s.absmax)
    h3b.h3b_quantize_rows(s.hidden, a_f, s.scales, absmax=s.absmax)
    h3b.h3b_gemm_i8_dequant(a_f, s.scales, t["w2"], t["s2"], t.get("b2"), y)
    h3b.h3b_residual_norm(s.after, y, norms.get("post_mlp"), gate_m, xf, xf, None, None)
