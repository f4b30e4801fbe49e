"""Plain 64-bit implementations of the per-head norm with rotary positions, the key block
selection, the attention over selected blocks and the gated residual norms, in loops over
items, heads and blocks. They share no code with the library and run on the inputs' device."""
import math

import torch


def qk_norm_rope(qkv, B, L, heads, kv_heads, head_dim, rope, wq, wk, pos, theta=10000.0, eps=1e-6):
    """(q, k, v) head-major, float64, and the magnitudes |a| + |b| each rotated lane is formed from."""
    x = qkv[:, : (heads + 2 * kv_heads) * head_dim].double().view(B, L, heads + 2 * kv_heads, head_dim)
    out, mag = [], []
    for first, n, w in ((0, heads, wq), (heads, kv_heads, wk), (heads + kv_heads, kv_heads, None)):
        y = x[:, :, first:first + n].clone()
        if w is not None:
            y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
        z, m = y.clone(), y.abs()
        if pos is not None and first < heads + kv_heads:
            lane = 0
            for axis, r in enumerate(rope):
                for j in range(r // 2):
                    a = pos[:, :, axis].double() * theta ** (-2.0 * j / r)
                    c, s = torch.cos(a)[..., None], torch.sin(a)[..., None]
                    e, o = y[..., lane], y[..., lane + 1]
                    z[..., lane], z[..., lane + 1] = e * c - o * s, e * s + o * c
                    m[..., lane] = m[..., lane + 1] = e.abs() + o.abs()
                    lane += 2
        out.append(z.transpose(1, 2).contiguous())
        mag.append(m.transpose(1, 2).contiguous())
    return out, mag


def _len(lens, b, L):
    return L if lens is None else min(max(int(lens[b]), 0), L)


def select_blocks(q, k, block_k, topk, q_lens=None, kv_lens=None, first=0, local=0):
    B, H, Lq, dh = q.shape
    KV, Lk = k.shape[1:3]
    nqb, nkb = -(-Lq // 128), -(-Lk // block_k)
    blocks = torch.full((B, H, nqb, topk), -1, dtype=torch.int32)
    counts = torch.zeros((B, H, nqb), dtype=torch.int32)
    for b in range(B):
        qn, kn = _len(q_lens, b, Lq), _len(kv_lens, b, Lk)
        cand = -(-kn // block_k)
        for h in range(H):
            qd, kd = q[b, h, :qn].double(), k[b, h // (H // KV), :kn].double()
            km = [kd[j * block_k:(j + 1) * block_k].mean(0) for j in range(cand)]
            for i in range(-(-qn // 128)):
                if not cand:
                    continue
                score = (torch.stack(km) @ qd[i * 128:(i + 1) * 128].mean(0)).tolist()
                lo, hi = i * 128 // block_k - local + 1, (i * 128 + 127) // block_k + local - 1

                def rank(j):
                    kept = j < first or (local > 0 and lo <= j <= hi)
                    nan = score[j] != score[j]
                    return (0 if kept else 1, 1 if nan else 0, 0.0 if kept or nan else -score[j], j)

                best = sorted(sorted(range(cand), key=rank)[:topk])
                blocks[b, h, i, :len(best)] = torch.tensor(best, dtype=torch.int32)
                counts[b, h, i] = len(best)
    return blocks, counts


def attention_blocks(q, k, v, blocks, counts, block_k, q_lens=None, kv_lens=None):
    """(o, weight): o float64 [B][Lq][H*dh]; weight is the softmax-weighted mean of |v|, the scale that an
    error relative to each probability has in o. Rows behind q_lens are NaN in both."""
    B, H, Lq, dh = q.shape
    KV, Lk = k.shape[1:3]
    nkb, topk = -(-Lk // block_k), blocks.shape[-1]
    o = torch.full((B, Lq, H, dh), math.nan, dtype=torch.float64, device=q.device)
    mag = o.clone()
    bl = blocks.cpu()
    ct = None if counts is None else counts.cpu()
    for b in range(B):
        qn, kn = _len(q_lens, b, Lq), _len(kv_lens, b, Lk)
        for h in range(H):
            kd, vd = k[b, h // (H // KV)].double(), v[b, h // (H // KV)].double()
            for i in range(-(-qn // 128)):
                n = topk if ct is None else min(max(int(ct[b, h, i]), 0), topk)
                keys = []
                for j in bl[b, h, i, :n].tolist():
                    if 0 <= j < nkb:
                        keys += range(j * block_k, min((j + 1) * block_k, kn))
                rows = slice(i * 128, min((i + 1) * 128, qn))
                if not keys:
                    o[b, rows, h] = mag[b, rows, h] = 0.0
                    continue
                at = torch.tensor(keys, device=q.device)
                w = torch.softmax(q[b, h, rows].double() @ kd[at].T / math.sqrt(dh), -1)
                o[b, rows, h], mag[b, rows, h] = w @ vd[at], w @ vd[at].abs()
    return o.view(B, Lq, H * dh), mag.view(B, Lq, H * dh)


def normed(x, kind, eps):
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    return x if kind == "none" else x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)


def residual_out(y, w_post, gate, x, alpha, post, eps, rows_per_item):
    """x + alpha * gate * (post_norm(y) * w_post) in float64 (before its rounding), and the added part."""
    r = normed(y.double(), post, eps)
    if w_post is not None:
        r = r * w_post.double()
    if gate is not None:
        item = torch.arange(y.shape[0], device=y.device) // rows_per_item
        r = r * gate.double()[item]
    return x.double() + alpha * r, alpha * r


def modulated(x_out, shift, scale, pre, eps, rows_per_item):
    h = normed(x_out.double(), pre, eps)
    item = torch.arange(h.shape[0], device=h.device) // rows_per_item
    if scale is not None:
        h = h * (1 + scale.double()[item])
    if shift is not None:
        h = h + shift.double()[item]
    return h


def quantized(h):
    """The per-row quantizer's decision in binary32 on bf16 rows: (codes int8, scales fp32)."""
    h = h.float()
    s = h.abs().amax(-1) / torch.tensor(127.0, device=h.device)
    q = torch.where(s[:, None] > 0, h / s[:, None], 0.0).round().clamp(-127, 127)
    return q.to(torch.int8), s
