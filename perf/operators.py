"""The operators of a block-sparse, per-head-normalised DiT block, as they are measured.

Four operators, each over the range of sizes that a user of this library meets:

  rope     per-head RMSNorm of Q and K and rotary positions on three axes (time, height, width) given
           per token, from token-major projections to the head-major layout attention reads
  select   which key blocks each block of 128 queries attends: the score of a pair of blocks is the
           product of the blocks' mean query and mean key, the best `topk` key blocks are listed
  attend   softmax attention of each block of 128 queries over its listed key blocks
  resnorm  a branch's output normalised, gated and added to the residual stream, and the next
           branch's norm, modulation and int8 quantizer, in one pass over the rows

`own` selects what `run` does: the plain form in elementary torch operations, or the library's entry
points on the same state.
"""
import math

import torch

own = False

QB = 128  # queries per block of the selection


# ------------------------------------------------------------------------------------------- cases

def _rope(name, B, L, heads, kv_heads, head_dim, rope, pad=0, norm=True, fractional=False, offset=0):
    return {"name": name, "op": "rope", "B": B, "L": L, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim,
            "rope_t": rope[0], "rope_h": rope[1], "rope_w": rope[2], "pad": pad, "norm": norm,
            "fractional": fractional, "offset": offset}


def _select(name, B, Lq, Lk, heads, kv_heads, head_dim, block_k, topk, first=0, local=0, ragged=False):
    return {"name": name, "op": "select", "B": B, "Lq": Lq, "Lk": Lk, "heads": heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "block_k": block_k, "topk": topk, "first": first, "local": local, "ragged": ragged}


def _attend(name, B, Lq, Lk, heads, kv_heads, head_dim, block_k, topk, ragged=False, absmax=False):
    return {"name": name, "op": "attend", "B": B, "Lq": Lq, "Lk": Lk, "heads": heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "block_k": block_k, "topk": topk, "ragged": ragged, "absmax": absmax}


def _resnorm(name, B, L, d, post, pre, int8, weight=True, alpha=1.0):
    return {"name": name, "op": "resnorm", "B": B, "L": L, "d": d, "post": post, "pre": pre, "int8": int8,
            "weight": weight, "alpha": alpha}


def listed():
    return [
        # the smallest grid of the library's workloads (2x16x16 tokens, 4 heads of 64): latency
        _rope("rope_d256_L512", 1, 512, 4, 4, 64, (16, 24, 24)),
        # the largest single-latent workload: 8x48x48 tokens, 40 heads of 128
        _rope("rope_d5120_L18432", 1, 18432, 40, 40, 128, (32, 48, 48)),
        # three ragged clips with shared key heads, half the lanes rotated, a padded projection, the
        # fractional far positions of merged tokens late in a long video
        _rope("rope_shared_padded", 3, 1001, 10, 2, 128, (16, 24, 24), pad=64, fractional=True, offset=20000),
        # two short clips of different lengths, a text block always kept
        _select("select_two_clips", 2, 777, 777, 4, 4, 64, 64, 5, first=1, local=1, ragged=True),
        # the largest latent at one key block in eight
        _select("select_d5120_L18432", 1, 18432, 18432, 40, 40, 128, 64, 36, local=1),
        # the smallest grid, half of its key blocks
        _attend("attend_d256_L512", 1, 512, 512, 4, 4, 64, 64, 4),
        # one new token of four streams over a long latent, key heads shared by five query heads
        _attend("attend_one_token", 4, 1, 18432, 40, 8, 128, 64, 72),
        # three clips padded to one length, with query blocks that no key block is listed for; the row
        # maxima that the int8 output projection takes its scales from
        _attend("attend_padded_clips", 3, 2500, 2500, 8, 2, 128, 128, 6, ragged=True, absmax=True),
        # the largest latent at one key block in eight
        _attend("attend_d5120_L18432", 1, 18432, 18432, 40, 40, 128, 64, 36),
        # the smallest grid: latency
        _resnorm("resnorm_d256_L512", 1, 512, 256, "rms", "layer", False),
        # odd rows, RMS norms on both sides, a damped residual, ahead of an int8 projection
        _resnorm("resnorm_odd_rows_int8", 3, 1001, 1552, "rms", "rms", True, alpha=0.7),
        # the largest latent, ahead of a bf16 projection
        _resnorm("resnorm_d5120_L18432", 1, 18432, 5120, "rms", "layer", False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "select", "attend", "resnorm"])
    head_dim = rng.choice([64, 128])
    if op == "resnorm":
        d = 8 * _log(rng, 32, 1024)
        B = rng.randint(1, 4)
        L = _log(rng, 1, max(1, min(20000, 18432 * 5120 // (B * d))))
        c = _resnorm("", B, L, d, rng.choice(["rms", "layer", "none"]), rng.choice(["rms", "layer"]),
                     rng.random() < 0.5, rng.random() < 0.7, rng.choice([1.0, 0.5, 0.25]))
    else:
        kv = rng.choice([1, 2, 3, 4, 5, 8])
        heads = kv * rng.choice([1, 1, 2, 4])
        B = rng.randint(1, 3)
        if op == "rope":
            L = _log(rng, 1, min(20000, 18432 * 40 * 128 // (B * heads * head_dim)))
            half = head_dim // 2
            rope = rng.choice([(head_dim // 4, 3 * head_dim // 8, 3 * head_dim // 8), (0, half, half),
                               (head_dim // 8, head_dim // 4, head_dim // 4), (head_dim, 0, 0)])
            c = _rope("", B, L, heads, kv, head_dim, rope, rng.choice([0, 8, 64]), rng.random() < 0.8,
                      rng.random() < 0.5, rng.choice([0, 100, 50000]))
        else:
            block_k = rng.choice([64, 128])
            if rng.random() < 0.25:  # few queries over a long latent
                Lq, Lk = rng.randint(1, 200), _log(rng, 2000, 40000)
            else:
                Lq = Lk = _log(rng, 1, 12000)
            nkb = -(-Lk // block_k)
            most = 40 * 18432 * 36 * 64 // (B * heads * -(-Lq // QB) * QB * block_k)
            topk = max(1, min(nkb, most, _log(rng, 1, 64)))
            ragged = rng.random() < 0.4
            if op == "select":
                local = rng.choice([0, 0, 1]) if topk >= 4 else 0
                first = rng.choice([0, 1]) if topk >= 4 else 0
                c = _select("", B, Lq, Lk, heads, kv, head_dim, block_k, topk, first, local, ragged)
            else:
                c = _attend("", B, Lq, Lk, heads, kv, head_dim, block_k, topk, ragged, rng.random() < 0.3)
    del c["name"]
    return c


# ------------------------------------------------------------------------------------------ inputs

def _lens(B, L, ragged, gen):
    """Valid tokens of each item: the first is full, the others lose up to half."""
    if not ragged:
        return None
    n = L - (torch.rand(B, generator=gen, device="cuda") * (L / 2)).to(torch.int32)
    n[0] = L
    return n.to(torch.int32)


def _field(B, heads, L, head_dim, gen, smooth):
    """Head-major rows as a video's are: neighbouring tokens share a part, each has its own."""
    base = torch.randn((B, heads, -(-L // 48), head_dim), generator=gen, device="cuda")
    x = torch.randn((B, heads, L, head_dim), generator=gen, device="cuda")
    return (x + smooth * base.repeat_interleave(48, dim=2)[:, :, :L]).to(torch.bfloat16)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    s = {"case": c}
    if c["op"] == "rope":
        B, L, H, KV, hd = c["B"], c["L"], c["heads"], c["kv_heads"], c["head_dim"]
        stride = (H + 2 * KV) * hd + c["pad"]
        s["qkv"] = randn(B * L, stride).to(torch.bfloat16)
        s["wq"] = 1 + 0.1 * randn(hd) if c["norm"] else None
        s["wk"] = 1 + 0.1 * randn(hd) if c["norm"] else None
        side = max(1, int(round(L ** (1 / 3))))
        i = torch.arange(L, device="cuda")
        pos = torch.stack([i // (side * side) + c["offset"], i // side % side, i % side], 1).to(torch.float32)
        if c["fractional"]:
            pos[:, 2] = 2 * pos[:, 2] + 0.5
            pos[:, 0] += torch.rand(1, generator=gen, device="cuda")
        s["pos"] = pos.expand(B, L, 3).contiguous()
        for n, h in (("q", H), ("k", KV), ("v", KV)):
            s[n] = torch.empty((B, h, L, hd), dtype=torch.bfloat16, device="cuda")
    elif c["op"] in ("select", "attend"):
        B, Lq, Lk, H, KV, hd = c["B"], c["Lq"], c["Lk"], c["heads"], c["kv_heads"], c["head_dim"]
        nqb, nkb, topk = -(-Lq // QB), -(-Lk // c["block_k"]), c["topk"]
        s["q"], s["k"] = _field(B, H, Lq, hd, gen, 1.0), _field(B, KV, Lk, hd, gen, 1.0)
        s["kv_lens"] = _lens(B, Lk, c["ragged"], gen)
        s["q_lens"] = _lens(B, Lq, c["ragged"], gen) if Lq != Lk else s["kv_lens"]
        if c["op"] == "select":
            s["blocks"] = torch.empty((B, H, nqb, topk), dtype=torch.int32, device="cuda")
            s["counts"] = torch.empty((B, H, nqb), dtype=torch.int32, device="cuda")
        else:
            s["v"] = _field(B, KV, Lk, hd, gen, 0.5)
            pick = torch.rand((B, H, nqb, nkb), generator=gen, device="cuda").topk(topk, dim=-1).indices
            s["blocks"] = pick.sort(dim=-1).values.to(torch.int32)
            s["counts"] = torch.full((B, H, nqb), topk, dtype=torch.int32, device="cuda")
            if c["ragged"]:  # lists of different lengths, empty ones among them
                s["counts"] = torch.randint(0, topk + 1, (B, H, nqb), generator=gen, device="cuda").to(torch.int32)
            s["o"] = torch.zeros((B, Lq, H * hd), dtype=torch.bfloat16, device="cuda")
            s["absmax"] = torch.zeros(B * Lq, dtype=torch.float32, device="cuda") if c["absmax"] else None
    else:
        B, L, d = c["B"], c["L"], c["d"]
        s["y"] = (3 * randn(B * L, d)).to(torch.bfloat16)
        s["x"] = randn(B * L, d).to(torch.bfloat16)
        s["x"][:, :: max(1, d // 50)] *= 16  # the residual stream's outlier channels
        s["w_post"] = 1 + 0.1 * randn(d) if c["weight"] else None
        s["mod"] = 0.5 * randn(B, 3, d)  # gate, shift, scale of each item
        s["x_out"] = torch.empty_like(s["x"])
        if c["int8"]:
            s["codes"] = torch.empty((B * L, d), dtype=torch.int8, device="cuda")
            s["scales"] = torch.empty(B * L, dtype=torch.float32, device="cuda")
        s["h"] = torch.empty_like(s["x"])
    return s


# -------------------------------------------------------------------------------------- plain forms

def _angles(c, pos):
    """The angle of each rotated pair of lanes, [..., pairs], in 64 bits."""
    parts = []
    for axis, r in enumerate((c["rope_t"], c["rope_h"], c["rope_w"])):
        j = torch.arange(r // 2, device=pos.device, dtype=torch.float64)
        parts.append(pos[..., axis, None].double() * 10000.0 ** (-2 * j / max(r, 1)))
    return torch.cat(parts, -1)


def _plain_rope(s):
    c = s["case"]
    B, L, H, KV, hd = c["B"], c["L"], c["heads"], c["kv_heads"], c["head_dim"]
    ang = _angles(c, s["pos"])[:, None]
    cos, sin = ang.cos().float(), ang.sin().float()
    n = 2 * cos.shape[-1]
    x = s["qkv"][:, : (H + 2 * KV) * hd].view(B, L, H + 2 * KV, hd).transpose(1, 2)

    def turn(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
        a, b = x[..., 0:n:2], x[..., 1:n:2]
        r = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        return torch.cat([r, x[..., n:]], -1).to(torch.bfloat16)

    return {"q": turn(x[:, :H], s["wq"]), "k": turn(x[:, H: H + KV], s["wk"]), "v": x[:, H + KV:].contiguous()}


def _valid(lens, B, L, device):
    """[B][L]: whether a token is one of its item's."""
    i = torch.arange(L, device=device)
    return (i < (lens[:, None] if lens is not None else L)).expand(B, L)


def _block_means(x, lens, size):
    """Mean of each block's valid rows, in 64 bits, and how many there are."""
    B, H, L, hd = x.shape
    n = -(-L // size)
    ok = _valid(lens, B, L, x.device)
    x = torch.where(ok[:, None, :, None], x.double(), 0.0)
    x = torch.nn.functional.pad(x, (0, 0, 0, n * size - L)).view(B, H, n, size, hd).sum(3)
    num = torch.nn.functional.pad(ok, (0, n * size - L)).view(B, n, size).sum(2)
    return x / num.clamp(min=1)[:, None, :, None], num


def _plain_select(s):
    c = s["case"]
    B, H, KV, bk, topk = c["B"], c["heads"], c["kv_heads"], c["block_k"], c["topk"]
    qm, qn = _block_means(s["q"], s["q_lens"], QB)
    km, kn = _block_means(s["k"], s["kv_lens"], bk)
    nqb, nkb = qn.shape[1], kn.shape[1]
    score = torch.matmul(qm.view(B, KV, H // KV, nqb, -1), km[:, :, None].transpose(-1, -2)).view(B, H, nqb, nkb)
    i, j = torch.arange(nqb, device=score.device)[:, None], torch.arange(nkb, device=score.device)
    keep = j < c["first"]
    if c["local"]:
        keep = keep | ((j >= i * QB // bk - c["local"] + 1) & (j <= (i * QB + QB - 1) // bk + c["local"] - 1))
    score = torch.where(keep, math.inf, score)
    score = torch.where((kn > 0)[:, None, None], score, -math.inf)
    order = score.sort(dim=-1, descending=True, stable=True).indices[..., :topk]
    count = torch.minimum((kn > 0).sum(1), torch.tensor(topk, device=score.device))[:, None, None].expand(B, H, nqb)
    count = torch.where((qn > 0)[:, None], count, 0)
    listed_ = torch.arange(topk, device=score.device) < count[..., None]
    order = torch.where(listed_, order, nkb).sort(dim=-1).values
    return {"blocks": torch.where(listed_, order, -1).int(), "counts": count.int()}


def _plain_attend(s):
    c = s["case"]
    B, Lq, Lk, H, KV, hd, bk = (c[n] for n in ("B", "Lq", "Lk", "heads", "kv_heads", "head_dim", "block_k"))
    nqb, topk = s["counts"].shape[-1], c["topk"]
    dev = s["q"].device
    q = torch.nn.functional.pad(s["q"], (0, 0, 0, nqb * QB - Lq)).view(B, H, nqb, QB, hd).float()
    key = (s["blocks"][..., None] * bk + torch.arange(bk, device=dev)).flatten(-2)
    slot = torch.arange(topk * bk, device=dev) // bk < s["counts"][..., None]
    top = s["kv_lens"].view(B, 1, 1, 1) if s["kv_lens"] is not None else Lk
    ok = slot & (key >= 0) & (key < top)
    key = key.clamp(0, Lk - 1).long()
    b = torch.arange(B, device=dev).view(B, 1, 1, 1)
    h = (torch.arange(H, device=dev) // (H // KV)).view(1, H, 1, 1)
    score = torch.matmul(q, s["k"][b, h, key].float().transpose(-1, -2)) / math.sqrt(hd)
    score = score.masked_fill(~ok[..., None, :], -math.inf)
    m = score.amax(-1, keepdim=True)
    p = (score - torch.where(m == -math.inf, 0.0, m)).exp()
    del score
    o = torch.matmul(p, torch.where(ok[..., None], s["v"][b, h, key].float(), 0.0))
    total = p.sum(-1, keepdim=True)
    o = torch.where(total > 0, o / total, 0.0).view(B, H, nqb * QB, hd)[:, :, :Lq].transpose(1, 2).reshape(B, Lq, H * hd)
    o = torch.where(_valid(s["q_lens"], B, Lq, dev)[..., None], o, 0.0).to(torch.bfloat16)
    if s["absmax"] is None:
        return {"o": o}
    return {"o": o, "absmax": o.abs().amax(-1).view(-1)}


def _normed(x, kind, eps=1e-6):
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    if kind != "none":
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)
    return x


def _plain_resnorm(s):
    c = s["case"]
    gate, shift, scale = (s["mod"][:, i, None] for i in range(3))
    r = _normed(s["y"].float(), c["post"])
    if s["w_post"] is not None:
        r = r * s["w_post"]
    x = s["x"].float().view(c["B"], c["L"], -1) + c["alpha"] * gate * r.view(c["B"], c["L"], -1)
    x = x.to(torch.bfloat16)
    h = (_normed(x.float(), c["pre"]) * (1 + scale) + shift).to(torch.bfloat16)
    x, h = x.view(s["x"].shape), h.view(s["x"].shape)
    if not c["int8"]:
        return {"x": x, "h": h}
    sc = h.float().abs().amax(-1, keepdim=True) / 127
    code = torch.where(sc > 0, h.float() / sc, 0.0).round().clamp(-127, 127)
    return {"x": x, "h": (code * sc).to(torch.bfloat16)}


# ----------------------------------------------------------------------------------- the library's

def _own_rope(s):
    from video_diffusion_transformer_adaln_b200 import h3b
    c = s["case"]
    if "plan" not in s:
        s["plan"] = h3b.make_qk(c["B"], c["L"], c["heads"], c["kv_heads"], c["head_dim"],
                                (c["rope_t"], c["rope_h"], c["rope_w"]), row_stride=s["qkv"].shape[1])
    h3b.h3b_qk_norm_rope(s["plan"], s["qkv"], s["wq"], s["wk"], s["pos"], s["q"], s["k"], s["v"])
    return {"q": s["q"], "k": s["k"], "v": s["v"]}


def _sparse_plan(s):
    from video_diffusion_transformer_adaln_b200 import h3b
    c = s["case"]
    if "plan" not in s:
        s["plan"] = h3b.make_sparse(c["B"], c["heads"], c["kv_heads"], c["head_dim"], c["Lq"], c["Lk"], c["block_k"],
                                    c["topk"], c.get("first", 0), c.get("local", 0))
        s["ws"] = torch.empty(h3b.h3b_sparse_workspace_size(s["plan"]), dtype=torch.uint8, device="cuda")
    return h3b


def _own_select(s):
    h3b = _sparse_plan(s)
    h3b.h3b_select_blocks(s["plan"], s["q"], s["k"], s["q_lens"], s["kv_lens"], s["blocks"], s["counts"], s["ws"])
    return {"blocks": s["blocks"], "counts": s["counts"]}


def _own_attend(s):
    h3b = _sparse_plan(s)
    if s["absmax"] is not None:
        s["absmax"].zero_()
    h3b.h3b_attention_blocks(s["plan"], s["q"], s["k"], s["v"], s["q_lens"], s["kv_lens"], s["blocks"], s["counts"],
                             s["o"], s["absmax"], s["ws"])
    if s["absmax"] is None:
        return {"o": s["o"]}
    return {"o": s["o"], "absmax": s["absmax"].to(torch.bfloat16)}  # maxima of bf16 values


def _own_resnorm(s):
    from video_diffusion_transformer_adaln_b200 import h3b
    c = s["case"]
    if "plan" not in s:
        s["plan"] = h3b.make_residual_norm(c["B"] * c["L"], c["d"], c["L"], 3 * c["d"], post=c["post"], pre=c["pre"],
                                           alpha=c["alpha"])
    gate, shift, scale = (s["mod"][:, i] for i in range(3))
    if not c["int8"]:
        h3b.h3b_residual_norm(s["plan"], s["y"], s["w_post"], gate, s["x"], s["x_out"], shift, scale, h_out=s["h"])
        return {"x": s["x_out"], "h": s["h"]}
    h3b.h3b_residual_norm(s["plan"], s["y"], s["w_post"], gate, s["x"], s["x_out"], shift, scale, q=s["codes"],
                          s=s["scales"])
    torch.mul(s["codes"], s["scales"][:, None], out=s["h"])  # the values that the codes stand for
    return {"x": s["x_out"], "h": s["h"]}


def run(state):
    op = state["case"]["op"]
    if own:
        f = {"rope": _own_rope, "select": _own_select, "attend": _own_attend, "resnorm": _own_resnorm}[op]
    else:
        f = {"rope": _plain_rope, "select": _plain_select, "attend": _plain_attend, "resnorm": _plain_resnorm}[op]
    return f(state)


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["B"] * c["L"] * (c["heads"] + 2 * c["kv_heads"]) * c["head_dim"]
        return {"bytes": 4 * n + 12 * c["B"] * c["L"], "flops": 8 * n}
    if c["op"] == "resnorm":
        n = c["B"] * c["L"] * c["d"]
        return {"bytes": (7 if c["int8"] else 8) * n + 12 * c["B"] * c["d"], "flops": 12 * n}
    B, Lq, Lk, H, KV, hd, bk, topk = (c[n] for n in ("B", "Lq", "Lk", "heads", "kv_heads", "head_dim", "block_k",
                                                     "topk"))
    nqb, nkb = -(-Lq // QB), -(-Lk // bk)
    lists = 4 * B * H * nqb * (topk + 1)
    if c["op"] == "select":
        return {"bytes": 2 * hd * B * (H * Lq + KV * Lk) + lists,
                "flops": hd * B * (H * Lq + KV * Lk) + 2 * hd * B * H * nqb * nkb}
    share = 0.5 if c["ragged"] else 1.0  # listed keys, on average
    keys = min(KV * Lk, share * H * nqb * topk * bk)  # distinct key rows at most
    return {"bytes": 2 * hd * B * (2 * H * Lq + 2 * keys) + lists,
            "flops": 4 * hd * B * H * Lq * min(Lk, share * topk * bk)}


# --------------------------------------------------------------------------------------- in 64 bits

def _exact_rope(s):
    c = s["case"]
    B, L, H, KV, hd = c["B"], c["L"], c["heads"], c["kv_heads"], c["head_dim"]
    out = {}
    freq, axis = [], []
    for a, r in enumerate((c["rope_t"], c["rope_h"], c["rope_w"])):
        freq += [10000.0 ** (-2 * j / r) for j in range(r // 2)]
        axis += [a] * (r // 2)
    freq = torch.tensor(freq, dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       s["pos"].double()[:, :, axis] * freq)  # [B][L][pairs]
    n = 2 * len(axis)
    first = 0
    for name, heads, w in (("q", H, s["wq"]), ("k", KV, s["wk"]), ("v", KV, None)):
        got = torch.empty((B, heads, L, hd), dtype=torch.float64, device="cuda")
        for h in range(heads):
            x = s["qkv"][:, (first + h) * hd: (first + h + 1) * hd].double().reshape(B, L, hd)
            if w is not None:
                x = x / (x.square().sum(-1, keepdim=True) / hd + 1e-6).sqrt() * w.double()
            if name != "v":
                z = torch.view_as_complex(x[..., :n].reshape(B, L, -1, 2).contiguous()) * turn
                x = torch.cat([torch.view_as_real(z).reshape(B, L, n), x[..., n:]], -1)
            got[:, h] = x
        out[name] = got
        first += heads
    return out


def _exact_attend(s):
    c = s["case"]
    B, Lq, Lk, H, KV, hd, bk = (c[n] for n in ("B", "Lq", "Lk", "heads", "kv_heads", "head_dim", "block_k"))
    o = torch.zeros((B, Lq, H, hd), dtype=torch.float64, device="cuda")
    for b in range(B):
        kv_n = Lk if s["kv_lens"] is None else int(s["kv_lens"][b])
        q_n = Lq if s["q_lens"] is None else int(s["q_lens"][b])
        for h in range(H):
            k, v = (s[n][b, h // (H // KV), :kv_n].double() for n in ("k", "v"))
            q = s["q"][b, h, :q_n].double()
            n = -(-q_n // QB)
            at = torch.stack([s["blocks"][b, h, :n].long() * bk + e for e in range(bk)], -1)  # [n][topk][bk]
            for slot in range(at.shape[1]):
                at[:, slot][s["counts"][b, h, :n] <= slot] = -1
            at[at >= kv_n] = -1
            at = at.view(n, -1)
            qs = torch.zeros((n * QB, hd), dtype=torch.float64, device="cuda")
            qs[:q_n] = q
            if kv_n:
                ks, vs = k[at.clamp(min=0)], v[at.clamp(min=0)]
                w = torch.bmm(qs.view(-1, QB, hd), ks.transpose(1, 2)) / hd ** 0.5
                w = w.masked_fill((at < 0)[:, None], -math.inf).softmax(-1).nan_to_num(0.0)
                o[b, :q_n, h] = torch.bmm(w, vs).view(-1, hd)[:q_n]
    o = o.view(B, Lq, H * hd)
    return {"o": o} if s["absmax"] is None else {"o": o, "absmax": o.abs().amax(-1).view(-1)}


def _exact_resnorm(s):
    c = s["case"]
    rows, d = s["y"].shape
    x_out, h_out = (torch.empty((rows, d), dtype=torch.float64, device="cuda") for _ in range(2))
    for b in range(c["B"]):
        at = slice(b * c["L"], (b + 1) * c["L"])
        gate, shift, scale = s["mod"][b].double()
        y, x = s["y"][at].double(), s["x"][at].double()
        if c["post"] == "rms":
            y = y / (y.square().sum(1, keepdim=True) / d + 1e-6).sqrt()
        elif c["post"] == "layer":
            y = (y - y.sum(1, keepdim=True) / d) / (y.var(1, unbiased=False, keepdim=True) + 1e-6).sqrt()
        if s["w_post"] is not None:
            y = y * s["w_post"].double()
        x_out[at] = x + c["alpha"] * gate * y
        z = x_out[at].to(torch.bfloat16).double()  # the stream is held in bf16: the next norm reads that
        if c["pre"] == "layer":
            z = z - z.sum(1, keepdim=True) / d
        z = z / (z.square().sum(1, keepdim=True) / d + 1e-6).sqrt()
        z = z * (1 + scale) + shift
        if c["int8"]:  # the quantizer's input is the bf16 activation
            z = z.to(torch.bfloat16).double()
            step = z.abs().amax(1, keepdim=True) / 127
            z = (z / step.clamp(min=1e-300)).round() * step
        h_out[at] = z
    return {"x": x_out, "h": h_out}


def exact(case, seed):
    if case["op"] == "select":
        return None  # whole numbers
    s = prepare(case, seed)
    return {"rope": _exact_rope, "attend": _exact_attend, "resnorm": _exact_resnorm}[case["op"]](s)
