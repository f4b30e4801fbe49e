"""The operators beside the block in the checked build (every computed global index tested against its buffer)
and without programmatic dependent launch: the same bits as the normal build's, and a clear error word. The child
process loads the other library (or launch mode); see test_gpu_checked.py for the block's own cases."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from gpu_helpers import bf16_host, require_gpu

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def run_cases():
    from video_diffusion_transformer_adaln_b200 import h3b

    out = {}
    g = torch.Generator(device="cuda").manual_seed(1)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    bf = lambda *s: randn(*s).to(torch.bfloat16)  # noqa: E731
    # rotary positions: cut boxes of heads and tokens, padded rows
    for n, (B, L, H, KV, dh, rope, pad) in enumerate([(2, 77, 6, 2, 128, (16, 24, 24), 8), (1, 3001, 18, 18, 64, (16, 24, 24), 0)]):
        stride = (H + 2 * KV) * dh + pad
        o = [torch.zeros((B, h, L, dh), dtype=torch.bfloat16, device="cuda") for h in (H, KV, KV)]
        h3b.h3b_qk_norm_rope(h3b.make_qk(B, L, H, KV, dh, rope, row_stride=stride), bf(B * L, stride), 1 + randn(dh),
                             1 + randn(dh), 50 * randn(B, L, 3), *o)
        out.update({f"rope{n}_{p}": bf16_host(t) for p, t in zip("qkv", o)})
    # selection and attention: padded items, split lists, many pairs per CTA, one token
    for n, (B, H, KV, dh, Lq, Lk, bk, topk) in enumerate([(2, 4, 2, 128, 777, 777, 64, 5), (3, 32, 8, 64, 1024, 900, 128, 7),
                                                          (2, 3, 1, 128, 5, 9000, 64, 100), (4, 8, 2, 128, 1, 3000, 64, 20),
                                                          (1, 1, 1, 64, 130, 64 * 1600, 64, 30)]):
        q, k, v = bf(B, H, Lq, dh), bf(B, KV, Lk, dh), bf(B, KV, Lk, dh)
        d = h3b.make_sparse(B, H, KV, dh, Lq, Lk, bk, topk, 1)
        lens = torch.tensor([max(1, Lk - 70 * b) for b in range(B)], dtype=torch.int32, device="cuda")
        ws = torch.zeros(h3b.h3b_sparse_workspace_size(d), dtype=torch.uint8, device="cuda")
        blocks = torch.zeros((B, H, d.nqb, topk), dtype=torch.int32, device="cuda")
        counts = torch.zeros((B, H, d.nqb), dtype=torch.int32, device="cuda")
        h3b.h3b_select_blocks(d, q, k, None, lens, blocks, counts, ws)
        o = torch.zeros((B, Lq, H * dh), dtype=torch.bfloat16, device="cuda")
        am = torch.zeros(B * Lq, device="cuda")
        h3b.h3b_attention_blocks(d, q, k, v, None, lens, blocks, counts, o, am, ws)
        out[f"select{n}"], out[f"counts{n}"] = blocks.cpu().numpy(), counts.cpu().numpy()
        out[f"attend{n}"], out[f"absmax{n}"] = bf16_host(o), am.cpu().numpy()
    # residual norms: every number of vectors per thread, staged and direct vectors
    for n, (rows, d, rpi) in enumerate([(37, 1552, 20), (13, 8184, 13), (9, 8, 2), (10000, 256, 5000), (4000, 1280, 4000)]):
        x_out, h = bf(rows, d), bf(rows, d)
        q, s = torch.zeros((rows, d), dtype=torch.int8, device="cuda"), torch.zeros(rows, device="cuda")
        items = -(-rows // rpi)
        mod = randn(items, 3, d)
        h3b.h3b_residual_norm(h3b.make_residual_norm(rows, d, rpi, 3 * d), bf(rows, d), 1 + randn(d), mod[:, 0], bf(rows, d),
                              x_out, mod[:, 1], mod[:, 2], h_out=h, q=q, s=s)
        out[f"rn_x{n}"], out[f"rn_h{n}"], out[f"rn_q{n}"], out[f"rn_s{n}"] = (bf16_host(x_out), bf16_host(h), q.cpu().numpy(),
                                                                             s.cpu().numpy())
    torch.cuda.synchronize()
    out["error_word"] = np.array([h3b.h3b_device_error(clear=True)], np.uint32)
    out["checked"] = np.array([int(h3b.h3b_checked_build())], np.int32)
    return out


def child(path):
    np.savez(path, **run_cases())


@pytest.mark.parametrize("env,checked", [({"H3B_CHECKED": "1"}, 1), ({"H3B_PDL": "0"}, 0)])
def test_same_bits(tmp_path, env, checked):
    require_gpu()
    from video_diffusion_transformer_adaln_b200 import build
    build.build(checked=True)
    ref = run_cases()
    assert ref["checked"][0] == 0 and ref["error_word"][0] == 0
    path = str(tmp_path / "other.npz")
    full = {k: v for k, v in os.environ.items() if k not in ("H3B_CHECKED", "H3B_PDL")}
    code = f"import sys; sys.path[:0] = [{HERE!r}, {os.path.dirname(HERE)!r}]; import test_gpu_operators_checked as t; t.child({path!r})"
    r = subprocess.run([sys.executable, "-c", code], env=dict(full, **env), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    got = dict(np.load(path))
    assert got["checked"][0] == checked and got["error_word"][0] == 0
    for k, v in ref.items():
        if k != "checked":
            assert np.array_equal(got[k], v), k
