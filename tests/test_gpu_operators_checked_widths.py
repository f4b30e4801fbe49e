"""The gated residual norms at widths of two vectors per thread (264 to 512 channels), the item's vectors staged and
read row by row, in the checked build and without programmatic dependent launch: the bits of the normal build, and a
clear error word."""
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
    g = torch.Generator(device="cuda").manual_seed(2)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    bf = lambda *s: randn(*s).to(torch.bfloat16)  # noqa: E731
    for n, (rows, d, rpi) in enumerate([(37, 264, 20), (700, 264, 350), (41, 392, 7), (3000, 392, 3000), (9, 512, 9),
                                        (1201, 512, 601)]):
        x_out, h = bf(rows, d), bf(rows, d)
        q, s = torch.zeros((rows, d), dtype=torch.int8, device="cuda"), torch.zeros(rows, device="cuda")
        mod = randn(-(-rows // rpi), 3, d)
        h3b.h3b_residual_norm(h3b.make_residual_norm(rows, d, rpi, 3 * d), bf(rows, d), 1 + randn(d), mod[:, 0], bf(rows, d),
                              x_out, mod[:, 1], mod[:, 2], h_out=h, q=q, s=s)
        out[f"x{n}"], out[f"h{n}"], out[f"q{n}"], out[f"s{n}"] = bf16_host(x_out), bf16_host(h), q.cpu().numpy(), s.cpu().numpy()
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
    code = (f"import sys; sys.path[:0] = [{HERE!r}, {os.path.dirname(HERE)!r}]; "
            f"import test_gpu_operators_checked_widths as t; t.child({path!r})")
    r = subprocess.run([sys.executable, "-c", code], env=dict(full, **env), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    got = dict(np.load(path))
    assert got["checked"][0] == checked and got["error_word"][0] == 0
    for k, v in ref.items():
        if k != "checked":
            assert np.array_equal(got[k], v), k
