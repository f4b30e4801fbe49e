"""The gated residual with norms on both sides against the formula in 64 bits.

Tolerances: x_out is one bf16 rounding (2^-8) of an fp32 sum whose added part is off by less
than 2^-19 of it (a norm over at most 8192 channels by a tree of fp32 sums, a root, a division
and three products). h is compared with the norm of the x_out that was written: one rounding,
and an fp32 error below 2^-18 of (|x| + |mean|) rstd |1 + scale| + |shift|. The codes and scales
are those of the written h exactly."""
import pytest
import torch

import operator_refs as R
from gpu_helpers import no_device_error, require_gpu
from video_diffusion_transformer_adaln_b200 import h3b

pytestmark = pytest.mark.gpu


def make(rows, d, items, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    y, x = (3 * r(rows, d) + 0.5).to(torch.bfloat16), (r(rows, d) + 0.25).to(torch.bfloat16)
    x[:, :: max(1, d // 10)] *= 16
    return y, x, 1 + 0.2 * r(d), 0.5 * r(items, 3, d)


def check(rows, d, post, pre, rpi, alpha=1.0, weight=True, gated=True, modulated=True, in_place=False, seed=0):
    items = -(-rows // rpi)
    y, x, w, mod = make(rows, d, items, seed)
    w = w if weight else None
    gate, shift, scale = mod[:, 0], mod[:, 1], mod[:, 2]
    gate = gate if gated else None
    shift, scale = (shift, scale) if modulated else (None, None)
    dims = h3b.make_residual_norm(rows, d, rpi, 3 * d, post, pre, 1e-6, 1e-5, alpha)
    x_in = x.clone()
    x_out = x if in_place else torch.full_like(x, 7.0)
    h = torch.full_like(x, 7.0)
    q = torch.full((rows, d), 77, dtype=torch.int8, device="cuda")
    s = torch.full((rows,), 7.0, device="cuda")
    zero = torch.full((rows,), 7.0, device="cuda")
    h3b.h3b_residual_norm(dims, y, w, gate, x, x_out, shift, scale, h_out=h, q=q, s=s, absmax_zero=zero)
    ref, added = R.residual_out(y, w, gate, x_in, alpha, post, 1e-6, rpi)
    if not in_place:
        assert torch.equal(x, x_in)
    assert ((x_out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -19 * (added.abs() + x_in.double().abs())).all()
    hr = R.modulated(x_out, shift, scale, pre, 1e-5, rpi)
    xd = x_out.double()
    mean = xd.mean(-1, keepdim=True) if pre == "layer" else torch.zeros_like(xd[:, :1])
    rstd = 1.0 if pre == "none" else 1 / torch.sqrt(((xd - mean) ** 2).mean(-1, keepdim=True) + 1e-5)
    item = torch.arange(rows, device="cuda") // rpi
    size = (xd.abs() + mean.abs()) * rstd
    if modulated:
        size = size * (1 + scale.double()[item]).abs() + shift.double()[item].abs()
    assert ((h.double() - hr).abs() <= 2.0 ** -8 * hr.abs() + 2.0 ** -18 * size).all()
    qr, sr = R.quantized(h)
    assert torch.equal(s, sr) and torch.equal(q, qr)
    assert (zero == 0).all()
    no_device_error()
    # without h the codes are the same, without codes h is
    x2 = x_in.clone()
    q2, s2, h2 = torch.empty_like(q), torch.empty_like(s), torch.empty_like(h)
    h3b.h3b_residual_norm(dims, y, w, gate, x2, x2, shift, scale, q=q2, s=s2)
    assert torch.equal(q2, q) and torch.equal(s2, s) and torch.equal(x2, x_out)
    x3 = torch.empty_like(x_in)
    h3b.h3b_residual_norm(dims, y, w, gate, x_in, x3, shift, scale, h_out=h2)
    assert torch.equal(h2, h) and torch.equal(x3, x_out)
    x4 = torch.empty_like(x_in)
    h3b.h3b_residual_norm(dims, y, w, gate, x_in, x4, shift, scale)
    assert torch.equal(x4, x_out)


@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
def test_norm_kinds(post, pre):
    require_gpu()
    check(37, 1552, post, pre, 20, alpha=0.7)


@pytest.mark.parametrize("d", [8, 16, 24, 248, 256, 264, 1024, 1032, 1544, 2048, 2056, 4096, 4104, 5120, 8184, 8192])
def test_widths(d):
    require_gpu()
    check(13, d, "rms", "layer", 13, seed=d)


@pytest.mark.parametrize("rows,rpi", [(1, 1), (1, 5), (3, 1), (130, 33), (2000, 777), (5000, 5000)])
def test_rows_and_items(rows, rpi):
    require_gpu()
    check(rows, 256, "rms", "layer", rpi, in_place=True)


@pytest.mark.parametrize("rows,d,rpi", [(9600, 256, 2400), (9500, 264, 9500), (2500, 5120, 833), (5000, 2056, 2500),
                                        (1300, 8192, 1300)])
def test_many_rows_share_an_item(rows, d, rpi):
    """The item's vectors folded in shared memory; items end inside a pass."""
    require_gpu()
    check(rows, d, "rms", "layer", rpi, alpha=0.7, in_place=True)


@pytest.mark.parametrize("weight,gated,modulated", [(False, True, True), (True, False, True), (True, True, False),
                                                    (False, False, False)])
def test_optional_vectors(weight, gated, modulated):
    require_gpu()
    check(29, 768, "rms", "rms", 10, weight=weight, gated=gated, modulated=modulated)
    check(29, 5120, "layer", "layer", 29, weight=weight, gated=gated, modulated=modulated)
    check(9600, 128, "layer", "rms", 4800, weight=weight, gated=gated, modulated=modulated)


def test_rows_without_spread_and_zero_rows():
    """A zero branch adds nothing, a constant stream row has LayerNorm zero and h = shift."""
    require_gpu()
    rows, d = 4, 512
    y, x, w, mod = make(rows, d, 1, 3)
    y[0], x[1], x[2], y[2] = 0, 0, 2.0, 0
    y[1] = 0
    dims = h3b.make_residual_norm(rows, d, rows, 3 * d, "rms", "layer")
    x_out, h = torch.empty_like(x), torch.empty_like(x)
    q, s = torch.empty((rows, d), dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    h3b.h3b_residual_norm(dims, y, w, mod[:, 0], x, x_out, mod[:, 1], mod[:, 2], h_out=h, q=q, s=s)
    assert torch.equal(x_out[:3], x[:3])
    assert torch.equal(h[2], mod[0, 1].to(torch.bfloat16)) and torch.equal(h[1], h[2])
    qr, sr = R.quantized(h)
    assert torch.equal(q, qr) and torch.equal(s, sr)
    z = torch.zeros_like(x)
    h3b.h3b_residual_norm(dims, z, None, None, z, x_out, None, None, h_out=h, q=q, s=s)
    assert (x_out == 0).all() and (h == 0).all() and (q == 0).all() and (s == 0).all()


def test_a_non_finite_row_stays_in_its_row():
    require_gpu()
    rows, d = 40, 264
    y, x, w, mod = make(rows, d, 1, 4)
    dims = h3b.make_residual_norm(rows, d, rows, 3 * d, "rms", "layer")
    out = [torch.empty_like(x) for _ in range(4)]
    h3b.h3b_residual_norm(dims, y, w, mod[:, 0], x, out[0], mod[:, 1], mod[:, 2], h_out=out[1])
    y[11, 100], x[23, 3] = float("inf"), float("nan")
    h3b.h3b_residual_norm(dims, y, w, mod[:, 0], x, out[2], mod[:, 1], mod[:, 2], h_out=out[3])
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[11] = keep[23] = False
    assert torch.equal(out[0][keep], out[2][keep]) and torch.equal(out[1][keep], out[3][keep])
    assert out[3][23].isnan().all() and not out[2][11].isfinite().all()


def test_neighbours_are_not_written():
    require_gpu()
    rows, d = 9, 1544
    y, x, w, mod = make(rows, d, 1, 5)
    dims = h3b.make_residual_norm(rows, d, rows, 3 * d)
    bufs = [torch.full((rows * d + 128,), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    codes = torch.full((rows * d + 128,), 5, dtype=torch.int8, device="cuda")
    s = torch.full((rows + 8,), 5.0, device="cuda")
    xo, h = (b[64:-64].view(rows, d) for b in bufs)
    h3b.h3b_residual_norm(dims, y, w, mod[:, 0], x, xo, mod[:, 1], mod[:, 2], h_out=h,
                          q=codes[64:-64].view(rows, d), s=s[4:-4])
    for b in (*bufs, codes):
        assert (b[:64] == 5).all() and (b[-64:] == 5).all()
    assert (s[:4] == 5).all() and (s[-4:] == 5).all()


def test_on_another_stream_and_in_a_graph():
    require_gpu()
    rows, d = 600, 1024
    y, x, w, mod = make(rows, d, 2, 6)
    dims = h3b.make_residual_norm(rows, d, 300, 3 * d, "layer", "rms")
    want, got = [torch.empty_like(x) for _ in range(2)], [torch.empty_like(x) for _ in range(2)]

    def call(out, stream=None):
        h3b.h3b_residual_norm(dims, y, w, mod[:, 0], x, out[0], mod[:, 1], mod[:, 2], h_out=out[1], stream=stream)

    call(want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    call(got, side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(got)
    x.copy_(x.flip(0))
    call(want)
    for _ in range(2):
        [t.zero_() for t in got]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("rpi", [65, 10 ** 6, 2 ** 31 - 1])
@pytest.mark.parametrize("rows,d", [(64, 256), (5, 5120), (1, 8)])
def test_items_longer_than_the_rows(rows, d, rpi):
    require_gpu()
    check(rows, d, "rms", "layer", rpi)


def test_non_finite_rows_have_non_finite_scales():
    require_gpu()
    rows, d = 24, 528
    y, x, w, mod = make(rows, d, 1, 7)
    x[3, 5], x[7, 9], y[11, 0] = float("nan"), float("inf"), float("-inf")
    x[15, 500], x[15, 7] = float("nan"), float("inf")
    for pre in ("none", "layer"):
        dims = h3b.make_residual_norm(rows, d, rows, 3 * d, "rms", pre)
        x_out, h = torch.empty_like(x), torch.empty_like(x)
        q, s = torch.empty((rows, d), dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
        h3b.h3b_residual_norm(dims, y, w, mod[:, 0], x, x_out, mod[:, 1], mod[:, 2], h_out=h, q=q, s=s)
        assert torch.equal(s.isnan(), h.isnan().any(-1)) and torch.equal(s.isfinite(), h.isfinite().all(-1))
        ok = h.isfinite().all(-1)
        assert int(ok.sum()) == rows - 4
        qr, sr = R.quantized(h[ok])
        assert torch.equal(q[ok], qr) and torch.equal(s[ok], sr)
