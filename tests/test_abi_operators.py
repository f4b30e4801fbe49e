"""The host side of the operators beside the block (no GPU): refusals before any launch, empty
problems, workspace sizes, and what the binding passes to the C entry points."""
import ctypes as C

import pytest
import torch

from video_diffusion_transformer_adaln_b200 import build, h3b

ARG, SHAPE, ALIGN, WORKSPACE = -1, -2, -3, -4
P = 0x10000  # a placeholder device pointer: never dereferenced, every refusal comes before a launch


@pytest.fixture(scope="module")
def L():
    build.build()
    return h3b.lib()


def edit(d, kw):
    for k, v in kw.items():
        setattr(d, k, v)
    return d


# ---- h3b_qk_norm_rope

def qk(**kw):
    return edit(h3b.make_qk(2, 10, 4, 2, 64, (16, 24, 24)), kw)


def call_qk(L, d, qkv=P, wq=P, wk=P, pos=P, q=P, k=P, v=P):
    return L.h3b_qk_norm_rope(None if d is None else C.byref(d), qkv, wq, wk, pos, q, k, v, None)


@pytest.mark.parametrize("kw,status", [
    ({"head_dim": 96}, SHAPE), ({"n_heads": 0}, SHAPE), ({"n_kv_heads": 0}, SHAPE), ({"n_heads": 1023}, SHAPE),
    ({"n_heads": 2 ** 31 - 1}, SHAPE), ({"B": -1}, SHAPE), ({"L": -1}, SHAPE), ({"B": 2 ** 16, "L": 2 ** 15}, SHAPE),
    ({"rope_t": 15}, SHAPE), ({"rope_t": 32}, SHAPE), ({"rope_w": -2}, SHAPE), ({"rope_t": 2 ** 31 - 2}, SHAPE),
    ({"rope_theta": 0.0}, ARG), ({"rope_theta": float("nan")}, ARG), ({"norm_eps": -1.0}, ARG),
    ({"row_stride": 8 * 64 - 8}, SHAPE), ({"row_stride": 8 * 64 + 4}, SHAPE), ({"row_stride": 2 ** 40}, SHAPE),
])
def test_qk_refuses_dimensions(L, kw, status):
    assert call_qk(L, qk(**kw)) == status
    assert L.h3b_last_error_detail()


def test_qk_refuses_pointers(L):
    assert call_qk(L, None) == ARG
    for name in ("qkv", "q", "k", "v"):
        assert call_qk(L, qk(), **{name: None}) == ARG
    for name in ("qkv", "wq", "wk", "pos", "q", "k", "v"):
        assert call_qk(L, qk(), **{name: P + 8}) == ALIGN


@pytest.mark.parametrize("kw", [{"B": 0}, {"L": 0}])
def test_qk_empty_problem(L, kw):
    assert call_qk(L, qk(**kw), *[None] * 7) == 0


# ---- h3b_select_blocks, h3b_attention_blocks

def sparse(**kw):
    return edit(h3b.make_sparse(2, 4, 2, 64, 300, 1000, 64, 5), kw)


def call_select(L, d, q=P, k=P, q_lens=P, kv_lens=P, blocks=P, counts=P, ws=P, n=1 << 40):
    return L.h3b_select_blocks(None if d is None else C.byref(d), q, k, q_lens, kv_lens, blocks, counts, ws, n, None)


def call_attend(L, d, q=P, k=P, v=P, q_lens=P, kv_lens=P, blocks=P, counts=P, o=P, absmax=P, ws=P, n=1 << 40):
    return L.h3b_attention_blocks(None if d is None else C.byref(d), q, k, v, q_lens, kv_lens, blocks, counts, o,
                                  absmax, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    ({"head_dim": 80}, SHAPE), ({"block_k": 32}, SHAPE), ({"block_k": 256}, SHAPE), ({"n_heads": 3}, SHAPE),
    ({"n_heads": 0}, SHAPE), ({"n_kv_heads": 0}, SHAPE), ({"n_kv_heads": -1}, SHAPE), ({"B": -1}, SHAPE),
    ({"Lq": -1}, SHAPE), ({"Lk": 0}, SHAPE), ({"B": 20000}, SHAPE), ({"B": 4096, "Lq": 2 ** 19}, SHAPE),
    ({"Lk": 64 * 4096 + 1}, SHAPE), ({"topk": 0}, SHAPE), ({"topk": 17}, SHAPE), ({"keep_first": -1}, ARG),
    ({"keep_local": -1}, ARG), ({"keep_first": 6}, SHAPE), ({"keep_local": 3}, SHAPE),
    ({"keep_local": 2 ** 31 - 1}, SHAPE), ({"keep_first": 4, "keep_local": 1}, SHAPE),
])
def test_sparse_refuses_dimensions(L, kw, status):
    n = C.c_size_t(0)
    assert L.h3b_sparse_workspace_size(C.byref(sparse(**kw)), C.byref(n)) == status
    assert call_select(L, sparse(**kw)) == status
    assert call_attend(L, sparse(**kw)) == status


def test_sparse_limits_are_reached(L):
    for kw in ({"Lk": 64 * 4096}, {"Lk": 128 * 4096, "block_k": 128}, {"topk": 16}, {"keep_first": 3, "keep_local": 1},
               {"topk": 16, "keep_first": 16, "keep_local": 16}, {"B": 16383}):
        n = C.c_size_t(0)
        assert L.h3b_sparse_workspace_size(C.byref(sparse(**kw)), C.byref(n)) == 0


def test_sparse_refuses_pointers_and_workspaces(L):
    d = sparse()
    need = h3b.h3b_sparse_workspace_size(d)
    assert need > 0 and need % 256 == 0
    assert L.h3b_sparse_workspace_size(C.byref(d), None) == ARG
    assert call_select(L, None) == ARG and call_attend(L, None) == ARG
    for name in ("q", "k", "blocks", "counts", "ws"):
        assert call_select(L, d, **{name: None}) == ARG
    for name in ("q", "k", "v", "blocks", "o", "ws"):
        assert call_attend(L, d, **{name: None}) == ARG
    for name in ("q", "k", "blocks", "counts", "q_lens", "kv_lens"):
        assert call_select(L, d, **{name: P + 4}) == ALIGN
    for name in ("q", "k", "v", "blocks", "counts", "q_lens", "kv_lens", "o", "absmax"):
        assert call_attend(L, d, **{name: P + 4}) == ALIGN
    for call in (call_select, call_attend):
        assert call(L, d, ws=P + 16) == ALIGN
        assert call(L, d, n=need - 1) == WORKSPACE


@pytest.mark.parametrize("kw", [{"B": 0}, {"Lq": 0}])
def test_sparse_empty_problem(L, kw):
    assert call_select(L, sparse(**kw), *[None] * 7) == 0
    assert call_attend(L, sparse(**kw), *[None] * 10) == 0


# ---- h3b_residual_norm

def rn(**kw):
    return edit(h3b.make_residual_norm(20, 256, 10, 768), kw)


def call_rn(L, d, y=P, w=P, gate=P, x=P, x_out=P, shift=P, scale=P, h=P, q=P, s=P, zero=P):
    return L.h3b_residual_norm(None if d is None else C.byref(d), y, w, gate, x, x_out, shift, scale, h, q, s, zero,
                               None)


@pytest.mark.parametrize("kw,status", [
    ({"rows": -1}, SHAPE), ({"d": 0}, SHAPE), ({"d": 12}, SHAPE), ({"d": 8200}, SHAPE), ({"rows_per_item": 0}, ARG),
    ({"mod_stride": -4}, ARG), ({"mod_stride": 770}, ARG), ({"post_norm": 3}, ARG), ({"pre_norm": -1}, ARG),
    ({"post_eps": -1.0}, ARG), ({"pre_eps": float("nan")}, ARG),
])
def test_residual_norm_refuses_dimensions(L, kw, status):
    assert call_rn(L, rn(**kw)) == status


def test_residual_norm_refuses_pointers(L):
    assert call_rn(L, None) == ARG
    for name in ("y", "x", "x_out", "q", "s"):  # codes and scales go together
        assert call_rn(L, rn(), **{name: None}) == ARG
    for name in ("y", "w", "gate", "x", "x_out", "shift", "scale", "h", "q", "s", "zero"):
        assert call_rn(L, rn(), **{name: P + 8}) == ALIGN


def test_residual_norm_empty_problem(L):
    assert call_rn(L, rn(rows=0), *[None] * 11) == 0


# ---- the binding

class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def fn(*args):
            self.calls.append((name, args))
            return 0
        return fn


def test_binding_passes_the_arguments_in_order(monkeypatch):
    rec = Recorder()
    monkeypatch.setattr(h3b, "_LIB", rec)
    t = [torch.empty(4) for _ in range(12)]
    p = [x.data_ptr() for x in t]
    d = qk()
    assert d.row_stride == 8 * 64 and d.norm_eps == pytest.approx(1e-6) and d.rope_theta == 10000.0
    h3b.h3b_qk_norm_rope(d, t[0], None, t[1], t[2], t[3], t[4], t[5], stream=3)
    name, args = rec.calls[-1]
    assert name == "h3b_qk_norm_rope" and args[0]._obj is d and args[1:] == (p[0], None, *p[1:6], 3)
    d = sparse()
    assert (d.nqb, d.nkb) == (3, 16)
    ws = torch.empty(100, dtype=torch.uint8)
    h3b.h3b_select_blocks(d, t[0], t[1], None, t[2], t[3], t[4], ws, stream=3)
    name, args = rec.calls[-1]
    assert name == "h3b_select_blocks" and args[1:] == (p[0], p[1], None, *p[2:5], ws.data_ptr(), 100, 3)
    h3b.h3b_attention_blocks(d, t[0], t[1], t[2], t[3], None, t[4], None, t[5], None, ws, stream=3)
    name, args = rec.calls[-1]
    assert name == "h3b_attention_blocks"
    assert args[1:] == (*p[:4], None, p[4], None, p[5], None, ws.data_ptr(), 100, 3)
    d = h3b.make_residual_norm(20, 256, 10, 768, post="layer", pre="none", alpha=0.5)
    assert (d.post_norm, d.pre_norm, d.alpha) == (2, 0, 0.5)
    h3b.h3b_residual_norm(d, *t[:7], h_out=t[7], q=t[8], s=t[9], absmax_zero=t[10], stream=3)
    name, args = rec.calls[-1]
    assert name == "h3b_residual_norm" and args[1:] == (*p[:11], 3)
    h3b.h3b_residual_norm(d, *t[:7], stream=3)
    assert rec.calls[-1][1][8:] == (None, None, None, None, 3)


def test_structs_have_the_header_layout():
    """Field for field as include/h3b.h declares them (ints, then floats, 8-byte stride last)."""
    assert C.sizeof(h3b.QkDims) == 48 and h3b.QkDims.row_stride.offset == 40 and h3b.QkDims.rope_theta.offset == 32
    assert C.sizeof(h3b.SparseDims) == 40 and h3b.SparseDims.keep_local.offset == 36
    assert C.sizeof(h3b.ResidualNormDims) == 36 and h3b.ResidualNormDims.post_eps.offset == 24


def test_grid_positions():
    from video_diffusion_transformer_adaln_b200.runtime import grid_positions
    d = h3b.make_dims(2, 2, 3, 4, 256, 4, 64, 256, (16, 24, 24))
    pos = grid_positions(d, offset=(10.0, 0.0, 0.5), step=(0.5, 1.0, 2.0), device="cpu")
    assert pos.shape == (2, 24, 3) and pos.dtype == torch.float32 and pos.is_contiguous()
    for l in range(24):
        assert pos[1, l].tolist() == [10.0 + 0.5 * (l // 12), float(l // 4 % 3), 0.5 + 2.0 * (l % 4)]


@pytest.mark.parametrize("bad", [
    dict(pos=torch.zeros(1, 8, 3)),                             # of one item where the grid has two
    dict(pos=torch.zeros(1, 8, 3).expand(2, -1, -1)),           # not laid out
    dict(pos=torch.zeros(2, 8, 3, dtype=torch.float64)),
    dict(x=torch.zeros(2, 8, 256)),                             # fp32
    dict(x=torch.zeros(2, 8, 512, dtype=torch.bfloat16)[..., :256]),
    dict(c=torch.zeros(1, 256)),
])
def test_sparse_block_refuses_tensors_that_do_not_fit(L, bad):
    from types import SimpleNamespace
    from video_diffusion_transformer_adaln_b200.runtime import SparseBlockState, sparse_block_forward
    dims = h3b.make_dims(2, 1, 2, 4, 256, 4, 64, 512, (16, 24, 24))
    state = SparseBlockState(dims, device="cpu")
    good = dict(c=torch.zeros(2, 256), x=torch.zeros(2, 8, 256, dtype=torch.bfloat16), pos=torch.zeros(2, 8, 3))
    with pytest.raises(ValueError, match=next(iter(bad))):
        sparse_block_forward(state, SimpleNamespace(tensors={}), {}, **{**good, **bad})
