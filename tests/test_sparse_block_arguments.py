"""What sparse_block_forward refuses before anything is launched (no GPU): tensors on another device than the state's, norm
weights and projections of another type, length or layout than the kernels read, names that it does not know. A recording
stand-in takes the library's calls once the state is made."""
from types import SimpleNamespace

import pytest
import torch

from video_diffusion_transformer_adaln_b200 import build, h3b
from video_diffusion_transformer_adaln_b200.runtime import SparseBlockState, sparse_block_forward

D, F = 256, 512


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def fn(*args):
            self.calls.append(name)
            return 0
        return fn


@pytest.fixture
def call(monkeypatch):
    build.build()
    state = SparseBlockState(h3b.make_dims(2, 1, 2, 4, D, 4, 64, F, (16, 24, 24)), device="cpu")
    rec = Recorder()
    monkeypatch.setattr(h3b, "_LIB", rec)
    monkeypatch.setattr(h3b, "_s", lambda stream: 0)
    i8, f32 = torch.int8, torch.float32
    tensors = {"w_ada": torch.zeros(6 * D, D, dtype=torch.bfloat16), "b_ada": torch.zeros(6 * D)}
    for w, s, b, n, k in (("wqkv", "sqkv", "bqkv", 3 * D, D), ("wo", "so", "bo", D, D), ("w1", "s1", "b1", F, D),
                          ("w2", "s2", "b2", D, F)):
        tensors.update({w: torch.zeros(n, k, dtype=i8), s: torch.zeros(n, dtype=f32), b: torch.zeros(n, dtype=f32)})
    norms = {"q": torch.zeros(64), "k": torch.zeros(64), "post_attn": torch.zeros(D), "post_mlp": torch.zeros(D)}
    args = dict(c=torch.zeros(2, D), x=torch.zeros(2, 8, D, dtype=torch.bfloat16), pos=torch.zeros(2, 8, 3))

    def run(norm=None, weight=None, **kw):
        n, w = {**norms, **(norm or {})}, {**tensors, **(weight or {})}
        w = {k: v for k, v in w.items() if v is not None}
        sparse_block_forward(state, SimpleNamespace(tensors=w), n, **{**args, **kw})
        return rec.calls

    run.calls, run.state = rec.calls, state
    return run


def refused(call, name, **kw):
    with pytest.raises(ValueError, match=name):
        call(**kw)
    assert call.calls == []


def test_fitting_tensors_pass(call):
    assert len(call()) == 13 and call.calls.count("h3b_residual_norm") == 2
    call(norm={"q": None, "post_mlp": None}, weight={"b_ada": None, "bqkv": None, "bo": None, "b1": None, "b2": None})
    call(norm={"q": torch.zeros(1, 64)}, x=torch.zeros(2, 1, 2, 4, D, dtype=torch.bfloat16))


@pytest.mark.parametrize("name,n", [("q", 64), ("k", 64), ("post_attn", D), ("post_mlp", D)])
def test_norm_weights(call, name, n):
    for bad in (torch.zeros(n, dtype=torch.bfloat16), torch.zeros(n, dtype=torch.float64), torch.zeros(n - 8), torch.zeros(n + 8),
                torch.zeros(2 * n)[::2], torch.zeros(1).expand(n), torch.zeros(n, device="meta"), torch.zeros(n + 8)[1:n + 1]):
        refused(call, name, norm={name: bad})


@pytest.mark.parametrize("name", ["post_attention", "Q", "norm_q"])
def test_unknown_norms(call, name):
    refused(call, name, norm={name: torch.zeros(64)})


@pytest.mark.parametrize("name", ["x", "pos", "c"])
def test_another_device(call, name):
    good = dict(c=torch.zeros(2, D), x=torch.zeros(2, 8, D, dtype=torch.bfloat16), pos=torch.zeros(2, 8, 3))
    refused(call, name, **{name: good[name].to("meta")})


@pytest.mark.parametrize("name", ["x", "pos", "c"])
def test_no_16_byte_boundary(call, name):
    """Else the call would fail half way, with x updated by the first branch."""
    shape, dtype = {"c": ((2, D), torch.float32), "x": ((2, 8, D), torch.bfloat16), "pos": ((2, 8, 3), torch.float32)}[name]
    n = torch.Size(shape).numel()
    refused(call, name, **{name: torch.zeros(n + 1, dtype=dtype)[1:].view(shape)})


@pytest.mark.parametrize("name", ["w_ada", "b_ada", "wqkv", "sqkv", "bqkv", "wo", "so", "bo", "w1", "s1", "b1", "w2", "s2", "b2"])
def test_projections(call, name):
    good = torch.zeros({"w_ada": (6 * D, D), "wqkv": (3 * D, D), "wo": (D, D), "w1": (F, D), "w2": (D, F)}.get(
        name, ({"b_ada": 6 * D, "sqkv": 3 * D, "bqkv": 3 * D, "s1": F, "b1": F}.get(name, D),)))
    dtype = torch.bfloat16 if name == "w_ada" else torch.int8 if name[0] == "w" else torch.float32
    bad = [good.to(torch.float16), good.to(dtype)[:-16], torch.cat([good, good]).to(dtype)[::2], good.to(dtype).to("meta")]
    if good.dim() == 2:
        bad += [good.to(dtype).T.contiguous().T, good.to(dtype).view(-1), good.to(dtype)[:, :-16].contiguous()]
    for t in bad:
        refused(call, name, weight={name: t})


@pytest.mark.parametrize("name", ["w_ada", "wqkv", "sqkv", "wo", "so", "w1", "s1", "w2", "s2"])
def test_missing_projections(call, name):
    refused(call, name, weight={name: None})


def test_the_weights_of_another_width(call):
    """A block whose MLP is wider than the state's: its output would not fit the state's buffer."""
    refused(call, "w1", weight={"w1": torch.zeros(2 * F, D, dtype=torch.int8), "s1": torch.zeros(2 * F),
                                "b1": torch.zeros(2 * F), "w2": torch.zeros(D, 2 * F, dtype=torch.int8)})


def test_a_state_on_another_device_than_the_current_one(call, monkeypatch):
    """The kernels run on the current device's stream."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    call.state.device = torch.device("cuda", 1)
    refused(call, "device")
