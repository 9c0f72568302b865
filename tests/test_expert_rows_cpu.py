"""Refusals of the grouped products, the activation and the norm, on the host: by the C entry points with fake device
addresses, and by the Python functions with tensors without memory."""
from __future__ import annotations

import contextlib
from types import SimpleNamespace

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from combine_moe_get_gb300 import binding as moe

A = 0x7F0000000000          # 256-byte aligned
BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def at(i):
    return A + i * 0x100000


LINEAR = dict(x=at(0), xs=None, M=8, K=256, w=at(1), ws=None, E=4, N=128, prefix=at(2), type=0, out=at(3), status=at(4))
GRAD_X = dict(grad=at(0), M=8, N=128, w=at(1), E=4, K=256, prefix=at(2), out=at(3), status=at(4))
GRAD_W = dict(grad=at(0), x=at(1), M=8, N=128, K=256, E=4, prefix=at(2), type=0, add=0, out=at(3), status=at(4))
SWIGLU = dict(gu=at(0), M=8, I=256, rw=at(1), rows=at(2), out=at(3), scales=None, status=at(4))
BACKWARD = dict(gu=at(0), grad=at(5), M=8, I=256, rw=at(1), rows=at(2), out=at(3), gw=at(6), status=at(4))
NORM = dict(x=at(0), res=at(1), T=8, H=256, weight=at(2), type=0, eps=1e-6, out=at(3), res_out=at(5), codes=at(6),
            scales=at(7), status=at(4))
NORM_BACKWARD = dict(h=at(0), weight=at(2), type=0, grad=at(1), gr=at(5), T=8, H=256, eps=1e-6, gx=at(3), gw=at(6),
                     ws=at(7), ws_bytes=1 << 30, status=at(4))
ENTRIES = dict(moe_grouped_linear=LINEAR, moe_grouped_linear_grad_x=GRAD_X, moe_grouped_linear_grad_w=GRAD_W,
               moe_swiglu=SWIGLU, moe_swiglu_backward=BACKWARD, moe_add_rms_norm=NORM,
               moe_add_rms_norm_backward=NORM_BACKWARD)

SIZES = [(dict(M=-1), 1), (dict(M=(1 << 30) + 1), 1), (dict(E=0), 1), (dict(E=8193), 1), (dict(K=0), 1), (dict(K=252), 1),
         (dict(K=(1 << 20) + 8), 1), (dict(N=0), 1), (dict(N=12), 1), (dict(N=(1 << 20) + 8), 1), (dict(prefix=None), 1),
         (dict(w=None), 1), (dict(out=None), 1), (dict(status=None), 1), (dict(prefix=A + 2), 2), (dict(out=A + 8), 2),
         (dict(status=A + 2), 2)]
GRAD_W_SIZES = [b for b in SIZES if "w" not in b[0]]
ROWS = [(dict(M=-1), 1), (dict(M=(1 << 30) + 1), 1), (dict(I=0), 1), (dict(I=12), 1), (dict(I=(1 << 20) + 8), 1),
        (dict(gu=None), 1), (dict(out=None), 1), (dict(status=None), 1), (dict(gu=A + 8), 2), (dict(out=A + 8), 2),
        (dict(rw=A + 2), 2), (dict(rows=A + 2), 2), (dict(status=A + 2), 2)]
NORMS = [(dict(T=-1), 1), (dict(T=(1 << 30) + 1), 1), (dict(H=0), 1), (dict(H=12), 1), (dict(H=16392), 1), (dict(type=2), 1),
         (dict(weight=None), 1), (dict(status=None), 1), (dict(weight=A + 8), 2), (dict(status=A + 2), 2)]
BAD = dict(
    moe_grouped_linear=SIZES + [
        (dict(type=2), 1), (dict(type=1), 1), (dict(type=1, xs=A), 1), (dict(type=1, ws=A), 1), (dict(xs=A), 1),
        (dict(ws=A), 1), (dict(type=1, xs=A, ws=A, K=264), 1), (dict(x=None), 1), (dict(x=A + 8), 2), (dict(w=A + 8), 2),
        (dict(type=1, xs=A + 2, ws=A), 2), (dict(type=1, xs=A, ws=A + 2), 2)],
    moe_grouped_linear_grad_x=SIZES + [(dict(grad=None), 1), (dict(grad=A + 8), 2), (dict(w=A + 8), 2)],
    moe_grouped_linear_grad_w=GRAD_W_SIZES + [(dict(type=2), 1), (dict(type=-1), 1), (dict(add=2), 1), (dict(grad=None), 1),
                                              (dict(x=None), 1), (dict(grad=A + 8), 2), (dict(x=A + 8), 2)],
    moe_swiglu=ROWS + [(dict(scales=A, I=264), 1), (dict(scales=A + 2), 2), (dict(scales=A, out=A + 4), 2)],
    moe_swiglu_backward=ROWS + [(dict(grad=None), 1), (dict(grad=A + 8), 2), (dict(gw=A + 2), 2)],
    moe_add_rms_norm=NORMS + [
        (dict(x=None), 1), (dict(codes=None), 1), (dict(scales=None), 1), (dict(H=264), 1), (dict(res=None), 1),
        (dict(out=None, res_out=None, codes=None, scales=None), 1), (dict(x=A + 8), 2), (dict(res=A + 8), 2),
        (dict(out=A + 8), 2), (dict(res_out=A + 8), 2), (dict(codes=A + 4), 2), (dict(scales=A + 2), 2)],
    moe_add_rms_norm_backward=NORMS + [
        (dict(h=None), 1), (dict(grad=None), 1), (dict(gx=None), 1), (dict(gw=None), 1), (dict(ws=None), 1),
        (dict(h=A + 8), 2), (dict(grad=A + 8), 2), (dict(gr=A + 8), 2), (dict(gx=A + 8), 2), (dict(gw=A + 2), 2),
        (dict(ws=A + 8), 2), (dict(ws_bytes=8 * 256 * 4 - 1), 7)])


@pytest.mark.parametrize("name,kw,code", [(n, kw, c) for n in BAD for kw, c in BAD[n]])
def test_entry_rejects_bad_arguments(name, kw, code):
    assert set(kw) <= set(ENTRIES[name])
    assert getattr(moe.LIB, name)(*dict(ENTRIES[name], **kw).values(), None) == code


def test_no_rows_is_nothing_to_do():
    """... and needs no rows, on a machine without a GPU too."""
    none = dict(M=0, T=0)
    for name in ("moe_grouped_linear", "moe_grouped_linear_grad_x", "moe_swiglu", "moe_swiglu_backward", "moe_add_rms_norm"):
        d = ENTRIES[name]
        assert getattr(moe.LIB, name)(*dict(d, **{k: v for k, v in none.items() if k in d}).values(), None) == moe.MOE_OK


def test_status_string():
    assert moe.status_string(moe.MOE_ERR_BAD_PREFIX) == "MOE_ERR_BAD_PREFIX"


def test_norm_workspace_sizes():
    size = moe.moe_add_rms_norm_backward_workspace_size
    assert size(1, 8) >= 32 and size(1 << 30, 16384) > 0
    assert all(size(t, 1024) <= size(t + 100, 1024) for t in range(1, 1000, 50))   # enough for fewer rows
    for bad in ((-1, 8), (1, 12), (1, 16392), ((1 << 30) + 1, 8), (1 + 2 ** 32, 8), (1, 8 + 2 ** 32)):
        assert size(*bad) == 0


# ------------------------------------------------------------------ the Python functions

TENSORS = {
    "linear": (moe.moe_grouped_linear, dict(x=(8, 16, BF), w=(3, 24, 16, BF), expert_prefix=(4, I32), out=(8, 24, BF),
                                            status=(1, I32))),
    "E4M3 linear": (moe.moe_grouped_linear, dict(
        x=(8, 128, U8), w=(3, 24, 128, U8), expert_prefix=(4, I32), x_scales=(8, 1, F32), w_scales=(3, 24, 1, F32),
        out=(8, 24, BF), status=(1, I32))),
    "grad_x": (moe.moe_grouped_linear_grad_x, dict(grad=(8, 24, BF), w=(3, 24, 16, BF), expert_prefix=(4, I32),
                                                   out=(8, 16, BF), status=(1, I32))),
    "grad_w": (moe.moe_grouped_linear_grad_w, dict(grad=(8, 24, BF), x=(8, 16, BF), expert_prefix=(4, I32),
                                                   out=(3, 24, 16, F32), status=(1, I32))),
    "swiglu": (moe.moe_swiglu, dict(gate_up=(8, 32, BF), row_weights=(8, F32), num_rows=(1, I32), out=(8, 16, BF),
                                    status=(1, I32))),
    "E4M3 swiglu": (moe.moe_swiglu, dict(gate_up=(8, 256, BF), row_weights=(8, F32), num_rows=(1, I32), out=(8, 128, U8),
                                         out_scales=(8, 1, F32), quantize_fp8=True, status=(1, I32))),
    "swiglu_backward": (moe.moe_swiglu_backward, dict(
        gate_up=(8, 32, BF), grad=(8, 16, BF), row_weights=(8, F32), num_rows=(1, I32), out=(8, 32, BF),
        grad_row_weights=(8, F32), status=(1, I32))),
    "norm": (moe.moe_add_rms_norm, dict(
        x=(8, 128, BF), weight=(128, BF), residual=(8, 128, BF), out=(8, 128, BF), residual_out=(8, 128, BF), codes=(8, 128, U8),
        scales=(8, 1, F32), quantize_fp8=True, status=(1, I32))),
    "norm_backward": (moe.moe_add_rms_norm_backward, dict(
        h=(8, 16, BF), weight=(16, F32), grad=(8, 16, BF), grad_residual=(8, 16, BF), out=(8, 16, BF), grad_weight=(16, F32),
        workspace=(4096, U8), status=(1, I32))),
}


@pytest.fixture(autouse=True)
def no_context_for_tensors_without_memory(monkeypatch):
    """On a machine with one GPU there is none for cuda:1."""
    monkeypatch.setattr("torch._subclasses.fake_tensor.init_gpu_context", lambda device: None, raising=False)


def fake(spec, device="cuda:0"):
    if isinstance(spec, bool):
        return spec
    with FakeTensorMode():
        return torch.empty(*spec[:-1], dtype=spec[-1], device=device)


def call(name, device_of=lambda n: "cuda:0", **changed):
    f, specs = TENSORS[name]
    return f(**{n: fake(s, device_of(n)) if not torch.is_tensor(s) else s for n, s in dict(specs, **changed).items()})


PLACES = [(n, t) for n in TENSORS for t, s in TENSORS[n][1].items() if not isinstance(s, bool)]


@pytest.mark.parametrize("name,tensor", PLACES)
def test_one_tensor_on_another_device(name, tensor):
    with pytest.raises(ValueError, match="is on cuda:"):
        call(name, lambda n: "cuda:1" if n == tensor else "cuda:0")


@pytest.mark.gpu
@pytest.mark.parametrize("name", TENSORS)
def test_all_tensors_on_another_device_than_the_current(name):
    with pytest.raises(ValueError, match="tensors on cuda:1, the current device is cuda:0"):
        call(name, lambda n: "cuda:1")


@pytest.mark.parametrize("name,tensor", [(n, t) for n, t in PLACES if t != "workspace"])
def test_another_type(name, tensor):
    with pytest.raises(ValueError):
        call(name, **{tensor: TENSORS[name][1][tensor][:-1] + (torch.float64,)})


@pytest.mark.parametrize("name,tensor", [(n, t) for n, t in PLACES if t not in ("workspace", "status")])
def test_another_shape(name, tensor):
    spec = TENSORS[name][1][tensor]
    for i in range(len(spec) - 1):
        with pytest.raises(ValueError):
            call(name, **{tensor: spec[:i] + (spec[i] + 1,) + spec[i + 1:]})
    with pytest.raises(ValueError):
        call(name, **{tensor: spec[:-1] + (1, spec[-1])})


@pytest.mark.parametrize("name,tensor", [(n, t) for n, t in PLACES if len(TENSORS[n][1][t]) > 2])
def test_not_contiguous(name, tensor):
    spec = TENSORS[name][1][tensor]
    with FakeTensorMode():
        t = torch.empty(*spec[:-2], spec[-2] * 2, dtype=spec[-1], device="cuda:0")[..., ::2]
    if t.is_contiguous():
        pytest.skip("one element a row")
    with pytest.raises(ValueError, match="contiguous"):
        call(name, **{tensor: t})


@pytest.mark.parametrize("name,tensor,dim", [(n, t, i) for n, t in PLACES for i in range(len(TENSORS[n][1][t]) - 1)
                                             if list(TENSORS[n][1]).index(t) < 2 and t != "weight"])
def test_sizes_beyond_32_bits(name, tensor, dim):
    spec = TENSORS[name][1][tensor]
    with pytest.raises(ValueError):
        call(name, **{tensor: spec[:dim] + (2 ** 32 + spec[dim],) + spec[dim + 1:]})


def test_combinations_that_have_no_meaning():
    for name, kw, match in [
            ("linear", dict(x_scales=(8, 1, F32)), "take no scales"),
            ("E4M3 linear", dict(w=(3, 24, 128, BF)), "w is torch.uint8"),
            ("swiglu", dict(out_scales=(8, 1, F32)), "not written"),
            ("swiglu", dict(quantize_fp8=True, out=(8, 16, U8)), "multiple of 128"),
            ("norm", dict(bf16_out=False), "out is not written"),
            ("norm", dict(quantize_fp8=False), "codes is not written")]:
        with pytest.raises(ValueError, match=match):
            call(name, **kw)
    with pytest.raises(ValueError, match="need x_scales"):
        moe.moe_grouped_linear(fake((8, 128, U8)), fake((3, 24, 128, U8)), fake((4, I32)), status=fake((1, I32)))
    with pytest.raises(ValueError, match="residual_out is not written"):
        moe.moe_add_rms_norm(fake((8, 16, BF)), fake((16, BF)), residual_out=fake((8, 16, BF)), out=fake((8, 16, BF)),
                             status=fake((1, I32)))
    with pytest.raises(ValueError, match="adds to out"):
        moe.moe_grouped_linear_grad_w(fake((8, 24, BF)), fake((8, 16, BF)), fake((4, I32)), accumulate=True)
    with pytest.raises(ValueError, match="float32 or torch.bfloat16"):
        moe.moe_grouped_linear_grad_w(fake((8, 24, BF)), fake((8, 16, BF)), fake((4, I32)), dtype=torch.float16)


# status for all of them, the norm's backward takes a workspace too
@pytest.mark.parametrize("name,least", [(n, 2 if n == "norm_backward" else 1) for n in TENSORS])
def test_allocates_under_the_given_stream(monkeypatch, name, least):
    """What a function allocates in Python, it allocates under the stream of the call."""
    f, specs = TENSORS[name]
    given = {n: s if isinstance(s, bool) else torch.zeros(*s[:-1], dtype=s[-1]) for n, s in specs.items()
             if n not in ("status", "workspace")}
    under, made = [None], []

    @contextlib.contextmanager
    def stream(s):
        under.append(s)
        yield
        under.pop()

    def recording(make):
        def made_here(*args, **kw):
            made.append(under[-1])
            return make(*args, **kw)
        return made_here

    side = SimpleNamespace(cuda_stream=0x1000)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    for n in ("empty", "zeros"):
        monkeypatch.setattr(torch, n, recording(getattr(torch, n)))
    with pytest.raises(ValueError, match="CUDA tensors only"):   # after the allocations
        f(**given, stream=side)
    assert len(made) >= least and set(map(id, made)) == {id(side)}, made
