"""Refusals of the gate, expert and adapter entry points: every call below fails
validation on the host, before any CUDA call, with fake device addresses."""
from __future__ import annotations

import pytest

from combine_moe_get_gb300 import build as cuda_build

A = 0x7F0000000000          # 256-byte aligned
MIS = A + 2


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    from combine_moe_get_gb300 import binding
    return binding


def test_new_status_strings(lib):
    assert lib.status_string(lib.MOE_ERR_BAD_LOGIT) == "MOE_ERR_BAD_LOGIT"


def _gate(lib, logits=A, ltype=0, bias=None, T=8, k=2, E=16, mode=0, idx=A + 0x1000, w=A + 0x2000, status=A + 0x3000):
    return lib.LIB.moe_topk_gate(logits, ltype, bias, T, k, E, mode, 1.0, idx, w, status, None)


def _gate_backward(lib, logits=A, ltype=0, T=8, k=2, E=16, mode=0, idx=A + 0x1000, w=A + 0x2000, out=A + 0x4000,
                   status=A + 0x3000):
    return lib.LIB.moe_topk_gate_backward(logits, ltype, idx, w, T, k, E, mode, 1.0, out, status, None)


GATE_BAD = [(dict(k=0), 1), (dict(k=33, E=64), 1), (dict(k=17), 1), (dict(E=0), 1), (dict(E=8193), 1), (dict(T=-1), 1),
            (dict(T=1 << 30), 1), (dict(ltype=2), 1), (dict(ltype=-1), 1), (dict(mode=2), 1), (dict(mode=0x200), 1),
            (dict(mode=0x102), 1), (dict(mode=-1), 1), (dict(logits=None), 1), (dict(idx=None), 1), (dict(w=None), 1),
            (dict(status=None), 1), (dict(logits=MIS), 2), (dict(logits=A + 1, ltype=1), 2), (dict(idx=A + 4), 2),
            (dict(w=MIS), 2), (dict(status=MIS), 2)]


@pytest.mark.parametrize("kw,code", GATE_BAD + [(dict(bias=MIS), 2)])
def test_gate_rejects_bad_arguments(lib, kw, code):
    assert _gate(lib, **kw) == code


@pytest.mark.parametrize("kw,code", GATE_BAD + [(dict(out=None), 1), (dict(out=MIS), 2), (dict(out=A + 1, ltype=1), 2)])
def test_gate_backward_rejects_bad_arguments(lib, kw, code):
    assert _gate_backward(lib, **kw) == code


def test_adapter_status_string(lib):
    assert lib.status_string(lib.MOE_ERR_BAD_ADAPTER) == "MOE_ERR_BAD_ADAPTER"


def test_operator_workspace_sizes(lib):
    ws = lib.moe_experts_workspace_size
    assert ws(128, 256, 256, 2, 16) > 0 and ws(1024, 7168, 2048, 8, 256) > 0
    assert ws(1025, 256, 256, 2, 16) == 0 and ws(8, 260, 256, 2, 16) == 0 and ws(8, 256, 4, 2, 16) == 0
    assert ws(8, 256, 256, 33, 64) == 0 and ws(-1, 256, 256, 2, 16) == 0 and ws(8, 256, 256, 2, 8193) == 0
    ws = lib.moe_adapter_linear_workspace_size
    assert ws(128, 7168, 7168, 48, 16) > 0 and ws(1 << 20, 64, 64, 1, 8) > 0
    assert ws(-1, 64, 64, 1, 8) == 0 and ws(8, 60, 64, 1, 8) == 0 and ws(8, 64, 60, 1, 8) == 0
    assert ws(8, 64, 64, 0, 8) == 0 and ws(8, 64, 64, 8193, 8) == 0 and ws(8, 64, 64, 1, 136) == 0
    assert ws(8, 64, 64, 1, 12) == 0 and ws((1 << 20) + 1, 64, 64, 1, 8) == 0


EXPERT = dict(x=A, T=8, H=256, idx=A + 0x10000, w=A + 0x20000, k=2, E=16, w13=A + 0x100000, s13=None, w2=A + 0x200000,
              s2=None, I=128, wtype=0, out=A + 0x30000, ws=A + 0x400000, ws_bytes=1 << 30, status=A + 0x40000)


def _experts(lib, **kw):
    d = dict(EXPERT, **kw)
    return lib.LIB.moe_experts(d["x"], d["T"], d["H"], d["idx"], d["w"], d["k"], d["E"], d["w13"], d["s13"], d["w2"],
                               d["s2"], d["I"], d["wtype"], d["out"], d["ws"], d["ws_bytes"], d["status"], None)


def _layer(lib, logits=A + 0x50000, ltype=0, bias=None, mode=0, **kw):
    d = dict(EXPERT, **kw)
    return lib.LIB.moe_layer(d["x"], d["T"], d["H"], logits, ltype, bias, d["k"], d["E"], mode, 1.0, d["idx"], d["w"],
                             d["w13"], d["s13"], d["w2"], d["s2"], d["I"], d["wtype"], d["out"], d["ws"], d["ws_bytes"],
                             d["status"], None)


S = A + 0x500000
EXPERT_BAD = [(dict(T=-1), 1), (dict(T=1025), 1), (dict(H=0), 1), (dict(H=252), 1), (dict(I=0), 1), (dict(I=12), 1),
              (dict(H=(1 << 20) + 8), 1), (dict(k=0), 1), (dict(k=33, E=64), 1), (dict(E=0), 1), (dict(E=8193), 1),
              (dict(E=8192, I=1 << 18), 1), (dict(wtype=2), 1), (dict(wtype=-1), 1), (dict(wtype=1), 1),
              (dict(wtype=1, s13=S), 1), (dict(s13=S, s2=S), 1), (dict(wtype=1, s13=S, s2=S, H=264), 1),
              (dict(wtype=1, s13=S, s2=S, I=136), 1), (dict(x=None), 1), (dict(idx=None), 1), (dict(w=None), 1),
              (dict(w13=None), 1), (dict(w2=None), 1), (dict(out=None), 1), (dict(ws=None), 1), (dict(status=None), 1),
              (dict(x=A + 8), 2), (dict(idx=A + 4), 2), (dict(w=MIS), 2), (dict(w13=A + 8), 2), (dict(w2=A + 8), 2),
              (dict(out=A + 8), 2), (dict(ws=A + 8), 2), (dict(status=MIS), 2), (dict(wtype=1, s13=MIS, s2=S), 2),
              (dict(ws_bytes=16), 7)]


@pytest.mark.parametrize("kw,code", EXPERT_BAD)
def test_experts_reject_bad_arguments(lib, kw, code):
    assert _experts(lib, **kw) == code


@pytest.mark.parametrize("kw,code", EXPERT_BAD + [(dict(logits=None), 1), (dict(ltype=2), 1), (dict(mode=2), 1),
                                                  (dict(k=17), 1), (dict(logits=MIS), 2), (dict(bias=MIS), 2)])
def test_layer_rejects_bad_arguments(lib, kw, code):
    assert _layer(lib, **kw) == code


def _adapter(lib, x=A, T=8, K=256, w=A + 0x100000, N=128, idx=A + 0x10000, a=A + 0x200000, b=A + 0x300000,
             s=A + 0x20000, L=4, r=16, out=A + 0x30000, ws=A + 0x400000, ws_bytes=1 << 30, status=A + 0x40000):
    return lib.LIB.moe_adapter_linear(x, T, K, w, N, idx, a, b, s, L, r, out, ws, ws_bytes, status, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(T=(1 << 20) + 1), 1), (dict(K=0), 1), (dict(K=252), 1), (dict(N=0), 1), (dict(N=12), 1),
    (dict(L=0), 1), (dict(L=8193), 1), (dict(L=2048, N=1 << 20), 1), (dict(r=0), 1), (dict(r=12), 1), (dict(r=136), 1), (dict(x=None), 1),
    (dict(w=None), 1), (dict(idx=None), 1), (dict(a=None), 1), (dict(b=None), 1), (dict(s=None), 1), (dict(out=None), 1),
    (dict(ws=None), 1), (dict(status=None), 1), (dict(x=A + 8), 2), (dict(w=A + 8), 2), (dict(idx=MIS), 2),
    (dict(a=A + 8), 2), (dict(b=A + 8), 2), (dict(s=MIS), 2), (dict(out=A + 8), 2), (dict(ws=A + 8), 2),
    (dict(status=MIS), 2), (dict(ws_bytes=16), 7),
])
def test_adapter_rejects_bad_arguments(lib, kw, code):
    assert _adapter(lib, **kw) == code
