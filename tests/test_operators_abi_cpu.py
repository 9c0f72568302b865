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
