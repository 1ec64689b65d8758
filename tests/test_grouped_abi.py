"""Argument checks of the experts' products backward and in 8-bit integers: every refusal comes back before any device
work, so no GPU is needed (the addresses below are never dereferenced)."""
import contextlib
import ctypes
import subprocess

import pytest
import torch

import moe_dispatch_expert_amd as mk

A, B, C, D, F, G = (ctypes.c_void_p(0x10000 * (i + 1)) for i in range(6))
ODD = ctypes.c_void_p(0x90008)    # 8-byte aligned only
WORD = ctypes.c_void_p(0xA0004)   # a word inside an array
BYTE = ctypes.c_void_p(0xA0002)

NAMES = ("mk_expert_layout", "mk_expert_layout_workspace_bytes", "mk_combine_backward", "mk_swiglu_backward",
         "mk_grouped_gemm_dgrad", "mk_grouped_gemm_wgrad", "mk_quant_i8", "mk_swiglu_i8", "mk_grouped_gemm_i8")


def test_new_entry_points_are_exported():
    out = subprocess.run(["nm", "-D", "--defined-only", mk.LIB_PATH], capture_output=True, text=True, check=True).stdout
    for name in NAMES:
        assert f" T {name}\n" in out, name
        assert callable(getattr(mk, name))


def _caller(name, order, ok):
    """A call of entry point `name` with the arguments `ok`, some of them changed."""
    f = getattr(mk.load(), name)

    def call(**kw):
        assert not set(kw) - set(order), kw
        v = dict(ok, **kw)
        return f(*(v[a] for a in order), None)
    return call


def _refused(call, status, *changes):
    for kw in changes:
        assert call(**kw) == status, kw


def test_layout_refusals():
    need = mk.mk_expert_layout_workspace_bytes(100, 4, 8)
    call = _caller("mk_expert_layout", ("ids", "T", "k", "e0", "E", "slot", "off", "rt", "ws", "n"),
                   dict(ids=A, T=100, k=4, e0=0, E=8, slot=B, off=C, rt=D, ws=F, n=need))
    assert need > 0
    _refused(call, mk.MK_EINVAL, dict(T=-1), dict(k=0), dict(e0=-1), dict(E=0), dict(ids=None), dict(slot=None),
             dict(off=None), dict(ws=None), dict(ids=ODD), dict(slot=ODD), dict(off=ODD), dict(rt=ODD), dict(ws=ODD),
             dict(slot=A), dict(off=B), dict(rt=B), dict(rt=F), dict(T=1 << 30))
    _refused(call, mk.MK_EUNSUPPORTED, dict(k=33), dict(E=1025))
    _refused(call, mk.MK_EWORKSPACE, dict(n=need - 1), dict(n=0))
    f = mk.mk_expert_layout_workspace_bytes
    assert f(-1, 4, 8) == 0 and f(4, 33, 8) == 0 and f(4, 4, 0) == 0 and f(1 << 30, 4, 8) == 0 and f(0, 4, 8) > 0
    assert f(1 << 20, 8, 256) >= 128 * 256 * 4 and f(1 << 25, 8, 256) == f(1 << 24, 8, 256)


def test_combine_backward_refusals():
    call = _caller("mk_combine_backward", ("dout", "y", "rows", "slot", "w", "T", "k", "N", "dy", "dw"),
                   dict(dout=A, y=B, rows=8, slot=C, w=D, T=4, k=2, N=64, dy=F, dw=G))
    assert call(T=0) == mk.MK_OK and call(T=0, dout=None, y=None, slot=None, w=None, dy=None, dw=None) == mk.MK_OK
    _refused(call, mk.MK_EINVAL, dict(T=-1), dict(k=0), dict(k=33), dict(rows=-1), dict(N=0), dict(N=-8), dict(N=60),
             dict(dout=None), dict(y=None), dict(slot=None), dict(w=None), dict(dy=None), dict(dout=ODD), dict(y=ODD),
             dict(slot=ODD), dict(w=ODD), dict(dy=ODD), dict(dw=ODD), dict(dy=A), dict(dy=C), dict(dy=D), dict(dw=A),
             dict(dw=B), dict(dw=C), dict(dw=D), dict(dw=F))


def test_swiglu_backward_refusals():
    call = _caller("mk_swiglu_backward", ("gu", "dh", "rows", "F", "rv", "dgu", "h"),
                   dict(gu=A, dh=B, rows=4, F=64, rv=None, dgu=C, h=D))
    assert call(rows=0) == mk.MK_OK and call(rows=0, gu=None, dh=None, dgu=None, h=None) == mk.MK_OK
    _refused(call, mk.MK_EINVAL, dict(rows=-1), dict(F=0), dict(F=-8), dict(F=12), dict(gu=None), dict(dh=None),
             dict(dgu=None), dict(gu=ODD), dict(dh=ODD), dict(dgu=ODD), dict(h=ODD), dict(rv=BYTE), dict(dgu=B),
             dict(h=A), dict(h=C), dict(rv=C), dict(rv=D))


def test_dgrad_refusals():
    call = _caller("mk_grouped_gemm_dgrad", ("dy", "rows", "off", "E", "w", "K", "N", "da"),
                   dict(dy=A, rows=4, off=B, E=8, w=C, K=64, N=64, da=D))
    assert call(rows=0) == mk.MK_OK and call(rows=0, dy=None, da=None) == mk.MK_OK
    _refused(call, mk.MK_EINVAL, dict(rows=-1), dict(E=0), dict(K=0), dict(N=0), dict(K=-8), dict(N=-8), dict(K=60),
             dict(N=60), dict(dy=None), dict(off=None), dict(w=None), dict(da=None), dict(dy=ODD), dict(off=ODD),
             dict(w=ODD), dict(da=ODD), dict(da=A), dict(da=B), dict(da=C))
    _refused(call, mk.MK_EUNSUPPORTED, dict(E=1025), dict(K=(1 << 20) + 8), dict(N=(1 << 20) + 8))


def test_wgrad_refusals():
    call = _caller("mk_grouped_gemm_wgrad", ("dy", "a", "rows", "off", "E", "rt", "ar", "K", "N", "dw", "f32", "acc"),
                   dict(dy=A, a=B, rows=4, off=C, E=8, rt=D, ar=4, K=64, N=64, dw=F, f32=1, acc=0))
    _refused(call, mk.MK_EINVAL, dict(rows=-1), dict(E=0), dict(K=0), dict(N=0), dict(K=60), dict(N=60), dict(dy=None),
             dict(a=None), dict(a=None, rt=None), dict(off=None), dict(dw=None), dict(dy=ODD), dict(a=ODD),
             dict(off=ODD), dict(rt=ODD), dict(dw=ODD), dict(dw=A), dict(dw=B), dict(dw=C), dict(dw=D), dict(f32=2),
             dict(f32=-1), dict(acc=2), dict(acc=-1), dict(acc=1, f32=0), dict(ar=-1))
    _refused(call, mk.MK_EUNSUPPORTED, dict(E=1025), dict(K=(1 << 20) + 8), dict(N=(1 << 20) + 8),
             dict(ar=1 << 25))


def test_quant_refusals():
    for name in ("mk_quant_i8", "mk_swiglu_i8"):
        call = _caller(name, ("x", "rows", "d", "rv", "q", "s"), dict(x=A, rows=4, d=64, rv=None, q=B, s=C))
        assert call(rows=0) == mk.MK_OK and call(rows=0, x=None, q=None, s=None) == mk.MK_OK
        _refused(call, mk.MK_EINVAL, dict(rows=-1), dict(d=0), dict(d=-8), dict(d=12), dict(x=None), dict(q=None),
                 dict(s=None), dict(x=ODD), dict(q=ODD), dict(s=ODD), dict(rv=BYTE), dict(q=A), dict(s=A), dict(s=B),
                 dict(rv=B), dict(rv=C))
        _refused(call, mk.MK_EUNSUPPORTED, dict(d=32776))


def test_i8_refusals():
    call = _caller("mk_grouped_gemm_i8", ("a", "s", "rows", "off", "E", "rt", "ar", "w", "ws", "K", "N", "y"),
                   dict(a=A, s=B, rows=4, off=C, E=8, rt=None, ar=0, w=D, ws=F, K=64, N=64, y=G))
    assert call(rows=0) == mk.MK_OK and call(rows=0, a=None, s=None, y=None) == mk.MK_OK
    _refused(call, mk.MK_EINVAL, dict(rows=-1), dict(E=0), dict(K=0), dict(N=0), dict(K=72), dict(N=60), dict(a=None),
             dict(s=None), dict(off=None), dict(w=None), dict(ws=None), dict(y=None), dict(a=ODD), dict(s=ODD),
             dict(off=ODD), dict(rt=ODD), dict(w=ODD), dict(ws=ODD), dict(y=ODD), dict(y=A), dict(y=B), dict(y=C),
             dict(y=D), dict(y=F), dict(rt=G), dict(rt=WORD), dict(rt=ODD, ar=-1))
    _refused(call, mk.MK_EUNSUPPORTED, dict(E=1025), dict(K=1 << 17), dict(N=(1 << 20) + 8),
             dict(rt=ctypes.c_void_p(0xB0000), ar=1 << 26))


I32, BF = torch.int32, torch.bfloat16
X = torch.zeros(4, 64, dtype=BF)
W = torch.zeros(2, 32, 64, dtype=BF)
OFF = torch.tensor([0, 2, 4], dtype=I32)
SLOTS, GATES = torch.zeros(4, 2, dtype=I32), torch.zeros(4, 2)
Q, S = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
CALLS = {
    "mk_expert_layout": lambda s: mk.mk_expert_layout(SLOTS, 8, stream=s),
    "mk_combine_backward": lambda s: mk.mk_combine_backward(X, X, SLOTS, GATES, stream=s),
    "mk_swiglu_backward": lambda s: mk.mk_swiglu_backward(torch.zeros(4, 128, dtype=BF), X, h=True, stream=s),
    "mk_grouped_gemm_dgrad": lambda s: mk.mk_grouped_gemm_dgrad(torch.zeros(4, 32, dtype=BF), OFF, W, stream=s),
    "mk_grouped_gemm_wgrad": lambda s: mk.mk_grouped_gemm_wgrad(torch.zeros(4, 32, dtype=BF), X, OFF, stream=s),
    "mk_quant_i8": lambda s: mk.mk_quant_i8(X, stream=s),
    "mk_swiglu_i8": lambda s: mk.mk_swiglu_i8(X, stream=s),
    "mk_grouped_gemm_i8": lambda s: mk.mk_grouped_gemm_i8(Q, S, OFF, torch.zeros(2, 32, 64, dtype=torch.int8),
                                                          torch.zeros(2, 32), stream=s),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_allocations_are_made_on_the_calls_stream(name, monkeypatch):
    """On the CPU: the calls refuse these tensors, after they have allocated what they were not given."""
    inside, made = [], []
    other = object()

    @contextlib.contextmanager
    def stream_context(s):
        assert s is other
        inside.append(s)
        yield
        inside.pop()

    real = torch.empty

    def watch(*args, **kw):
        made.append(bool(inside))
        return real(*args, **kw)

    monkeypatch.setattr(torch.cuda, "stream", stream_context)
    monkeypatch.setattr(torch, "empty", watch)
    for s in (other, None):
        with pytest.raises(ValueError, match="device tensors"):
            CALLS[name](s)
        assert made and all(m == (s is other) for m in made), made
        made.clear()


def test_binding_names_the_wrong_tensor():
    """Types, shapes and layouts that the C ABI cannot see."""
    for fn, word in ((lambda: mk.mk_expert_layout(SLOTS.long(), 8), "topk_ids"),
                     (lambda: mk.mk_expert_layout(SLOTS, 8, out={"row_token": SLOTS}), "row_token"),
                     (lambda: mk.mk_combine_backward(X, X[:, :32].contiguous(), SLOTS, GATES), "y_perm"),
                     (lambda: mk.mk_combine_backward(X, X, SLOTS, GATES[:2]), "topk_w"),
                     (lambda: mk.mk_combine_backward(X.float(), X, SLOTS, GATES), "dout"),
                     (lambda: mk.mk_swiglu_backward(X, X), "gate_up"),
                     (lambda: mk.mk_swiglu_backward(torch.zeros(4, 128, dtype=BF), X, rows_valid=OFF), "rows_valid"),
                     (lambda: mk.mk_grouped_gemm_dgrad(X, OFF, W), "dy"),
                     (lambda: mk.mk_grouped_gemm_dgrad(X[:, :32], OFF, W), "dy"),
                     (lambda: mk.mk_grouped_gemm_dgrad(X[:, :32].contiguous(), OFF[:2], W), "expert_offsets"),
                     (lambda: mk.mk_grouped_gemm_wgrad(X, X[:2], OFF), "a"),
                     (lambda: mk.mk_grouped_gemm_wgrad(X, X, OFF, dtype=torch.float16), "dtype"),
                     (lambda: mk.mk_grouped_gemm_wgrad(X, X, OFF, accumulate=True), "accumulate"),
                     (lambda: mk.mk_grouped_gemm_wgrad(X, X, OFF, row_token=OFF), "row_token"),
                     (lambda: mk.mk_grouped_gemm_wgrad(X, X, OFF, out=W), "out"),
                     (lambda: mk.mk_quant_i8(X.t()), "x"),
                     (lambda: mk.mk_swiglu_i8(torch.zeros(4, 63, dtype=BF)), "2F"),
                     (lambda: mk.mk_quant_i8(X, out={"q": Q.to(torch.uint8)}), "q"),
                     (lambda: mk.mk_grouped_gemm_i8(Q, S[:2], OFF, Q.view(2, 2, 64), torch.zeros(2, 2)), "a_scale"),
                     (lambda: mk.mk_grouped_gemm_i8(Q, S, OFF, Q.view(2, 2, 64), S), "w_scale")):
        with pytest.raises(ValueError, match=word):
            fn()


def test_rows_whose_tiles_would_pass_32_bits_are_refused():
    for rows, st in ((2 ** 31 - 4096, mk.MK_EINVAL), (2 ** 31 - 4095, mk.MK_EUNSUPPORTED), (2 ** 31 - 1, mk.MK_EUNSUPPORTED)):
        for name, names, args in (
                ("mk_grouped_gemm_dgrad", ("dy", "rows", "off", "E", "w", "K", "N", "da"),
                 dict(dy=None, off=C, E=8, w=D, K=64, N=64, da=F)),
                ("mk_grouped_gemm_wgrad", ("dy", "a", "rows", "off", "E", "rt", "ar", "K", "N", "dw", "fp32", "acc"),
                 dict(dy=None, a=B, off=C, E=8, rt=None, ar=0, K=64, N=64, dw=D, fp32=1, acc=0)),
                ("mk_grouped_gemm_i8", ("a", "s", "rows", "off", "E", "rt", "ar", "w", "ws", "K", "N", "y"),
                 dict(a=None, s=B, off=C, E=8, rt=None, ar=0, w=D, ws=F, K=64, N=64, y=G))):
            assert _caller(name, names, dict(rows=rows, **args))() == st, (name, rows)
