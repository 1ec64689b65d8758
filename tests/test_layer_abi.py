"""Argument checks of mk_add_rmsnorm and the few-token MoE layer: every refusal comes back before any device work, so
no GPU is needed (the addresses below are never dereferenced)."""
import ctypes
import subprocess

import moe_dispatch_expert_amd as mk

A, B, C, D, F, G = (ctypes.c_void_p(0x10000 * (i + 1)) for i in range(6))
ODD = ctypes.c_void_p(0x90008)   # 8-byte aligned only


def test_new_entry_points_are_exported():
    out = subprocess.run(["nm", "-D", "--defined-only", mk.LIB_PATH], capture_output=True, text=True, check=True).stdout
    for name in ("mk_add_rmsnorm",):
        assert f" T {name}\n" in out, name


def test_norm_refusals():
    f = mk.load().mk_add_rmsnorm
    ok = dict(x=A, residual=None, gamma=B, T=4, d=256, eps=1e-6, residual_out=None, y=C, q=None, qs=None)

    def call(**kw):
        v = dict(ok, **kw)
        return f(v["x"], v["residual"], v["gamma"], v["T"], v["d"], v["eps"], v["residual_out"], v["y"], v["q"],
                 v["qs"], None)

    assert call(T=0) == mk.MK_OK
    assert call(T=0, x=None, gamma=None) == mk.MK_OK
    for bad in (dict(T=-1), dict(d=0), dict(d=-8), dict(d=12), dict(eps=-1.0), dict(eps=float("nan")),
                dict(y=None),                                   # no output
                dict(q=D), dict(qs=D),                          # codes without scales, scales without codes
                dict(q=D, qs=F, d=136),                         # groups of 128
                dict(x=None), dict(gamma=None), dict(x=ODD), dict(gamma=ODD), dict(y=ODD), dict(residual=ODD),
                dict(q=ODD, qs=F), dict(q=D, qs=ODD),
                dict(y=B), dict(residual_out=C), dict(q=C, qs=F), dict(q=D, qs=D), dict(q=A, qs=F),
                dict(residual=G, q=G, qs=F), dict(q=D, qs=A)):
        assert call(**bad) == mk.MK_EINVAL, bad
    assert call(d=32776) == mk.MK_EUNSUPPORTED
