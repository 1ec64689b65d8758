"""Argument checks of mk_add_rmsnorm and the few-token MoE layer: every refusal comes back before any device work, so
no GPU is needed (the addresses below are never dereferenced)."""
import ctypes
import subprocess

import moe_dispatch_expert_amd as mk

A, B, C, D, F, G = (ctypes.c_void_p(0x10000 * (i + 1)) for i in range(6))
ODD = ctypes.c_void_p(0x90008)   # 8-byte aligned only


def test_new_entry_points_are_exported():
    out = subprocess.run(["nm", "-D", "--defined-only", mk.LIB_PATH], capture_output=True, text=True, check=True).stdout
    for name in ("mk_add_rmsnorm", "mk_moe_layer", "mk_moe_layer_q8", "mk_moe_layer_workspace_bytes"):
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


def _layer(q8, shape, **kw):
    lib = mk.load()
    v = dict(x=A, xq=B, xs=C, wr=D, bias=None, ids=None, w=None, gu=F, gs=G, dn=A, ds=B, tv=None, out=C, ido=None,
             wo=None, ws=D, nbytes=1 << 40)
    v.update(kw)
    s = ctypes.byref(mk.MkShape(*shape))
    if q8:
        return lib.mk_moe_layer_q8(s, v["x"], v["xq"], v["xs"], v["wr"], v["bias"], v["ids"], v["w"], v["gu"], v["gs"],
                                   v["dn"], v["ds"], v["tv"], v["out"], v["ido"], v["wo"], v["ws"], v["nbytes"], None)
    return lib.mk_moe_layer(s, v["x"], v["wr"], v["bias"], v["ids"], v["w"], v["gu"], v["dn"], v["tv"], v["out"],
                            v["ido"], v["wo"], v["ws"], v["nbytes"], None)


def test_layer_refusals():
    ok = (4, 256, 8, 2, 0, 8, 64)   # T, d, E, k, e_begin, E_local, N = 2F
    for q8 in (False, True):
        assert _layer(q8, (0,) + ok[1:]) == mk.MK_OK
        assert _layer(q8, (0,) + ok[1:], x=None, out=None, ws=None) == mk.MK_OK
        for shape in ((-1, 256, 8, 2, 0, 8, 64), (4, 0, 8, 2, 0, 8, 64), (4, 250, 8, 2, 0, 8, 64),
                      (4, 256, 8, 9, 0, 8, 64), (4, 256, 8, 0, 0, 8, 64), (4, 256, 8, 2, 1, 8, 64),
                      (4, 256, 8, 2, -1, 8, 64), (4, 256, 8, 2, 0, 0, 64), (4, 256, 8, 2, 0, 8, 0),
                      (4, 256, 8, 2, 0, 8, 72)):
            assert _layer(q8, shape) == mk.MK_EINVAL, shape
        for shape in ((129, 256, 8, 2, 0, 8, 64), (4, 136, 8, 2, 0, 8, 64), (4, 32896, 8, 2, 0, 8, 64),
                      (4, 256, 2048, 2, 0, 8, 64), (4, 256, 64, 33, 0, 8, 64), (4, 8192, 8, 2, 0, 8, 1 << 18)):
            assert _layer(q8, shape) == mk.MK_EUNSUPPORTED, shape
        for kw in (dict(wr=None), dict(ids=A), dict(w=A), dict(x=None), dict(gu=None), dict(dn=None), dict(out=None),
                   dict(ws=None), dict(x=ODD), dict(wr=ODD), dict(bias=ODD), dict(ids=ODD, w=A), dict(ids=A, w=ODD),
                   dict(gu=ODD), dict(dn=ODD), dict(tv=ODD), dict(out=ODD), dict(ido=ODD), dict(wo=ODD), dict(ws=ODD)):
            assert _layer(q8, ok, **kw) == mk.MK_EINVAL, kw
        need = mk.mk_moe_layer_workspace_bytes(4, 256, 8, 2, 0, 8, 32)
        assert need > 0 and _layer(q8, ok, nbytes=need - 1) == mk.MK_EWORKSPACE
    for kw in (dict(xq=None), dict(xs=None), dict(gs=None), dict(ds=None), dict(xq=ODD), dict(xs=ODD), dict(gs=ODD),
               dict(ds=ODD)):
        assert _layer(True, ok, **kw) == mk.MK_EINVAL, kw
    assert _layer(True, (4, 256, 8, 2, 0, 8, 48)) == mk.MK_EINVAL          # F = 24: a multiple of 8 only
    assert _layer(False, (4, 8192, 8, 2, 0, 8, 1 << 17)) == mk.MK_EUNSUPPORTED   # 2F d 2 = 2^31


def test_layer_workspace_bytes():
    f = mk.mk_moe_layer_workspace_bytes
    assert f(129, 256, 8, 2, 0, 8, 32) == 0 and f(4, 256, 8, 9, 0, 8, 32) == 0 and f(4, 256, 8, 2, 0, 8, 12) == 0
    # router partial sums and the rows' h: what the call cannot do without
    assert f(128, 7168, 256, 8, 0, 32, 2048) >= 8 * 128 * 256 * 4 + 128 * 8 * 2048 * 2
    assert f(128, 7168, 256, 8, 0, 4, 2048) < f(128, 7168, 256, 8, 0, 8, 2048) == f(128, 7168, 256, 8, 0, 32, 2048)
