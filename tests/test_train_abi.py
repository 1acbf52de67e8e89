"""Refusals of the gated block, layer normalisation and AdamW: every bad argument is
answered with its status before anything is launched (no GPU needed)."""
import ctypes

import tiled_newton_schulz_amd as H
from tiled_newton_schulz_amd import shape_descriptor as sd

OK, INVALID, UNSUPPORTED, LAYOUT, OVERLAP, WORKSPACE = 0, 1, 2, 3, 4, 5
P = 1 << 30
UNSET = object()


def at(k):
    return P + (k << 24)


def ref(d):
    return None if d is None else ctypes.byref(d)


def mats(ds):
    return (H.himuon_matrix_t * max(len(ds), 1))(*ds)


def empty(cols):
    return H.himuon_matrix_t(None, 0, cols, cols)


def gated(x=sd(10, 64, ptr=at(0)), w=None, n=None, tr=0, ends=at(5), h=sd(10, 16, ptr=at(1)), p=sd(10, 32, ptr=at(4)), act=0,
          dt=H.BF16):
    w = [sd(64, 32, ptr=at(2)), sd(64, 32, ptr=at(3))] if w is None else w
    return H.lib.himuon_grouped_gated_mm(ref(x), mats(w) if w else None, len(w) if n is None else n, tr, ends, ref(h), ref(p),
                                         act, dt, None)


def gated_grad(dy=sd(10, 64, ptr=at(0)), w=None, n=None, tr=0, ends=at(5), p=sd(10, 32, ptr=at(1)), d=sd(10, 32, ptr=at(4)),
               h=sd(10, 16, ptr=at(6)), act=0, dt=H.BF16):
    w = [sd(16, 64, ptr=at(2)), sd(16, 64, ptr=at(3))] if w is None else w
    return H.lib.himuon_grouped_gated_mm_grad(ref(dy), mats(w) if w else None, len(w) if n is None else n, tr, ends, ref(p),
                                              ref(d), ref(h), act, dt, None)


def test_gated_refusals():
    assert gated(x=None) == gated(h=None) == gated(w=[]) == gated(ends=None) == gated(n=0) == INVALID
    assert gated(dt=H.BF16_PRECISE) == gated(act=4) == gated(act=-1) == UNSUPPORTED
    assert gated(w=[sd(64, 33, ptr=at(2))]) == INVALID                      # an odd number of columns
    assert gated(h=sd(10, 17, ptr=at(1))) == gated(h=sd(9, 16, ptr=at(1))) == INVALID
    assert gated(p=sd(10, 31, ptr=at(4))) == gated(p=sd(11, 32, ptr=at(4))) == INVALID
    assert gated(x=sd(10, 63, ptr=at(0))) == gated(tr=1) == INVALID
    assert gated(w=[sd(64, 32, ptr=at(2)), sd(64, 30, ptr=at(3))]) == INVALID
    assert gated(ends=at(5) + 2) == gated(h=sd(10, 16, ptr=at(1) + 1)) == LAYOUT
    assert gated(h=sd(10, 16, ptr=at(0))) == gated(p=sd(10, 32, ptr=at(3))) == gated(p=sd(10, 32, ptr=at(1))) == OVERLAP
    assert gated(h=sd(10, 16, ld=48, ptr=at(4)), p=sd(10, 32, ld=40, ptr=at(4) + 32)) == OVERLAP
    assert gated(ends=at(1)) == gated(ends=at(4)) == OVERLAP
    assert gated(x=empty(64), h=empty(16), p=empty(32)) == gated(x=empty(64), h=empty(16), p=None) == OK
    huge = (1 << 31) - 1
    assert gated(x=sd(huge, 64, ptr=1 << 40), h=sd(huge, 16, ptr=1 << 50), p=None) == LAYOUT


def test_gated_grad_refusals():
    assert gated_grad(dy=None) == gated_grad(p=None) == gated_grad(d=None) == gated_grad(w=[]) == gated_grad(ends=None) == INVALID
    assert gated_grad(dt=7) == gated_grad(act=9) == UNSUPPORTED
    assert gated_grad(p=sd(10, 30, ptr=at(1))) == gated_grad(d=sd(10, 16, ptr=at(4))) == gated_grad(h=sd(10, 32, ptr=at(6))) == INVALID
    assert gated_grad(tr=1) == gated_grad(dy=sd(10, 16, ptr=at(0))) == gated_grad(d=sd(9, 32, ptr=at(4))) == INVALID
    assert gated_grad(d=sd(10, 32, ptr=at(4) + 1)) == LAYOUT
    # D may be P, but nothing else may overlap
    assert gated_grad(d=sd(10, 32, ptr=at(1) + 64)) == gated_grad(d=sd(10, 32, ld=40, ptr=at(1))) == OVERLAP
    assert gated_grad(d=sd(10, 32, ptr=at(0))) == gated_grad(d=sd(10, 32, ptr=at(2))) == gated_grad(d=sd(10, 32, ptr=at(5))) == OVERLAP
    assert gated_grad(h=sd(10, 16, ptr=at(1))) == gated_grad(h=sd(10, 16, ptr=at(4))) == gated_grad(h=sd(10, 16, ptr=at(0))) == OVERLAP
    assert gated_grad(dy=empty(64), p=empty(32), d=empty(32), h=empty(16)) == OK


def norm(x=sd(6, 100, ptr=at(0)), w=at(1), b=at(2), eps=1e-5, y=sd(6, 100, ptr=at(3)), stats=at(4), dt=H.FP32):
    return H.lib.himuon_layer_norm(ref(x), w, b, eps, ref(y), stats, dt, None)


def norm_grad(x=sd(6, 100, ptr=at(0)), w=at(1), stats=at(4), dy=sd(6, 100, ptr=at(5)), dx=sd(6, 100, ptr=at(6)), dw=at(7), db=at(8),
              dt=H.FP32, ws=at(9), nbytes=1 << 20):
    return H.lib.himuon_layer_norm_grad(ref(x), w, stats, ref(dy), ref(dx), dw, db, dt, ws, nbytes, None)


def test_norm_refusals():
    assert norm(x=None) == norm(y=None) == norm(eps=-1.0) == norm(eps=float("nan")) == norm(eps=float("inf")) == INVALID
    assert norm(y=sd(6, 99, ptr=at(3))) == norm(y=sd(5, 100, ptr=at(3))) == INVALID
    big = H.MAX_NORM_COLS + 1
    assert norm(dt=H.BF16_PRECISE) == norm(x=sd(6, big, ptr=at(0)), y=sd(6, big, ptr=at(3))) == UNSUPPORTED
    assert norm(w=at(1) + 2) == norm(stats=at(4) + 4) == norm(x=sd(6, 100, ptr=at(0) + 1)) == LAYOUT
    assert norm(y=sd(6, 100, ptr=at(0) + 400)) == norm(y=sd(6, 100, ld=104, ptr=at(0))) == OVERLAP
    assert norm(y=sd(6, 100, ptr=at(1))) == norm(stats=at(0)) == norm(stats=at(3)) == norm(stats=at(2)) == OVERLAP
    assert norm(x=empty(100), y=empty(100), stats=None) == OK


def test_norm_grad_refusals():
    assert norm_grad(x=None) == norm_grad(dy=None) == norm_grad(stats=None) == INVALID
    assert norm_grad(dy=sd(6, 99, ptr=at(5))) == norm_grad(dx=sd(7, 100, ptr=at(6))) == INVALID
    assert norm_grad(dt=5) == UNSUPPORTED
    assert norm_grad(dw=at(7) + 2) == norm_grad(ws=at(9) + 8) == LAYOUT
    assert norm_grad(dx=sd(6, 100, ptr=at(5) + 4)) == norm_grad(dw=at(8)) == norm_grad(db=at(0)) == norm_grad(dw=at(4)) == OVERLAP
    assert norm_grad(dx=sd(6, 100, ptr=at(1))) == norm_grad(ws=at(5)) == norm_grad(ws=at(6)) == OVERLAP
    need = ctypes.c_size_t(0)
    size = lambda x, dt=H.FP32: H.lib.himuon_layer_norm_grad_workspace(ref(x), dt, ctypes.byref(need))
    assert size(sd(6, 100)) == OK and 0 < need.value <= 512 * 2 * 100 * 4
    assert norm_grad(nbytes=need.value - 1) == norm_grad(ws=None) == WORKSPACE
    assert size(sd(1 << 20, 32768)) == OK and need.value <= 512 * 2 * 32768 * 4
    assert size(None) == size(sd(-1, 10)) == size(sd(6, 0)) == INVALID
    assert size(sd(6, 32769)) == size(sd(6, 10), H.BF16_PRECISE) == UNSUPPORTED
    assert H.lib.himuon_layer_norm_grad_workspace(ref(sd(6, 10)), H.FP32, None) == INVALID
    # nothing asked for, or no rows and no sums: nothing to do
    assert norm_grad(dx=None, dw=None, db=None, ws=None, nbytes=0) == OK
    assert norm_grad(x=empty(100), dy=empty(100), dx=empty(100), dw=None, db=None, stats=None, ws=None) == OK


def adamw(w=UNSET, g=UNSET, s=UNSET, n=None, bits=32, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.1, step=1, scale=None, wdt=H.FP32,
          gdt=H.FP32):
    w = [sd(4, 100, ptr=at(0)), sd(1, 300, ptr=at(1))] if w is UNSET else w
    g = [sd(4, 100, ptr=at(2)), sd(1, 300, ptr=at(3))] if g is UNSET else g
    s = [(at(4), at(5), at(8), at(9)), (at(6), at(7), at(10), at(11))] if s is UNSET else s
    states = None if s is None else (H.himuon_adamw_state_t * max(len(s), 1))(*[H.himuon_adamw_state_t(*x) for x in s])
    return H.lib.himuon_adamw_step(None if w is None else mats(w), None if g is None else mats(g), states,
                                   len(w or []) if n is None else n, bits, lr, b1, b2, eps, wd, step, scale, wdt, gdt, None)


def test_adamw_refusals():
    assert adamw(w=None, n=2) == adamw(g=None) == adamw(s=None) == adamw(n=-1) == INVALID
    assert adamw(bits=16) == adamw(wdt=H.BF16_PRECISE) == adamw(gdt=9) == UNSUPPORTED
    nan, inf = float("nan"), float("inf")
    for k, bad in {"lr": (nan, inf), "wd": (nan, -inf), "b1": (1.0, -0.1, nan), "b2": (1.0, 2.0, nan), "eps": (0.0, -1e-8, nan, inf, 1e39, 1e-39),
                   "step": (0, -5)}.items():
        for v in bad:
            assert adamw(**{k: v}) == INVALID, (k, v)
    assert adamw(g=[sd(4, 100, ptr=at(2)), sd(300, 1, ptr=at(3))]) == INVALID
    assert adamw(w=[sd(4, 100, ptr=at(0)), H.himuon_matrix_t(None, 1, 300, 300)]) == INVALID
    assert adamw(s=[(at(4), at(5), None, None), (at(6), None, None, None)]) == INVALID
    assert adamw(bits=8, s=[(at(4), at(5), at(8), at(9)), (at(6), at(7), at(10), None)]) == INVALID
    assert adamw(s=[(at(4) + 2, at(5), None, None), (at(6), at(7), None, None)]) == adamw(scale=at(20) + 1) == LAYOUT
    assert adamw(w=[sd(4, 100, ptr=at(0)), sd(1, 300, ptr=at(0) + 1200)]) == OVERLAP
    assert adamw(g=[sd(4, 100, ptr=at(0)), sd(1, 300, ptr=at(3))]) == OVERLAP
    assert adamw(s=[(at(4), at(4) + 1596, None, None), (at(6), at(7), None, None)]) == OVERLAP
    assert adamw(s=[(at(4), at(5), None, None), (at(6), at(0), None, None)]) == OVERLAP
    assert adamw(bits=8, s=[(at(4), at(5), at(8), at(9)), (at(6), at(7), at(8) + 4, at(11))]) == OVERLAP
    assert adamw(scale=at(0)) == adamw(scale=at(5) + 4) == OVERLAP
    # one weight twice, in the same call
    assert adamw(w=[sd(4, 100, ptr=at(0))] * 2, g=[sd(4, 100, ptr=at(2)), sd(4, 100, ptr=at(3))]) == OVERLAP
    big = (1 << 31) - 1
    assert adamw(w=[sd(big, big, ptr=1 << 40)], g=[sd(big, big, ptr=1 << 40)], s=[(at(4), at(5), None, None)]) != OK
    assert adamw(w=[], g=[], s=[]) == adamw(w=None, g=None, s=None, n=0) == OK
