"""Refusals of the feature operators, on the host, before any HIP call: the
C ABI with pointers that are never read, and the binding with CPU tensors."""

import ctypes
from types import SimpleNamespace

import pytest
import torch

import group_shared_fixed_amd as hs
from group_shared_fixed_amd import binding as hb

NULL, DIM, UNSUP, ALIGN, WS = -1, -2, -3, -4, -5
P = ctypes.c_void_p
A, MIS = P(0x100000), P(0x100008)
ODD = P(0x100001)


@pytest.fixture(scope="module")
def L():
    return hb.lib()


def drop(L, x=A, r=None, y=A, rows=4, cols=24, ldx=24, ldr=24, p=0.1, od=None, dt=0):
    return L.haste_dropout(x, r, y, rows, cols, ldx, ldr, p, 1, 2, od, dt, None)


def test_dropout_refuses(L):
    assert drop(L, x=None) == NULL and drop(L, y=None) == NULL
    assert drop(L, rows=0) == DIM and drop(L, cols=0) == DIM and drop(L, rows=-3) == DIM
    assert drop(L, ldx=23) == DIM and drop(L, r=A, ldr=23) == DIM
    assert drop(L, p=-0.1) == DIM and drop(L, p=1.0001) == DIM and drop(L, p=float("nan")) == DIM
    assert drop(L, dt=3) == UNSUP and drop(L, dt=-1) == UNSUP
    assert drop(L, rows=1 << 41) == UNSUP and drop(L, cols=1 << 21, ldx=1 << 21) == UNSUP
    assert drop(L, x=ODD) == ALIGN and drop(L, y=MIS) == ALIGN and drop(L, r=ODD) == ALIGN
    assert drop(L, dt=2, x=P(0x100002)) == ALIGN
    assert drop(L, od=P(0x100004)) == ALIGN


def norm(L, x=A, r=A, g=A, s=A, y=A, q=None, qs=None, rstd=A, rows=4, cols=24, ldx=24, ldr=24, eps=1e-6, p=0.0, dt=0):
    return L.haste_add_norm(x, r, g, s, y, q, qs, rstd, rows, cols, ldx, ldr, eps, p, 0, 0, None, dt, None)


def test_add_norm_refuses(L):
    assert norm(L, x=None) == NULL and norm(L, g=None) == NULL and norm(L, y=None) == NULL
    assert norm(L, q=A, qs=None) == NULL
    assert norm(L, rows=0) == DIM and norm(L, ldx=8) == DIM and norm(L, ldr=8) == DIM
    assert norm(L, eps=-1.0) == DIM and norm(L, eps=float("nan")) == DIM and norm(L, eps=float("inf")) == DIM
    assert norm(L, p=2.0) == DIM
    assert norm(L, cols=32769, ldx=32769, ldr=32769) == UNSUP and norm(L, dt=4) == UNSUP
    assert norm(L, rows=1 << 31) == UNSUP
    assert norm(L, g=MIS) == ALIGN and norm(L, s=MIS) == ALIGN and norm(L, rstd=MIS) == ALIGN
    assert norm(L, q=MIS, qs=A) == ALIGN and norm(L, x=ODD) == ALIGN


def nbwd(L, dy=A, s=A, g=A, rstd=A, ds=A, dres=A, dx=A, dg=A, rows=64, cols=24, lddy=24, ldds=24, p=0.0, dt=0, ws=A,
         wsb=1 << 20):
    return L.haste_add_norm_bwd(dy, s, g, rstd, ds, dres, dx, dg, rows, cols, lddy, ldds, p, 0, 0, None, dt, ws, wsb,
                                None)


def test_add_norm_bwd_refuses(L):
    for k in ("dy", "s", "g", "rstd", "dres"):
        assert nbwd(L, **{k: None}) == NULL
    assert nbwd(L, rows=0) == DIM and nbwd(L, lddy=2) == DIM and nbwd(L, ldds=2) == DIM and nbwd(L, p=-1.0) == DIM
    assert nbwd(L, cols=40000, lddy=40000, ldds=40000) == UNSUP and nbwd(L, dt=9) == UNSUP
    assert nbwd(L, s=MIS) == ALIGN and nbwd(L, dx=MIS) == ALIGN and nbwd(L, dg=MIS) == ALIGN
    assert nbwd(L, ws=None) == WS and nbwd(L, ws=P(0x100010)) == WS
    assert nbwd(L, wsb=L.haste_add_norm_workspace_size(64, 24) - 1) == WS
    assert L.haste_add_norm_workspace_size(0, 24) == 0 and L.haste_add_norm_workspace_size(4, 40000) == 0


def test_quantize_and_score_refuse(L):
    def quant(x=A, q=A, s=A, rows=3, cols=16, ld=16, dt=0):
        return L.haste_quantize_rows(x, q, s, rows, cols, ld, dt, None)
    assert quant(x=None) == NULL and quant(q=None) == NULL and quant(s=None) == NULL
    assert quant(rows=0) == DIM and quant(ld=15) == DIM and quant(dt=7) == UNSUP
    assert quant(cols=40000, ld=40000) == UNSUP and quant(q=MIS) == ALIGN

    def score(hq=A, h=A, Wq=A, w=A, Z=A, B=2, H=32, n=5):
        return L.haste_score_a8w8(hq, h, Wq, w, Z, B, H, n, None)
    for k in ("hq", "h", "Wq", "w", "Z"):
        assert score(**{k: None}) == NULL and score(**{k: MIS}) == ALIGN
    assert score(B=0) == DIM and score(H=0) == DIM and score(n=0) == DIM
    assert score(H=24) == UNSUP and score(H=1 << 15) == UNSUP and score(B=(1 << 20) + 1) == UNSUP
    assert score(n=2**31 - 64) == UNSUP and score(B=1 << 20, n=2**31 - 65) == UNSUP


def soft(L, grad=True, h=A, W=A, rp=A, col=A, scale=1.0, dW=A, dh=A, rl=A, lse=A, loss=A, B=40, H=64, n=1000, ldh=64,
         ldw=64, dt=0, ws=A, wsb=1 << 30):
    if grad:
        return L.haste_softmax_step(h, W, rp, col, scale, dW, dh, rl, lse, loss, B, H, n, ldh, ldw, dt, ws, wsb, None)
    return L.haste_softmax_loss(h, W, rp, col, scale, rl, lse, loss, B, H, n, ldh, ldw, dt, ws, wsb, None)


@pytest.mark.parametrize("grad", [True, False])
def test_softmax_refuses(L, grad):
    names = ["h", "W", "rp", "col", "rl", "lse", "loss"] + (["dW", "dh"] if grad else [])
    for k in names:
        assert soft(L, grad, **{k: None}) == NULL and soft(L, grad, **{k: MIS}) == ALIGN, k
    assert soft(L, grad, B=0) == DIM and soft(L, grad, n=0) == DIM and soft(L, grad, H=0) == DIM
    assert soft(L, grad, ldh=56) == DIM and soft(L, grad, ldw=56) == DIM
    assert soft(L, grad, scale=float("inf")) == DIM and soft(L, grad, scale=float("nan")) == DIM
    assert soft(L, grad, H=60) == UNSUP and soft(L, grad, ldh=68) == UNSUP and soft(L, grad, ldw=68) == UNSUP
    assert soft(L, grad, dt=2) == UNSUP and soft(L, grad, B=(1 << 20) + 1) == UNSUP
    assert soft(L, grad, n=2**31 - 64) == UNSUP and soft(L, grad, H=16392, ldh=16392, ldw=16392) == UNSUP
    assert soft(L, grad, ws=None) == WS and soft(L, grad, ws=P(0x100010)) == WS
    least = L.haste_softmax_workspace_min(40, 64, 1000, int(grad))
    assert soft(L, grad, wsb=least - 1) == WS
    assert 0 < least <= L.haste_softmax_workspace_size(40, 64, 1000, int(grad))
    assert L.haste_softmax_workspace_size(0, 64, 10, 1) == 0 and L.haste_softmax_workspace_size(4, 60, 10, 1) == 0


def test_softmax_workspace_is_bounded(L):
    # the gradient matrix of 4096 x 131072 would be 1 GiB; a piece of it is at most 256 MiB
    full, least = (f(4096, 1024, 131072, 1) for f in (L.haste_softmax_workspace_size, L.haste_softmax_workspace_min))
    assert full - least <= 256 << 20
    # asked for, the whole of it: two bytes per logit more than the least, for a step that can keep it
    whole = L.haste_softmax_workspace_whole(4096, 1024, 131072)
    assert 1 << 30 <= whole - least + (2 << 20) <= (1 << 30) + (16 << 20)
    assert L.haste_softmax_workspace_whole(128, 1024, 131072) == L.haste_softmax_workspace_size(128, 1024, 131072, 1)
    assert L.haste_softmax_workspace_whole(4096, 1023, 131072) == 0
    assert hs.softmax_workspace_size(4096, 1024, 131072, whole=True) == whole


def test_binding_refuses():
    x = torch.zeros(4, 24, dtype=torch.bfloat16)
    g = torch.zeros(24, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        hs.dropout(x.t(), 0.1, 1)                                    # columns contiguous
    with pytest.raises(TypeError):
        hs.dropout(x.double(), 0.1, 1)
    with pytest.raises(ValueError):
        hs.dropout(x, 0.1, 1, residual=x.float())
    with pytest.raises(ValueError):
        hs.dropout(x[:1].expand(4, 24), 0.1, 1)                      # rows on one another
    with pytest.raises(ValueError):
        hs.dropout(x, 0.1, 1, out=torch.zeros(4, 25, dtype=x.dtype))
    st = SimpleNamespace(cuda_stream=0)
    with pytest.raises(hb.HasteError):
        hs.dropout(x, 1.5, 1, stream=st)
    with pytest.raises(hb.HasteError):
        hs.dropout(torch.zeros(0, 24, dtype=x.dtype), 0.5, 1, stream=st)
    with pytest.raises(ValueError):
        hs.dropout(x, 0.5, 1, residual=torch.empty(4, 24, dtype=x.dtype, device="meta"))   # another device
    with pytest.raises(ValueError):
        hs.add_norm(x, g[:8])
    with pytest.raises(ValueError):
        hs.add_norm(x, g.float())
    with pytest.raises(hb.HasteError):
        hs.add_norm(x, g, want_y=False, stream=st)                              # neither y nor codes
    with pytest.raises(ValueError):
        hs.add_norm_bwd(x, x, g, torch.zeros(3))
    with pytest.raises(ValueError):
        hs.score_a8w8(x, torch.zeros(4), x, torch.zeros(4))          # not codes
    rp, col = torch.zeros(5, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        hs.softmax_step(x, torch.zeros(9, 16, dtype=x.dtype), rp, col, 1.0)
    with pytest.raises(ValueError):
        hs.softmax_step(x, torch.zeros(9, 24), rp, col, 1.0)          # W of another type
    with pytest.raises(ValueError):
        hs.softmax_step(x, torch.zeros(9, 24, dtype=x.dtype), rp[:4], col, 1.0)
    with pytest.raises(TypeError):
        hs.softmax_loss(x, torch.zeros(9, 24, dtype=x.dtype), rp.long(), col, 1.0)
