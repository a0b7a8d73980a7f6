"""Host-side refusals of the recurrence, slot and conv-gradient entry points.  Every call below must be rejected (or have
nothing to do) before a launch: its placeholder pointers are never dereferenced."""
import ctypes

import pytest
import torch

import gated_deltanet_gdr_b200 as gdr
from gated_deltanet_gdr_b200 import build as gbuild

NUL = None


def at(k):
    """aligned, non-NULL placeholders, a gigabyte apart"""
    return ctypes.c_void_p((k + 1) << 30)


@pytest.fixture(scope="module")
def L():
    gbuild.build()
    return gdr.lib()


def fwd(L, **kw):
    a = dict(x=at(0), g=at(1), h0=NUL, lens=NUL, B=2, N=3, S=8, D=16, dt=gdr.GDR_BF16, gt=gdr.GDR_F32, mode=0, out=at(2),
             fin=at(3), ck=NUL)
    a.update(kw)
    return L.gdr_scan_fwd(*a.values(), None)


def bwd(L, **kw):
    a = dict(x=at(0), g=at(1), ck=at(2), dout=at(3), df=NUL, lens=NUL, B=2, N=3, S=8, D=16, dt=gdr.GDR_BF16, gt=gdr.GDR_F32,
             mode=0, dx=at(4), dg=at(5), di=at(6))
    a.update(kw)
    return L.gdr_scan_bwd(*a.values(), None)


def step(L, **kw):
    a = dict(x=at(0), g=at(1), pool=at(2), slots=4, idx=at(3), lens=NUL, acc=NUL, B=2, N=3, S=1, D=16, dt=gdr.GDR_BF16,
             gt=gdr.GDR_F32, mode=0, per=0, out=at(4))
    a.update(kw)
    return L.gdr_scan_step(*a.values(), None)


def conv(L, **kw):
    a = dict(x=at(0), w=at(1), bias=NUL, s0=NUL, lens=NUL, dq=at(2), dk=at(3), dv=at(4), ds=NUL, B=1, S=8, Nk=2, Nv=4, Dk=128,
             Dv=128, K=4, dt=gdr.GDR_BF16, dx=at(5), dw=at(6), db=at(7), dsi=NUL, ws=at(8), nb=1 << 30)
    a.update(kw)
    return L.gdr_conv1d_bwd(*a.values(), None)


@pytest.mark.parametrize("f", [fwd, bwd, step])
def test_scan_sizes_types_and_modes(L, f):
    assert f(L, B=-1) == gdr.GDR_ERR_SHAPE
    assert f(L, N=0) == gdr.GDR_ERR_SHAPE
    assert f(L, D=0) == gdr.GDR_ERR_SHAPE
    assert f(L, S=-1) == gdr.GDR_ERR_SHAPE
    assert f(L, mode=2) == gdr.GDR_ERR_SHAPE
    assert f(L, B=1 << 15, N=1 << 8, D=1 << 8) == gdr.GDR_ERR_SHAPE
    assert f(L, B=1, N=1 << 15, D=1 << 16) == gdr.GDR_ERR_SHAPE
    assert f(L, dt=3) == gdr.GDR_ERR_DTYPE
    assert f(L, gt=gdr.GDR_F16) == gdr.GDR_ERR_DTYPE
    assert f(L, dt=gdr.GDR_F32, gt=gdr.GDR_BF16) == gdr.GDR_ERR_DTYPE
    assert f(L, x=NUL) == gdr.GDR_ERR_NULL
    assert f(L, g=NUL) == gdr.GDR_ERR_NULL
    assert f(L, g=ctypes.c_void_p((2 << 30) + 8)) == gdr.GDR_ERR_ALIGN
    assert f(L, lens=ctypes.c_void_p((20 << 30) + 4)) == gdr.GDR_ERR_ALIGN
    assert f(L, B=0) == gdr.GDR_OK


def test_scan_buffers(L):
    assert fwd(L, B=1, N=1, D=(1 << 26) + 1) == gdr.GDR_ERR_SHAPE
    assert bwd(L, B=1, N=1, D=(1 << 26) + 1) == gdr.GDR_ERR_SHAPE
    assert fwd(L, out=NUL) == gdr.GDR_ERR_NULL
    assert fwd(L, out=at(0)) == gdr.GDR_ERR_SHAPE  # in place
    assert fwd(L, out=ctypes.c_void_p((2 << 30) + 64)) == gdr.GDR_ERR_SHAPE  # inside g
    assert fwd(L, ck=at(3)) == gdr.GDR_ERR_SHAPE  # two outputs in one place
    assert fwd(L, h0=ctypes.c_void_p((4 << 30) + 16)) == gdr.GDR_ERR_SHAPE  # a state half over the other
    assert fwd(L, S=0, fin=NUL, x=NUL, g=NUL, out=NUL) == gdr.GDR_OK
    assert bwd(L, ck=NUL) == gdr.GDR_ERR_NULL
    assert bwd(L, dout=NUL) == gdr.GDR_ERR_NULL
    assert bwd(L, dg=at(4)) == gdr.GDR_ERR_SHAPE
    assert bwd(L, dx=at(3)) == gdr.GDR_ERR_SHAPE
    assert bwd(L, S=0, di=NUL, x=NUL, g=NUL, ck=NUL, dout=NUL, dx=NUL, dg=NUL) == gdr.GDR_OK
    assert step(L, S=9) == gdr.GDR_ERR_SHAPE
    assert step(L, S=0) == gdr.GDR_ERR_SHAPE
    assert step(L, slots=0) == gdr.GDR_ERR_SHAPE
    assert step(L, pool=NUL) == gdr.GDR_ERR_NULL
    assert step(L, idx=NUL) == gdr.GDR_ERR_NULL
    assert step(L, out=at(0)) == gdr.GDR_ERR_SHAPE


def test_conv1d_bwd(L):
    need = L.gdr_conv1d_bwd_workspace(1, 8, 2, 4, 128, 128, 4)
    assert need >= 1024 * 5 * 4 and L.gdr_conv1d_bwd_workspace(1, 8, 2, 4, 128, 128, 9) == 0
    assert L.gdr_conv1d_bwd_workspace(0, 8, 2, 4, 128, 128, 4) == 0
    assert conv(L, K=0) == gdr.GDR_ERR_SHAPE
    assert conv(L, K=9) == gdr.GDR_ERR_SHAPE
    assert conv(L, Nv=3) == gdr.GDR_ERR_SHAPE
    assert conv(L, B=70000) == gdr.GDR_ERR_SHAPE
    assert conv(L, dt=4) == gdr.GDR_ERR_DTYPE
    assert conv(L, Dv=48) == gdr.GDR_ERR_UNSUPPORTED
    for name in ("x", "w", "dq", "dk", "dv", "dx", "dw", "ws"):
        assert conv(L, **{name: NUL}) == gdr.GDR_ERR_NULL, name
    assert conv(L, nb=need - 1) == gdr.GDR_ERR_WORKSPACE
    assert conv(L, db=ctypes.c_void_p((8 << 30) + 4)) == gdr.GDR_ERR_ALIGN
    assert conv(L, dx=at(0)) == gdr.GDR_ERR_SHAPE
    assert conv(L, ws=at(6)) == gdr.GDR_ERR_SHAPE


def pool(*p):
    a = (gdr.GdrPoolStruct * len(p))()
    for i, (d, n) in enumerate(p):
        a[i].data, a[i].slot_bytes = d, n
    return a


def test_slots(L):
    one = pool((1 << 40, 64))
    calls = {
        "copy": lambda p=one, k=1, s=4, n=2, a=at(0), b=at(1): L.gdr_slot_copy(p, k, s, a, b, n, None),
        "fork": lambda p=one, k=1, s=4, n=2, a=at(0), b=at(1), c=at(2): L.gdr_slot_fork(p, k, s, a, b, n, c, None),
        "compact": lambda p=one, k=1, s=4, a=at(0), b=at(1), c=at(2): L.gdr_slot_compact(p, k, s, a, b, c, None),
        "free": lambda p=one, k=1, s=4, n=2, a=at(0), b=NUL: L.gdr_slot_free(p, k, s, a, n, b, None),
    }
    for name, f in calls.items():
        assert f(k=0) == gdr.GDR_ERR_SHAPE, name
        assert f(k=65) == gdr.GDR_ERR_SHAPE, name
        assert f(s=0) == gdr.GDR_ERR_SHAPE, name
        assert f(s=1 << 24) == gdr.GDR_ERR_SHAPE, name
        assert f(p=None) == gdr.GDR_ERR_NULL, name
        assert f(a=NUL) == gdr.GDR_ERR_NULL, name
        assert f(a=ctypes.c_void_p((1 << 30) + 4)) == gdr.GDR_ERR_ALIGN, name
        assert f(p=pool((None, 64))) == gdr.GDR_ERR_NULL, name
        assert f(p=pool(((1 << 40) + 8, 64))) == gdr.GDR_ERR_ALIGN, name
        assert f(p=pool((1 << 40, 0))) == gdr.GDR_ERR_SHAPE, name
        assert f(p=pool((1 << 40, (1 << 37) + 1))) == gdr.GDR_ERR_SHAPE, name
        assert f(p=pool((1 << 40, 64), ((1 << 40) + 128, 64)), k=2) == gdr.GDR_ERR_SHAPE, name  # they overlap
        if name != "compact":
            assert f(n=-1) == gdr.GDR_ERR_SHAPE, name
            assert f(n=65537) == gdr.GDR_ERR_SHAPE, name
            assert f(n=0) == gdr.GDR_OK, name
        assert f(p=pool((1 << 30, 64))) == gdr.GDR_ERR_SHAPE, name  # the first index array lies in the pool
    assert calls["copy"](b=NUL) == gdr.GDR_ERR_NULL
    assert calls["fork"](n=16385) == gdr.GDR_ERR_SHAPE
    assert calls["fork"](c=at(0)) == gdr.GDR_ERR_SHAPE
    assert calls["fork"](c=at(1)) == gdr.GDR_ERR_SHAPE
    assert calls["compact"](s=262145) == gdr.GDR_ERR_SHAPE
    assert calls["compact"](b=at(0)) == gdr.GDR_ERR_SHAPE
    assert calls["compact"](c=at(0)) == gdr.GDR_ERR_SHAPE
    assert calls["free"](b=at(0)) == gdr.GDR_ERR_SHAPE


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device status; on a GPU host the placeholder pointers "
                    "would be launched on")
def test_no_device_status(L):
    assert fwd(L) == bwd(L) == step(L) == conv(L) == gdr.GDR_ERR_DEVICE
    assert L.gdr_slot_copy(pool((1 << 40, 64)), 1, 4, at(0), at(1), 2, None) == gdr.GDR_ERR_DEVICE
