"""include/gmm_experts.h refuses bad arguments on the host before launching
anything, and accepts empty problems without one.  CPU only: no call here
reaches a kernel."""
import ctypes

import pytest
import torch

from soft_clustering_amd import experts, gmm

LIB = gmm._lib
P = 4096          # stands for a device pointer; never dereferenced on the host
ARG, WORK, OK = gmm.GMM_E_ARG, gmm.GMM_E_WORKSPACE, gmm.GMM_OK


def routes(n=10, m=2, k=3, offsets=P, entry=P, slot=P):
    return ctypes.byref(experts._CRoutes(n, m, k, offsets, entry, slot))


def desc(d_in=16, d_out=24, ldx=None, ldy=None, lddx=None, dtype=0, sorted_rows=0):
    pick = lambda v, d: d if v is None else v   # noqa: E731
    return ctypes.byref(experts._CLinear(d_in, d_out, pick(ldx, d_in), pick(ldy, d_out), pick(lddx, d_in), dtype, sorted_rows))


BAD_SHAPES = [dict(n=-1), dict(m=0), dict(m=17), dict(k=0), dict(k=4097), dict(n=(1 << 30) + 1, m=1), dict(n=1 << 29, m=3),
              dict(n=1 << 62, m=16)]


@pytest.mark.parametrize("kw", BAD_SHAPES)
def test_bad_shapes(kw):
    s = dict(n=10, m=2, k=3) | kw
    need = ctypes.c_size_t(0)
    assert LIB.gmm_route_workspace_bytes(s["n"], s["m"], s["k"], ctypes.byref(need)) == ARG
    assert LIB.gmm_route(s["n"], s["m"], s["k"], P, P, 1 << 40, P, P, P, None) == ARG
    assert LIB.gmm_dispatch(routes(**s), 8, 0, P, 8, P, 8, None) == ARG
    assert LIB.gmm_combine(routes(**s), 8, 0, P, 8, P, P, 8, None) == ARG
    assert LIB.gmm_linear(routes(**s), desc(), P, P, P, P, None) == ARG
    assert LIB.gmm_linear_backward_workspace_bytes(s["n"], s["m"], s["k"], desc(), ctypes.byref(need)) == ARG
    assert LIB.gmm_linear4(s["n"], s["m"], s["k"], 32, 8, 32, 0, P, 32, P, P, P, P, P, P, 8, None) == ARG


def test_route_refusals():
    need = ctypes.c_size_t(0)
    assert LIB.gmm_route_workspace_bytes(10, 2, 3, None) == ARG
    assert LIB.gmm_route_workspace_bytes(10, 2, 3, ctypes.byref(need)) == OK and need.value == 0
    assert LIB.gmm_route_workspace_bytes(10 ** 6, 2, 300, ctypes.byref(need)) == OK and need.value > 0
    ok = (10 ** 6, 2, 300, P)
    assert LIB.gmm_route(*ok, None, need.value, P, P, P, None) == ARG
    assert LIB.gmm_route(*ok, P + 1, need.value, P, P, P, None) == ARG
    assert LIB.gmm_route(*ok, P, need.value - 1, P, P, P, None) == WORK
    for args in [(None, P, P, P), (P, None, P, P), (P, P, None, P), (P, P, P, None)]:
        assert LIB.gmm_route(10, 2, 3, args[0], None, 0, *args[1:], None) == ARG


def test_route_workspace_far_below_points_times_lists():
    """One counter a list for every 8192 entries (16384 with more than 1024 lists); never the
    N x K matrix."""
    b = ctypes.c_size_t(0)
    for n, m, k in [(10 ** 7, 2, 256), (10 ** 8, 1, 4096), (1 << 30, 1, 4096), (10 ** 6, 16, 1024)]:
        assert LIB.gmm_route_workspace_bytes(n, m, k, ctypes.byref(b)) == OK
        assert b.value <= (n * m / 8192 + 2) * k * 4


def test_rows_refusals():
    assert LIB.gmm_dispatch(None, 8, 0, P, 8, P, 8, None) == ARG
    for f in (LIB.gmm_dispatch, LIB.gmm_dispatch_backward):
        for r in (routes(offsets=None), routes(entry=None), routes(slot=None)):
            assert f(r, 8, 0, P, 8, P, 8, None) == ARG
        for d, t, x, ldx, y, ldy in [(0, 0, P, 8, P, 8), ((1 << 20) + 1, 0, P, 1 << 21, P, 1 << 21), (8, -1, P, 8, P, 8),
                                     (8, 3, P, 8, P, 8), (8, 0, P, 7, P, 8), (8, 0, P, 8, P, 7), (8, 0, P, 1 << 23, P, 8),
                                     (8, 0, None, 8, P, 8), (8, 0, P, 8, None, 8)]:
            assert f(routes(), d, t, x, ldx, y, ldy, None) == ARG
    for z, g, o in [(None, P, P), (P, None, P), (P, P, None)]:
        assert LIB.gmm_combine(routes(), 8, 0, z, 8, g, o, 8, None) == ARG
    cb = lambda dout=P, lddo=8, z=P, ldz=8, g=P, dz=P, lddz=8, dg=P: LIB.gmm_combine_backward(   # noqa: E731
        routes(), 8, 0, dout, lddo, z, ldz, g, dz, lddz, dg, None)
    for kw in (dict(dout=None), dict(z=None), dict(g=None), dict(lddo=7), dict(ldz=7), dict(lddz=7)):
        assert cb(**kw) == ARG
    assert cb(dz=None, dg=None) == OK          # nothing asked for


def test_linear_refusals():
    for kw in (dict(d_in=0), dict(d_out=0), dict(d_in=(1 << 20) + 1), dict(dtype=3), dict(dtype=-1), dict(sorted_rows=2),
               dict(ldx=15), dict(ldy=23)):
        assert LIB.gmm_linear(routes(), desc(**kw), P, P, P, P, None) == ARG
    assert LIB.gmm_linear(routes(), None, P, P, P, P, None) == ARG
    for a in ((None, P, P, P), (P, None, P, P), (P, P, P, None)):
        assert LIB.gmm_linear(routes(), desc(), *a, None) == ARG
    back = lambda r=routes(), d=desc(), dy=P, x=P, w=P, dx=P, dw=P, db=P, ws=P, nb=1 << 40: LIB.gmm_linear_backward(   # noqa: E731
        r, d, dy, x, w, dx, dw, db, ws, nb, None)
    for kw in (dict(dy=None), dict(x=None), dict(w=None), dict(dw=None), dict(d=desc(lddx=15)), dict(d=desc(ldx=15)),
               dict(d=desc(ldy=23)), dict(r=routes(entry=None))):
        assert back(**kw) == ARG
    need = ctypes.c_size_t(0)
    big = routes(n=10 ** 6)
    assert LIB.gmm_linear_backward_workspace_bytes(10 ** 6, 2, 3, desc(), ctypes.byref(need)) == OK and need.value > 0
    assert back(r=big, ws=None) == ARG and back(r=big, ws=P + 16) == ARG and back(r=big, nb=need.value - 1) == WORK
    assert LIB.gmm_linear_backward_workspace_bytes(10, 2, 3, desc(), None) == ARG


def test_linear4_refusals():
    call = lambda n=4, m=2, k=3, di=64, do=8, group=32, t=0, x=P, ldx=64, idx=P, g=P, c=P, s=P, o=P, ldo=8: (   # noqa: E731
        LIB.gmm_linear4(n, m, k, di, do, group, t, x, ldx, idx, g, c, s, None, o, ldo, None))
    for kw in (dict(n=1025), dict(n=-1), dict(group=16), dict(group=0), dict(group=256), dict(di=0), dict(do=0), dict(t=3),
               dict(ldx=63), dict(ldo=7), dict(x=None), dict(idx=None), dict(g=None), dict(c=None), dict(s=None),
               dict(o=None)):
        assert call(**kw) == ARG
    q = lambda rows=4, d=64, group=32, t=0, w=P, c=P, s=P: LIB.gmm_quantize4(rows, d, group, t, w, c, s, None)   # noqa: E731
    for kw in (dict(rows=-1), dict(d=0), dict(group=40), dict(t=5), dict(w=None), dict(c=None), dict(s=None)):
        assert q(**kw) == ARG


def test_no_points_need_nothing():
    r = routes(n=0, offsets=None, entry=None, slot=None)
    assert LIB.gmm_dispatch(r, 8, 0, None, 8, None, 8, None) == OK
    assert LIB.gmm_dispatch_backward(r, 8, 0, None, 8, None, 8, None) == OK
    assert LIB.gmm_combine(r, 8, 0, None, 8, None, None, 8, None) == OK
    assert LIB.gmm_combine_backward(r, 8, 0, None, 8, None, 8, None, P, 8, P, None) == OK
    assert LIB.gmm_linear(r, desc(), None, None, None, None, None) == OK
    assert LIB.gmm_linear_backward(r, desc(), None, None, None, P, None, None, None, 0, None) == OK
    assert LIB.gmm_linear4(0, 2, 3, 64, 8, 32, 0, None, 64, None, None, None, None, None, None, 8, None) == OK
    assert LIB.gmm_quantize4(0, 64, 32, 0, None, None, None, None) == OK


def test_cpu_tensors_are_refused():
    idx = torch.zeros((4, 2), dtype=torch.int32)
    r = experts.Routes(torch.zeros(4, dtype=torch.int32), torch.zeros(8, dtype=torch.int32), idx)
    x = torch.zeros((4, 8))
    for f in (lambda: experts.route(idx, 3), lambda: experts.dispatch(x, r), lambda: experts.quantize4(x, 32),
              lambda: experts.combine(torch.zeros((8, 8)), torch.zeros((4, 2)), r)):
        with pytest.raises(ValueError):
            f()
