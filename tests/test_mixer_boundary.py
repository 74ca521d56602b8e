"""Host-side checks of the layer-norm and recurrence entry points: bad
arguments are refused before any launch (no GPU needed)."""
import ctypes

import pytest
import torch

from linear_attention_delta_gb300 import kla

INVALID, UNSUPPORTED, OK = -1, -2, 0
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def lib():
    return kla.load_library()


def at(i):
    return ctypes.c_void_p(0x1000000 * i)


def ln_fwd(lib, **kw):
    a = dict(x=at(1), xs=64, res=None, rs=0, w=at(3), b=at(4), eps=1e-5,
             y=at(5), sum=None, mean=at(7), rstd=at(8), rows=4, D=64,
             dtype=BF16, wdtype=BF16)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.kla_layernorm_fwd(*a.values(), None)


def ln_bwd(lib, **kw):
    a = dict(dy=at(1), dys=64, x=at(2), xs=64, w=at(3), mean=at(4),
             rstd=at(5), ds=None, dss=0, dx=at(6), dw=at(7), db=at(8),
             rows=4, D=64, dtype=BF16, wdtype=BF16, ws=at(9),
             ws_bytes=1 << 22)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.kla_layernorm_bwd(*a.values(), None)


def glr_fwd(lib, **kw):
    a = dict(x=at(1), xsb=640, xst=64, la=at(2), asb=640, ast=64, h0=None,
             o=at(4), hT=at(5), cu=None, B=2, T=10, D=64, dtype=BF16,
             gdtype=F32)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.kla_glr_fwd(*a.values(), None)


def glr_bwd(lib, **kw):
    a = dict(o=at(1), osb=640, ost=64, la=at(2), asb=640, ast=64, h0=at(3),
             do=at(4), gsb=640, gst=64, dhT=None, dx=at(5), dla=at(6),
             dh0=at(7), cu=None, B=2, T=10, D=64, dtype=BF16, gdtype=F32)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.kla_glr_bwd(*a.values(), None)


def glr_step(lib, **kw):
    a = dict(x=at(1), xs=64, la=at(2), as_=64, S=at(3), o=at(4), N=4, D=64,
             dtype=BF16, gdtype=F32)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.kla_glr_step(*a.values(), None)


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(D=0), dict(xs=-64), dict(rs=-1), dict(eps=-1.0),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(dtype=2),
    dict(wdtype=7), dict(x=None), dict(y=None), dict(sum=at(6)),
    dict(y=at(1)), dict(x=ctypes.c_void_p(0x1000001)),
    dict(dtype=F32, y=ctypes.c_void_p(0x5000002)),
    dict(w=ctypes.c_void_p(0x3000001)),
    dict(wdtype=F32, b=ctypes.c_void_p(0x4000002)),
    dict(mean=ctypes.c_void_p(0x7000002)), dict(mean=at(8)),
    dict(res=at(2), sum=at(2)), dict(y=at(3)),
    # the last row of a strided x reaches into y
    dict(x=ctypes.c_void_p(0x5000000 - 3 * 2 * 1000), xs=1000),
])
def test_layernorm_fwd_refuses(lib, bad):
    assert ln_fwd(lib, **bad) == INVALID


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(D=0), dict(dys=-1), dict(xs=-1), dict(dss=-1),
    dict(dtype=5), dict(wdtype=-1), dict(dy=None), dict(x=None),
    dict(mean=None), dict(rstd=None), dict(dx=None), dict(ws=None),
    dict(ws_bytes=8), dict(ws=ctypes.c_void_p(0x9000008)), dict(ws=at(1)),
    dict(dx=at(1)), dict(dx=at(2)), dict(dw=at(8)), dict(ds=at(6)),
    dict(dw=ctypes.c_void_p(0x7000001)),
])
def test_layernorm_bwd_refuses(lib, bad):
    assert ln_bwd(lib, **bad) == INVALID


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(T=-1), dict(D=0), dict(xsb=-1), dict(xst=-1),
    dict(asb=-1), dict(ast=-1), dict(dtype=2), dict(gdtype=2), dict(x=None),
    dict(la=None), dict(o=None), dict(o=at(1)), dict(o=at(2)),
    dict(hT=at(1)), dict(hT=at(4)), dict(h0=at(4)),
    dict(h0=at(5), hT=ctypes.c_void_p(0x5000004)),
    dict(x=ctypes.c_void_p(0x1000001)), dict(la=ctypes.c_void_p(0x2000002)),
    dict(h0=ctypes.c_void_p(0x3000002)), dict(cu=ctypes.c_void_p(0x9000002)),
    dict(cu=at(9), B=0), dict(cu=at(4)),
])
def test_glr_fwd_refuses(lib, bad):
    assert glr_fwd(lib, **bad) == INVALID


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(T=-1), dict(D=0), dict(gst=-1), dict(gsb=-1),
    dict(dtype=2), dict(gdtype=2), dict(o=None), dict(la=None),
    dict(do=None), dict(dx=None), dict(dla=None), dict(dx=at(1)),
    dict(dla=at(2)), dict(dx=at(6)), dict(dh0=at(3)),
    dict(dhT=at(7)), dict(dh0=ctypes.c_void_p(0x7000002)),
])
def test_glr_bwd_refuses(lib, bad):
    assert glr_bwd(lib, **bad) == INVALID


@pytest.mark.parametrize("bad", [
    dict(N=-1), dict(D=0), dict(xs=-1), dict(as_=-1), dict(dtype=2),
    dict(gdtype=2), dict(x=None), dict(la=None), dict(S=None), dict(o=None),
    dict(o=at(3)), dict(o=at(1)), dict(S=at(2)),
    dict(S=ctypes.c_void_p(0x3000002)), dict(x=ctypes.c_void_p(0x1000001)),
])
def test_glr_step_refuses(lib, bad):
    assert glr_step(lib, **bad) == INVALID


def test_empty_problems_are_no_ops(lib):
    assert ln_fwd(lib, rows=0, x=None, y=None) == OK
    assert ln_bwd(lib, rows=0, x=None, dy=None, dx=None, dw=None, db=None,
                  ws=None) == OK
    assert glr_fwd(lib, B=0, x=None, la=None, o=None) == OK
    assert glr_bwd(lib, B=0, o=None, la=None, do=None, dx=None,
                   dla=None) == OK
    assert glr_step(lib, N=0, x=None, la=None, S=None, o=None) == OK


def test_workspace_sizes(lib):
    n = ctypes.c_size_t(0)
    f = lib.kla_layernorm_bwd_workspace_size
    assert f(1000, 64, BF16, ctypes.byref(n)) == OK
    assert n.value >= 2 * 64 * 4
    assert f(-1, 64, BF16, ctypes.byref(n)) == INVALID
    assert f(1, 0, BF16, ctypes.byref(n)) == INVALID
    assert f(1, 64, 9, ctypes.byref(n)) == INVALID
    assert f(1, 64, BF16, None) == INVALID


@pytest.mark.parametrize("dtype,elt", [(BF16, 2), (F32, 4)])
def test_workspace_of_wide_rows_is_a_row_of_sums_a_block(lib, dtype, elt):
    """A row a block where one block fills an SM of the 152."""
    n, f = ctypes.c_size_t(0), lib.kla_layernorm_bwd_workspace_size
    for D in (8192 // elt + 1, 16384, 100000):
        assert f(1 << 20, D, dtype, ctypes.byref(n)) == OK
        assert n.value <= 152 * 2 * D * 4
    assert f(400, 64, dtype, ctypes.byref(n)) == OK
    assert n.value <= 128 * 2 * 64 * 4


def test_glr_refuses_more_tokens_than_it_counts(lib):
    assert glr_fwd(lib, T=0x7fffffff) == UNSUPPORTED
    assert glr_bwd(lib, T=0x7fffffff) == UNSUPPORTED


def test_refuses_more_channels_and_sequences_than_it_counts(lib):
    """A thread's column would pass 2^31.  (At the limit itself the call gets
    as far as the overlap of these buffers.)"""
    n, most = ctypes.c_size_t(0), 0x7fffffff - 4096
    size = lib.kla_layernorm_bwd_workspace_size
    for D, want in ((most, INVALID), (most + 1, UNSUPPORTED),
                    (0x7fffffff, UNSUPPORTED)):
        assert ln_fwd(lib, rows=1, D=D) == want
        assert ln_bwd(lib, rows=1, D=D, ws_bytes=1 << 40) == want
        assert glr_fwd(lib, B=1, T=1, D=D) == want
        assert glr_bwd(lib, B=1, T=1, D=D) == want
        assert glr_step(lib, N=1, D=D) == want
        assert glr_fwd(lib, cu=at(9), B=D) == want
        assert glr_bwd(lib, cu=at(9), B=D) == want
        assert size(1, D, BF16, ctypes.byref(n)) == (
            OK if D == most else UNSUPPORTED)


def test_binding_refuses_sizes_that_c_would_cut_off():
    n = 2 ** 31 + 5
    for rows, D in ((n, 1), (1, n)):
        with pytest.raises(ValueError, match="2.31"):
            kla.layernorm_bwd_workspace_size(rows, D, torch.float32)


def test_binding_refuses_cpu_tensors():
    x, s = torch.zeros(1, 4, 16), torch.zeros(4, 16)
    for call in (lambda: kla.layernorm_fwd(x),
                 lambda: kla.layernorm_bwd(x, x, None, x[..., 0], x[..., 0]),
                 lambda: kla.glr_fwd(x, x), lambda: kla.glr_bwd(x, x, x),
                 lambda: kla.glr_step(s, s, s)):
        with pytest.raises(TypeError):
            call()
