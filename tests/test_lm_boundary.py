"""Host-side checks of the linear-attention and log-probability entry points:
bad arguments are refused before any launch (no GPU needed)."""
import ctypes

import pytest
import torch

from linear_attention_delta_gb300 import kla

INVALID, UNSUPPORTED, OK = -1, -2, 0
F32, BF16 = 0, 1
LIMIT = 0x7fffffff - 4096


@pytest.fixture(scope="module")
def lib():
    return kla.load_library()


def at(i):
    return ctypes.c_void_p(0x10000000 * i)


def odd(i, n=1):
    return ctypes.c_void_p(0x10000000 * i + n)


def heads(**kw):
    """Strides of a contiguous [2, 10, 3, 64]."""
    out = {}
    for n, p in kw.items():
        out.update({n: p, n + "b": 1920, n + "t": 192, n + "h": 64})
    return out


def call(fn, a, kw):
    assert set(kw) <= set(a), kw
    a.update(kw)
    return fn(*a.values(), None)


def la_fwd(lib, **kw):
    return call(lib.kla_linattn_fwd, dict(
        **heads(q=at(1), k=at(2), v=at(3)), la=at(4), h0=at(5), o=at(6),
        hT=at(7), B=2, T=10, H=3, dk=64, dv=64, dtype=BF16, ws=at(15),
        ws_bytes=1 << 30), kw)


def la_bwd(lib, **kw):
    return call(lib.kla_linattn_bwd, dict(
        **heads(q=at(1), k=at(2), v=at(3)), la=at(4), h0=at(5),
        **heads(g=at(6)), dhT=at(7), dq=at(8), dk_=at(9), dv_=at(10),
        dh0=at(11), B=2, T=10, H=3, dk=64, dv=64, dtype=BF16, ws=at(15),
        ws_bytes=1 << 30), kw)


def la_step(lib, **kw):
    return call(lib.kla_linattn_step, dict(
        q=at(1), qn=192, qh=64, k=at(2), kn=192, kh=64, v=at(3), vn=192,
        vh=64, la=at(4), S=at(5), o=at(6), N=2, H=3, dk=64, dv=64,
        dtype=BF16), kw)


def lp_fwd(lib, **kw):
    return call(lib.kla_logprob_fwd, dict(
        x=at(1), stride=100, tokens=at(2), scale=1.0, logp=at(3), ent=at(4),
        lse=at(5), top_logp=at(6), top_ids=at(7), N=4, V=100, top=5,
        dtype=BF16), kw)


def lp_bwd(lib, **kw):
    return call(lib.kla_logprob_bwd, dict(
        x=at(1), stride=100, tokens=at(2), scale=1.0, lse=at(3), ent=at(4),
        g=at(5), ge=at(6), dx=at(7), N=4, V=100, dtype=BF16), kw)


SIZES = [dict(B=-1), dict(T=-1), dict(H=-1), dict(dk=0), dict(dv=0),
         dict(dtype=2), dict(qb=-1), dict(qt=-1), dict(kh=-1), dict(vb=-2),
         dict(q=None), dict(k=None), dict(v=None), dict(la=None),
         dict(q=odd(1)), dict(la=odd(4, 2)), dict(h0=odd(5, 2))]


@pytest.mark.parametrize("bad", SIZES + [
    dict(o=None), dict(o=odd(6)), dict(hT=odd(7, 2)), dict(o=at(1)),
    dict(o=at(3)), dict(hT=at(2)), dict(hT=at(6)), dict(hT=at(4)),
    dict(hT=odd(5, 16)), dict(o=at(5)),
    # the last token of a strided k reaches into o
    dict(k=ctypes.c_void_p(0x60000000 - 9 * 2 * 4096), kt=4096),
    # 16 heads of 65536 tokens need a workspace
    dict(T=65536, ws=None), dict(T=65536, ws_bytes=64),
    dict(T=65536, ws=odd(15, 8)), dict(T=65536, ws=at(5)),
])
def test_linattn_fwd_refuses(lib, bad):
    assert la_fwd(lib, **bad) == INVALID


@pytest.mark.parametrize("bad", SIZES + [
    dict(g=None), dict(gt=-1), dict(dq=None), dict(dk_=None), dict(dv_=None),
    dict(dhT=odd(7, 1)), dict(dh0=odd(11, 2)), dict(dq=at(1)),
    dict(dk_=at(8)), dict(dv_=at(6)), dict(dh0=at(5)), dict(dh0=at(7)),
    dict(dq=at(4)), dict(T=65536, ws=None), dict(T=65536, ws_bytes=64),
    dict(T=65536, ws=odd(15, 8)), dict(T=65536, ws=at(8)),
])
def test_linattn_bwd_refuses(lib, bad):
    assert la_bwd(lib, **bad) == INVALID


@pytest.mark.parametrize("bad", [
    dict(N=-1), dict(H=-1), dict(dk=0), dict(dv=0), dict(dtype=3),
    dict(qn=-1), dict(kh=-1), dict(vn=-1), dict(q=None), dict(k=None),
    dict(v=None), dict(la=None), dict(S=None), dict(o=None), dict(o=at(5)),
    dict(o=at(1)), dict(S=at(2)), dict(S=odd(5, 2)), dict(v=odd(3)),
    dict(S=at(4)),
])
def test_linattn_step_refuses(lib, bad):
    assert la_step(lib, **bad) == INVALID


def test_linattn_refuses_what_it_has_no_kernel_for(lib):
    for bad in (dict(dk=257), dict(dv=257), dict(H=1 << 24)):
        for f in (la_fwd, la_bwd, la_step):
            assert f(lib, **bad) == UNSUPPORTED
    for f in (la_fwd, la_bwd):
        assert f(lib, T=LIMIT + 1) == UNSUPPORTED
    n = ctypes.c_size_t(0)
    f = lib.kla_linattn_workspace_size
    assert f(1, LIMIT + 1, 1, 64, 64, BF16, 0, ctypes.byref(n)) == UNSUPPORTED
    assert f(1, 8, 1, 64, 257, BF16, 0, ctypes.byref(n)) == UNSUPPORTED
    for bad in ((-1, 8, 1, 64, 64, BF16), (1, 8, 1, 0, 64, BF16),
                (1, 8, 1, 64, 64, 2)):
        assert f(*bad, 0, ctypes.byref(n)) == INVALID
    assert f(1, 8, 1, 64, 64, BF16, 0, None) == INVALID


def test_linattn_workspace(lib):
    """Many or short sequences need none; long ones some, a state a part of
    each of the passes at most."""
    size = kla.linattn_workspace_size
    for back in (False, True):
        assert size(64, 4096, 16, 128, 128, torch.bfloat16, back) == 0
        assert size(1, 64, 1, 64, 64, torch.float32, back) == 0
        assert size(1, 128, 1, 64, 64, torch.bfloat16, back) <= 3 * 4 * 64 * 64 * 4
        n = size(1, 65536, 4, 128, 64, torch.bfloat16, back)
        assert 0 < n <= (3 if back else 1) * 64 * 4 * 128 * 64 * 4


@pytest.mark.parametrize("bad", [
    dict(N=-1), dict(V=0), dict(stride=-1), dict(top=-1), dict(top=101),
    dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(dtype=2), dict(x=None), dict(tokens=None),
    dict(logp=None), dict(top_logp=None), dict(top_ids=None),
    dict(x=odd(1)), dict(tokens=odd(2, 4)), dict(logp=odd(3, 2)),
    dict(ent=odd(4, 1)), dict(lse=odd(5, 2)), dict(top_logp=odd(6, 2)),
    dict(top_ids=odd(7, 4)), dict(logp=at(1)), dict(ent=at(3)),
    dict(lse=at(2)), dict(top_ids=at(6)), dict(top_logp=odd(1, 8)),
    dict(x=ctypes.c_void_p(0x30000000 - 3 * 2 * 1000), stride=1000),
])
def test_logprob_fwd_refuses(lib, bad):
    assert lp_fwd(lib, **bad) == INVALID


@pytest.mark.parametrize("bad", [
    dict(N=-1), dict(V=0), dict(stride=-1), dict(scale=0.0),
    dict(scale=float("nan")), dict(dtype=2), dict(x=None), dict(tokens=None),
    dict(lse=None), dict(dx=None), dict(ent=None), dict(lse=odd(3, 2)),
    dict(g=odd(5, 2)), dict(ge=odd(6, 1)), dict(dx=odd(7)),
    dict(dx=odd(1, 2)), dict(dx=at(1), stride=101), dict(dx=at(3)),
    dict(dx=at(2)), dict(dx=at(5)), dict(dx=at(4)),
])
def test_logprob_bwd_refuses(lib, bad):
    assert lp_bwd(lib, **bad) == INVALID


def test_logprob_refuses_what_it_has_no_kernel_for(lib):
    assert lp_fwd(lib, V=1000, top=129) == UNSUPPORTED
    assert lp_fwd(lib, N=1, V=LIMIT + 1) == UNSUPPORTED
    assert lp_bwd(lib, N=1, V=LIMIT + 1) == UNSUPPORTED


def test_empty_problems_are_no_ops(lib):
    none = dict(q=None, k=None, v=None, la=None, o=None)
    for n in ("B", "H"):
        assert la_fwd(lib, **none, **{n: 0}) == OK
        assert la_bwd(lib, q=None, k=None, v=None, la=None, g=None, dq=None,
                      dk_=None, dv_=None, **{n: 0}) == OK
    assert la_fwd(lib, **none, T=0, hT=at(5)) == OK      # hT is h0
    assert la_fwd(lib, **none, T=0, hT=None) == OK
    for n in ("N", "H"):
        assert la_step(lib, **none, S=None, **{n: 0}) == OK
    assert lp_fwd(lib, N=0, x=None, tokens=None, logp=None) == OK
    assert lp_bwd(lib, N=0, x=None, tokens=None, lse=None, dx=None) == OK


def test_binding_refuses_cpu_tensors():
    x, a = torch.zeros(1, 4, 2, 16), torch.zeros(2)
    y, t = torch.zeros(3, 8), torch.zeros(3, dtype=torch.int64)
    S = torch.zeros(4, 2, 16, 16)
    for f in (lambda: kla.linattn_fwd(x, x, x, a),
              lambda: kla.linattn_bwd(x, x, x, a, x),
              lambda: kla.linattn_step(x[0], x[0], x[0], a, S),
              lambda: kla.logprob_fwd(y, t),
              lambda: kla.logprob_bwd(y, t, y[:, 0])):
        with pytest.raises(TypeError):
            f()


def test_binding_refuses_sizes_that_c_would_cut_off():
    with pytest.raises(ValueError, match="2.31"):
        kla.linattn_workspace_size(1, 2 ** 31 + 5, 1, 64, 64, torch.float32)
