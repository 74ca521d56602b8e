"""Gated linear recurrence (kla_glr_fwd / _bwd / _step) against the fp64
oracle.  Bounds per element: the running error bound of a 32-bit evaluation
(oracle.mixer.glr_fwd_bound, glr_bwd_bound), plus half a unit of the output's
type."""
import numpy as np
import pytest
import torch

from linear_attention_delta_gb300 import kla
from oracle import mixer
from oracle.mixer import U16, U32

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TYPES = [(F32, F32), (BF16, BF16), (BF16, F32), (F32, BF16)]


@pytest.fixture(scope="module", autouse=True)
def cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    kla.load_library()
    yield
    assert kla.device_status() == 0


def normal(shape, dtype, seed):
    r = np.random.default_rng(seed)
    return torch.from_numpy(
        r.standard_normal(shape).astype(np.float32)).cuda().to(dtype)


def gates(shape, dtype, seed, lo=1e-4, hi=3.0):
    """Log decays from almost none to almost all, mixed over channels and
    tokens."""
    r = np.random.default_rng(seed)
    rate = np.exp(r.uniform(np.log(lo), np.log(hi), shape[-1:]))
    g = -(rate * 2 * r.random(shape)).astype(np.float32)
    return torch.from_numpy(g).cuda().to(dtype)


def assert_within(name, got, ref, bound, dtype):
    got = mixer.f64(got)
    assert got.shape == ref.shape, name
    bound = bound + (U16 * 1.01 if dtype == BF16 else U32) * np.abs(ref)
    bad = ~(np.abs(got - ref) <= bound)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(
            f"{name}: {bad.sum()} of {bad.size} outside, first at {i}: got "
            f"{got[i]}, expected {ref[i]} +- {bound[i]}")


def offsets(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)


def check_fwd(x, la, h0=None, cu=None):
    o, hT = kla.glr_fwd(x, la, h0, None if cu is None else cu.cuda())
    ro, rh = mixer.glr_fwd(x, la, h0, cu)
    bo, bh = mixer.glr_fwd_bound(x, la, h0, cu)
    assert_within("o", o, ro, bo, x.dtype)
    assert_within("hT", hT, rh, bh, F32)
    assert o.dtype == x.dtype and hT.dtype == F32
    return o, hT


def check_bwd(o, la, do, dhT=None, h0=None, cu=None):
    g = kla.glr_bwd(o, la, do, dhT, h0, None if cu is None else cu.cuda())
    ref = mixer.glr_bwd(o, la, do, dhT, h0, cu)
    bound = mixer.glr_bwd_bound(o, la, do, dhT, h0, cu)
    for name, r, b, dt in zip(("x_grad", "log_alpha_grad", "h0_grad"), ref,
                              bound, (o.dtype, la.dtype, F32)):
        assert_within(name, g[name], r, b, dt)
        assert g[name].dtype == dt
    return g


SHAPES = [(1, 1, 1), (2, 1, 7), (1, 2, 64), (5, 3, 33), (3, 17, 130),
          (2, 128, 64), (2, 129, 256), (1, 1000, 33), (1, 5000, 8),
          (2, 257, 2048), (40, 65, 96), (1, 1025, 1001)]


@pytest.mark.parametrize("dtype,gtype", TYPES)
@pytest.mark.parametrize("B,T,D", SHAPES)
def test_sizes_and_types(B, T, D, dtype, gtype):
    seed = B * 1000 + T + D
    x, la = normal((B, T, D), dtype, seed), gates((B, T, D), gtype, seed + 1)
    h0, dhT = normal((B, D), F32, seed + 2), normal((B, D), F32, seed + 3)
    do = normal((B, T, D), dtype, seed + 4)
    check_fwd(x, la)
    o, _ = check_fwd(x, la, h0)
    check_bwd(o, la, do)
    check_bwd(o, la, do, dhT, h0)


LENGTHS = [[5], [0], [0, 0], [0, 1, 0], [1] * 40, [3, 0, 0, 130, 1, 0],
           [0, 0, 127, 1, 128, 129, 2], [300, 1, 0, 511, 64, 64, 64, 1, 1],
           [0, 2000, 0, 0, 1, 700, 0], [16] * 30 + [15, 17, 1]]


@pytest.mark.parametrize("dtype,gtype", TYPES)
@pytest.mark.parametrize("k", range(len(LENGTHS)))
def test_packed(k, dtype, gtype):
    lens = LENGTHS[k]
    cu, T, N = offsets(lens), sum(lens), len(lens)
    for D in (1, 64, 131):
        seed = 100 * k + D
        x, la = normal((T, D), dtype, seed), gates((T, D), gtype, seed + 1)
        h0, dhT = normal((N, D), F32, seed + 2), normal((N, D), F32, seed + 3)
        do = normal((T, D), dtype, seed + 4)
        check_fwd(x, la, None, cu)
        o, _ = check_fwd(x, la, h0, cu)
        check_bwd(o, la, do, None, None, cu)
        check_bwd(o, la, do, dhT, h0, cu)


def test_packed_many_empty_sequences():
    r = np.random.default_rng(0)
    lens = [int(v) if r.random() < 0.02 else 0
            for v in r.integers(1, 400, 3000)]
    cu, T = offsets(lens), sum(lens)
    x, la = normal((T, 70), BF16, 1), gates((T, 70), F32, 2)
    h0 = normal((3000, 70), F32, 3)
    o, _ = check_fwd(x, la, h0, cu)
    check_bwd(o, la, x, h0, h0, cu)


@pytest.mark.parametrize("dtype,gtype", TYPES)
def test_strided_views(dtype, gtype):
    """Slices of wider tensors (odd offsets among them), sequences and tokens
    in swapped order, a gate repeated over the batch."""
    B, T, D = 3, 150, 96
    wide, wide_a = normal((B, T, 2 * D + 1), dtype, 5), \
        gates((B, T, 2 * D + 1), gtype, 6)
    h0 = normal((B, D), F32, 7)
    for off in (0, 1, 2, D):
        x, la = wide[..., off:off + D], wide_a[..., off:off + D]
        o, _ = check_fwd(x, la, h0)
        check_bwd(x, la, wide[..., D:2 * D], h0, h0)
    x, la = (v[..., :D].transpose(0, 1).contiguous().transpose(0, 1)
             for v in (wide, wide_a))
    assert not x.is_contiguous()
    check_fwd(x, la, h0)
    check_bwd(x, la, x, h0, h0)
    la = wide_a[:1, :, :D].expand(B, T, D)
    check_fwd(x, la, h0)
    check_bwd(x, la, x, h0, h0)
    la = wide_a[:, :1, :D].expand(B, T, D)       # one gate for all tokens
    check_fwd(x, la, h0)
    cut = wide[:, 5:, :D], wide_a[:, 5:, :D]
    check_fwd(*cut, h0)
    cu = offsets([40, 0, 110])
    check_fwd(wide[0, :, 3:3 + D], wide_a[0, :, 3:3 + D], h0, cu)


@pytest.mark.parametrize("dtype,gtype", TYPES)
@pytest.mark.parametrize("width", [129, 133, 200])
def test_one_token_of_a_strided_view(width, dtype, gtype):
    """One token a sequence, cut out of rows of odd width: the distance
    between tokens, which no step is taken with, says nothing about how the
    token lines up."""
    for B, T in ((1, 4), (2, 2), (2, 3)):
        wide = normal((B, T, width), dtype, 5)
        wide_a = gates((B, T, width), gtype, 6)
        for D, at in ((64, 0), (66, 0), (64, 2), (66, 1), (34, 4), (63, 1)):
            h0, dhT = normal((B, D), F32, 7), normal((B, D), F32, 8)
            x, la = (v[:, 1:2, at:at + D] for v in (wide, wide_a))
            dx, da = x.contiguous().clone(), la.contiguous().clone()
            for v, g in ((x, la), (x, da), (dx, la)):
                o, _ = check_fwd(v, g, h0)
                check_bwd(v, g, dx, dhT, h0)
                check_bwd(o, g, x, dhT, h0)
            # the same tokens packed: one token in all
            cu = offsets([0, 1])
            h0, dhT = normal((2, D), F32, 9), normal((2, D), F32, 10)
            for v, g in ((x[0], la[0]), (x[0], da[0]), (dx[0], la[0])):
                o, _ = check_fwd(v, g, h0, cu)
                check_bwd(v, g, dx[0], dhT, h0, cu)
                check_bwd(o, g, x[0], dhT, h0, cu)


@pytest.mark.parametrize("T", [5, 128, 700])
def test_extreme_gates(T):
    D = 64
    x, h0 = normal((2, T, D), F32, 8), normal((2, D), F32, 9)
    la = gates((2, T, D), F32, 10)
    la[:, ::7] = -float("inf")                   # forget
    la[:, 3::11] = torch.finfo(F32).min
    la[:, 1::5] = 0.0                            # keep everything
    la[:, 2::13] = -1e-30
    o, hT = check_fwd(x, la, h0)
    check_bwd(o, la, x, h0, h0)
    check_fwd(x, torch.zeros_like(la), h0)
    check_fwd(x, torch.full_like(la, 1e-3), h0)   # growth
    check_fwd(x, torch.full_like(la, -100.0), h0)


def test_growth_past_the_range_starts_from_zero():
    """exp(log_alpha) whose product over many tokens overflows, on a state
    that stays zero: 0, not 0 * inf."""
    x = torch.zeros(1, 600, 64, device="cuda")
    la = torch.ones_like(x)
    o, hT = kla.glr_fwd(x, la)
    assert (o == 0).all() and (hT == 0).all()
    g = kla.glr_bwd(x, la, x)
    assert (g["x_grad"] == 0).all() and (g["log_alpha_grad"] == 0).all()


def check_growth(x, la, h0, do=None, dhT=None, cu=None):
    """Forward (and backward, with do) where decays above 1 have products
    past the range of fp32 and states stay inside it.  A decay's error is
    that of l log2 e, two roundings of its size, besides the 8 units of the
    other bounds; the smallest numbers are rounded to 2^-149, bf16's to
    2^-133."""
    small = {F32: 0.0, BF16: 2.0 ** -134}
    dcu, f = None if cu is None else cu.cuda(), mixer.f64
    k = (8 + 2 * np.abs(np.maximum(f(la), -88.0))) * U32
    ab = lambda v: None if v is None else np.abs(f(v))  # noqa: E731
    o, hT = kla.glr_fwd(x, la, h0, dcu)
    mag, _ = mixer.glr_fwd(ab(x), la, ab(h0), cu)
    bo, bh = mixer.glr_fwd(k * mag + 1e-44, la, None, cu)
    ro, rh = mixer.glr_fwd(x, la, h0, cu)
    assert np.abs(ro).max() < 3e38
    assert_within("o", o, ro, bo + small[x.dtype], x.dtype)
    assert_within("hT", hT, rh, bh, F32)
    if do is None:
        return
    g = kla.glr_bwd(o, la, do, dhT, h0, dcu)
    ref = mixer.glr_bwd(o, la, do, dhT, h0, cu)
    mag, da, d0 = mixer.glr_bwd(ab(o), la, ab(do), ab(dhT), ab(h0), cu)
    e, ea, e0 = mixer.glr_bwd(ab(o), la, k * mag + 1e-44, None, ab(h0), cu)
    for name, r, b, dt in zip(
            ("x_grad", "log_alpha_grad", "h0_grad"), ref,
            (e, ea + k * da + 1e-44, e0 + k.max() * d0),
            (o.dtype, la.dtype, F32)):
        assert np.abs(r).max() < 3e38
        assert_within(name, g[name], r, b + small[dt], dt)


@pytest.mark.parametrize("dtype,gtype", TYPES)
@pytest.mark.parametrize("B,T,D", [(2, 150, 64), (1, 1000, 66), (2, 700, 33),
                                   (1, 9000, 128), (300, 160, 96)])
def test_growth_of_a_small_state(B, T, D, dtype, gtype):
    """Up by some e^150 and down again: the product of a tile's decays
    overflows, the state does not."""
    r = np.random.default_rng(66)
    up = np.where(np.arange(T) // 150 % 2 == 0, 1.0, -1.0)
    la = torch.from_numpy((up[:, None] * r.uniform(0.8, 1.1, D)).astype(
        np.float32)).cuda().to(gtype).expand(B, T, D).contiguous()
    x, do = normal((B, T, D), dtype, 67) * 1e-36, \
        normal((B, T, D), dtype, 68) * 1e-36
    h0, dhT = normal((B, D), F32, 69) * 1e-36, normal((B, D), F32, 70) * 1e-36
    check_growth(x, la, h0, do, dhT)
    check_growth(torch.zeros_like(x), la, h0, torch.zeros_like(x), dhT)
    if B == 1:                           # sequences that begin on the way up
        cu = offsets([T // 3, 0, 1, T - T // 3 - 41, 40])
        h0, dhT = normal((5, D), F32, 71) * 1e-36, \
            normal((5, D), F32, 72) * 1e-36
        check_growth(x[0], la[0], h0, do[0], dhT, cu)


@pytest.mark.parametrize("dtype,gtype", TYPES)
@pytest.mark.parametrize("D", [64, 33])
def test_growth_in_few_tokens(D, dtype, gtype):
    T = 400
    la = torch.zeros(1, T, D, device="cuda", dtype=gtype)
    la[:, 5:9], la[:, 30:34] = 40.0, -40.0       # within a warp's tokens
    la[:, 90:94], la[:, 310:314] = 42.0, -42.0   # and tiles apart
    la[:, 200::50] += 0.5
    h0, dhT = normal((1, D), F32, 73) * 1e-37, normal((1, D), F32, 74) * 1e-37
    x = normal((1, T, D), dtype, 75) * 1e-38
    check_growth(x, la, h0, torch.zeros_like(x), dhT)
    # growth that is then forgotten, in one warp's tokens and in two tiles'
    la = torch.zeros(1, T, D, device="cuda", dtype=gtype)
    la[:, 2:14] = la[:, 60:200:12] = 10.0
    la[:, 16] = la[:, 250] = -float("inf")
    x = normal((1, T, D), dtype, 76)
    x[:, :251] = 0.0
    x[:, 17] = 1e-37
    check_growth(x, la, h0)


def test_growth_past_the_range_is_infinite():
    x = torch.zeros(2, 500, 64, device="cuda")
    la = torch.ones_like(x)
    o, hT = kla.glr_fwd(x, la, torch.ones(2, 64, device="cuda"))
    ref = np.exp(np.arange(1, 501.0))
    assert (o[:, ref > 4e38] == float("inf")).all() and hT.isinf().all()
    assert o[:, ref < 3e38].isfinite().all()


@pytest.mark.parametrize("dtype,gtype", TYPES)
def test_bad_sequences_stay_their_own(dtype, gtype):
    """NaN and infinities of one packed sequence, in x, in the gates or in
    its initial state, reach no other sequence."""
    lens = [100, 33, 0, 260, 1, 90]
    cu, T, D = offsets(lens), sum(lens), 66
    x, la = normal((T, D), dtype, 11), gates((T, D), gtype, 12)
    h0, do = normal((6, D), F32, 13), normal((T, D), dtype, 14)
    o, hT = kla.glr_fwd(x, la, h0, cu.cuda())
    g = kla.glr_bwd(o, la, do, h0, h0, cu.cuda())
    x2, la2, h2, do2, o2 = x.clone(), la.clone(), h0.clone(), do.clone(), \
        o.clone()
    x2[40] = float("nan")                        # sequence 0
    x2[150, ::2] = float("inf")                  # sequence 3
    do2[60], do2[300] = float("inf"), float("nan")
    o2[99] = float("nan")
    h2[1] = float("inf")
    la2[110] = float("nan")                      # sequence 1
    oo, hh = kla.glr_fwd(x2, la2, h2, cu.cuda())
    gg = kla.glr_bwd(o2, la2, do2, h2, h2, cu.cuda())
    for n in (2, 4, 5):
        q = slice(int(cu[n]), int(cu[n + 1]))
        assert torch.equal(oo[q], o[q]) and torch.equal(hh[n], hT[n])
        assert torch.equal(gg["x_grad"][q], g["x_grad"][q])
        assert torch.equal(gg["log_alpha_grad"][q], g["log_alpha_grad"][q])
        assert torch.equal(gg["h0_grad"][n], g["h0_grad"][n])
    assert oo[40:100].isnan().all()


def test_bad_offsets_stay_inside():
    """Offsets that run backwards or past the tokens: whatever the result,
    every access stays inside the tensors (the guard rows keep their value)
    and the call returns."""
    T, D = 300, 64
    buf = torch.full((T + 512, D), 3.0, device="cuda")
    o = buf[256:256 + T]
    x, la = normal((T, D), F32, 15), gates((T, D), F32, 16)
    for cu in ([0, 500, 20, 300], [5, 2, 1, 0], [-7, 90, 10 ** 9, 300],
               [300, 300, 300, 300], [0, 0, 0, 0], [200, 300, 400, 500]):
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        kla.glr_fwd(x, la, normal((3, D), F32, 17), c, o=o)
        kla.glr_bwd(x, la, x, normal((3, D), F32, 17), None, c)
        assert (buf[:256] == 3).all() and (buf[256 + T:] == 3).all()
    assert kla.device_status() == 0


def test_zero_tokens_and_zero_sequences():
    h0 = normal((3, 50), F32, 18)
    x = torch.empty(3, 0, 50, device="cuda")
    o, hT = kla.glr_fwd(x, x, h0)
    assert o.shape == x.shape and torch.equal(hT, h0)
    assert (kla.glr_fwd(x, x)[1] == 0).all()
    assert torch.equal(kla.glr_bwd(x, x, x, h0)["h0_grad"], h0)
    e = torch.empty(0, 7, 50, device="cuda")
    o, hT = kla.glr_fwd(e, e)
    assert o.shape == e.shape and hT.shape == (0, 50)


def test_state_in_place_and_carried_over():
    """hT written over h0; a sequence in two calls equals one call within
    rounding; tokens one by one through glr_step equal the scan."""
    B, T, D = 3, 200, 320
    x, la = normal((B, T, D), BF16, 19), gates((B, T, D), F32, 20)
    h0 = normal((B, D), F32, 21)
    o, hT = check_fwd(x, la, h0)
    s = h0.clone()
    o2, s2 = kla.glr_fwd(x, la, s, hT=s)
    assert s2 is s and torch.equal(s, hT) and torch.equal(o2, o)
    _, mid = kla.glr_fwd(x[:, :77], la[:, :77], h0)
    _, end = kla.glr_fwd(x[:, 77:], la[:, 77:], mid)
    ref, bound = mixer.glr_fwd(x, la, h0)[1], \
        mixer.glr_fwd_bound(x, la, h0)[1]
    assert_within("hT in two calls", end, ref, bound, F32)
    S = h0.clone()
    out = torch.stack([kla.glr_step(x[:, t], la[:, t], S) for t in range(T)],
                      1)
    ro, bo = mixer.glr_fwd(x, la, h0)[0], mixer.glr_fwd_bound(x, la, h0)[0]
    assert_within("steps", out, ro, bo, BF16)
    assert_within("S", S, ref, bound, F32)
    cu = offsets([150, 0, 50])
    p, pa = x[0], la[0]
    ref = kla.glr_fwd(p, pa, h0, cu.cuda())
    s = h0.clone()
    got = kla.glr_fwd(p, pa, s, cu.cuda(), hT=s)
    assert torch.equal(got[0], ref[0]) and torch.equal(s, ref[1])


@pytest.mark.parametrize("dtype,gtype", TYPES)
@pytest.mark.parametrize("N,D", [(1, 1), (1, 2048), (7, 33), (300, 130),
                                 (256, 2048), (70000, 3)])
def test_step(N, D, dtype, gtype):
    x, la = normal((N, D + 5), dtype, 22), gates((N, D + 5), gtype, 23)
    for off in (0, 3):
        xs, as_ = x[:, off:off + D], la[:, off:off + D]
        if off == 0:
            xs, as_ = xs.contiguous(), as_.contiguous()
        S = normal((N, D), F32, 24)
        a, s0 = np.exp(mixer.f64(as_)), mixer.f64(S)
        ref = a * s0 + mixer.f64(xs)
        bound = 8 * U32 * (np.abs(a * s0) + np.abs(ref)) + 1e-30
        o = kla.glr_step(xs, as_, S)
        assert_within("S", S, ref, bound, F32)
        assert_within("o", o, ref, bound, dtype)


@pytest.mark.parametrize("packed", [False, True])
def test_gradients_are_the_differences(packed):
    """fp32 gradients against central differences of the fp64 forward."""
    r = np.random.default_rng(25)
    lens = [60, 0, 1, 199] if packed else None
    cu = offsets(lens) if packed else None
    shape, N = ((260, 5), 4) if packed else ((2, 130, 5), 2)
    x, la = normal(shape, F32, 26), gates(shape, F32, 27, 1e-2)
    h0, dhT = normal((N, 5), F32, 28), normal((N, 5), F32, 29)
    do = normal(shape, F32, 30)
    dcu = cu.cuda() if packed else None
    o, _ = kla.glr_fwd(x, la, h0, dcu)
    g = kla.glr_bwd(o, la, do, dhT, h0, dcu)
    args = [mixer.f64(v) for v in (x, la, h0)]
    fdo, fdh = mixer.f64(do), mixer.f64(dhT)

    def loss(x, la, h0):
        o, hT = mixer.glr_fwd(x, la, h0, cu)
        return (o * fdo).sum() + (hT * fdh).sum()

    for k, name in enumerate(("x_grad", "log_alpha_grad", "h0_grad")):
        got = mixer.f64(g[name])
        v, h = r.standard_normal(got.shape), 1e-6
        up, dn = list(args), list(args)
        up[k], dn[k] = args[k] + h * v, args[k] - h * v
        slope = (loss(*up) - loss(*dn)) / (2 * h)
        # fp32: some 1e-6 of the terms; the differences: 1e-9
        assert abs((got * v).sum() - slope) <= 1e-5 * (
            np.abs(got * v).sum() + 1), name


@pytest.mark.parametrize("B,T,D", [(1, 20000, 64), (2, 4096, 512)])
def test_same_bits_every_call_and_on_another_stream(B, T, D):
    x, la = normal((B, T, D), BF16, 31), gates((B, T, D), F32, 32)
    h0, do = normal((B, D), F32, 33), normal((B, T, D), BF16, 34)
    o, hT = kla.glr_fwd(x, la, h0)
    g = kla.glr_bwd(o, la, do, h0, h0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i in range(10):
        s = side if i % 2 else None
        o2, h2 = kla.glr_fwd(x, la, h0, stream=s)
        g2 = kla.glr_bwd(o, la, do, h0, h0, stream=s)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(o, o2) and torch.equal(hT, h2)
        assert all(torch.equal(g[k], g2[k]) for k in g)


def test_long_sequence_with_long_memory():
    """65536 tokens, decays down to 1e-4 a token."""
    x, la = normal((1, 65536, 16), F32, 35), gates((1, 65536, 16), F32, 36)
    o, _ = check_fwd(x, la, normal((1, 16), F32, 37))
    check_bwd(o, la, x)


@pytest.mark.parametrize("dtype,gtype", TYPES)
@pytest.mark.parametrize("D", [64, 66, 131, 1024])
def test_few_channels_and_many_tokens(D, dtype, gtype):
    """Few channels for the whole GPU: many blocks share a run of tokens."""
    T = 20000
    x, la = normal((1, T, D), dtype, 48), gates((1, T, D), gtype, 49)
    h0 = normal((1, D), F32, 50)
    o, _ = check_fwd(x, la, h0)
    check_bwd(o, la, x, h0, h0)


def uneven_lengths(kind):
    r = np.random.default_rng(54)
    if kind == "random":
        return [int(v) for v in r.integers(0, 700, 40)]
    if kind == "one long":               # most parts of the tokens are empty
        return [0, 0, 9000] + [1, 0] * 20 + [3]
    if kind == "long last":
        return [1, 0] * 20 + [9000]
    return [0, 411, 0, 0] * 30 + [0]     # empty ones at every boundary


@pytest.mark.parametrize("dtype,gtype", TYPES)
@pytest.mark.parametrize("D", [64, 66, 1001])
@pytest.mark.parametrize("kind", ["random", "one long", "long last",
                                  "empty between"])
def test_packed_tokens_in_parts(kind, D, dtype, gtype):
    """Many tokens of few channels: the sequences are shared out among more
    blocks than could share one."""
    lens = uneven_lengths(kind)
    cu, T, N = offsets(lens), sum(lens), len(lens)
    x, la = normal((T, D), dtype, 55), gates((T, D), gtype, 56)
    h0, dhT = normal((N, D), F32, 57), normal((N, D), F32, 58)
    o, hT = check_fwd(x, la, h0, cu)
    g = check_bwd(o, la, x, dhT, h0, cu)
    s = h0.clone()
    o2, _ = kla.glr_fwd(x, la, s, cu.cuda(), hT=s)
    n = torch.tensor(lens).cuda() > 0            # an empty one keeps its state
    assert torch.equal(s[n], hT[n]) and torch.equal(s[~n], h0[~n])
    assert torch.equal(o2, o)
    x[int(cu[N // 2]):int(cu[N // 2 + 1])] = float("nan")
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[int(cu[N // 2]):int(cu[N // 2 + 1])] = True
    o2, _ = kla.glr_fwd(x, la, h0, cu.cuda())
    assert torch.equal(o2[~bad], o[~bad]) and o2[bad].isnan().all()


@pytest.mark.parametrize("dtype,gtype", TYPES)
@pytest.mark.parametrize("D", [64, 66, 1001])
@pytest.mark.parametrize("kind", ["random", "one long", "long last",
                                  "empty between"])
def test_bad_sequences_of_tokens_in_parts(kind, D, dtype, gtype):
    """Every second sequence that holds tokens (then the others) is NaN in all
    that it has: its neighbours, on both sides of every cut, keep their bits,
    forward and backward."""
    lens = uneven_lengths(kind)
    cu, T, N = offsets(lens), sum(lens), len(lens)
    x, la = normal((T, D), dtype, 77), gates((T, D), gtype, 78)
    do = normal((T, D), dtype, 79)
    h0, dhT = normal((N, D), F32, 80), normal((N, D), F32, 81)
    dcu, nan = cu.cuda(), float("nan")
    o, hT = kla.glr_fwd(x, la, h0, dcu)
    g = kla.glr_bwd(o, la, do, dhT, h0, dcu)
    held = [n for n in range(N) if lens[n]]
    for first in (0, 1):
        seqs = torch.zeros(N, dtype=torch.bool)
        seqs[held[first::2]] = True
        rows = seqs.repeat_interleave(torch.tensor(lens)).cuda()
        seqs = seqs.cuda()
        assert rows.any() and not rows.all()
        x2, la2, do2, o2, h2, d2 = (v.clone() for v in (x, la, do, o, h0,
                                                        dhT))
        for v in (x2, do2, o2):
            v[rows] = nan
        h2[seqs], d2[seqs] = nan, nan
        for gate in (la, la2):
            oo, hh = kla.glr_fwd(x2, gate, h2, dcu)
            gg = kla.glr_bwd(o2, gate, do2, d2, h2, dcu)
            assert torch.equal(oo[~rows], o[~rows])
            assert torch.equal(hh[~seqs], hT[~seqs])
            for name in ("x_grad", "log_alpha_grad"):
                assert torch.equal(gg[name][~rows], g[name][~rows]), name
                assert gg[name][rows].isnan().all(), name
            assert torch.equal(gg["h0_grad"][~seqs], g["h0_grad"][~seqs])
            assert oo[rows].isnan().all() and hh[seqs].isnan().all()
            la2[rows] = nan


@pytest.mark.parametrize("dtype,gtype", TYPES)
@pytest.mark.parametrize("D", [64, 70, 131])
def test_many_sequences_of_a_token_beside_a_long_one(D, dtype, gtype):
    """Single tokens of many sequences and a prompt in one call, states in
    place."""
    lens = [1] * 200 + [0, 2, 0, 0, 3] * 10 + [500] + [1, 0] * 30
    cu, T, N = offsets(lens), sum(lens), len(lens)
    x, la = normal((T, D), dtype, 63), gates((T, D), gtype, 64)
    h0 = normal((N, D), F32, 65)
    o, hT = check_fwd(x, la, h0, cu)
    check_bwd(o, la, x, h0, h0, cu)
    s = h0.clone()
    o2, _ = kla.glr_fwd(x, la, s, cu.cuda(), hT=s)
    assert torch.equal(s, hT) and torch.equal(o2, o)


def test_bad_offsets_of_many_tokens_stay_inside():
    T, D, N = 9000, 64, 30
    buf = torch.full((T + 512, D), 3.0, device="cuda")
    o = buf[256:256 + T]
    x, la = normal((T, D), F32, 59), gates((T, D), F32, 60)
    h = normal((N, D), F32, 61)
    r = np.random.default_rng(62)
    for cu in (r.integers(-100, 20000, N + 1), np.arange(N, -1, -1) * 300,
               np.full(N + 1, T), np.zeros(N + 1), np.full(N + 1, -5)):
        c = torch.tensor(cu.astype(np.int32), device="cuda")
        kla.glr_fwd(x, la, h, c, o=o)
        kla.glr_bwd(x, la, x, h, None, c)
        assert (buf[:256] == 3).all() and (buf[256 + T:] == 3).all()
    assert kla.device_status() == 0


@pytest.mark.parametrize("B,T,D", [(500, 70, 64), (30, 130, 2048),
                                   (700, 66, 70)])
def test_more_channels_than_blocks(B, T, D):
    x, la = normal((B, T, D), BF16, 51), gates((B, T, D), F32, 52)
    h0 = normal((B, D), F32, 53)
    o, _ = check_fwd(x, la, h0)
    check_bwd(o, la, x, h0, h0)


def test_a_wait_that_runs_out_is_reported_then_cleared():
    """A block whose team's maps never come gives up, reports it once, and the
    context and the next calls are as before."""
    assert kla.device_status() == 0
    assert kla.selftest_glr_timeout() == 0
    assert kla.device_status() == -4
    assert kla.device_status() == 0
    x, la = normal((1, 300, 64), F32, 60), gates((1, 300, 64), F32, 61)
    check_fwd(x, la)


def test_two_streams_at_once():
    """Calls that overlap on two streams, each with its own workspace."""
    x, la = normal((1, 30000, 256), BF16, 38), gates((1, 30000, 256), F32, 39)
    ref, _ = kla.glr_fwd(x, la)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [kla.glr_fwd(x, la, stream=streams[i % 2])[0] for i in range(12)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)


def test_graph_replay_equals_eager():
    x, la = normal((2, 3000, 128), BF16, 40), gates((2, 3000, 128), F32, 41)
    S0 = normal((2, 128), F32, 42)
    ref, hT = kla.glr_fwd(x, la, S0)
    gref = kla.glr_bwd(ref, la, x, S0, S0)
    S = S0.clone()
    sref = kla.glr_step(x[:, 0], la[:, 0], S)
    S.copy_(S0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, h = kla.glr_fwd(x, la, S0)
        g = kla.glr_bwd(o, la, x, S0, S0)
        so = kla.glr_step(x[:, 0], la[:, 0], S)
    for _ in range(3):
        S.copy_(S0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, ref) and torch.equal(h, hT)
        assert all(torch.equal(g[k], gref[k]) for k in g)
        assert torch.equal(so, sref)


def test_offsets_past_32_bits():
    T, D = 1100000, 2048               # 2.25e9 elements
    x = torch.zeros(T, D, dtype=BF16, device="cuda")
    la = torch.zeros(T, D, dtype=BF16, device="cuda")
    x[0] = 1.0                         # carried unchanged to the last block
    x[-300:], la[-300:] = normal((300, D), BF16, 43), gates((300, D), BF16,
                                                            44)
    o, hT = kla.glr_fwd(x[None], la[None])
    one = torch.ones(1, D, device="cuda")
    ro, rh = mixer.glr_fwd(x[None, -300:], la[None, -300:], one)
    bo, bh = mixer.glr_fwd_bound(x[None, -300:], la[None, -300:], one)
    assert (o[0, 1000000] == 1).all()
    assert_within("o", o[:, -300:], ro, bo, BF16)
    assert_within("hT", hT, rh, bh, F32)
    g = kla.glr_bwd(o, la[None], x[None])
    ref = mixer.glr_bwd(o[None, 0, -300:], la[None, -300:], x[None, -300:],
                        None, one)
    b = mixer.glr_bwd_bound(o[None, 0, -300:], la[None, -300:],
                            x[None, -300:], None, one)
    assert_within("x_grad", g["x_grad"][:, -300:], ref[0], b[0], BF16)
    assert_within("log_alpha_grad", g["log_alpha_grad"][:, -300:], ref[1],
                  b[1], BF16)


def test_refuses_more_than_it_counts():
    one, n = torch.zeros(1, 1, 1, device="cuda", dtype=BF16), 2 ** 31 + 5
    for x in (one.expand(n, 1, 1), one.expand(1, n, 1)):
        for call in (lambda: kla.glr_fwd(x, x), lambda: kla.glr_bwd(x, x, x)):
            with pytest.raises(ValueError, match="2.31"):
                call()
    x = one[0].expand(n, 1)
    cu = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="2.31"):
        kla.glr_fwd(x, x, cu_seqlens=cu)
    with pytest.raises(ValueError, match="2.31"):
        kla.glr_step(x, x, one[0].float().expand(n, 1))


def test_refusals():
    x, la = normal((2, 9, 64), BF16, 45), gates((2, 9, 64), F32, 46)
    h0 = normal((2, 64), F32, 47)
    o, _ = kla.glr_fwd(x, la, h0)
    cu = torch.tensor([0, 9], dtype=torch.int32, device="cuda")
    for bad in (lambda: kla.glr_fwd(x.half(), la),
                lambda: kla.glr_fwd(x, la.double()),
                lambda: kla.glr_fwd(x, la, h0.bfloat16()),
                lambda: kla.glr_fwd(x.cpu(), la),
                lambda: kla.glr_fwd(x[0], la[0], None, cu.long()),
                lambda: kla.glr_bwd(o, la, o.float()),
                lambda: kla.glr_step(x[:, 0], la[:, 0], h0.bfloat16())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: kla.glr_fwd(x[0], la[0]),
                lambda: kla.glr_fwd(x, la, None, cu),
                lambda: kla.glr_fwd(x, la[:, :8]),
                lambda: kla.glr_fwd(x, la, h0[:1]),
                lambda: kla.glr_fwd(x.transpose(1, 2), la.transpose(1, 2)),
                lambda: kla.glr_fwd(x, la, hT=h0.t()),
                lambda: kla.glr_bwd(o, la, o[:1]),
                lambda: kla.glr_step(x, la, h0)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(kla.KlaError):
        kla.glr_fwd(x, la, h0, o=x)              # over its own input
    empty = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(kla.KlaError):            # tokens of no sequence
        kla.glr_fwd(x[0], la[0], None, empty)
    f = torch.zeros(4, 8, device="cuda")
    with pytest.raises(kla.KlaError):
        kla.glr_step(f, f, f)
