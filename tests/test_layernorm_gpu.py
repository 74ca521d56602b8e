"""Layer norm (kla_layernorm_fwd / _bwd) against the fp64 oracle.

Bounds per element, from the arithmetic: a sum of D terms is made of chains of
at most D / 32 additions and a tree, and rounding errors of a chain are at
most its length in units u = 2^-24 of the sum of magnitudes; K = 32 + D / 32
units cover it with the few roundings around it.  A bf16 result adds its own
rounding, at most 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

from linear_attention_delta_gb300 import kla
from oracle import mixer
from oracle.mixer import U16, U32

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    kla.load_library()
    yield
    assert kla.device_status() == 0


def normal(shape, dtype, seed, scale=1.0, shift=0.0):
    r = np.random.default_rng(seed)
    v = r.standard_normal(shape) * scale + shift
    return torch.from_numpy(v.astype(np.float32)).cuda().to(dtype)


def rounding(ref, dtype):
    """The output's own rounding, with the fp32 value's behind it."""
    return (U16 * 1.01 if dtype == BF16 else U32) * np.abs(ref)


def assert_within(name, got, ref, bound):
    got = mixer.f64(got)
    assert got.shape == ref.shape, name
    bad = ~(np.abs(got - ref) <= bound)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(
            f"{name}: {bad.sum()} of {bad.size} outside, first at {i}: got "
            f"{got[i]}, expected {ref[i]} +- {bound[i]}")


def check_fwd(x, w, b, eps=1e-5, residual=None, got=None):
    """The forward (or results that it gave already) against the oracle."""
    if got is None:
        got = kla.layernorm_fwd(x, w, b, eps=eps, residual=residual)
    y, s, mean, rstd = got
    ry, rs, rm, rr = mixer.ln_fwd(x, w, b, eps, residual)
    D = x.shape[-1]
    K = (32 + D / 32) * U32
    top = np.abs(rs).max(-1)
    aw = 1.0 if w is None else np.abs(mixer.f64(w))
    # relative error of rstd: the variance's, from s - mean and its squares
    drel = K * (1 + top * rr)
    assert_within("mean", mean, rm, K * top)
    assert_within("rstd", rstd, rr, rr * drel)
    xh = np.abs(rs - rm[..., None]) * rr[..., None]
    ab = 0.0 if b is None else np.abs(mixer.f64(b))
    # xh's own error and the last addition's roundings, relative to its terms
    err = aw * ((K * top * rr)[..., None] + xh * drel[..., None]) \
        + 4 * U32 * (aw * xh + ab)
    assert_within("y", y, ry, err + rounding(ry, x.dtype))
    assert y.dtype == x.dtype and mean.dtype == rstd.dtype == F32
    if residual is None:
        assert s is None
    else:
        assert_within("sum", s, rs, U32 * top[..., None] +
                      rounding(rs, x.dtype))
    return y, s, mean, rstd


def check_bwd(dy, x, w, ds=None, eps=1e-5, got=None, stats=None):
    """The backward (or gradients that it gave already for the statistics
    ``stats``) against the oracle."""
    s = mixer.f64(x)
    m = s.mean(-1)
    r = 1 / np.sqrt(((s - m[..., None]) ** 2).mean(-1) + eps)
    mean, rstd = stats or (torch.from_numpy(np.asarray(v, np.float32)).cuda()
                           for v in (m, r))
    if got is None:
        got = kla.layernorm_bwd(dy, x, w, mean, rstd, sum_grad=ds)
    dx, dw, db = mixer.ln_bwd(dy, x, w, mean, rstd, ds)
    D, rows = x.shape[-1], x.numel() // x.shape[-1]
    K = (32 + D / 32) * U32
    f = mixer.f64
    r = f(rstd)[..., None]
    xh = np.abs(s - f(mean)[..., None]) * r
    g = np.abs(f(dy)) * (1.0 if w is None else np.abs(f(w)))
    c1, c2 = (g * xh).mean(-1, keepdims=True), g.mean(-1, keepdims=True)
    err = K * r * (g + c2 + xh * c1) + \
        (0 if ds is None else U32 * np.abs(f(ds)))
    assert_within("x_grad", got["x_grad"], dx, err + rounding(dx, x.dtype))
    if got["weight_grad"] is None:
        return got
    # the rows' sum: chains of rows and slices, at most rows + 64 additions
    wt = dy.dtype if w is None else w.dtype
    axes = tuple(range(dy.ndim - 1))
    n = (rows + 64) * U32
    aw = (np.abs(f(dy)) * xh).sum(axes)
    ab = np.abs(f(dy)).sum(axes)
    assert_within("weight_grad", got["weight_grad"], dw,
                  n * aw + 4 * U32 * aw + rounding(dw, wt))
    assert_within("bias_grad", got["bias_grad"], db,
                  n * ab + rounding(db, wt))
    assert got["weight_grad"].dtype == got["bias_grad"].dtype == wt
    return got


ROWS = [1, 3, 130]
WIDTHS = [1, 2, 7, 31, 64, 128, 200, 1000, 1001, 1024, 2048, 4100, 8192,
          8200, 20000, 40001]


@pytest.mark.parametrize("dtype,wtype", [(F32, F32), (BF16, BF16),
                                         (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("D", WIDTHS)
def test_sizes_and_types(D, dtype, wtype):
    for rows in ROWS:
        seed = D * 7 + rows
        x = normal((rows, D), dtype, seed, 2.0, 0.5)
        w = normal((D,), wtype, seed + 1, 0.2, 1.0)
        b = normal((D,), wtype, seed + 2)
        res = normal((rows, D), dtype, seed + 3)
        check_fwd(x, w, b)
        check_fwd(x, w, b, residual=res)
        check_bwd(normal((rows, D), dtype, seed + 4), x, w)
        check_bwd(normal((rows, D), dtype, seed + 4), x, w, ds=res)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_rows(dtype):
    x, dy = normal((5001, 384), dtype, 1), normal((5001, 384), dtype, 2)
    w = normal((384,), F32, 3, 0.2, 1.0)
    check_fwd(x, w, None)
    check_bwd(dy, x, w, ds=x)


# Widths of each number of threads a row (in elements of bf16; half of it in
# fp32), aligned rows first, and rows enough for a group of threads to take a
# dozen even where an SM holds 2048 threads: the rings go round.
RINGS = [(256, 32), (512, 32), (1000, 64), (2048, 128), (4096, 256),
         (8192, 512), (8208, 640), (10240, 640), (12288, 512), (16384, 512)]
LOOSE = [(127, 32), (255, 32), (511, 64), (1001, 128), (2047, 256),
         (4095, 512)]


def ring_rows(threads):
    return 12 * 152 * (2048 // threads) + 5


def assert_close(name, got, ref, bound):
    """As assert_within, on the GPU; bound already has the rounding."""
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bad.any(), (name, int(bad.sum()), bad.nonzero()[0].tolist())


def integers(g, lo, hi, shape, dtype):
    return torch.randint(lo, hi + 1, shape, device="cuda",
                         generator=g).to(dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("k", range(len(RINGS) + 2 * len(LOOSE)))
def test_rings_of_rows(k, dtype):
    """Forward and backward over many rows of every width of the rings, all
    different: a place that is read too early or twice, or a row left out of
    the weight gradients, shows.  The loose widths also as slices at an odd
    offset of wider rows.  In the backward, x, dy and the statistics are such
    that the weight gradients' terms and sums are exact in fp32."""
    if k < len(RINGS):
        D, threads = RINGS[k]
        D = D if dtype == BF16 else D // 2
        wider = 0
    else:
        D, threads = LOOSE[(k - len(RINGS)) % len(LOOSE)]
        wider = 0 if k - len(RINGS) < len(LOOSE) else 6
    rows, g = ring_rows(threads), torch.Generator(device="cuda")
    g.manual_seed(1000 * k + D)

    def cut(t):
        return t[:, wider // 2:wider // 2 + D]

    u = U16 * 1.01 if dtype == BF16 else U32
    x = cut(torch.randn(rows, D + wider, device="cuda", generator=g).to(dtype))
    res = cut(torch.randn(rows, D + wider, device="cuda",
                          generator=g).to(dtype))
    w = 1 + 0.2 * torch.randn(D, device="cuda", generator=g)
    b = torch.randn(D, device="cuda", generator=g)
    K = (32 + D / 32) * U32
    for r in (None, res):
        y, s, mean, rstd = kla.layernorm_fwd(x, w, b, residual=r)
        exact = x.double() if r is None else x.double() + r.double()
        var, m = torch.var_mean(exact, 1, correction=0, keepdim=True)
        rr = (var + 1e-5).rsqrt()
        xh = (exact - m) * rr
        top = exact.abs().amax(1, keepdim=True)
        drel = K * (1 + top * rr)
        assert_close("mean", mean[:, None], m, K * top)
        assert_close("rstd", rstd[:, None], rr, rr * (drel + U32))
        wd, bd = w.double(), b.double()
        ref = xh * wd + bd
        a = xh.abs() * wd.abs()
        assert_close("y", y, ref, wd.abs() * (K * top * rr) + a * drel
                     + 4 * U32 * (a + bd.abs()) + u * ref.abs())
        if r is not None:
            assert torch.equal(s, (x.float() + r.float()).to(dtype))
        del exact, xh, ref, a
    x = cut(integers(g, -8, 8, (rows, D + wider), dtype))
    dy = cut(integers(g, -3, 3, (rows, D + wider), dtype))
    mean = integers(g, -2, 2, (rows,), F32)
    rstd = 2.0 ** integers(g, -1, 1, (rows,), F32)
    xh = (x.double() - mean[:, None]) * rstd[:, None]
    gd = dy.double() * w.double()
    c1, c2 = (gd * xh).mean(1, keepdim=True), gd.mean(1, keepdim=True)
    a1, a2 = (gd * xh).abs().mean(1, keepdim=True), \
        gd.abs().mean(1, keepdim=True)
    dx = rstd[:, None] * (gd - c2 - xh * c1)
    err = K * rstd[:, None] * (gd.abs() + a2 + xh.abs() * a1)
    for ds in (None, res):
        got = kla.layernorm_bwd(dy, x, w, mean, rstd, sum_grad=ds)
        ref = dx if ds is None else dx + ds.double()
        assert_close("x_grad", got["x_grad"], ref, err + u * ref.abs() + (
            0 if ds is None else U32 * ds.double().abs()))
        assert torch.equal(got["weight_grad"].double(),
                           (dy.double() * xh).sum(0))
        assert torch.equal(got["bias_grad"].double(), dy.double().sum(0))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows", [1, 3, 129, 700, 5000])
def test_workspace_of_the_stated_size_suffices(rows, dtype):
    """Every width of the rings and of the loops: nothing is written past the
    workspace, and more of it changes nothing."""
    for D, _ in RINGS + LOOSE + [(4097, 0), (20001, 0)]:
        g = torch.Generator(device="cuda").manual_seed(D)
        x = torch.randn(rows, D, device="cuda", generator=g).to(dtype)
        mean, rstd = torch.zeros(rows, device="cuda"), \
            torch.ones(rows, device="cuda")
        n = kla.layernorm_bwd_workspace_size(rows, D, dtype)
        ws = torch.full((n + 65536,), 77, dtype=torch.uint8, device="cuda")
        got = kla.layernorm_bwd(x, x, None, mean, rstd, workspace=ws[:n])
        assert (ws[n:] == 77).all(), D
        more = torch.empty(4 * n, dtype=torch.uint8, device="cuda")
        ref = kla.layernorm_bwd(x, x, None, mean, rstd, workspace=more)
        assert all(torch.equal(got[k], ref[k]) for k in got), D


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [128, 1001, 2048])
def test_without_weight_or_bias(D, dtype):
    x, dy = normal((9, D), dtype, 4), normal((9, D), dtype, 5)
    w, b = normal((D,), F32, 6), normal((D,), F32, 7)
    check_fwd(x, None, None)
    check_fwd(x, w, None)
    check_fwd(x, None, b)
    check_bwd(dy, x, None)
    y, s, mean, rstd = kla.layernorm_fwd(x, w, b, want_stats=False)
    assert s is None and mean is None and rstd is None
    _, _, mean, rstd = kla.layernorm_fwd(x)
    g = kla.layernorm_bwd(dy, x, w, mean, rstd, want_weight_grads=False)
    assert g["weight_grad"] is None and g["bias_grad"] is None
    full = kla.layernorm_bwd(dy, x, w, mean, rstd)
    assert torch.equal(g["x_grad"], full["x_grad"])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_layouts_give_the_same_bits(dtype):
    """Slices, odd offsets, repeated rows and more axes against contiguous
    copies, when the same vector width applies; else within bounds."""
    D = 640
    big = normal((12, 3 * D + 1), dtype, 8)
    w, b = normal((D,), dtype, 9), normal((D,), dtype, 10)
    dy = normal((12, 3 * D + 1), dtype, 11)
    for off in (0, 1, 3, D, D + 1):
        x, g = big[:, off:off + D], dy[:, off:off + D]
        check_fwd(x, w, b, residual=g)
        check_bwd(g, x, w, ds=x)
    x = normal((5, D), dtype, 12)
    y0 = kla.layernorm_fwd(x, w, b)[0]
    y1 = kla.layernorm_fwd(x.view(5, 1, D), w, b)[0]
    assert y1.shape == (5, 1, D) and torch.equal(y1[:, 0], y0)
    y2, _, m, _ = kla.layernorm_fwd(x[0], w, b)
    assert y2.shape == (D,) and m.shape == () and torch.equal(y2, y0[0])
    rep = x[:1].expand(6, D)
    y3 = kla.layernorm_fwd(rep, w, b)[0]
    assert all(torch.equal(r, y0[0]) for r in y3)
    odd = torch.empty(5 * D + 1, dtype=dtype, device="cuda")[1:].view(5, D)
    res = normal((5, D), dtype, 13)
    _, s, _, _ = kla.layernorm_fwd(x, w, b, residual=res, y=odd)
    ref, *_ = kla.layernorm_fwd(x, w, b, residual=res)
    assert torch.allclose(odd.float(), ref.float(), rtol=1e-2, atol=1e-5)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [256, 1001, 40001])
def test_offset_rows_keep_their_variance(D, dtype):
    # mean 1000 times the spread: E[s^2] - m^2 would lose it
    check_fwd(normal((4, D), dtype, 14, 0.05, 50.0), None, None)


def test_constant_rows():
    x = torch.full((3, 512), 7.0, device="cuda")
    y, _, mean, rstd = kla.layernorm_fwd(x, None, None, eps=1e-5)
    assert (y == 0).all() and (mean == 7).all()
    assert torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows", [3, 20000])
@pytest.mark.parametrize("D", [96, 100, 250, 1000, 1001, 1025])
def test_constant_rows_of_any_width(D, rows, dtype):
    """Sums that are exact: the mean is the value and y the bias, however many
    rows there are."""
    v = torch.tensor([1.0, 3.0, 7.0, 10.0, 100.0, 1000.0, 0.5, -3.0],
                     device="cuda").repeat(rows)[:rows]
    x = v[:, None].to(dtype).expand(rows, D).contiguous()
    b = normal((D,), dtype, 28)
    y, _, mean, _ = kla.layernorm_fwd(x, None, b)
    assert torch.equal(mean, x[:, 0].float())
    assert torch.equal(y, b.expand(rows, D))


def test_infinite_rows_keep_their_mean():
    x = normal((20000, 384), BF16, 29)
    x[::100, 7] = float("inf")
    mean = kla.layernorm_fwd(x)[2]
    assert mean[::100].isinf().all() and mean.isinf().sum() == 200


@pytest.mark.parametrize("D", [96, 512, 1001, 8192, 40001])
def test_bad_rows_stay_their_own(D):
    """A row with a NaN or an infinity is NaN; its neighbours are not."""
    x = normal((8, D), BF16, 15)
    clean = kla.layernorm_fwd(x)[0].clone()
    x[2, D // 2] = float("nan")
    x[5, D - 1] = float("inf")
    y = kla.layernorm_fwd(x)[0]
    assert y[2].isnan().all() and y[5].isnan().any()
    for i in (0, 1, 3, 4, 6, 7):
        assert torch.equal(y[i], clean[i])


def test_no_rows():
    w = normal((64,), F32, 16)
    x = torch.empty(0, 64, device="cuda")
    y, _, mean, _ = kla.layernorm_fwd(x, w, w)
    assert y.shape == (0, 64) and mean.shape == (0,)
    g = kla.layernorm_bwd(x, x, w, mean, mean)
    assert (g["weight_grad"] == 0).all() and (g["bias_grad"] == 0).all()


@pytest.mark.parametrize("rows,D", [(6, 48), (3, 1001), (5, 512)])
def test_gradients_are_the_differences(rows, D):
    """fp32 gradients against central differences of the fp64 forward: the
    kernel's error is some 1e-6 of the terms' magnitude, the differences'
    1e-8."""
    r = np.random.default_rng(D)
    x, w = r.standard_normal((rows, D)), r.standard_normal(D)
    dy, ds = r.standard_normal((rows, D)), r.standard_normal((rows, D))
    t = [torch.from_numpy(v.astype(np.float32)).cuda()
         for v in (x, w, dy, ds)]
    x, w, dy, ds = (mixer.f64(v) for v in t)
    _, _, mean, rstd = kla.layernorm_fwd(t[0], t[1], t[1])
    g = kla.layernorm_bwd(t[2], t[0], t[1], mean, rstd, sum_grad=t[3])

    def loss(x, w, b):
        y, s, _, _ = mixer.ln_fwd(x, w, b)
        return (y * dy).sum() + (s * ds).sum()

    args, h = (x, w, w), 1e-5
    for k, name in enumerate(("x_grad", "weight_grad", "bias_grad")):
        got = mixer.f64(g[name])
        v = r.standard_normal(got.shape)
        up, dn = list(args), list(args)
        up[k], dn[k] = args[k] + h * v, args[k] - h * v
        slope = (loss(*up) - loss(*dn)) / (2 * h)
        scale = np.abs(got * v).sum() + np.abs(dy).sum()
        assert abs((got * v).sum() - slope) <= 1e-5 * scale, name


def test_same_bits_every_call_and_on_another_stream():
    x, dy = normal((777, 2048), BF16, 17), normal((777, 2048), BF16, 18)
    w = normal((2048,), BF16, 19)
    y, _, mean, rstd = kla.layernorm_fwd(x, w, w)
    g = kla.layernorm_bwd(dy, x, w, mean, rstd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, _, mean2, rstd2 = kla.layernorm_fwd(x, w, w, stream=side)
    g2 = kla.layernorm_bwd(dy, x, w, mean2, rstd2, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, y2) and torch.equal(rstd, rstd2)
    assert all(torch.equal(g[k], g2[k]) for k in g)


def test_graph_replay_equals_eager():
    x, res = normal((4, 2048), BF16, 20), normal((4, 2048), BF16, 21)
    w = normal((2048,), BF16, 22)
    ref = kla.layernorm_fwd(x, w, w, residual=res)
    gref = kla.layernorm_bwd(res, x, w, ref[2], ref[3])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = kla.layernorm_fwd(x, w, w, residual=res)
        g = kla.layernorm_bwd(res, x, w, out[2], out[3])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, ref))
    assert all(torch.equal(g[k], gref[k]) for k in g)


def test_offsets_past_32_bits():
    rows, D = 1100000, 2048            # 2.25e9 elements
    x = torch.empty(rows, D, dtype=BF16, device="cuda")
    x.fill_(1.0)
    x[-3:] = normal((3, D), BF16, 23)
    w = normal((D,), BF16, 24)
    out = kla.layernorm_fwd(x, w, w)
    y, _, mean, rstd = out
    tail = [None if v is None else v[-3:].clone() for v in out]
    check_fwd(x[-3:], w, w, got=tail)
    assert (y[:4].float() == w.float()).all()
    g = kla.layernorm_bwd(x, x, w, mean, rstd, want_weight_grads=False)
    g["x_grad"] = g["x_grad"][-3:].clone()
    check_bwd(x[-3:].clone(), x[-3:].clone(), w, got=g,
              stats=(tail[2], tail[3]))


def test_weight_gradients_of_more_than_2_30_columns():
    """The partial sums' place of column c of the bias's gradient is D + c,
    past 2^31.  With one row the gradients are dy xh and dy."""
    D = 2 ** 30 + 1000
    g = torch.Generator(device="cuda").manual_seed(27)
    x = torch.randn(1, D, device="cuda", generator=g, dtype=BF16)
    dy = torch.randn(1, D, device="cuda", generator=g, dtype=BF16)
    mean = torch.full((1,), 0.25, device="cuda")
    rstd = torch.full((1,), 0.75, device="cuda")
    got = kla.layernorm_bwd(dy, x, None, mean, rstd)
    assert torch.equal(got["bias_grad"], dy[0])
    for i in range(0, D, 1 << 28):
        q = slice(i, i + (1 << 28))
        xh = (x[0, q].float() - 0.25) * 0.75
        ref = dy[0, q].float() * xh
        err = (got["weight_grad"][q].float() - ref).abs()
        # the result's own rounding; xh's and the product's in fp32
        assert (err <= (U16 * 1.01 + 4 * U32) * ref.abs()).all()


def test_refuses_more_rows_than_it_counts():
    x = torch.zeros(1, 1, device="cuda", dtype=BF16).expand(2 ** 31 + 5, 1)
    with pytest.raises(ValueError, match="2.31"):
        kla.layernorm_fwd(x)
    mean = torch.zeros(1, device="cuda").expand(2 ** 31 + 5)
    with pytest.raises(ValueError, match="2.31"):
        kla.layernorm_bwd(x, x, None, mean, mean)


def test_refusals():
    x, w = normal((4, 64), BF16, 25), normal((64,), BF16, 26)
    _, _, mean, rstd = kla.layernorm_fwd(x, w, w)
    with pytest.raises(TypeError):
        kla.layernorm_fwd(x.half(), w, w)
    with pytest.raises(TypeError):
        kla.layernorm_fwd(x, w.cpu(), w)
    with pytest.raises(TypeError):
        kla.layernorm_fwd(x, w, w.float())
    with pytest.raises(ValueError):
        kla.layernorm_fwd(x, w[:63], w[:63])
    with pytest.raises(ValueError):
        kla.layernorm_fwd(x.t(), None, None)
    with pytest.raises(ValueError):
        kla.layernorm_fwd(x.view(2, 2, 64).transpose(0, 1), w, w)
    with pytest.raises(ValueError):
        kla.layernorm_fwd(x, w, w, residual=x[:2])
    with pytest.raises(ValueError):
        kla.layernorm_fwd(x, w, w, sum=x)
    with pytest.raises(kla.KlaError):
        kla.layernorm_fwd(x, w, w, eps=-1.0)
    with pytest.raises(kla.KlaError):
        kla.layernorm_fwd(x, w, w, y=x)
    with pytest.raises(TypeError):
        kla.layernorm_bwd(x.float(), x, w, mean, rstd)
    with pytest.raises(ValueError):
        kla.layernorm_bwd(x, x, w, mean[:2], rstd)
    with pytest.raises(kla.KlaError):
        kla.layernorm_bwd(x, x, w, mean, rstd, workspace=torch.empty(
            16, dtype=torch.uint8, device="cuda"))
