"""Log probabilities of given tokens, entropies, alternatives and their
gradient on the GPU against the fp64 oracle."""
import math

import numpy as np
import pytest
import torch

from linear_attention_delta_gb300 import kla
from oracle import mixer

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
U32, U16 = mixer.U32, mixer.U16


def rows(N, V, dtype, seed=0, masked=0.0):
    gen = torch.Generator().manual_seed(seed + V)
    x = torch.randn(N, V, generator=gen) * 3 * torch.exp(
        0.7 * torch.randn(N, 1, generator=gen)) + 2
    if masked:
        x[torch.rand(N, V, generator=gen) < masked] = -math.inf
        x[:, V // 2] = 1.0
    tokens = torch.randint(0, V, (N,), generator=gen)
    return x.to(dtype).cuda(), tokens.cuda()


def check_fwd(x, tokens, out, top=0, scale=1.0):
    scale32 = float(np.float32(scale))
    lp, ent, lse, tlp, ids = mixer.lp_fwd(x, tokens, top, scale32)
    V = x.shape[1]
    z = np.abs(scale32 * mixer.f64(x))
    m = np.where(np.isfinite(z), z, 0).max(1)
    # sums: a thread's terms and the joins; exp and its argument (a rounding
    # of a difference of up to 104, after which exp is 0); every rounding of a
    # logit or a logarithm of up to m + 12
    s = (V / 128 + 64 + 104) * U32
    base = s + 4 * U32 * (m + math.log(V) + 1)
    logp, entropy, l, tl, ti = out
    for got, want in ((logp, lp), (l, lse)):
        got = mixer.f64(got)
        inf = np.isinf(want)
        assert (got[inf] == want[inf]).all()
        with np.errstate(invalid="ignore"):
            off = np.where(inf, 0, np.abs(got - want))
            assert (off <= base + 4 * U32 * np.where(inf, 0, np.abs(want))
                    ).all()
    # the mean distance from the maximum, its relative error twice that of a sum
    mean = np.abs(np.where(np.isinf(lse), 0, ent) + m + np.log(V))
    assert (np.abs(mixer.f64(entropy) - ent) <=
            2 * s * (1 + mean) + 4 * U32 * (m + 12)).all()
    if top:
        assert (ti.cpu().numpy() == ids).all()
        got = mixer.f64(tl)
        inf = np.isinf(tlp)
        assert (got[inf] == tlp[inf]).all()
        with np.errstate(invalid="ignore"):
            off = np.where(inf, 0, np.abs(got - tlp))
            assert (off <= base[:, None] + 4 * U32 * np.where(
                inf, 0, np.abs(tlp))).all()
    else:
        assert tl is None and ti is None


def check_bwd(x, tokens, lse, ent, g, ge, out, scale=1.0):
    scale32 = float(np.float32(scale))
    want = mixer.lp_bwd(x, tokens, lse, ent, g, ge, scale32)
    z = scale32 * mixer.f64(x)
    l64 = mixer.f64(lse)
    with np.errstate(invalid="ignore"):
        lp = z - l64[:, None]
    p = np.where(np.isneginf(l64)[:, None] | np.isnan(lp), 0, np.exp(lp))
    lp = np.where(p > 0, lp, 0)
    gm = np.abs(mixer.f64(g))[:, None] if g is not None else 0.0
    gem = np.abs(mixer.f64(ge))[:, None] if ge is not None else 0.0
    H = np.abs(mixer.f64(ent))[:, None] if ent is not None else 0.0
    # exp's argument (a difference of numbers up to |z| + |lse|) and exp; the
    # factors' products and sums; the term of the token itself
    arg = 2 * U32 * (np.where(p > 0, np.abs(z), 0) +
                     np.where(np.isinf(l64), 0, np.abs(l64))[:, None]) + 6 * U32
    size = p * (gm + gem * (np.abs(lp) + H))
    bound = scale32 * ((arg + 8 * U32) * size + gem * p * arg +
                       4 * U32 * gm * (p > 0)) + 1e-37
    if x.dtype == BF16:
        bound = bound + U16 * (np.abs(want) + bound)
    got = mixer.f64(out)
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= bound + 4 * U32 * np.abs(want)).all()


SIZES = [(1, 1), (3, 2), (5, 31), (4, 257), (2, 1000), (7, 4097), (3, 32000),
         (1, 50001), (2, 131072), (300, 640), (1000, 64)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,V", SIZES)
def test_forward(N, V, dtype):
    for scale, top in ((1.0, 0), (0.7, min(V, 20)), (1.25, 1)):
        x, t = rows(N, V, dtype)
        check_fwd(x, t, kla.logprob_fwd(x, t, top, scale), top, scale)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,V", SIZES)
def test_backward(N, V, dtype):
    x, t = rows(N, V, dtype)
    t[::3] = -1
    gen = torch.Generator().manual_seed(1)
    g = torch.randn(N, generator=gen).cuda()
    ge = torch.randn(N, generator=gen).cuda()
    for scale in (1.0, 0.7):
        _, ent, lse, _, _ = kla.logprob_fwd(x, t, scale=scale)
        for a, b in ((g, ge), (g, None), (None, ge)):
            out = kla.logprob_bwd(x, t, lse, ent if b is not None else None,
                                  a, b, scale)
            check_bwd(x, t, lse, ent, a, b, out, scale)
        assert (kla.logprob_bwd(x, t, lse, scale=scale) == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [40, 5003, 40000])
def test_masked_logits(V, dtype):
    x, t = rows(9, V, dtype, masked=0.6)
    low = torch.finfo(dtype).min
    x[4] = -math.inf                      # nothing left
    x[5, :] = low                         # all of the type's lowest value
    x[6, 1:] = low
    x[7, :-3] = -math.inf                 # fewer left than asked for
    t[7] = V - 1
    top = 12
    out = kla.logprob_fwd(x, t, top)
    check_fwd(x, t, out, top)
    assert out[0][4] == -math.inf and out[2][4] == -math.inf
    assert out[1][4] == 0 and out[4][4].tolist() == list(range(top))
    g = torch.ones(9, device="cuda")
    d = kla.logprob_bwd(x, t, out[2], out[1], g, g)
    check_bwd(x, t, out[2], out[1], g, g, d)
    assert (d[4] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [7, 3000, 70001])
@pytest.mark.parametrize("values", [1, 2, 40])
def test_ties_go_to_the_lowest_id(V, values, dtype):
    gen = torch.Generator().manual_seed(V)
    x = torch.randint(0, values, (6, V), generator=gen).to(dtype).cuda()
    x[0] = torch.where(x[0] == 0, -0.0, x[0])     # -0 and 0 are equal
    x[1] = torch.where(torch.arange(V, device="cuda") % 2 == 0, -0.0, 0.0)
    t = torch.zeros(6, dtype=torch.int64, device="cuda")
    top = min(V, 128)
    check_fwd(x, t, kla.logprob_fwd(x, t, top), top)


@pytest.mark.parametrize("order", ["up", "down"])
def test_sorted_rows(order):
    V, top = 20000, 50
    x = torch.arange(V, device="cuda", dtype=F32).div(V).repeat(3, 1)
    x = x if order == "up" else x.flip(1).contiguous()
    t = torch.zeros(3, dtype=torch.int64, device="cuda")
    check_fwd(x, t, kla.logprob_fwd(x, t, top), top)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_not_finite_rows_leave_the_others(dtype):
    x, t = rows(6, 3000, dtype)
    want = kla.logprob_fwd(x, t, 5)
    x[1, 17] = math.nan
    x[3, 5] = math.inf
    x[4, 9] = -math.nan
    got = kla.logprob_fwd(x, t, 5)
    for r in range(6):
        for a, b in zip(got[:4], want[:4]):
            if r in (1, 3, 4):
                assert torch.isnan(a[r]).all()
            else:
                assert torch.equal(a[r], b[r])
    assert [got[4][r, 0].item() for r in (1, 3, 4)] == [17, 5, 9]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("off,wide", [(0, 8), (1, 3), (5, 57)])
def test_strided_rows(off, wide, dtype):
    x, t = rows(9, 1003, dtype)
    buf = torch.zeros(9, 1003 + wide + off, dtype=dtype, device="cuda")
    y = buf[:, off:off + 1003]
    y.copy_(x)
    a, b = kla.logprob_fwd(y, t, 4), kla.logprob_fwd(x, t, 4)
    check_fwd(x, t, a, 4)
    assert torch.equal(a[4], b[4])
    g = torch.rand(9, device="cuda")
    check_bwd(x, t, a[2], a[1], g, g,
              kla.logprob_bwd(y, t, a[2], a[1], g, g))
    one = x[:1].expand(9, 1003)           # one row for all
    check_fwd(one, t, kla.logprob_fwd(one, t, 4), 4)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradient_in_place(dtype):
    x, t = rows(5, 2050, dtype)
    _, ent, lse, _, _ = kla.logprob_fwd(x, t)
    g = torch.rand(5, device="cuda")
    want = kla.logprob_bwd(x, t, lse, ent, g, g)
    assert kla.logprob_bwd(x, t, lse, ent, g, g, out=x) is x
    assert torch.equal(x, want)


def test_tokens_outside_the_vocabulary():
    x, t = rows(6, 300, F32)
    t[:5] = torch.tensor([-1, -100, 300, 2 ** 40, -2 ** 40])
    logp = kla.logprob_fwd(x, t)[0]
    assert (logp[:5] == 0).all() and logp[5] < 0
    lse = kla.logprob_fwd(x, t)[2]
    d = kla.logprob_bwd(x, t, lse, logp_grad=torch.ones(6, device="cuda"))
    assert (d[:5] == 0).all() and (d[5] != 0).any()


def test_shapes_streams_and_graphs():
    x, t = rows(12, 5000, BF16)
    x, t = x.view(3, 4, 5000), t.view(3, 4)
    g = torch.rand(3, 4, device="cuda")

    def run():
        out = kla.logprob_fwd(x, t, 7)
        return [*out, kla.logprob_bwd(x, t, out[2], out[1], g, g)]

    want = run()
    assert want[0].shape == (3, 4) and want[4].shape == (3, 4, 7)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = kla.logprob_fwd(x, t, 7, stream=s)
    with torch.cuda.stream(s):
        run()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for o in out:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    empty = kla.logprob_fwd(x[:0], t[:0], 2)
    assert empty[0].shape == (0, 4) and empty[3].shape == (0, 4, 2)


def test_offsets_beyond_32_bits():
    """Rows 2^31 elements apart."""
    V, far = 1000, 2 ** 31 + 40
    buf = torch.empty(far + V, dtype=BF16, device="cuda")
    x, t = rows(2, V, BF16)
    y = buf.as_strided((2, V), (far, 1))
    y.copy_(x)
    out = kla.logprob_fwd(y, t, 3)
    check_fwd(x, t, out, 3)
    g = torch.ones(2, device="cuda")
    check_bwd(x, t, out[2], out[1], g, None,
              kla.logprob_bwd(y, t, out[2], None, g))


def test_binding_refuses():
    x, t = rows(4, 10, F32)
    g = torch.ones(4, device="cuda")
    with pytest.raises(ValueError):
        kla.logprob_fwd(x, t[:3])
    with pytest.raises(TypeError):
        kla.logprob_fwd(x, t.int())
    with pytest.raises(TypeError):
        kla.logprob_fwd(x.half(), t)
    with pytest.raises(kla.KlaError):
        kla.logprob_fwd(x, t, top=11)
    with pytest.raises(kla.KlaError):
        kla.logprob_fwd(x, t, scale=0.0)
    with pytest.raises(ValueError):
        kla.logprob_bwd(x, t, g, None, g, g)
    with pytest.raises(ValueError):
        kla.logprob_bwd(x, t, g, out=torch.empty(4, 20, device="cuda")[:, ::2])
    with pytest.raises(kla.KlaError):
        kla.logprob_fwd(torch.zeros(2, 500, device="cuda"),
                        t[:2], top=129)


def peaked(V, dtype, peaks, seed=0):
    """Rows around 0 with one logit far above the others, early and late."""
    gen = torch.Generator().manual_seed(seed + V)
    n = len(peaks)
    x = torch.randn(n, V, generator=gen)
    at = torch.tensor([0, V // 3, V - 1 - V // 50, V - 1, V // 2]).repeat(
        n)[:n]
    x[torch.arange(n), at] = torch.tensor(peaks, dtype=F32)
    return x.to(dtype).cuda(), at.cuda()


PEAKS = [12.0, 13.5, 15.0, 17.0, 18.0, 20.0, 22.5, 25.0, 27.0, 30.0, 32.0,
         35.0, 37.0, 39.0]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [1000, 32000, 131072])
@pytest.mark.parametrize("scale", [1.0, 0.8, 1.3])
def test_confident_rows_keep_their_digits(V, scale, dtype):
    """Entropies and log probabilities near 0, and their signs."""
    x, t = peaked(V, dtype, PEAKS)
    scale32, top = float(np.float32(scale)), 4
    want = mixer.lp_fwd(x, t, top, scale32)
    out = kla.logprob_fwd(x, t, top, scale)
    logp, ent, lse, tlp = (mixer.f64(o) for o in out[:4])
    # Relative to the largest logit all terms of a sum have one sign.  A row's
    # sum meets some 100 roundings of half a step, 2^-24, at most: they add up
    # to 32 of them where their signs are any (more than three times the square
    # root of their number).  The quotient, the logarithm and the last sum are
    # roundings of what is returned.
    step = 32 * U32
    assert (np.abs(ent - want[1]) <= step + 4 * U32 * want[1]).all()
    assert (np.abs(logp - want[0]) <= step + 4 * U32 * np.abs(want[0])).all()
    assert (np.abs(lse - want[2]) <= step + 2 * U32 * np.abs(want[2])).all()
    assert (np.abs(tlp - want[3]) <= step + 4 * U32 * np.abs(want[3])).all()
    assert (out[4].cpu().numpy() == want[4]).all()
    # what no rounding may turn round
    assert (ent >= 0).all() and (logp <= 0).all() and (tlp <= 0).all()
    assert (lse >= scale32 * mixer.f64(x).max(1)).all()
    g = torch.ones(len(PEAKS), device="cuda")
    d = mixer.f64(kla.logprob_bwd(x, t, out[2], logp_grad=g, scale=scale))
    own = d[np.arange(len(PEAKS)), t.cpu().numpy()]
    assert (own >= 0).all()
    assert (np.delete(d, t.cpu().numpy(), 1).max() <= 0)
    # 1 - p, of an lse rounded once more, and rounded to logits' type
    exact = -np.expm1(want[0]) * scale32
    bound = scale32 * (step + 4 * U32 * (1 + np.abs(want[2])))
    if dtype == BF16:
        bound = bound + U16 * (exact + bound)
    assert (np.abs(own - exact) <= bound).all()


@pytest.mark.parametrize("V", [700, 32000, 131072])
def test_a_shift_of_all_logits_changes_lse_alone(V):
    gen = torch.Generator().manual_seed(V)
    # multiples of 2^-10 below 2^13: exact with the shift
    x = (torch.randn(5, V, generator=gen) * 4096).round().div(1024)
    x[2, V - 3] = 30.0
    x, t = x.cuda(), torch.randint(0, V, (5,), generator=gen).cuda()
    a, b = kla.logprob_fwd(x, t, 6), kla.logprob_fwd(x + 4096, t, 6)
    for i in (0, 1, 3, 4):
        assert torch.equal(a[i], b[i])
    assert ((b[2] - 4096 - a[2]).abs() <= 2 * U32 * 4200).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scaled_logits_below_the_range_are_masked(dtype):
    x = torch.full((3, 2000), torch.finfo(dtype).min, dtype=dtype,
                   device="cuda")
    x[1, 7] = 1.0
    x[2, :1999] = -math.inf
    t = torch.full((3,), 7, dtype=torch.int64, device="cuda")
    logp, ent, lse, tlp, ids = kla.logprob_fwd(x, t, 2, scale=2.0)
    inf = math.inf
    assert logp.tolist() == [-inf, 0, -inf] and ent.tolist() == [0, 0, 0]
    assert lse.tolist() == [-inf, 2, -inf]
    assert tlp.tolist() == [[-inf, -inf], [0, -inf], [-inf, -inf]]
    assert ids.tolist() == [[0, 1], [7, 0], [1999, 0]]
    d = kla.logprob_bwd(x, t, lse, ent, torch.ones_like(lse),
                        torch.ones_like(lse), scale=2.0)
    assert (d == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [1000, 3000, 70001])
def test_nan_at_the_first_id(V, dtype):
    """NaN ranks first, equal logits by rising id, whichever way the row is
    searched (more candidates than a block holds: round by round)."""
    x = torch.zeros(5, V, dtype=dtype, device="cuda")
    x[0] = math.nan
    x[1, 0] = math.nan                       # above V - 1 equal logits
    x[2] = -math.inf
    x[2, 0] = math.nan                       # the only one not masked
    x[3, V - 1] = math.nan
    t = torch.ones(5, dtype=torch.int64, device="cuda")
    _, _, _, tlp, ids = kla.logprob_fwd(x, t, 6)
    first = list(range(6))
    assert [r.tolist() for r in ids] == [first, first, first,
                                         [V - 1] + first[:5], first]
    assert torch.isnan(tlp[:4]).all() and torch.isfinite(tlp[4]).all()


def far_rows(V, dtype, seed=0):
    """Rows far from 0: some neighbouring numbers of the type each, from one to
    the next the same step; the last ones all of the type's lowest value."""
    gen = torch.Generator().manual_seed(seed + V)
    bits = 23 if dtype == F32 else 7
    at, rows = [300.0, -900.0, 5000.0, -70000.0, 3e9, -2e20, -1e38], []
    for x in at:
        step = 2.0 ** (math.floor(math.log2(abs(x))) - bits)
        base = round(x / step) * step
        n = max(1.0, round(0.5 / step)) if step < 1 else 1.0
        j = torch.randint(-8, 9, (V,), generator=gen).double()
        rows.append(base + step * n * j)
    low = torch.full((2, V), torch.finfo(dtype).min, dtype=torch.float64)
    x = torch.cat([torch.stack(rows), low])
    out = x.to(dtype)
    assert torch.equal(out.double(), x)
    return out.cuda(), torch.randint(0, V, (len(x),), generator=gen).cuda()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [1, 2, 700, 5003, 40000])
@pytest.mark.parametrize("scale", [1.0, 0.6, 0.9])
def test_rows_far_from_zero(V, scale, dtype):
    x, t = far_rows(V, dtype)
    top = min(V, 5)
    logp, ent, lse, tlp, ids = kla.logprob_fwd(x, t, top, scale)
    # 64 bits hold the differences from the largest logit
    scale32 = float(np.float32(scale))
    x64 = mixer.f64(x)
    m = x64.max(1, keepdims=True)
    z = scale32 * (x64 - m)
    ls = np.log(np.exp(z).sum(1, keepdims=True))
    p = np.exp(z - ls)
    n = np.arange(len(x64))
    want = (z - ls)[n, t.cpu().numpy()]
    H = ls[:, 0] - (p * z).sum(1)
    # 32 roundings of a sum's own (see above); each e is off by three half
    # steps (of the difference, the factor and the product), which moves ls by
    # the mean of |z|, and the entropy by that of z^2, of as many
    far = 32 * U32 + 3 * U32 * ((p * np.abs(z)).sum(1) + (p * z * z).sum(1))
    assert (np.abs(mixer.f64(logp) - want) <= far + 4 * U32 * np.abs(want)
            ).all()
    assert (np.abs(mixer.f64(ent) - H) <= far + 4 * U32 * H).all()
    l64 = scale32 * m[:, 0] + ls[:, 0]
    assert (np.abs(mixer.f64(lse) - l64) <= far + 2 * U32 * np.abs(l64)).all()
    assert (mixer.f64(lse) >= scale32 * m[:, 0]).all()
    order = np.argsort(-x64, axis=1, kind="stable")[:, :top]
    assert (ids.cpu().numpy() == order).all()
    want = np.take_along_axis(z - ls, order, 1)
    assert (np.abs(mixer.f64(tlp) - want) <= far[:, None] +
            4 * U32 * np.abs(want)).all()


@pytest.mark.parametrize("scale", [0.7, 1.3])
def test_a_shift_of_all_logits_at_other_scales(scale):
    gen = torch.Generator().manual_seed(5)
    x = (torch.randn(5, 9000, generator=gen) * 4096).round().div(1024).cuda()
    x[1, ::2] = -math.inf
    t = torch.randint(0, 9000, (5,), generator=gen).cuda()
    a, b = kla.logprob_fwd(x, t, 6, scale), kla.logprob_fwd(x + 4096, t, 6,
                                                            scale)
    for i in (0, 1, 3, 4):
        assert torch.equal(a[i], b[i])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_extreme_scales(dtype):
    x = torch.full((3, 900), -1.0, dtype=dtype, device="cuda")
    x[0, 300:302] = -0.5                  # two of the same
    x[1, 500:] = -math.inf                # 500 of the same
    x[2, 7] = -0.5
    t = torch.full((3,), 300, dtype=torch.int64, device="cuda")
    logp, ent, lse, tlp, ids = kla.logprob_fwd(x, t, 2, 3e38)
    ln2, ln500 = math.log(2), math.log(500)
    assert (ent.cpu() - torch.tensor([ln2, ln500, 0.0])).abs().max() <= 1e-6
    assert (logp[:2].cpu() + torch.tensor([ln2, ln500])).abs().max() <= 1e-6
    assert logp[2] == torch.tensor(-0.5 * 3e38) and lse[2] == logp[2]
    assert ids.tolist() == [[300, 301], [0, 1], [7, 0]]
    logp, ent, lse, tlp, ids = kla.logprob_fwd(x, t, 2, 1e-38)
    ln = torch.tensor([900.0, 500.0, 900.0]).log()
    for got in (ent, -logp, lse, -tlp[:, 0], -tlp[:, 1]):
        # (a sum of 900 equal terms, and the roundings above)
        assert (got.cpu() - ln).abs().max() <= (32 + 8 * 7) * U32


def exact_gradient(x, t, g, ge, scale32):
    """(gradient, p, z, log p, H, mean |z|, mean z^2) in 64 bits, from
    differences of logits; z: scaled distances from the largest."""
    x64 = mixer.f64(x)
    z = scale32 * (x64 - x64.max(1, keepdims=True))
    lp = z - np.log(np.exp(z).sum(1, keepdims=True))
    p = np.exp(lp)
    H = -(p * lp).sum(1, keepdims=True)
    g, ge = (mixer.f64(a)[:, None] for a in (g, ge))
    d = -p * (g + ge * (lp + H))
    n = np.arange(len(x64))
    d[n, t.cpu().numpy()] += g[:, 0]
    mean = [(p * y).sum(1, keepdims=True) for y in (np.abs(z), z * z)]
    return scale32 * d, p, z, lp, H, *mean


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [1, 2, 700, 5003, 40000])
@pytest.mark.parametrize("scale", [1.0, 0.6])
def test_gradient_of_rows_far_from_zero(V, scale, dtype):
    x, t = far_rows(V, dtype)
    gen = torch.Generator().manual_seed(3)
    g, ge = (torch.randn(len(x), generator=gen).cuda() for _ in range(2))
    _, ent, lse, _, _ = kla.logprob_fwd(x, t, scale=scale)
    got = kla.logprob_bwd(x, t, lse, ent, g, ge, scale)
    scale32 = float(np.float32(scale))
    want, p, z, lp, H, d1, d2 = exact_gradient(x, t, g, ge, scale32)
    # log p: three half steps of z, those of log s (as in the forward), and,
    # where it is small enough to be used, of lse; then exp and the products
    small = np.abs(mixer.f64(lse))[:, None]
    small = np.where(small < 1024, small, 0)
    e = 3 * U32 * np.abs(z) + (32 + 3 * d1 + 3 * d2 + small) * U32
    gm, gem = (np.abs(mixer.f64(a))[:, None] for a in (g, ge))
    bound = scale32 * (p * (gm + gem * (np.abs(lp) + H)) * (e + 8 * U32) +
                       gem * p * (2 * e + 4 * U32 * (np.abs(lp) + H)) +
                       4 * U32 * gm * (p > 0)) + 1e-37
    if dtype == BF16:
        bound = bound + U16 * (np.abs(want) + bound)
    off = np.abs(mixer.f64(got) - want)
    assert (off <= bound + 4 * U32 * np.abs(want)).all()
    y = x.clone()
    kla.logprob_bwd(y, t, lse, ent, g, ge, scale, out=y)
    assert torch.equal(y, got)


def test_gradient_of_part_of_a_vocabulary():
    """The whole's lse with a part's logits, far from 0: taken as given."""
    gen = torch.Generator().manual_seed(8)
    x = (torch.randn(6, 9000, generator=gen) * 2 + 5000).cuda()
    t = torch.randint(0, 4000, (6,), generator=gen).cuda()
    _, ent, lse, _, _ = kla.logprob_fwd(x, t)
    g = torch.ones(6, device="cuda")
    part = x[:, :4000]
    check_bwd(part, t, lse, ent, g, g,
              kla.logprob_bwd(part, t, lse, ent, g, g))
