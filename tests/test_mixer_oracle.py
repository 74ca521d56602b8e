"""Pins of the fp64 oracle of layer norm and the gated linear recurrence:
closed forms, central differences of the forward, packed against batched."""
import numpy as np
import pytest

from oracle import mixer


def rng(seed):
    return np.random.default_rng(seed)


def test_ln_hand_worked():
    # s = (1, 3): mean 2, variance 1; eps 0.44 -> rstd = 1 / 1.2
    y, s, mean, rstd = mixer.ln_fwd(np.array([[0.0, 1.0]]),
                                    weight=np.array([3.0, 6.0]),
                                    bias=np.array([1.0, -1.0]), eps=0.44,
                                    residual=np.array([[1.0, 2.0]]))
    assert s.tolist() == [[1.0, 3.0]] and mean.tolist() == [2.0]
    assert np.allclose(rstd, 1 / 1.2) and np.allclose(y, [[-1.5, 4.0]])


def differences(f, args, k, v, h=1e-6):
    """Directional derivative of f along v in its k-th argument."""
    up, dn = list(args), list(args)
    up[k], dn[k] = args[k] + h * v, args[k] - h * v
    return (f(*up) - f(*dn)) / (2 * h)


@pytest.mark.parametrize("M,D", [(1, 2), (3, 5), (7, 16)])
def test_ln_gradients_are_the_differences(M, D):
    r = rng(M * 100 + D)
    x, w, b = r.normal(size=(M, D)), r.normal(size=D), r.normal(size=D)
    dy, ds = r.normal(size=(M, D)), r.normal(size=(M, D))

    def loss(x, w, b):
        y, s, _, _ = mixer.ln_fwd(x, w, b)
        return (y * dy).sum() + (s * ds).sum()

    _, _, mean, rstd = mixer.ln_fwd(x)
    grads = mixer.ln_bwd(dy, x, w, mean, rstd, ds)
    for k, g in enumerate(grads):
        v = r.normal(size=g.shape)
        # truncation h^2 and rounding 1e-16 / h, both about 1e-10
        assert abs(differences(loss, (x, w, b), k, v) - (g * v).sum()) \
            <= 1e-7 * (1 + np.abs(g).sum())


def test_glr_closed_form():
    # constant decay and input: h_t = x (1 - a^t) / (1 - a) + a^t h0
    T, a = 40, 0.8
    x, la = np.full((1, T, 1), 2.0), np.full((1, T, 1), np.log(a))
    o, hT = mixer.glr_fwd(x, la, np.array([[5.0]]))
    t = np.arange(1, T + 1)
    assert np.allclose(o[0, :, 0], 2 * (1 - a ** t) / (1 - a) + 5 * a ** t)
    assert hT[0, 0] == o[0, -1, 0]


def test_glr_forget_and_sum():
    x = rng(1).normal(size=(2, 9, 3))
    la = np.full_like(x, -np.inf)
    assert np.array_equal(mixer.glr_fwd(x, la, np.ones((2, 3)))[0], x)
    o, _ = mixer.glr_fwd(x, np.zeros_like(x))
    assert np.allclose(o, np.cumsum(x, 1))


@pytest.mark.parametrize("with_h0", [False, True])
def test_glr_gradients_are_the_differences(with_h0):
    r = rng(3)
    B, T, D = 2, 6, 3
    x, la = r.normal(size=(B, T, D)), -r.random((B, T, D))
    h0 = r.normal(size=(B, D)) if with_h0 else None
    do, dhT = r.normal(size=(B, T, D)), r.normal(size=(B, D))

    def loss(x, la, h0=None):
        o, hT = mixer.glr_fwd(x, la, h0)
        return (o * do).sum() + (hT * dhT).sum()

    o, _ = mixer.glr_fwd(x, la, h0)
    grads = mixer.glr_bwd(o, la, do, dhT, h0)
    args = (x, la) + ((h0,) if with_h0 else ())
    for k in range(len(args)):
        v = r.normal(size=grads[k].shape)
        assert abs(differences(loss, args, k, v) - (grads[k] * v).sum()) \
            <= 1e-7 * (1 + np.abs(grads[k]).sum())


def test_glr_packed_is_each_sequence_alone():
    r = rng(5)
    lens = [3, 0, 1, 7, 0]
    cu = np.concatenate([[0], np.cumsum(lens)])
    T, D = cu[-1], 4
    x, la = r.normal(size=(T, D)), -r.random((T, D))
    h0, dhT = r.normal(size=(5, D)), r.normal(size=(5, D))
    do = r.normal(size=(T, D))
    o, hT = mixer.glr_fwd(x, la, h0, cu)
    dx, dla, dh0 = mixer.glr_bwd(o, la, do, dhT, h0, cu)
    for n in range(5):
        q = slice(cu[n], cu[n + 1])
        o1, h1 = mixer.glr_fwd(x[q][None], la[q][None], h0[n:n + 1])
        g1 = mixer.glr_bwd(o1, la[q][None], do[q][None], dhT[n:n + 1],
                           h0[n:n + 1])
        assert np.array_equal(o[q], o1[0]) and np.array_equal(hT[n], h1[0])
        assert np.array_equal(dx[q], g1[0][0])
        assert np.array_equal(dla[q], g1[1][0])
        assert np.array_equal(dh0[n], g1[2][0])


def test_a_planted_mistake_exceeds_the_bounds():
    """The forward's and backward's bounds are tight enough to tell one
    dropped token, an undecayed carry or a shifted state from rounding."""
    r = rng(7)
    B, T, D = 1, 200, 4
    x, la = r.normal(size=(B, T, D)), -0.1 * r.random((B, T, D))
    o, hT = mixer.glr_fwd(x, la)
    bo, bh = mixer.glr_fwd_bound(x, la)
    y = x.copy()
    y[0, 50] = 0
    assert (np.abs(mixer.glr_fwd(y, la)[0] - o) > bo).any()
    do = r.normal(size=(B, T, D))
    bound = mixer.glr_bwd_bound(o, la, do)
    good = mixer.glr_bwd(o, la, do)
    shifted = mixer.glr_bwd(np.roll(o, 1, 1), la, do)
    assert (np.abs(shifted[1] - good[1]) > bound[1]).any()
    assert (np.abs(mixer.glr_bwd(o, la * 1.001, do)[0] - good[0])
            > bound[0]).any()
