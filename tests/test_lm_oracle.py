"""Pins of the fp64 oracle of linear attention with a decay for each head and
of token log probabilities (CPU)."""
import numpy as np
import pytest
import torch

from oracle import mixer

RNG = np.random.default_rng(5)


def rand(*shape):
    return torch.from_numpy(RNG.standard_normal(shape))


def inputs(B=2, T=7, H=3, dk=4, dv=5):
    a = torch.tensor([0.0, -0.3, -2.0], dtype=torch.float64)[:H]
    return (rand(B, T, H, dk), rand(B, T, H, dk), rand(B, T, H, dv), a,
            rand(B, H, dk, dv))


def quadratic(q, k, v, a, h0):
    """The same as sums over pairs of tokens, written apart."""
    T = q.shape[1]
    i = torch.arange(T)
    n = (i[:, None] - i[None, :]).clamp(min=0)
    w = torch.exp(a[:, None, None] * n) * (i[:, None] >= i[None, :])
    P = torch.einsum("bthd,bshd->bhts", q, k) * w
    o = torch.einsum("bhts,bshe->bthe", P, v)
    o = o + torch.einsum("bthd,bhde,th->bthe", q, h0,
                         torch.exp(a * (i[:, None] + 1)))
    hT = torch.exp(a * T)[:, None, None] * h0 + torch.einsum(
        "bshd,bshe,sh->bhde", k, v, torch.exp(a * (T - 1 - i[:, None])))
    return o, hT


def test_linattn_forward_is_the_sum_over_pairs():
    q, k, v, a, h0 = inputs()
    for got, want in zip(mixer.la_fwd(q, k, v, a, h0),
                         quadratic(q, k, v, a, h0)):
        np.testing.assert_allclose(got, want.numpy(), rtol=1e-12, atol=1e-12)


def test_linattn_worked_by_hand():
    """One head, 1 x 1, decay 1/2: S = 2 1/2 + 3 = 4, 4/2 + 2 5 = 12."""
    one = torch.ones(1, 2, 1, 1)
    k = torch.tensor([3.0, 2.0]).view(1, 2, 1, 1)
    v = torch.tensor([1.0, 5.0]).view(1, 2, 1, 1)
    o, hT = mixer.la_fwd(one, k, v, np.log([0.5]), torch.full((1, 1, 1, 1),
                                                             2.0))
    assert o.ravel().tolist() == pytest.approx([4.0, 12.0])
    assert hT.item() == pytest.approx(12.0)


def test_linattn_backward_is_autograd():
    q, k, v, a, h0 = inputs()
    for x in (q, k, v, h0):
        x.requires_grad_()
    o, hT = quadratic(q, k, v, a, h0)
    do, dhT = rand(*o.shape), rand(*hT.shape)
    want = torch.autograd.grad((o, hT), (q, k, v, h0), (do, dhT))
    got = mixer.la_bwd(q, k, v, a, do, dhT, h0)
    for x, y in zip(got, want):
        np.testing.assert_allclose(x, y.numpy(), rtol=1e-11, atol=1e-12)


def test_linattn_backward_is_differences():
    q, k, v, a, h0 = inputs(1, 3, 1, 2, 2)
    do, dhT = rand(*v.shape), rand(*h0.shape)

    def loss(*x):
        o, hT = mixer.la_fwd(*x[:3], a, x[3])
        return (o * do.numpy()).sum() + (hT * dhT.numpy()).sum()

    args = [q, k, v, h0]
    grads = mixer.la_bwd(q, k, v, a, do, dhT, h0)
    for n, g in enumerate(grads):
        for at in np.ndindex(*g.shape):
            d = 1e-6
            up, down = ([x.clone() for x in args] for _ in range(2))
            up[n][at] += d
            down[n][at] -= d
            assert (loss(*up) - loss(*down)) / (2 * d) == \
                pytest.approx(g[at], abs=1e-7, rel=1e-7)


def test_linattn_forgets_at_minus_infinity():
    q, k, v, _, h0 = inputs(1, 4, 1)
    o, hT = mixer.la_fwd(q, k, v, [-np.inf], h0)
    want = (q * k).sum(-1, keepdim=True) * v
    np.testing.assert_allclose(o, want.numpy(), rtol=1e-12)


def logits(N=5, V=11):
    x = rand(N, V) * 2
    x[1, 3:6] = -np.inf
    x[2] = -np.inf
    x[3, :] = 0.25
    tokens = torch.tensor([0, 2, 4, -1, 10])
    return x, tokens


def test_logprob_is_torchs():
    x, tokens = logits()
    logp, ent, lse, top, ids = mixer.lp_fwd(x, tokens, top=3, scale=0.7)
    rows = [0, 1, 4]
    want = torch.log_softmax(0.7 * x, 1)
    for r in rows:
        assert logp[r] == pytest.approx(want[r, tokens[r]].item())
        p = want[r].exp()
        assert ent[r] == pytest.approx(torch.special.entr(p).sum().item())
        assert lse[r] == pytest.approx(torch.logsumexp(0.7 * x[r], 0).item())
        np.testing.assert_allclose(top[r], want[r].topk(3).values.numpy())
        assert ids[r].tolist() == want[r].topk(3).indices.tolist()
    # nothing left: -inf, no entropy, the lowest ids; no token: 0; ties
    assert logp[2] == lse[2] == -np.inf and ent[2] == 0
    assert ids[2].tolist() == ids[3].tolist() == [0, 1, 2]
    assert np.isneginf(top[2]).all()
    assert logp[3] == 0 and ent[3] == pytest.approx(np.log(11))


def test_logprob_gradient_is_autograd():
    x, tokens = logits()
    keep = [0, 1, 3, 4]
    g, ge = rand(5), rand(5)
    _, ent, lse, _, _ = mixer.lp_fwd(x, tokens, scale=0.7)
    got = mixer.lp_bwd(x, tokens, lse, ent, g, ge, scale=0.7)
    assert (got[2] == 0).all()
    leaf = torch.where(torch.isinf(x), -1e4, x)[keep].requires_grad_()
    lp = torch.log_softmax(0.7 * leaf, 1)
    t = tokens[keep]
    picked = lp.gather(1, t.clamp(min=0)[:, None])[:, 0] * (t >= 0)
    H = -(lp.exp() * lp).sum(1)
    want, = torch.autograd.grad((picked * g[keep]).sum() +
                                (H * ge[keep]).sum(), leaf)
    np.testing.assert_allclose(got[keep], want.numpy(), atol=1e-13,
                               rtol=1e-11)
