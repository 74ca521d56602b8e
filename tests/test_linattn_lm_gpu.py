"""A language model of linear attention, layer norm and token log probabilities
together: it runs, and its gradients are those of the same model written with
torch in 64 bits."""
import pytest
import torch
import torch.nn.functional as F

pytestmark = pytest.mark.gpu


def test_example_runs_and_decodes_what_it_prefills():
    from examples import linattn_lm
    losses, worst, scale = linattn_lm.main(steps=3)
    assert len(losses) == 3 and all(x == x for x in losses)
    # bf16 activations: the prompt's and the tokens' own way round differently
    # (a few roundings of 2^-8 a block on a logit's sum)
    assert worst <= 16 * 2.0 ** -8 * scale


def reference(model, tokens, target):
    """The loss of the same model in 64 bits, written with torch alone."""
    T = tokens.shape[1]
    i = torch.arange(T, device="cuda")
    n = (i[:, None] - i[None, :]).clamp(min=0)
    w = torch.exp(model.log_decay.double()[:, None, None] * n) * (
        i[:, None] >= i[None, :])
    s = F.embedding(tokens, model.embed)
    for b in model.blocks:
        y = F.layer_norm(s, s.shape[-1:], b.w, b.b, 1e-5)
        q, k, v, z = model.inputs(b, y)
        P = torch.einsum("bthd,bshd->bhts", q, k) * w
        o = torch.einsum("bhts,bshe->bthe", P, v)
        s = s + (o * F.silu(z)).flatten(-2) @ b.out
    y = F.layer_norm(s, s.shape[-1:], model.w, model.b, 1e-5)
    return F.cross_entropy((y @ model.head).flatten(0, 1), target.flatten(),
                           ignore_index=-1)


def test_gradients_of_the_whole_model():
    from examples import linattn_lm
    torch.manual_seed(1)
    gen = torch.Generator(device="cuda").manual_seed(1)
    model = linattn_lm.Model(vocab=23, dim=48, heads=3, width=16,
                             dtype=torch.float32)
    tokens, target = linattn_lm.batch(2, 150, 23, 3, gen)
    logits, _ = model(tokens)
    loss = linattn_lm.TokenLoss.apply(logits, target)
    loss.backward()
    grads = {n: p.grad.double() for n, p in model.named_parameters()}
    exact = linattn_lm.Model(vocab=23, dim=48, heads=3, width=16,
                             dtype=torch.float64)
    exact.load_state_dict({n: x.double() for n, x in
                           model.state_dict().items()})
    want = reference(exact, tokens, target)
    want.backward()
    # some hundred roundings of 2^-24 (sums over 150 tokens, 48 to 192 wide,
    # through six products in a row), and TF32 is off
    assert not torch.backends.cuda.matmul.allow_tf32
    assert abs(loss.item() - want.item()) <= 1e-5 * abs(want.item())
    for n, p in exact.named_parameters():
        off = (grads[n] - p.grad).norm() / p.grad.norm()
        assert off <= 1e-5 * 10, (n, off.item())


def test_training_step_in_a_graph():
    """Forward, loss, backward and one decoded token captured and replayed:
    the same as run at once."""
    from linear_attention_delta_gb300 import kla
    B, T, H, d, V = 2, 200, 3, 64, 100
    q, k, v = (torch.randn(B, T, H, d, device="cuda").bfloat16()
               for _ in range(3))
    a = torch.tensor([-0.5, -0.05, 0.0], device="cuda")
    W = (torch.randn(H * d, V, device="cuda") * 0.1).bfloat16()
    t = torch.randint(-1, V, (B, T), device="cuda")
    S0 = torch.randn(B, H, d, d, device="cuda")

    def run():
        o, hT = kla.linattn_fwd(q, k, v, a, S0)
        logits = o.flatten(-2) @ W
        logp, _, lse, top, ids = kla.logprob_fwd(logits, t, top=4)
        dl = kla.logprob_bwd(logits, t, lse, logp_grad=torch.full_like(
            logp, -1.0))
        do = (dl @ W.t()).unflatten(-1, (H, d))
        g = kla.linattn_bwd(q, k, v, a, do, hT_grad=hT, h0=S0)
        S = hT.clone()
        o1 = kla.linattn_step(q[:, 0], k[:, 1], v[:, 2], a, S)
        return [o, hT, logp, top, ids, dl, *g.values(), S, o1]

    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for x in out:
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(out, want):
        assert torch.equal(x, y)


def test_second_derivatives_are_refused():
    """The backward passes are not differentiable themselves: asked for, that
    is an error and no wrong gradient."""
    from examples import linattn_lm, recurrent_lm
    B, T, H, d = 1, 12, 2, 16
    x = torch.randn(B, T, H, d, device="cuda", requires_grad=True)
    one = torch.ones(d, device="cuda", requires_grad=True)
    zero = torch.zeros(d, device="cuda", requires_grad=True)
    target = torch.zeros(B, T, H, dtype=torch.int64, device="cuda")
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    a = torch.full((H,), -0.1, device="cuda")
    for f in (lambda: linattn_lm.Attention.apply(x, x * x, x, a)[0],
              lambda: recurrent_lm.TokenLoss.apply(x * x, target),
              lambda: recurrent_lm.AddNorm.apply(x * x, None, one, zero)[0],
              lambda: recurrent_lm.Recurrence.apply(
                  x[0].flatten(1), -x[0].flatten(1).square(), cu)[0]):
        for g in (lambda y: y.sum(), lambda y: y.square().sum()):
            with pytest.raises(RuntimeError, match="second derivative"):
                dx, = torch.autograd.grad(g(f()), x, create_graph=True)
                torch.autograd.grad(dx.square().sum(), x)
