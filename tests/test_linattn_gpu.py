"""Linear attention with a decay for each head (forward, backward, single
token) on the GPU against the fp64 oracle."""
import math

import numpy as np
import pytest
import torch

from linear_attention_delta_gb300 import kla
from oracle import mixer

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
U32, U16 = mixer.U32, mixer.U16


def decays(H):
    """From 1 (no decay) to a token's worth of memory."""
    if H == 1:
        return torch.tensor([-0.03])
    a = -torch.exp2(-torch.linspace(0.0, 11.0, H))
    a[-1] = 0.0
    return a


def heads(gen, B, T, H, d, dtype, layout="bthd"):
    """[B, T, H, d] in a layout: contiguous, a slice of something wider in
    every axis, heads outside tokens, or the fused slice of a projection."""
    shape = {"bthd": (B, T, H, d), "wide": (B, T + 3, H + 1, d + 8),
             "bhtd": (B, H, T, d), "fused": (B, T, 3, H, d)}[layout]
    x = (torch.randn(shape, generator=gen) * d ** -0.25).to(dtype).cuda()
    if layout == "wide":
        return x[:, 2:T + 2, :H, 8:]
    if layout == "bhtd":
        return x.transpose(1, 2)
    return x[:, :, 1] if layout == "fused" else x


def make(B, T, H, dk, dv, dtype, state=True, layout="bthd", seed=0):
    gen = torch.Generator().manual_seed(seed + T + 7 * dk)
    mk = lambda d: heads(gen, B, T, H, d, dtype, layout)  # noqa: E731
    S = lambda: torch.randn(B, H, dk, dv, generator=gen).cuda()  # noqa: E731
    return dict(q=mk(dk), k=mk(dk), v=mk(dv), log_decay=decays(H).cuda(),
                h0=S() if state else None), dict(
        o_grad=mk(dv), hT_grad=S() if state else None)


def mag(t):
    return None if t is None else np.abs(mixer.f64(t))


def slack(T, dk, dv):
    """Roundings of 32 bits that a term of a sum of the chunked pass meets:
    the products' sums (width, chunk; a sum of n terms rounds n times), the
    state's two roundings a chunk of at least 32, the part states' sums, the
    powers of the decays (the exponent's rounding counts up to 104 times
    before the power itself leaves the range; exp to 2 units), the three parts
    a weighted value is split into."""
    return (max(dk, dv) + 2 * 128 + 2 * T / 32 + 32 + 104 + 16) * U32


def near(got, want, bound):
    got, bound = mixer.f64(got), bound + 1e-36
    assert got.shape == want.shape
    assert np.isfinite(got).all()
    over = (np.abs(got - want) / bound).max() if got.size else 0.0
    assert over <= 1.0, over


def out_bound(size, want, dtype, slack):
    """Half a step of the output's own rounding and, with 16-bit inputs, of
    the scores' or of the state's on their way into a product."""
    if dtype == F32:
        return slack * size
    return (U16 + 2 * slack) * size + U16 * np.abs(want)


def check_fwd(x, o, hT):
    B, T, H, dk = x["q"].shape
    dv = x["v"].shape[-1]
    want_o, want_h = mixer.la_fwd(**x)
    size_o, size_h = mixer.la_fwd(*(mag(x[n]) for n in "qkv"),
                                  x["log_decay"], mag(x["h0"]))
    s = slack(T, dk, dv)
    near(o, want_o, out_bound(size_o, want_o, x["q"].dtype, s))
    if hT is not None:
        near(hT, want_h, s * size_h)


def check_bwd(x, y, g):
    B, T, H, dk = x["q"].shape
    dv = x["v"].shape[-1]
    want = mixer.la_bwd(**x, **y)
    size = mixer.la_bwd(*(mag(x[n]) for n in "qkv"), x["log_decay"],
                        mag(y["o_grad"]), mag(y["hT_grad"]), mag(x["h0"]))
    s = slack(T, dk, dv)
    for n, w, m in zip(("q_grad", "k_grad", "v_grad"), want, size):
        assert g[n].dtype == x["q"].dtype and g[n].is_contiguous()
        near(g[n], w, out_bound(m, w, x["q"].dtype, s))
    if g["h0_grad"] is not None:
        near(g["h0_grad"], want[3], s * size[3])


# lengths around the chunks (32, 64, 128 tokens) and beyond a sequence's cut
LENGTHS = [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 257, 640, 1025]
WIDTHS = [(64, 64), (128, 128), (128, 64), (64, 128), (16, 16), (72, 40),
          (8, 120), (1, 1), (17, 33), (96, 129), (200, 56), (256, 256),
          (130, 65)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", LENGTHS)
def test_lengths(T, dtype):
    for d in (64, 128):
        x, y = make(2, T, 3, d, d, dtype)
        check_fwd(x, *kla.linattn_fwd(**x))
        check_bwd(x, y, kla.linattn_bwd(**x, **y))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk,dv", WIDTHS)
def test_widths(dk, dv, dtype):
    for state in (True, False):
        x, y = make(1, 150, 2, dk, dv, dtype, state)
        check_fwd(x, *kla.linattn_fwd(**x))
        check_bwd(x, y, kla.linattn_bwd(**x, **y))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("layout", ["wide", "bhtd", "fused"])
@pytest.mark.parametrize("d", [64, 128, 24])
def test_strides(layout, d, dtype):
    x, y = make(2, 133, 3, d, d, dtype, layout=layout)
    check_fwd(x, *kla.linattn_fwd(**x))
    check_bwd(x, y, kla.linattn_bwd(**x, **y))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_unaligned_and_repeated(dtype):
    """Rows that start at any element; one query for all heads, one key for
    all tokens (stride 0)."""
    B, T, H, d = 2, 70, 3, 64
    x, y = make(B, T, H, d, d, dtype)
    flat = torch.randn(B * T * H * (d + 3) + 1).to(dtype).cuda()
    x["q"] = flat[1:].view(B, T, H, d + 3)[..., :d]
    y["o_grad"] = flat[1:].view(B, T, H, d + 3)[..., 2:d + 2]
    check_fwd(x, *kla.linattn_fwd(**x))
    check_bwd(x, y, kla.linattn_bwd(**x, **y))
    x, y = make(B, T, H, d, d, dtype)
    x["q"] = x["q"][:, :, :1].expand(B, T, H, d)
    x["k"] = x["k"][:, :1].expand(B, T, H, d)
    x["v"] = x["v"][:1].expand(B, T, H, d)
    check_fwd(x, *kla.linattn_fwd(**x))
    check_bwd(x, y, kla.linattn_bwd(**x, **y))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T,H,d", [(1, 4099, 1, 128), (1, 2500, 3, 64),
                                     (2, 1537, 4, 128), (1, 6000, 2, 40)])
def test_long_sequences_in_parts(B, T, H, d, dtype):
    x, y = make(B, T, H, d, d, dtype)
    check_fwd(x, *kla.linattn_fwd(**x))
    check_bwd(x, y, kla.linattn_bwd(**x, **y))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [40, 3000])
def test_extreme_decays(T, dtype):
    """Forgetting at once, within a token, and growth within the range."""
    x, y = make(1, T, 5, 64, 64, dtype)
    x["log_decay"] = torch.tensor(
        [-math.inf, -200.0, -30.0, -1e-6, 10.0 / T]).cuda()
    check_fwd(x, *kla.linattn_fwd(**x))
    check_bwd(x, y, kla.linattn_bwd(**x, **y))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("a", [-0.65, -0.74, -0.76, -0.92, -1.5])
@pytest.mark.parametrize("scale,name", [(1e-14, "v"), (1e8, "qk")])
def test_range_of_the_decays_factors(scale, name, a, dtype):
    """Small values and states, large scores: a chunk's decays reach e^190,
    and no factor of theirs may take a 16-bit number out of its digits (the
    bounds are relative to the values)."""
    for d in (64, 128):
        x, y = make(1, 260, 2, d, d, dtype)
        x["log_decay"] = torch.full((2,), a).cuda()
        if name == "v":
            x["v"], x["h0"] = x["v"] * scale, x["h0"] * scale
        else:
            x["q"], x["k"] = x["q"] * scale, x["k"] * scale
        check_fwd(x, *kla.linattn_fwd(**x))
        check_bwd(x, y, kla.linattn_bwd(**x, **y))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [100, 4200])
def test_state_replaced_in_place(T, dtype):
    x, _ = make(1, T, 2, 128, 128, dtype)
    o, hT = kla.linattn_fwd(**x)
    h = x["h0"].clone()
    o2, h2 = kla.linattn_fwd(**{**x, "h0": h}, hT=h)
    assert h2 is h and torch.equal(h, hT) and torch.equal(o2, o)
    o3, none = kla.linattn_fwd(**x, want_state=False, o=torch.empty_like(o))
    assert none is None and torch.equal(o3, o)


@pytest.mark.parametrize("T", [90, 4200])
def test_handed_over_between_calls(T):
    """A prompt in two calls and the tokens one by one end in the same state
    as at once."""
    x, _ = make(2, T, 3, 64, 128, F32)
    cut = T - 40
    part = lambda a, b: {n: x[n][:, a:b] for n in "qkv"}  # noqa: E731
    w = dict(log_decay=x["log_decay"])
    o1, S = kla.linattn_fwd(**part(0, cut), **w, h0=x["h0"])
    o2, S = kla.linattn_fwd(**part(cut, T - 5), **w, h0=S)
    outs = [o1, o2]
    for t in range(T - 5, T):
        outs.append(kla.linattn_step(*(x[n][:, t] for n in "qkv"), **w, S=S)
                    [:, None])
    check_fwd(x, torch.cat(outs, 1), S)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_no_tokens_and_no_heads(dtype):
    x, y = make(2, 0, 3, 64, 64, dtype)
    o, hT = kla.linattn_fwd(**x)
    assert o.shape == (2, 0, 3, 64) and torch.equal(hT, x["h0"])
    g = kla.linattn_bwd(**x, **y)
    assert torch.equal(g["h0_grad"], y["hT_grad"])
    x, y = make(2, 0, 3, 64, 64, dtype, state=False)
    assert (kla.linattn_fwd(**x)[1] == 0).all()
    assert (kla.linattn_bwd(**x, **y)["h0_grad"] == 0).all()
    for B, H in ((0, 3), (2, 0)):
        x = dict(q=torch.empty(B, 5, H, 64, dtype=dtype, device="cuda"),
                 log_decay=torch.zeros(H, device="cuda"))
        x["k"] = x["v"] = x["q"]
        assert kla.linattn_fwd(**x)[0].shape == (B, 5, H, 64)
        assert kla.linattn_bwd(**x, o_grad=x["q"])["q_grad"].numel() == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("name", ["q", "k", "v"])
def test_what_is_not_finite_reaches_no_earlier_token(name, bad, dtype):
    """Nor another sequence or head; later tokens' outputs are not finite."""
    for T, at in ((200, 77), (200, 128), (1100, 700)):
        x, y = make(2, T, 2, 64, 64, dtype)
        x["log_decay"] = torch.tensor([-0.01, 0.0]).cuda()
        want, _ = kla.linattn_fwd(**x)
        x[name][1, at, 0, 5] = bad
        o, hT = kla.linattn_fwd(**x)
        fine = torch.ones(2, T, 2, dtype=torch.bool, device="cuda")
        fine[1, at:, 0] = False
        assert torch.equal(o[fine], want[fine])
        rest = o[1, at + 1:, 0]
        if name == "q":
            assert torch.equal(rest, want[1, at + 1:, 0])
            assert not torch.isfinite(o[1, at, 0]).any()
        elif name == "v":
            keep = torch.arange(64, device="cuda") != 5
            assert not torch.isfinite(o[1, at:, 0, 5]).any()
            assert not torch.isfinite(hT[1, 0, :, 5]).any()
            assert torch.equal(o[1, :, 0][:, keep], want[1, :, 0][:, keep])
        else:
            assert not torch.isfinite(o[1, at:, 0]).any()
            assert not torch.isfinite(hT[1, 0, 5]).any()
        assert torch.isfinite(hT[0]).all() and torch.isfinite(hT[1, 1]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradients_of_padding_stay_there(dtype):
    """NaN in o_grad behind a sequence's end reaches no q_grad before it, and
    NaN in v before a token no v_grad after it."""
    T, cut = 150, 90
    x, y = make(1, T, 2, 64, 64, dtype)
    want = kla.linattn_bwd(**x, **y)
    y["o_grad"][:, cut:] = math.nan
    g = kla.linattn_bwd(**x, **y)
    assert torch.equal(g["q_grad"][:, :cut], want["q_grad"][:, :cut])
    x, y = make(1, T, 2, 64, 64, dtype)
    x["q"][:, :cut] = math.nan
    g = kla.linattn_bwd(**x, **y)
    for n in ("k_grad", "v_grad"):
        assert torch.equal(g[n][:, cut:], want[n][:, cut:])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,H,dk,dv", [
    (1, 1, 128, 128), (3, 5, 64, 64), (40, 16, 128, 128), (2, 3, 72, 40),
    (2, 2, 17, 33), (1, 4, 256, 256), (5, 2, 1, 1), (2, 3, 128, 36),
    (350, 1, 16, 200)])
def test_step(N, H, dk, dv, dtype):
    x, _ = make(N, 2, H, dk, dv, dtype)
    a, S = x["log_decay"], x["h0"].clone()
    for layout in ("plain", "strided"):
        q, k, v = (x[n][:, 0].contiguous() if layout == "plain"
                   else x[n][:, 1] for n in "qkv")
        S0 = S.clone()
        o = kla.linattn_step(q, k, v, a, S)
        want_o, want_S = mixer.la_fwd(q[:, None], k[:, None], v[:, None], a,
                                      S0)
        size_o, size_S = mixer.la_fwd(mag(q[:, None]), mag(k[:, None]),
                                      mag(v[:, None]), a, mag(S0))
        # exp to 2 units, a product and two sums; the read-out's sum
        near(S, want_S, 6 * U32 * size_S)
        bound = (dk + 8) * U32 * size_o[:, 0]
        if dtype == BF16:
            bound = bound + U16 * np.abs(want_o[:, 0])
        near(o, want_o[:, 0], bound)


def test_step_unaligned_state():
    N, H, d = 3, 2, 64
    x, _ = make(N, 1, H, d, d, F32)
    S = torch.empty(N * H * d * d + 1, device="cuda")[1:].view(N, H, d, d)
    S.copy_(x["h0"])
    o = kla.linattn_step(*(x[n][:, 0] for n in "qkv"), x["log_decay"], S)
    want_o, want_S = mixer.la_fwd(**x)
    np.testing.assert_allclose(mixer.f64(S), want_S, rtol=1e-5, atol=1e-5)
    np.testing.assert_allclose(mixer.f64(o), want_o[:, 0], rtol=1e-4,
                               atol=1e-4)


def test_other_stream_and_own_workspace():
    x, y = make(1, 4200, 2, 128, 128, BF16)
    want, h = kla.linattn_fwd(**x)
    grads = kla.linattn_bwd(**x, **y)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for back in (False, True):
        n = kla.linattn_workspace_size(1, 4200, 2, 128, 128, BF16, back)
        ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        s.wait_stream(torch.cuda.current_stream())
        if back:
            g = kla.linattn_bwd(**x, **y, workspace=ws, stream=s)
        else:
            o, hT = kla.linattn_fwd(**x, workspace=ws, stream=s)
        s.synchronize()
    assert torch.equal(o, want) and torch.equal(hT, h)
    assert all(torch.equal(g[n], grads[n]) for n in g)
    with pytest.raises(kla.KlaError):
        kla.linattn_fwd(**x, workspace=ws[:64])


def test_same_bits_and_graph_replay():
    x, y = make(1, 4200, 2, 128, 128, BF16)
    S0 = x["h0"].clone()

    def run():
        S = S0.clone()
        o, _ = kla.linattn_fwd(**x, hT=None)
        g = kla.linattn_bwd(**x, **y)
        o1 = kla.linattn_step(*(x[n][:, 0] for n in "qkv"), x["log_decay"], S)
        return [o, *g.values(), o1, S]

    want = run()
    assert all(torch.equal(a, b) for a, b in zip(run(), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = []
    for g in graphs:                 # each graph has workspaces of its own
        with torch.cuda.graph(g):
            outs.append(run())
    for out in outs:
        for t in out:
            t.zero_()
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for out in outs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 72, 200, 33])
def test_outputs_at_any_alignment(d, dtype):
    """o one element off every wider piece it is written in."""
    x, _ = make(2, 130, 2, d, d, dtype)
    room = torch.full((2 * 130 * 2 * d + 2,), 7.0, dtype=dtype).cuda()
    o = room[1:-1].view(2, 130, 2, d)
    got, hT = kla.linattn_fwd(**x, o=o)
    assert got is o
    check_fwd(x, o, hT)
    assert room[0] == 7 and room[-1] == 7
    assert torch.equal(o, kla.linattn_fwd(**x)[0])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_two_streams_at_once(dtype):
    """Calls in flight beside one another, each with parts of its own."""
    xs = [make(1, 2500, 2, 64, 64, dtype, seed=i) for i in range(2)]
    alone = [(kla.linattn_fwd(**x), kla.linattn_bwd(**x, **y)) for x, y in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i, (x, y) in enumerate(xs):
            with torch.cuda.stream(streams[i]):
                got[i].append((kla.linattn_fwd(**x),
                               kla.linattn_bwd(**x, **y)))
    torch.cuda.synchronize()
    for i in range(2):
        for fwd, bwd in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(fwd, alone[i][0]))
            assert all(torch.equal(bwd[n], alone[i][1][n]) for n in bwd)


@pytest.mark.parametrize("d,dtype", [(64, BF16), (20, F32)])
def test_offsets_beyond_32_bits(d, dtype):
    """A second sequence that starts 2^31 elements on."""
    T, H = 130, 2
    far = 2 ** 31 + 64
    buf = torch.empty(far + T * H * d, dtype=dtype, device="cuda")
    x, y = make(2, T, H, d, d, dtype)
    q = buf.as_strided((2, T, H, d), (far, H * d, d, 1))
    q.copy_(x["q"])
    x["q"] = q
    check_fwd(x, *kla.linattn_fwd(**x))
    check_bwd(x, y, kla.linattn_bwd(**x, **y))


def test_binding_refuses():
    x, y = make(1, 8, 2, 16, 16, F32)
    S = x["h0"]
    with pytest.raises(ValueError):
        kla.linattn_fwd(**{**x, "k": x["k"][:, :4]})
    with pytest.raises(ValueError):
        kla.linattn_fwd(**{**x, "h0": S[:, :1]})
    with pytest.raises(ValueError):
        kla.linattn_fwd(**{**x, "q": x["q"].transpose(-1, -2)})
    with pytest.raises(TypeError):
        kla.linattn_fwd(**{**x, "v": x["v"].half()})
    with pytest.raises(TypeError):
        kla.linattn_fwd(**{**x, "v": x["v"].bfloat16()})
    with pytest.raises(ValueError):
        kla.linattn_fwd(**{**x, "log_decay": x["log_decay"][:1]})
    with pytest.raises(TypeError):
        kla.linattn_fwd(**{**x, "log_decay": x["log_decay"].double()})
    with pytest.raises(TypeError):
        kla.linattn_bwd(**x, o_grad=y["o_grad"].cpu())
    with pytest.raises(ValueError):
        kla.linattn_step(*(x[n] for n in "qkv"), x["log_decay"], S)
    with pytest.raises(ValueError):
        kla.linattn_step(*(x[n][:, 0] for n in "qkv"), x["log_decay"],
                         S.transpose(2, 3))
    big = torch.zeros(1, 2, 1, 257, device="cuda")
    with pytest.raises(kla.KlaError):
        kla.linattn_fwd(big, big, big, torch.zeros(1, device="cuda"))


def test_bounded_wait_runs_out_and_is_reported():
    assert kla.device_status() == 0
    assert kla.selftest_linattn_timeout() == 0
    assert kla.device_status() == -4
    assert kla.device_status() == 0
    x, _ = make(1, 200, 2, 64, 64, BF16)
    check_fwd(x, *kla.linattn_fwd(**x))
