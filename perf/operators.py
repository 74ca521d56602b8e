"""Measured cases of the token-mixer operators: layer norm (forward, backward)
and the gated linear recurrence (forward, backward, single token).

    layer norm   s = x + r (r optional),  m = mean(s),  v = mean((s - m)^2),
                 y = (s - m) / sqrt(v + eps) * w + b
    recurrence   h_t = exp(log_alpha_t) h_{t-1} + x_t  per channel, o_t = h_t,
                 each sequence from its own h0, packed sequences back to back

``run`` computes a case with the library when ``own`` is true, else from the
formulas with elementary torch operations in 32 bits, rounded once at the end.
``exact`` computes it in 64 bits, written apart from the plain form.
"""
import math
import random

import torch

own = False

F32, BF16 = "f32", "bf16"
TYPES = {F32: torch.float32, BF16: torch.bfloat16}
EPS = 1e-5
MOST = 1 << 25          # elements of the largest drawn case


def _ln(name, rows, D, dtype, wtype, back=False, residual=False, wide=False):
    return dict(name=name, op="ln_bwd" if back else "ln_fwd", rows=rows, D=D,
                dtype=dtype, wtype=wtype, residual=residual, wide=wide)


def _glr(name, B, T, D, dtype, gtype, op="glr_fwd", packed=0, state=True,
         wide=False):
    return dict(name=name, op=op, B=B, T=T, D=D, dtype=dtype, gtype=gtype,
                packed=packed, state=state, wide=wide)


def listed():
    return [
        # one new token of a 2048-wide model: residual add and norm, latency
        _ln("ln_fwd_token", 1, 2048, BF16, BF16, residual=True),
        # the training forward of a 2048-wide layer (batch 4, 4096 tokens)
        _ln("ln_fwd_layer1b", 16384, 2048, BF16, BF16, residual=True),
        # its backward, with the gradient that arrives through the residual
        _ln("ln_bwd_layer1b", 16384, 2048, BF16, BF16, back=True,
            residual=True),
        # odd width and row count, fp32: no vector loads line up
        _ln("ln_fwd_odd", 4099, 1001, F32, F32),
        # few, wide rows: the norm of a fused projection, x a slice of it
        _ln("ln_bwd_wide", 1023, 8200, BF16, F32, back=True, wide=True),
        # one decode step of 256 sequences
        _glr("glr_step_256", 256, 1, 2048, BF16, F32, op="glr_step"),
        # a short prompt: latency
        _glr("glr_fwd_prompt33", 1, 33, 2048, BF16, F32),
        # the training forward of a 2048-wide layer, gates in fp32
        _glr("glr_fwd_layer1b", 4, 4096, 2048, BF16, F32),
        # its backward
        _glr("glr_bwd_layer1b", 4, 4096, 2048, BF16, F32, op="glr_bwd"),
        # one long sequence: few channels to spread over the card
        _glr("glr_fwd_65k", 1, 65536, 2048, BF16, BF16),
        # packed prompts of ragged lengths (empty ones and single tokens
        # among them), x and the gate slices of one projection's output
        _glr("glr_fwd_packed", 1, 16411, 1024, BF16, BF16, packed=24,
             wide=True),
        # packed training batch, odd width, fp32
        _glr("glr_bwd_packed_odd", 1, 8191, 1001, F32, F32, op="glr_bwd",
             packed=9),
    ]


def _size(rng, lo, hi):
    """A whole number in [lo, hi], uniform in its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo),
                                                    math.log(hi + 1))))))


def draw(rng):
    dtype = rng.choice([BF16, BF16, F32])
    pick = rng.random()
    if pick < 0.45:
        D = _size(rng, 64, 16384)
        if rng.random() < 0.5:
            D = max(64, D // 64 * 64)
        rows = _size(rng, 1, min(32768, MOST // D))
        c = _ln("", rows, D, dtype, rng.choice([dtype, F32]),
                back=rng.random() < 0.5, residual=rng.random() < 0.5,
                wide=rng.random() < 0.25)
    elif pick < 0.55:
        c = _glr("", _size(rng, 1, 1024), 1, _size(rng, 64, 8192), dtype,
                 rng.choice([dtype, F32]), op="glr_step",
                 wide=rng.random() < 0.25)
    else:
        D = _size(rng, 64, 8192)
        if rng.random() < 0.5:
            D = max(64, D // 64 * 64)
        T = _size(rng, 2, min(65536, MOST // D))
        packed = rng.choice([0, 0, _size(rng, 2, 64)])
        B = 1 if packed else _size(rng, 1, max(1, min(64, MOST // (D * T))))
        c = _glr("", B, T, D, dtype, rng.choice([dtype, F32]),
                 op=rng.choice(["glr_fwd", "glr_bwd"]), packed=packed,
                 state=rng.random() < 0.5, wide=rng.random() < 0.25)
    del c["name"]
    return c


# --- inputs ----------------------------------------------------------------

def _rows(g, rows, D, dtype, wide, scale=1.0, shift=0.0):
    """[rows, D] normal values, a slice of a 2 D wide tensor when ``wide``."""
    x = torch.randn(rows, D, device="cuda", generator=g) * scale + shift
    if not wide:
        return x.to(dtype)
    out = torch.zeros(rows, 2 * D, device="cuda", dtype=dtype)
    out[:, D:] = x
    return out[:, D:]


def _lengths(total, n, rng):
    """n lengths that sum to total; about one in six is empty and one in six
    a single token."""
    w = [rng.choice([0.0, -1.0] + 4 * [rng.uniform(0.05, 1.0)])
         for _ in range(n)]
    if max(w) <= 0.0:
        w[0] = 1.0
    left = max(0, total - sum(v < 0 for v in w))
    s = sum(v for v in w if v > 0)
    lens = [min(1, total) if v < 0 else int(left * v / s) for v in w]
    big = max(range(n), key=lambda i: lens[i])
    lens[big] += total - sum(lens)
    return lens


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = TYPES[case["dtype"]]
    D = case["D"]
    st = dict(case=case)
    if case["op"].startswith("ln"):
        M, wt = case["rows"], TYPES[case["wtype"]]
        # a residual stream: rows of different scale and offset, a few
        # channels far larger than the rest
        scale = torch.exp(torch.randn(M, 1, device="cuda", generator=g))
        chan = torch.where(torch.rand(1, D, device="cuda", generator=g) <
                           0.01, 8.0, 1.0)
        st["x"] = _rows(g, M, D, dt, case["wide"], scale * chan, 0.1 * scale)
        st["weight"] = (1 + 0.1 * torch.randn(D, device="cuda",
                                              generator=g)).to(wt)
        st["bias"] = (0.1 * torch.randn(D, device="cuda", generator=g)).to(wt)
        if case["op"] == "ln_fwd":
            st["residual"] = _rows(g, M, D, dt, False) \
                if case["residual"] else None
        else:
            st["y_grad"] = _rows(g, M, D, dt, False, 0.1)
            st["residual_grad"] = _rows(g, M, D, dt, False, 0.1) \
                if case["residual"] else None
            x = st["x"].float()
            m = x.mean(1)
            v = (x - m[:, None]).square().mean(1)
            st["mean"], st["rstd"] = m, 1 / torch.sqrt(v + EPS)
        return st
    B, T = case["B"], case["T"]
    rows, gt = B * T, TYPES[case["gtype"]]
    # decays from a few tokens to about a thousand, modulated per token
    rate = torch.exp(torch.empty(1, D, device="cuda").uniform_(
        math.log(1e-3), 0.0, generator=g))
    gate = torch.sigmoid(torch.randn(rows, D, device="cuda", generator=g))
    la = (-2.0 * rate * gate).to(gt)
    if case["op"] == "glr_step":
        st["x"] = _rows(g, B, D, dt, case["wide"])
        st["log_alpha"] = la
        st["S"] = torch.randn(B, D, device="cuda", generator=g)
        return st
    N = case["packed"] or B
    lens = _lengths(rows, N, random.Random(seed)) if case["packed"] \
        else [T] * B
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    st["longest"] = max(lens)
    st["cu"] = torch.tensor(cu, device="cuda", dtype=torch.int32)
    st["h0"] = torch.randn(N, D, device="cuda", generator=g) \
        if case["state"] else None
    x = _rows(g, rows, D, dt, False)
    if case["op"] == "glr_bwd":
        o, hT = _glr_plain(x, la, st["h0"], st["cu"], st["longest"])
        st["o"] = o.to(dt)
        st["o_grad"] = _rows(g, rows, D, dt, case["wide"])
        st["hT_grad"] = torch.randn(N, D, device="cuda", generator=g) \
            if case["state"] else None
    elif case["wide"] and gt == dt:
        both = torch.cat([x, la], 1)
        x, la = both[:, :D], both[:, D:]
    if case["op"] == "glr_fwd":
        st["x"] = x
    st["log_alpha"] = la
    if not case["packed"]:
        for k in ("x", "log_alpha", "o", "o_grad"):
            if k in st:
                st[k] = st[k].unflatten(0, (B, T))
    return st


# --- one pass --------------------------------------------------------------

def run(st):
    case = st["case"]
    return (_run_own if own else _run_plain)(st, case, case["op"])


def _run_own(st, case, op):
    from linear_attention_delta_gb300 import kla
    if op == "ln_fwd":
        y, s, mean, rstd = kla.layernorm_fwd(
            st["x"], st["weight"], st["bias"], eps=EPS,
            residual=st["residual"])
        return dict(y=y, mean=mean, rstd=rstd,
                    **({} if s is None else dict(sum=s)))
    if op == "ln_bwd":
        return kla.layernorm_bwd(st["y_grad"], st["x"], st["weight"],
                                 st["mean"], st["rstd"],
                                 sum_grad=st["residual_grad"])
    if op == "glr_step":
        o = kla.glr_step(st["x"], st["log_alpha"], st["S"])
        return dict(o=o, S=st["S"])
    cu = st["cu"] if case["packed"] else None
    if op == "glr_fwd":
        o, hT = kla.glr_fwd(st["x"], st["log_alpha"], st["h0"],
                            cu_seqlens=cu)
        return dict(o=o, hT=hT)
    out = kla.glr_bwd(st["o"], st["log_alpha"], st["o_grad"], st["hT_grad"],
                      h0=st["h0"], cu_seqlens=cu,
                      want_h0_grad=case["state"])
    return {k: v for k, v in out.items() if v is not None}


def _run_plain(st, case, op):
    if op == "ln_fwd":
        x, dt = st["x"].float(), st["x"].dtype
        if st["residual"] is not None:
            x = x + st["residual"].float()
        D = x.shape[1]
        mean = x.sum(1) / D
        xc = x - mean[:, None]
        rstd = 1 / torch.sqrt((xc * xc).sum(1) / D + EPS)
        y = xc * rstd[:, None] * st["weight"].float() + st["bias"].float()
        out = dict(y=y.to(dt), mean=mean, rstd=rstd)
        if st["residual"] is not None:
            out["sum"] = x.to(dt)
        return out
    if op == "ln_bwd":
        dt, wt = st["x"].dtype, st["weight"].dtype
        dy, rstd = st["y_grad"].float(), st["rstd"][:, None]
        xh = (st["x"].float() - st["mean"][:, None]) * rstd
        D = xh.shape[1]
        wdy = dy * st["weight"].float()
        c1 = (wdy * xh).sum(1, keepdim=True) / D
        c2 = wdy.sum(1, keepdim=True) / D
        dx = rstd * (wdy - c2 - xh * c1)
        if st["residual_grad"] is not None:
            dx = dx + st["residual_grad"].float()
        return dict(x_grad=dx.to(dt), weight_grad=(dy * xh).sum(0).to(wt),
                    bias_grad=dy.sum(0).to(wt))
    if op == "glr_step":
        S = torch.exp(st["log_alpha"].float()) * st["S"] + st["x"].float()
        st["S"].copy_(S)
        return dict(o=S.to(st["x"].dtype), S=st["S"])
    shape = st["log_alpha"].shape
    la = st["log_alpha"].flatten(0, -2)
    if op == "glr_fwd":
        o, hT = _glr_plain(st["x"].flatten(0, -2), la, st["h0"], st["cu"],
                           st["longest"])
        return dict(o=o.to(st["x"].dtype).view(shape), hT=hT)
    dx, dla, dh0 = _glr_grad_plain(
        st["o"].flatten(0, -2), la, st["o_grad"].flatten(0, -2),
        st["hT_grad"], st["h0"], st["cu"], st["longest"])
    out = dict(x_grad=dx.to(st["o"].dtype).view(shape),
               log_alpha_grad=dla.to(la.dtype).view(shape))
    if case["state"]:
        out["h0_grad"] = dh0
    return out


def _scan(a, b, longest):
    """h_t = a_t h_{t-1} + b_t along the rows by doubling: after each round a
    row holds the map of twice as many steps."""
    s = 1
    while s < longest:
        b = torch.cat([b[:s], a[s:] * b[:-s] + b[s:]])
        a = torch.cat([a[:s], a[s:] * a[:-s]])
        s *= 2
    return b


def _starts(cu, rows):
    """1 at each row that begins a sequence ([rows, 1]); which sequences hold
    rows ([N, 1])."""
    first = torch.zeros(rows + 1, 1, device=cu.device)
    first.index_fill_(0, cu[:-1].long(), 1.0)
    return first[:rows], (cu[1:] > cu[:-1])[:, None]


def _spread(v, at, some, rows):
    """Rows of v at the row indexes ``at`` (empty sequences left out)."""
    out = torch.zeros(rows + 1, v.shape[1], device=v.device)
    return out.index_add_(0, at, torch.where(some, v, 0.0))[:rows]


def _glr_plain(x, la, h0, cu, longest):
    rows, D = x.shape
    a, x = torch.exp(la.float()), x.float()
    first, some = _starts(cu, rows)
    if h0 is None:
        h0 = torch.zeros(cu.numel() - 1, D, device=x.device)
    x = x + a * _spread(h0, cu[:-1].long(), some, rows)
    h = _scan(a * (1 - first), x, longest)
    hT = torch.where(some, h[(cu[1:].long() - 1).clamp(min=0)], h0)
    return h, hT


def _glr_grad_plain(o, la, do, dhT, h0, cu, longest):
    rows, D = o.shape
    a, h, do = torch.exp(la.float()), o.float(), do.float()
    first, some = _starts(cu, rows)
    zero = torch.zeros(cu.numel() - 1, D, device=o.device)
    h0, dhT = zero if h0 is None else h0, zero if dhT is None else dhT
    start, end = cu[:-1].long(), (cu[1:].long() - 1).clamp(min=0)
    g = do + _spread(dhT, end, some, rows)
    nxt = torch.cat([(a * (1 - first))[1:], torch.zeros_like(a[:1])])
    g = _scan(nxt.flip(0), g.flip(0), longest).flip(0)
    prev = torch.cat([torch.zeros_like(h[:1]), h[:-1]]) * (1 - first) + \
        _spread(h0, start, some, rows)
    ag = a * g
    dh0 = torch.where(some, ag[start.clamp(max=rows - 1)], dhT)
    return g, ag * prev, dh0


# --- the work a case cannot do without -------------------------------------

def work(case):
    e = 2 if case["dtype"] == BF16 else 4
    D = case["D"]
    if case["op"].startswith("ln"):
        M, w = case["rows"], 2 if case["wtype"] == BF16 else 4
        n, r = M * D, 1 if case["residual"] else 0
        if case["op"] == "ln_fwd":
            return dict(bytes=n * e * (2 + 2 * r) + 2 * D * w + 8 * M,
                        flops=(8 + r) * n)
        return dict(bytes=n * e * (3 + r) + 3 * D * w + 8 * M,
                    flops=(16 + r) * n)
    ge = 2 if case["gtype"] == BF16 else 4
    n = case["B"] * case["T"] * D
    N = case["packed"] or case["B"]
    if case["op"] == "glr_step":
        return dict(bytes=n * (2 * e + ge + 8), flops=3 * n)
    s = 8 * N * D if case["state"] else 4 * N * D
    if case["op"] == "glr_fwd":
        return dict(bytes=n * (2 * e + ge) + s, flops=3 * n)
    s = 12 * N * D if case["state"] else 0
    return dict(bytes=n * (3 * e + 2 * ge) + s, flops=5 * n)


# --- the definition in 64 bits ---------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    f = {k: v.double() for k, v in st.items()
         if isinstance(v, torch.Tensor) and v.is_floating_point()}
    op = case["op"]
    if op.startswith("ln"):
        x = f["x"] + f["residual"] if "residual" in f else f["x"].clone()
        x.requires_grad_(op == "ln_bwd")
        w, b = (f[k].requires_grad_(op == "ln_bwd")
                for k in ("weight", "bias"))
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        y = (x - mean) * torch.rsqrt(var + EPS) * w + b
        if op == "ln_fwd":
            out = dict(y=y, mean=mean[:, 0], rstd=(var[:, 0] + EPS) ** -0.5)
            if "residual" in f:
                out["sum"] = x
            return out
        dx, dw, db = torch.autograd.grad(y, (x, w, b), f["y_grad"])
        if "residual_grad" in f:
            dx = dx + f["residual_grad"]
        return dict(x_grad=dx, weight_grad=dw, bias_grad=db)
    if op == "glr_step":
        S = torch.addcmul(f["x"], f["log_alpha"].exp(), f["S"])
        return dict(o=S, S=S)
    D, shape = case["D"], f["log_alpha"].shape
    alpha = f["log_alpha"].reshape(-1, D).exp()
    cu = st["cu"].tolist()
    N = len(cu) - 1
    h0 = f.get("h0", torch.zeros(N, D, device="cuda", dtype=torch.float64))
    if not case["packed"]:
        # all sequences step together: [T, B, D]
        alpha = alpha.view(shape).transpose(0, 1).contiguous()
        flat = [(0, case["T"], alpha)]
    else:
        flat = [(i, j, alpha[i:j, None]) for i, j in zip(cu, cu[1:])]

    def steps(v):
        v = v.reshape(-1, D)
        if not case["packed"]:
            return [v.view(shape).transpose(0, 1).contiguous()]
        return [v[i:j, None] for i, j, _ in flat]

    def rows(v):
        v = torch.cat(v)
        return v.transpose(0, 1).reshape(shape) if not case["packed"] \
            else v.reshape(shape)

    states = [h0] if not case["packed"] else list(h0[:, None])
    if op == "glr_fwd":
        os, last = [], []
        for x, (_, _, a), h in zip(steps(f["x"]), flat, states):
            o = torch.empty_like(x)
            for t in range(x.shape[0]):
                h = torch.addcmul(x[t], a[t], h, out=o[t])
            os.append(o)
            last.append(h.reshape(-1, D))
        return dict(o=rows(os), hT=torch.cat(last))
    dhT = f.get("hT_grad", torch.zeros_like(h0))
    ends = [dhT] if not case["packed"] else list(dhT[:, None])
    gs, gla, g0 = [], [], []
    for do, o, (_, _, a), h, c in zip(steps(f["o_grad"]), steps(f["o"]),
                                      flat, states, ends):
        g, back = torch.empty_like(do), torch.empty_like(do)
        for t in range(do.shape[0] - 1, -1, -1):
            torch.add(do[t], c, out=g[t])
            c = torch.mul(a[t], g[t], out=back[t])
        gs.append(g)
        gla.append(back * torch.cat([h[None], o[:-1]])[:do.shape[0]])
        g0.append(c.reshape(-1, D))
    out = dict(x_grad=rows(gs), log_alpha_grad=rows(gla))
    if case["state"]:
        out["h0_grad"] = torch.cat(g0)
    return out
