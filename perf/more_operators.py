"""Measured cases of linear attention with a decay for each head (forward,
backward, single token) and of the log probabilities of given tokens (forward,
backward).

    linear attention    S_t = exp(a_h) S_{t-1} + k_t v_t^T,  o_t = S_t^T q_t
                        per sequence and head, from S_0 = h0
    log probabilities   z = scale * logits,  lse = log sum_j exp(z_j),
                        logp = z_token - lse,  entropy = -sum_j p_j log p_j,
                        the `top` largest z_j - lse and their ids

``run`` computes a case with the library when ``own`` is true, else from the
formulas with elementary torch operations in 32 bits (the decays' powers in
64), rounded once at the end.  ``exact`` computes it in 64 bits, written apart
from the plain form.
"""
import math

import torch

own = False

F32, BF16 = "f32", "bf16"
TYPES = {F32: torch.float32, BF16: torch.bfloat16}
MOST = 1 << 28          # elements of the largest drawn case


def _la(name, op, B, T, H, dk, dv, dtype, state=True, layout="bthd"):
    """layout: q, k, v as [B, T, H, d] of their own ("bthd"), slices of one
    projection's output ("fused") or heads outside tokens ("bhtd")."""
    return dict(name=name, op=op, B=B, T=T, H=H, dk=dk, dv=dv, dtype=dtype,
                state=state, layout=layout)


def _lp(name, op, N, V, dtype, top=0, scale=1.0, masked=False, pad=False,
        wide=False, entropy=True):
    """masked: a part of the vocabulary is -inf; pad: some rows have no
    token; wide: logits are a slice of a wider (padded) tensor; entropy: its
    gradient arrives too (backward)."""
    return dict(name=name, op=op, N=N, V=V, dtype=dtype, top=top, scale=scale,
                masked=masked, pad=pad, wide=wide, entropy=entropy)


def listed():
    return [
        # the prompt of a training-sized layer: batch 4, 4096 tokens, 16 heads
        _la("la_fwd_layer1b", "la_fwd", 4, 4096, 16, 128, 128, BF16),
        # one long prompt: few heads, the work has to be split along it
        _la("la_fwd_long", "la_fwd", 1, 65536, 16, 128, 128, BF16,
            state=False),
        # odd lengths and widths in fp32, slices of one projection
        _la("la_fwd_odd", "la_fwd", 3, 1001, 5, 72, 72, F32, layout="fused"),
        # the training backward of the layer above
        _la("la_bwd_layer1b", "la_bwd", 4, 4096, 16, 128, 128, BF16,
            state=False),
        # a backward of ragged length, narrower heads outside the tokens
        _la("la_bwd_ragged", "la_bwd", 2, 2049, 12, 64, 64, BF16,
            layout="bhtd"),
        # one token of one sequence: latency
        _la("la_step_one", "la_step", 1, 1, 16, 128, 128, BF16),
        # one token of 256 sequences, the decode batch of the layer
        _la("la_step_batch", "la_step", 256, 1, 16, 128, 128, BF16),
        # what one new token scored, with its alternatives: latency
        _lp("lp_fwd_token", "lp_fwd", 1, 32000, BF16, top=8),
        # a serving batch over a large vocabulary, 20 alternatives each,
        # part of the vocabulary masked, sampled at a temperature
        _lp("lp_fwd_top", "lp_fwd", 256, 131072, BF16, top=20, scale=1.25,
            masked=True),
        # the loss of a training batch: 2 x 4096 tokens
        _lp("lp_fwd_train", "lp_fwd", 8192, 32000, BF16, pad=True),
        # its gradient
        _lp("lp_bwd_train", "lp_bwd", 8192, 32000, BF16, pad=True,
            entropy=False),
        # odd vocabulary in fp32, a slice of a padded tensor, with entropy
        _lp("lp_bwd_odd", "lp_bwd", 1023, 10007, F32, scale=0.7, wide=True),
    ]


def _size(rng, lo, hi):
    """A whole number in [lo, hi], uniform in its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo),
                                                    math.log(hi + 1))))))


def _width(rng, dtype):
    """A head's width: mostly the usual ones, some odd."""
    if rng.random() < 0.6:
        return rng.choice([64, 128])
    return _size(rng, 8, 128) // 8 * 8 if dtype == BF16 else _size(rng, 8, 128)


def draw(rng):
    dtype = rng.choice([BF16, BF16, F32])
    pick = rng.random()
    if pick < 0.15:
        H = _size(rng, 1, 64)
        c = _la("", "la_step", _size(rng, 1, 4096 // H), 1, H,
                _width(rng, dtype), _width(rng, dtype), dtype)
    elif pick < 0.55:
        dk, dv = _width(rng, dtype), _width(rng, dtype)
        layout = rng.choice(["bthd", "fused", "bhtd"])
        if layout == "fused":
            dv = dk
        most = MOST // (4 if dtype == F32 else 1) // (dk + dv)
        T = _size(rng, 1, 65536)
        H = _size(rng, 1, min(64, most // (2 * T)))
        B = _size(rng, 1, max(1, min(32, most // (2 * T * H))))
        op = rng.choice(["la_fwd", "la_bwd"])
        if op == "la_bwd":
            T = max(1, T // 2)
        c = _la("", op, B, T, H, dk, dv, dtype, state=rng.random() < 0.5,
                layout=layout)
    else:
        V = _size(rng, 64, 131072)
        if rng.random() < 0.5:
            V = max(64, V // 64 * 64)
        N = _size(rng, 1, min(16384, MOST // 2 // V))
        op = rng.choice(["lp_fwd", "lp_bwd"])
        top = rng.choice([0, 1, 5, 20]) if N <= 512 and op == "lp_fwd" else 0
        c = _lp("", op, N, V, dtype, top=top,
                scale=rng.choice([1.0, 1.0, 0.7, 1.25]),
                masked=rng.random() < 0.25, pad=rng.random() < 0.5,
                wide=rng.random() < 0.25, entropy=rng.random() < 0.5)
    del c["name"]
    return c


# --- inputs ----------------------------------------------------------------

def _heads(g, case, d, n, scale=1.0):
    """n tensors [B, T, H, d] of normal values in the case's layout."""
    B, T, H = case["B"], case["T"], case["H"]
    dt = TYPES[case["dtype"]]
    if case["layout"] == "fused":
        x = torch.randn(B, T, n, H, d, device="cuda", generator=g) * scale
        return list(x.to(dt).unbind(2))
    shape = (B, H, T, d) if case["layout"] == "bhtd" else (B, T, H, d)
    out = []
    for _ in range(n):
        x = (torch.randn(shape, device="cuda", generator=g) * scale).to(dt)
        out.append(x.transpose(1, 2) if case["layout"] == "bhtd" else x)
    return out


def _prepare_la(case, g):
    B, H, dk, dv = (case[n] for n in ("B", "H", "dk", "dv"))
    st = dict(case=case)
    if case["layout"] == "fused":
        # dk = dv: queries, keys and values of one projection
        st["q"], st["k"], st["v"] = _heads(g, case, dk, 3, dk ** -0.25)
    else:
        st["q"], st["k"] = _heads(g, case, dk, 2, dk ** -0.25)
        st["v"], = _heads(g, case, dv, 1)
    # one decay a head, from about two tokens to a thousand
    at = torch.linspace(1.0, 10.0, H, device="cuda") if H > 1 else \
        torch.full((1,), 6.0, device="cuda")
    st["log_decay"] = -torch.exp2(-at)
    if case["op"] == "la_step":
        for n in ("q", "k", "v"):
            st[n] = st[n][:, 0]
        st["S"] = torch.randn(B, H, dk, dv, device="cuda", generator=g)
        return st
    s = case["state"]
    st["h0"] = torch.randn(B, H, dk, dv, device="cuda", generator=g) \
        if s else None
    if case["op"] == "la_bwd":
        st["o_grad"], = _heads(g, {**case, "layout": "bthd"}, dv, 1)
        st["hT_grad"] = torch.randn(B, H, dk, dv, device="cuda",
                                    generator=g) if s else None
    return st


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"].startswith("la"):
        return _prepare_la(case, g)
    N, V = case["N"], case["V"]
    # rows of different sharpness around a common shift
    sharp = torch.exp(0.5 * torch.randn(N, 1, device="cuda", generator=g))
    x = torch.randn(N, V, device="cuda", generator=g)
    x = (x * (2.0 * sharp)).add_(1.5)
    if case["masked"]:
        off = torch.rand(V, device="cuda", generator=g) < 0.3
        off[0] = False
        x.masked_fill_(off, -math.inf)
    dt = TYPES[case["dtype"]]
    if case["wide"]:
        logits = torch.zeros(N, V + 57, device="cuda", dtype=dt)
        logits[:, :V] = x
        logits = logits[:, :V]
    else:
        logits = x.to(dt)
    tokens = torch.randint(0, V, (N,), device="cuda", generator=g)
    if case["masked"]:
        tokens = torch.where(off[tokens], 0, tokens)
    if case["pad"]:
        none = torch.rand(N, device="cuda", generator=g) < 0.1
        tokens = torch.where(none, -1, tokens)
    st = dict(case=case, logits=logits, tokens=tokens)
    if case["op"] == "lp_bwd":
        z, lse = _normal(logits, case["scale"])
        st["lse"] = lse
        st["entropy"] = _entropy(z, lse)
        st["logp_grad"] = -torch.rand(N, device="cuda", generator=g) - 0.5
        st["entropy_grad"] = 0.1 * torch.randn(N, device="cuda", generator=g) \
            if case["entropy"] else None
    return st


# --- one pass --------------------------------------------------------------

def run(st):
    case = st["case"]
    return (_run_own if own else _run_plain)(st, case, case["op"])


def _run_own(st, case, op):
    from linear_attention_delta_gb300 import kla
    if op == "la_fwd":
        o, hT = kla.linattn_fwd(st["q"], st["k"], st["v"], st["log_decay"],
                                st["h0"])
        return dict(o=o, hT=hT)
    if op == "la_bwd":
        out = kla.linattn_bwd(st["q"], st["k"], st["v"], st["log_decay"],
                              st["o_grad"], hT_grad=st["hT_grad"],
                              h0=st["h0"], want_h0_grad=case["state"])
        return {n: x for n, x in out.items() if x is not None}
    if op == "la_step":
        o = kla.linattn_step(st["q"], st["k"], st["v"], st["log_decay"],
                             st["S"])
        return dict(o=o, S=st["S"])
    if op == "lp_fwd":
        logp, entropy, lse, top_logp, top_ids = kla.logprob_fwd(
            st["logits"], st["tokens"], top=case["top"], scale=case["scale"])
        out = dict(logp=logp, entropy=entropy, lse=lse)
        if case["top"]:
            out.update(top_logp=top_logp, top_ids=top_ids)
        return out
    return dict(logits_grad=kla.logprob_bwd(
        st["logits"], st["tokens"], st["lse"], st["entropy"],
        st["logp_grad"], st["entropy_grad"], scale=case["scale"]))


def _run_plain(st, case, op):
    if op.startswith("la"):
        dt = st["q"].dtype
        q, k, v = (st[n].float() for n in ("q", "k", "v"))
        if op == "la_step":
            decay = torch.exp(st["log_decay"])[:, None, None]
            S = decay * st["S"] + k[..., :, None] * v[..., None, :]
            st["S"].copy_(S)
            o = torch.matmul(q[..., None, :], S)[..., 0, :]
            return dict(o=o.to(dt), S=st["S"])
        # [B, H, T, d]
        q, k, v = (x.transpose(1, 2) for x in (q, k, v))
        a = st["log_decay"]
        if op == "la_fwd":
            o, hT = _attend(q, k, v, a, st["h0"], 1)
            return dict(o=_back(o, dt), hT=hT)
        do = st["o_grad"].float().transpose(1, 2)
        h0, dhT = st["h0"], st["hT_grad"]
        dq, _ = _attend(do, v, k, a, _swap(h0), 1)
        qr, kr, vr, dor = (x.flip(2) for x in (q, k, v, do))
        dk, _ = _attend(vr, dor, qr, a, _swap(dhT), 0)
        dv, dh0 = _attend(kr, qr, dor, a, dhT, 0)
        out = dict(q_grad=_back(dq, dt), k_grad=_back(dk.flip(2), dt),
                   v_grad=_back(dv.flip(2), dt))
        if case["state"]:
            out["h0_grad"] = dh0
        return out
    logits, tokens = st["logits"], st["tokens"]
    valid = tokens >= 0
    at = tokens.clamp(min=0)[:, None]
    if op == "lp_fwd":
        z, lse = _normal(logits, case["scale"])
        logp = torch.where(valid, z.gather(1, at)[:, 0] - lse, 0.0)
        out = dict(logp=logp, entropy=_entropy(z, lse), lse=lse)
        if case["top"]:
            ids = _largest(logits, case["top"])
            out.update(top_logp=z.gather(1, ids) - lse[:, None], top_ids=ids)
        return out
    z = logits.float() * case["scale"]
    lp = z - st["lse"][:, None]
    p = torch.exp(lp)
    g = torch.where(valid, st["logp_grad"], 0.0)
    d = -g[:, None] * p
    d.scatter_add_(1, at, g[:, None])
    if case["entropy"]:
        t = torch.where(p > 0, p * (lp + st["entropy"][:, None]), 0.0)
        d = d - st["entropy_grad"][:, None] * t
    return dict(logits_grad=(d * case["scale"]).to(logits.dtype))


def _swap(S):
    return None if S is None else S.transpose(-1, -2)


def _back(x, dt):
    return x.transpose(1, 2).to(dt).contiguous()


def _power(a, n):
    """exp(a_h n) of whole n: [H, *n.shape], formed in 64 bits."""
    return torch.exp(a.double().view(-1, *([1] * n.dim())) * n).float()


def _attend(q, k, v, a, S0, e):
    """o_i = sum_{j <= i} exp(a (i - j)) (q_i k_j) v_j + exp(a (i + e)) S0^T q_i
    and the state exp(a T) S0 + sum_j exp(a (T - e - j)) k_j v_j^T of
    [B, H, T, d] tensors, in chunks of 256 tokens."""
    B, H, T, dk = q.shape
    dv, C = v.shape[-1], 256
    N = -(-T // C)
    pad = N * C - T
    q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, pad))
               .reshape(B, H, N, C, x.shape[-1]) for x in (q, k, v))
    i = torch.arange(C, device=q.device)
    ij = i[:, None] - i[None, :]
    w = torch.where(ij >= 0, _power(a, ij.clamp(min=0)), 0.0)
    o = torch.matmul(torch.matmul(q, k.transpose(-1, -2)) * w[:, None], v)
    # each chunk's own contribution to the state at its end
    n = torch.arange(N, device=q.device)
    size = torch.clamp(T - n * C, max=C)
    w = _power(a, (size[:, None] - e - i[None, :]).clamp(min=0))
    U = torch.matmul((k * w[..., None]).transpose(-1, -2), v)
    # the states before the chunks, and after the last
    m = n[:, None] - 1 - n[None, :]
    w = torch.where(m >= 0, _power(a, C * m.clamp(min=0)), 0.0)
    S = torch.matmul(w, U.reshape(B, H, N, dk * dv)) \
        .view(B, H, N, dk, dv)
    if S0 is not None:
        S = S + _power(a, C * n)[..., None, None] * S0[:, :, None]
    o = o + _power(a, i + e)[:, None, :, None] * torch.matmul(q, S)
    last = T - (N - 1) * C
    ST = _power(a, torch.tensor(last, device=q.device)) \
        .view(H, 1, 1) * S[:, :, -1] + U[:, :, -1]
    return o.reshape(B, H, N * C, dv)[:, :, :T], ST


def _normal(logits, scale):
    """(scaled logits in 32 bits, log of the sum of their exponentials)."""
    z = logits.float() * scale
    m = z.max(1, keepdim=True).values
    return z, m[:, 0] + torch.log(torch.exp(z - m).sum(1))


def _entropy(z, lse):
    lp = z - lse[:, None]
    p = torch.exp(lp)
    return -torch.where(p > 0, p * lp, 0.0).sum(1)


def _largest(logits, top):
    """Ids of the largest logits of each row, ties to the lowest id: one key a
    logit, its order in the upper and its id in the lower bits."""
    bits = (logits.float() + 0.0).view(torch.int32).long()
    order = torch.where(bits >= 0, bits, -(bits & 0x7fffffff) - 1)
    V = logits.shape[1]
    ids = torch.arange(V, device=logits.device)
    key = torch.topk(order * (1 << 20) + (V - 1 - ids), top).values
    return V - 1 - (key & ((1 << 20) - 1))


# --- the work a case cannot do without -------------------------------------

def work(case):
    e = 2 if case["dtype"] == BF16 else 4
    op = case["op"]
    if op.startswith("la"):
        B, T, H, dk, dv = (case[n] for n in ("B", "T", "H", "dk", "dv"))
        n, s = B * T * H, B * H * dk * dv * 4
        if op == "la_step":
            return dict(bytes=n * 2 * (dk + dv) * e + 2 * s + 4 * H,
                        flops=5 * n * dk * dv)
        if op == "la_fwd":
            return dict(bytes=n * 2 * (dk + dv) * e +
                        s * (2 if case["state"] else 1),
                        flops=4 * n * dk * dv)
        return dict(bytes=n * (4 * dk + 3 * dv) * e +
                    (3 * s if case["state"] else 0),
                    flops=10 * n * dk * dv)
    n = case["N"] * case["V"]
    if op == "lp_fwd":
        return dict(bytes=n * e + case["N"] * (20 + 12 * case["top"]),
                    flops=5 * n)
    return dict(bytes=2 * n * e + 24 * case["N"],
                flops=(8 if case["entropy"] else 4) * n)


# --- the definition in 64 bits ---------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    f = {n: x.double() for n, x in st.items()
         if isinstance(x, torch.Tensor) and x.is_floating_point()}
    if not case["op"].startswith("la"):
        return _exact_lp(case, st, f)
    B, H, dk, dv, T = (case[n] for n in ("B", "H", "dk", "dv", "T"))
    lam = f["log_decay"].exp().repeat(B)[:, None, None]
    if case["op"] == "la_step":
        S = f["S"].view(B * H, dk, dv) * lam + torch.einsum(
            "nd,ne->nde", f["k"].reshape(B * H, dk), f["v"].reshape(B * H, dv))
        o = torch.einsum("nd,nde->ne", f["q"].reshape(B * H, dk), S)
        return dict(o=o.view(B, H, dv), S=S.view(B, H, dk, dv))

    def steps(x):
        return x.transpose(0, 1).reshape(T, B * H, x.shape[-1])

    def whole(x):
        return x.view(T, B, H, -1).transpose(0, 1)

    def state(name):
        return f[name].view(B * H, dk, dv).clone() if name in f else \
            torch.zeros(B * H, dk, dv, device="cuda", dtype=torch.float64)

    q, k, v = steps(f["q"]), steps(f["k"]), steps(f["v"])
    S = state("h0")
    if case["op"] == "la_fwd":
        o = torch.empty_like(v)
        for t in range(T):
            S.mul_(lam).baddbmm_(k[t, :, :, None], v[t, :, None, :])
            torch.bmm(q[t, :, None, :], S, out=o[t, :, None, :])
        return dict(o=whole(o), hT=S.view(B, H, dk, dv))
    do, dS = steps(f["o_grad"]), state("hT_grad")
    dq, dk_, dv_ = (torch.empty_like(x) for x in (q, k, v))
    for t in range(T):
        S.mul_(lam).baddbmm_(k[t, :, :, None], v[t, :, None, :])
        torch.bmm(S, do[t, :, :, None], out=dq[t, :, :, None])
    for t in range(T - 1, -1, -1):
        dS.baddbmm_(q[t, :, :, None], do[t, :, None, :])
        torch.bmm(dS, v[t, :, :, None], out=dk_[t, :, :, None])
        torch.bmm(k[t, :, None, :], dS, out=dv_[t, :, None, :])
        dS.mul_(lam)
    out = dict(q_grad=whole(dq), k_grad=whole(dk_), v_grad=whole(dv_))
    if case["state"]:
        out["h0_grad"] = dS.view(B, H, dk, dv)
    return out


def _exact_lp(case, st, f):
    tokens, N = st["tokens"], case["N"]
    rows = torch.arange(N, device="cuda")
    some = tokens >= 0
    if case["op"] == "lp_fwd":
        logits = f["logits"]
        p = torch.softmax(case["scale"] * logits, 1)
        lse = torch.logsumexp(case["scale"] * logits, 1)
        logp = torch.zeros(N, device="cuda", dtype=torch.float64)
        logp[some] = (case["scale"] * logits[rows[some], tokens[some]] -
                      lse[some])
        out = dict(logp=logp, entropy=torch.special.entr(p).sum(1), lse=lse)
        if case["top"]:
            x, ids = torch.sort(logits, dim=1, descending=True, stable=True)
            out["top_logp"] = case["scale"] * x[:, :case["top"]] - \
                lse[:, None]
            out["top_ids"] = ids[:, :case["top"]].clone()
        return out
    # the function of the given sums: p from the given lse and entropy
    lp = (case["scale"] * f["logits"]).sub_(f["lse"][:, None])
    p = lp.exp()
    d = p * -(f["logp_grad"] * some)[:, None]
    d[rows[some], tokens[some]] += f["logp_grad"][some]
    if case["entropy"]:
        lp.add_(f["entropy"][:, None]).masked_fill_(p == 0, 0.0)
        d -= f["entropy_grad"][:, None] * p * lp
    return dict(logits_grad=d.mul_(case["scale"]))
