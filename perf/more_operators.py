"""The workloads by which the gated delta rule and the norm of queries and keys
are measured: the chunked form of a training step and of a prompt, the recurrent
form of a decoding step, and the norm with the position rotation in front of them.

Each case is one call (or one forward and backward) of a layer as a training
step, a prompt or a decoding step makes it.  ``run`` computes it either by
elementary torch operations in float32 (``own = False``) or by this package's
calls (``own = True``); ``exact`` computes it in float64 from the definition.
"""
import math

import torch

own = False

_F, _D = torch.float32, torch.float64
_TD = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # the delta rule of a layer of 24 value heads of 64 on 12 key heads of 128 in a training step
        dict(name="delta_train", op="delta", grad=True, dtype="bf16", B=4, T=4096, H=24, G=12, P=64,
             N=128, init=False, ragged=False),
        # two prompts of the hybrid layer (64 heads in 8 groups), going on from states
        dict(name="delta_prompt", op="delta", grad=False, dtype="bf16", B=2, T=8192, H=64, G=8, P=64,
             N=128, init=True, ragged=False),
        # one long prompt on few heads: 32768 tokens, as many key heads as value heads
        dict(name="delta_prompt_long", op="delta", grad=False, dtype="bf16", B=1, T=32768, H=16, G=16,
             P=128, N=128, init=False, ragged=False),
        # short sequences of unequal lengths, odd sizes, fp32, going on from states, trained on
        dict(name="delta_ragged_f32", op="delta", grad=True, dtype="f32", B=6, T=333, H=6, G=3, P=40,
             N=24, init=True, ragged=True),
        # one decoding step of one sequence: latency
        dict(name="delta_token_one", op="delta_step", dtype="bf16", B=1, H=24, G=12, P=64, N=128, slots=1),
        # one decoding step of a serving batch with empty rows
        dict(name="delta_token_batch", op="delta_step", dtype="bf16", B=128, H=32, G=16, P=128, N=128,
             slots=160),
        # queries and keys of a training step: RMS norm with weights and rotation of the whole head
        dict(name="qk_train", op="qk", grad=True, dtype="bf16", B=4, T=4096, HQ=24, HK=12, D=128, R=128,
             weights=True, l2=False, inter=False, far=False, wide=True),
        # unit queries and keys without rotation, as the delta rule of a prompt takes them
        dict(name="qk_prompt_unit", op="qk", grad=False, dtype="bf16", B=2, T=8192, HQ=16, HK=16, D=128,
             R=0, weights=False, l2=True, inter=False, far=False, wide=True),
        # odd heads, part of the head rotated in adjacent pairs, far positions, fp32, trained on
        dict(name="qk_odd_f32", op="qk", grad=True, dtype="f32", B=3, T=341, HQ=5, HK=1, D=74, R=38,
             weights=True, l2=False, inter=True, far=True, wide=False),
        # one decoding step of a serving batch, each row at its own position
        dict(name="qk_token", op="qk_step", dtype="bf16", B=64, HQ=32, HK=8, D=128, R=64, weights=True,
             l2=False, inter=False, far=True, wide=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "f32"])
    op = rng.choice(["delta", "delta", "delta", "delta_step", "delta_step", "qk", "qk", "qk_step"])
    flip = lambda: rng.random() < 0.5  # noqa: E731
    if op == "delta":
        grad = flip()
        N = rng.choice([16, 24, 40, 64, 64, 96, 100, 128, 128, 128])
        P = rng.choice([8, 24, 40, 64, 64, 72, 128, 128])
        G = _log(rng, 1, 16)
        H = G * rng.choice([1, 1, 2, 3, 8])
        T = _log(rng, 1, 4096 if grad else 16384)
        B = max(1, min(_log(rng, 1, 8), (4 * 4096 * 24 * 64) // (T * H * P)))
        T = max(1, min(T, (4 * 4096 * 24 * 64) // (B * H * P)))
        return dict(op=op, grad=grad, dtype=dtype, B=B, T=T, H=H, G=G, P=P, N=N, init=flip(), ragged=flip())
    if op == "delta_step":
        G = _log(rng, 1, 16)
        B = _log(rng, 1, 128)
        return dict(op=op, dtype=dtype, B=B, H=G * rng.choice([1, 2, 3]), G=G,
                    P=rng.choice([8, 40, 64, 64, 100, 128]), N=rng.choice([16, 33, 64, 100, 128, 128]),
                    slots=B + rng.randrange(0, 32))
    D = rng.choice([24, 32, 64, 74, 80, 128, 128, 128, 256])
    HQ, HK = _log(rng, 1, 32), _log(rng, 1, 32)
    R = rng.choice([0, D // 4 * 2, D // 2 * 2, D // 2 * 2])
    c = dict(op=op, dtype=dtype, HQ=HQ, HK=HK, D=D, R=R, weights=flip(), l2=flip(), inter=flip(),
             far=flip(), wide=flip())
    if op == "qk_step":
        return dict(c, B=_log(rng, 1, 512))
    T = _log(rng, 1, 8192)
    return dict(c, grad=flip(), T=T, B=max(1, min(_log(rng, 1, 16), (4 * 4096 * 36 * 128) // (T * (HQ + HK) * D))))


def work(case):
    """Bytes: each input and each output once (a pass forward and backward reads its
    inputs once).  Operations: those of the recurrence, token by token."""
    e, op = 2 if case["dtype"] == "bf16" else 4, case["op"]
    if op in ("delta", "delta_step"):
        B, H, G, P, N = (case[k] for k in "BHGPN")
        n = B * case.get("T", 1)
        row = 2 * G * N + H * P + 2 * H                     # q, k, v, dt, beta of one token
        st = B * H * P * N * 4
        by, fl = n * (row + H * P) * e, n * H * P * (7 * N + 4)
        by += 2 * st if op == "delta_step" or case["init"] else st
        if case.get("grad"):
            by += n * (row + H * P) * e + (st if case["init"] else 0)
            fl += n * H * P * (18 * N + 8)
        return {"bytes": by, "flops": fl}
    n = case["B"] * case.get("T", 1) * (case["HQ"] + case["HK"]) * case["D"]
    by, fl = 2 * n * e, 7 * n
    if case.get("grad"):
        by, fl = by + 2 * n * e, fl + 14 * n
    return {"bytes": by, "flops": fl}


# ------------------------------------------------------------------ inputs

class _Rng:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, *shape, dtype=_F, std=1.0):
        return (torch.randn(*shape, generator=self.g, device="cuda") * std).to(dtype)

    def uniform(self, lo, hi, *shape):
        return torch.rand(*shape, generator=self.g, device="cuda") * (hi - lo) + lo

    def ints(self, lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=self.g, device="cuda", dtype=torch.int32)

    def slots(self, batch, n):
        """A distinct cache slot for every row; where slots are left over, about
        one row in eight is empty (-1)."""
        s = torch.randperm(n, generator=self.g, device="cuda")[:batch].to(torch.int32)
        if n > batch:
            s = torch.where(self.uniform(0.0, 1.0, batch) < 0.125, torch.full_like(s, -1), s)
        return s


def _unit(v):
    return v / torch.sqrt((v * v).sum(-1, keepdim=True) + 1e-6)


def prepare(case, seed):
    r, td, op = _Rng(seed), _TD[case["dtype"]], case["op"]
    s = {"case": case}
    if op in ("delta", "delta_step"):
        B, H, G, P, N = (case[k] for k in "BHGPN")
        lead = (B, case["T"]) if op == "delta" else (B,)
        silu = lambda v: v / (1.0 + torch.exp(-v))  # noqa: E731
        # unit keys and queries after the convolution's SiLU; the values stay a column
        # range of the convolution's output (of the decoding step's: dense)
        s["q"] = _unit(silu(r.normal(*lead, G, N))).to(td)
        s["k"] = _unit(silu(r.normal(*lead, G, N))).to(td)
        if op == "delta":
            s["v"] = r.normal(*lead, 2 * G * N + H * P, dtype=td)[..., 2 * G * N:].unflatten(-1, (H, P))
        else:
            s["v"] = r.normal(*lead, H, P, dtype=td)
        step = lambda *sh: torch.exp(r.uniform(math.log(1e-3), math.log(1e-1), *sh))  # noqa: E731
        s["dt_bias"] = torch.log(torch.expm1(step(H)))
        s["dt"] = (torch.log(torch.expm1(step(*lead, H))) - s["dt_bias"]).to(td)
        s["A"] = -torch.exp(r.uniform(0.0, math.log(16.0), H))
        s["beta"] = r.normal(*lead, H, dtype=td)
        s["scale"] = N ** -0.5
        if op == "delta_step":
            # behind the last slot a spare one that the plain form writes empty rows to
            s["cache"] = r.normal(case["slots"] + 1, H, P, N, std=0.3)
            s["state"], s["slots"] = s["cache"][:-1], r.slots(B, case["slots"])
            return s
        s["init"] = r.normal(B, H, P, N, std=0.3) if case["init"] else None
        s["lengths"] = None
        if case["ragged"]:
            n = r.ints(0, case["T"] + 1, B)
            n[0] = case["T"]
            if B > 1:
                n[-1] = 0 if B > 2 else 1
            s["lengths"] = n
        if case["grad"]:
            s["dy"] = r.normal(*lead, H, P, dtype=td)
        return s
    HQ, HK, D, R = (case[k] for k in ("HQ", "HK", "D", "R"))
    lead = (case["B"], case["T"]) if op == "qk" else (case["B"],)
    if case["wide"]:  # column ranges of one projection, values behind them
        w = r.normal(*lead, (HQ + 2 * HK) * D, dtype=td)
        s["q"] = w[..., :HQ * D].unflatten(-1, (HQ, D))
        s["k"] = w[..., HQ * D:(HQ + HK) * D].unflatten(-1, (HK, D))
    else:
        s["q"], s["k"] = r.normal(*lead, HQ, D, dtype=td), r.normal(*lead, HK, D, dtype=td)
    s["w_q"] = 1.0 + r.normal(D, std=0.1) if case["weights"] else None
    s["w_k"] = 1.0 + r.normal(D, std=0.1) if case["weights"] else None
    s["freq"] = s["positions"] = None
    if R:
        s["freq"] = 10000.0 ** (-torch.arange(R // 2, device="cuda", dtype=_F) / (R // 2))
        if case["far"]:
            first = r.ints(0, 1 << 20, case["B"])
            s["positions"] = first if op == "qk_step" else \
                first[:, None] + torch.arange(case["T"], device="cuda", dtype=torch.int32)
        elif op == "qk_step":
            s["positions"] = r.ints(0, 4096, case["B"])
    if case.get("grad"):
        s["dq_out"], s["dk_out"] = r.normal(*lead, HQ, D, dtype=td), r.normal(*lead, HK, D, dtype=td)
    return s


# -------------------------------------------------------------- plain forms
# The delta rule by chunks of 64 tokens: with G the running sum of the log decays of
# a chunk, M[i, j] = b_i e^(G_i - G_j) k_i . k_j below the diagonal and S the state in
# front of the chunk, the chunk's corrections U solve (I + M) U = b (V - e^G K S^T).

_C = 64


def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _softplus(v):
    return torch.where(v > 20.0, v, torch.log1p(torch.exp(torch.minimum(v, torch.full_like(v, 20.0)))))


def _t(m):
    return m.transpose(-1, -2)


def _chunks(s):
    """Inputs by (batch, head, chunk, token), padded with tokens that do nothing."""
    c = s["case"]
    B, T, H, G = (c[k] for k in "BTHG")
    nc = (T + _C - 1) // _C
    ok = torch.ones(B, T, 1, dtype=torch.bool, device="cuda")
    if s["lengths"] is not None:
        ok = (torch.arange(T, device="cuda")[None, :] < s["lengths"][:, None])[:, :, None]

    def cut(v, heads):
        v = torch.where(ok if v.dim() == 3 else ok[..., None], v, torch.zeros_like(v))
        out = v.new_zeros(B, nc * _C, *v.shape[2:])
        out[:, :T] = v
        out = out.unflatten(1, (nc, _C)).movedim(3, 1)
        return out if heads == H else out.repeat_interleave(H // heads, 1)

    v = s["dt"].to(_F) + s["dt_bias"]
    d = dict(q=cut(s["q"].to(_F), G), k=cut(s["k"].to(_F), G), v=cut(s["v"].to(_F), H),
             delta=cut(_softplus(v), H), b=cut(_sigmoid(s["beta"].to(_F)), H))
    if c["grad"]:
        d["dy"] = cut(s["dy"].to(_F), H)
        d["slope"] = cut(_sigmoid(v), H)
    return d, ok


def _inverse(M):
    """(I + M)^-1 of strictly lower triangular M, row by row."""
    X = torch.eye(_C, device="cuda").expand_as(M).clone()
    for i in range(1, _C):
        X[..., i, :] -= (M[..., i, None, :i] @ X[..., :i, :])[..., 0, :]
    return X


def _plain_delta(s):
    c, td, sc = s["case"], s["v"].dtype, s["scale"]
    B, T, H, G, P, N = (c[k] for k in "BTHGPN")
    d, ok = _chunks(s)
    q, k, b = d["q"], d["k"], d["b"]
    nc = q.shape[2]
    Gs = (d["delta"] * s["A"][:, None, None]).cumsum(-1)
    low = torch.ones(_C, _C, device="cuda").tril()
    dec = torch.exp(torch.where(low > 0, Gs[..., :, None] - Gs[..., None, :], torch.full_like(low, -1e9)))
    M = (low.tril(-1) * dec) * (k @ _t(k)) * b[..., None]
    X = _inverse(M)
    eG, eC = torch.exp(Gs), torch.exp(Gs[..., -1:] - Gs)
    end = eG[..., -1, None, None]
    S = s["init"] if s["init"] is not None else q.new_zeros(B, H, P, N)
    states, us = [], []
    for i in range(nc):
        R = b[:, :, i, :, None] * (d["v"][:, :, i] - eG[:, :, i, :, None] * (k[:, :, i] @ _t(S)))
        U = X[:, :, i] @ R
        states.append(S)
        us.append(U)
        S = end[:, :, i] * S + _t(U * eC[:, :, i, :, None]) @ k[:, :, i]
    S0, U = torch.stack(states, 2), torch.stack(us, 2)
    Aqk = dec * (q @ _t(k)) * sc
    y = sc * eG[..., None] * (q @ _t(S0)) + Aqk @ U

    def flat(v):  # (batch, head, chunk, token, ...) -> (batch, token, head, ...), padding 0
        v = v.flatten(2, 3).movedim(1, 2)[:, :T]
        return torch.where(ok if v.dim() == 3 else ok[..., None], v, torch.zeros_like(v))

    out = [flat(y).to(td), S.clone()]
    if not c["grad"]:
        return out
    dy = d["dy"]
    E = _t(Aqk) @ dy
    dS = torch.zeros_like(S)
    dstates, drs = [None] * nc, [None] * nc
    for i in range(nc - 1, -1, -1):
        dstates[i] = dS
        dR = _t(X[:, :, i]) @ (E[:, :, i] + eC[:, :, i, :, None] * (k[:, :, i] @ _t(dS)))
        drs[i] = dR
        dS = end[:, :, i] * dS + _t(dy[:, :, i] * (sc * eG[:, :, i, :, None])) @ q[:, :, i] \
            - _t(dR * (b[:, :, i] * eG[:, :, i])[..., None]) @ k[:, :, i]
    dSc, dR = torch.stack(dstates, 2), torch.stack(drs, 2)
    dAqk = dy @ _t(U)
    W = dR @ _t(U)
    dQ, dK, dX = dy @ S0, U @ dSc, dR @ S0
    P1, P2 = dAqk * dec * sc, -(low.tril(-1) * W * dec) * b[..., None]
    dq = sc * eG[..., None] * dQ + P1 @ k
    dk = eC[..., None] * dK - (b * eG)[..., None] * dX + _t(P1) @ q + (P2 + _t(P2)) @ k
    cK = eC * (k * dK).sum(-1)
    pair = dAqk * Aqk - W * M
    dG = pair.sum(-1) - pair.sum(-2) + sc * eG * (q * dQ).sum(-1) - cK - b * eG * (k * dX).sum(-1)
    dG[..., -1] += cK.sum(-1) + eG[..., -1] * (dSc * S0).sum((-1, -2))
    dg = dG.flip(-1).cumsum(-1).flip(-1)
    dbeta = (1.0 - b) * torch.diagonal(W, dim1=-2, dim2=-1)
    dv = dg * s["A"][:, None, None] * d["slope"]
    group = lambda m: m.unflatten(1, (G, H // G)).sum(2)  # noqa: E731
    out += [flat(group(dq)).to(td), flat(group(dk)).to(td), flat(b[..., None] * dR).to(td), flat(dv).to(td),
            flat(dbeta).to(td), (dg * d["delta"]).sum((0, 2, 3)), dv.sum((0, 2, 3))]
    if s["init"] is not None:
        out.append(dS)
    return out


def _plain_delta_step(s):
    c, td = s["case"], s["v"].dtype
    rep = c["H"] // c["G"]
    sl = s["slots"].long()
    live = sl >= 0
    at = torch.where(live, sl, torch.full_like(sl, s["state"].shape[0]))
    q, k = (s[n].to(_F).repeat_interleave(rep, 1)[..., None] for n in "qk")
    a = torch.exp(_softplus(s["dt"].to(_F) + s["dt_bias"]) * s["A"])
    h = a[..., None, None] * s["cache"][at]
    u = _sigmoid(s["beta"].to(_F))[..., None, None] * (s["v"].to(_F)[..., None] - h @ k)
    h = h + u * _t(k)
    y = s["scale"] * (h @ q)[..., 0]
    y = torch.where(live[:, None, None], y, torch.zeros_like(y))
    s["cache"][at] = h
    return [y.to(td), s["state"]]


_EPS = 1e-6


def _angles(s, x, dt):
    """cos and sin (..., 1, R / 2) of the positions' rotation; the angles in 64 bits."""
    pos = s["positions"]
    if pos is None:
        pos = torch.arange(x.shape[1], device="cuda").expand(x.shape[:2])
    a = pos.to(_D)[..., None, None] * s["freq"].to(_D)
    return torch.cos(a).to(dt), torch.sin(a).to(dt)


def _pairs(c, v):
    """The two members of each rotated pair, and the columns that stay."""
    R = c["R"]
    if c["inter"]:
        return v[..., 0:R:2], v[..., 1:R:2], v[..., R:]
    return v[..., :R // 2], v[..., R // 2:R], v[..., R:]


def _join(c, a, b, rest):
    both = torch.stack([a, b], -1).flatten(-2) if c["inter"] else torch.cat([a, b], -1)
    return torch.cat([both, rest], -1)


def _plain_qk(s):
    c, fwd, bwd = s["case"], [], []
    for n in "qk":
        x = s[n].to(_F)
        ss = (x * x).sum(-1, keepdim=True)
        rs = 1.0 / torch.sqrt((ss if c["l2"] else ss / c["D"]) + _EPS)
        xh, w = x * rs, s["w_" + n]
        y = xh if w is None else xh * w
        if c["R"]:
            cs, sn = _angles(s, x, _F)
            a, b, rest = _pairs(c, y)
            y = _join(c, a * cs - b * sn, b * cs + a * sn, rest)
        fwd.append(y.to(s[n].dtype))
        if c.get("grad"):
            dy = s["d" + n + "_out"].to(_F)
            if c["R"]:
                a, b, rest = _pairs(c, dy)
                dy = _join(c, a * cs + b * sn, b * cs - a * sn, rest)
            g = dy if w is None else dy * w
            dot = (g * xh).sum(-1, keepdim=True)
            bwd.append((rs * (g - xh * (dot if c["l2"] else dot / c["D"]))).to(s[n].dtype))
            if w is not None:
                bwd.append((dy * xh).flatten(0, -2).sum(0))
    return fwd + bwd


# ----------------------------------------------------------- this package

def _own(s):
    import state_space_model_sm_gb300 as ssd
    c, op = s["case"], s["case"]["op"]
    if op in ("delta", "delta_step"):
        args = (s["q"], s["k"], s["v"], s["dt"], s["dt_bias"], s["A"], s["beta"])
        if op == "delta_step":
            return [ssd.gated_delta_step(*args, s["state"], slots=s["slots"], scale=s["scale"]), s["state"]]
        more = dict(init_states=s["init"], lengths=s["lengths"], scale=s["scale"])
        out = list(ssd.gated_delta_fwd(*args, **more))
        if c["grad"]:
            g = ssd.gated_delta_bwd(*args, s["dy"], **more)
            out += [g[n] for n in ("dq", "dk", "dv", "ddt", "dbeta", "dA", "ddt_bias")]
            if s["init"] is not None:
                out.append(g["dinit_states"])
        return out
    args = (s["q"], s["k"], s["w_q"], s["w_k"], s["freq"], s["positions"])
    more = dict(l2=c["l2"], interleaved=c["inter"], eps=_EPS)
    out = list(ssd.qk_norm_fwd(*args, **more))
    if c.get("grad"):
        g = ssd.qk_norm_bwd(*args, s["dq_out"], s["dk_out"], **more)
        out += [g[n] for n in ("dq", "dw_q", "dk", "dw_k") if n in g]
    return out


_PLAIN = {"delta": _plain_delta, "delta_step": _plain_delta_step, "qk": _plain_qk, "qk_step": _plain_qk}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------- float64, by definition
# The delta rule token by token, its gradients by automatic differentiation of that
# recurrence, one stretch of tokens at a time.

def _recur(c, h, q, k, v, a, b, scale):
    rep, ys = c["H"] // c["G"], []
    for qt, kt, vt, at, bt in zip(*(m.unbind(1) for m in (q, k, v, a, b))):
        kt, qt = kt.repeat_interleave(rep, 1), qt.repeat_interleave(rep, 1)
        h = at[..., None, None] * h
        u = bt[..., None] * (vt - torch.einsum("bhpn,bhn->bhp", h, kt))
        h = h + torch.einsum("bhp,bhn->bhpn", u, kt)
        ys.append(scale * torch.einsum("bhpn,bhn->bhp", h, qt))
    return torch.stack(ys, 1), h


def _exact_delta(c, d, live):
    B, T, H, P, N = (c[k] for k in "BTHPN")
    names = ["q", "k", "v", "dt", "beta"]
    h = d["init"] if c["init"] else torch.zeros(B, H, P, N, device="cuda", dtype=_D)
    step = 64

    def stretch(h, ins, par):
        q, k, v, dt, beta, on = ins
        delta = torch.nn.functional.softplus(dt + par[0], threshold=50.0) * on
        return _recur(c, h, q, k, v, torch.exp(delta * par[1]), torch.sigmoid(beta) * on, d["scale"])

    cut = lambda t: [d[n][:, t:t + step] for n in names] + [live[:, t:t + step, None]]  # noqa: E731
    par, starts, ys = [d["dt_bias"], d["A"]], [], []
    for t in range(0, T, step):
        starts.append(h)
        y, h = stretch(h, cut(t), par)
        ys.append(y * live[:, t:t + step, None, None])
    out = [torch.cat(ys, 1), h]
    if not c["grad"]:
        return out
    grads, dpar, dh = [], [torch.zeros_like(p) for p in par], torch.zeros_like(h)
    for t in range((T - 1) // step * step, -1, -step):
        with torch.enable_grad():
            leaf = [v.clone().requires_grad_() for v in [starts[t // step]] + cut(t)[:-1] + par]
            y, h = stretch(leaf[0], leaf[1:6] + [cut(t)[-1]], leaf[6:])
            on = live[:, t:t + step, None, None]
            L = (y * on * d["dy"][:, t:t + step]).sum() + (h * dh).sum()
            g = torch.autograd.grad(L, leaf)
        dh = g[0]
        grads.append(g[1:6])
        dpar = [p + v for p, v in zip(dpar, g[6:])]
    whole = [torch.cat([g[i] for g in grads[::-1]], 1) for i in range(5)]
    out += whole + [dpar[1], dpar[0]]
    return out + ([dh] if c["init"] else [])


def _exact_delta_step(c, d):
    y, state = d["v"].new_zeros(c["B"], c["H"], c["P"]), d["state"].clone()
    for i, n in enumerate(d["slots"].tolist()):
        if n >= 0:
            delta = torch.nn.functional.softplus(d["dt"][i] + d["dt_bias"], threshold=50.0)
            one = [d[m][i][None, None] for m in "qkv"] + [torch.exp(delta * d["A"])[None, None],
                                                          torch.sigmoid(d["beta"][i])[None, None]]
            o, h = _recur(c, d["state"][n][None], *one, d["scale"])
            y[i], state[n] = o[0, 0], h[0]
    return [y, state]


def _exact_qk(c, d):
    out, grads = [], []
    for n in "qk":
        x, w = d[n], d["w_" + n]
        size = x.square().sum(-1, keepdim=True) * (1.0 if c["l2"] else 1.0 / c["D"])
        y = x * (size + _EPS).pow(-0.5)
        y = y * w if w is not None else y
        if c["R"]:
            a, b, rest = _pairs(c, y)
            z = torch.complex(a, b) * torch.complex(*_angles(d, x, _D))
            y = _join(c, z.real, z.imag, rest)
        out.append(y)
        if c.get("grad"):
            wrt = [x] + ([w] if w is not None else [])
            grads += torch.autograd.grad((y * d["d" + n + "_out"]).sum(), wrt)
    return out + grads


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.to(_D) if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    if case["op"] == "delta":
        T = case["T"]
        n = torch.full((case["B"],), T, device="cuda") if d["lengths"] is None else d["lengths"]
        live = (torch.arange(T, device="cuda")[None, :] < n[:, None]).to(_D)
        return _exact_delta(case, d, live)
    if case["op"] == "delta_step":
        return _exact_delta_step(case, d)
    d["freq"] = s["freq"]
    if case.get("grad"):
        for k in ("q", "k", "w_q", "w_k"):
            if d[k] is not None:
                d[k].requires_grad_()
    with torch.set_grad_enabled(bool(case.get("grad"))):
        return [v.detach() for v in _exact_qk(case, d)]
