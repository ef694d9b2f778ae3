"""The workloads by which the layer operators are measured: the short causal
convolution, the selective scan, the single-token steps and the block norm.

Each case is one call (or one forward and backward) of a layer as a training
step, a prompt or a decoding step makes it.  ``run`` computes it either by
elementary torch operations in float32 (``own = False``) or by this package's
calls (``own = True``); ``exact`` computes it in float64 from the definition.
"""
import math

import torch

own = False

_F = torch.float32
_TD = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # the convolution of a Mamba-2 layer (24 heads of 64, plus B and C of 128) in a training step
        dict(name="conv_train", op="conv", grad=True, dtype="bf16", B=4, T=4096, C=1792, K=4,
             silu=True, bias=True, init=False, ragged=False),
        # a batch of right-padded prompts that go on from cached states, an odd channel count, fp32
        dict(name="conv_prompt_ragged", op="conv", grad=False, dtype="f32", B=5, T=1021, C=777, K=3,
             silu=True, bias=True, init=True, ragged=True),
        # one decoding step of a serving batch with empty rows
        dict(name="conv_token", op="conv_step", dtype="bf16", B=64, C=1792, K=4, silu=True, bias=True,
             slots=96),
        # the selective scan of a layer of 1536 channels in a training step
        dict(name="scan_train", op="scan", grad=True, dtype="bf16", B=4, T=4096, D=1536, N=16, G=1,
             z=True, init=False, ragged=False),
        # one long prompt: 65536 tokens, 2048 channels
        dict(name="scan_prompt_long", op="scan", grad=False, dtype="bf16", B=1, T=65536, D=2048, N=16,
             G=1, z=True, init=False, ragged=False),
        # short prompts of unequal lengths, odd sizes, two groups, fp32, going on from states, trained on
        dict(name="scan_ragged_f32", op="scan", grad=True, dtype="f32", B=6, T=333, D=202, N=24, G=2,
             z=False, init=True, ragged=True),
        # one decoding step of the selective scan
        dict(name="scan_token", op="scan_step", dtype="bf16", B=32, D=1536, N=16, G=1, z=True, slots=48),
        # one decoding step of the SSD layer, one sequence: latency
        dict(name="ssd_token_one", op="ssd_step", dtype="bf16", B=1, H=24, P=64, N=128, G=1, slots=1),
        # one decoding step of the hybrid layer (64 heads in 8 groups), a large serving batch
        dict(name="ssd_token_batch", op="ssd_step", dtype="bf16", B=256, H=64, P=64, N=128, G=8,
             slots=256),
        # between two layers of the hybrid width in a training step, residual kept in fp32
        dict(name="norm_train", op="norm", grad=True, dtype="bf16", res="f32", rows=16384, F=4096,
             post=True, gates=2, scale=0.5),
        # an odd width, fp32 throughout, without the norm after the block and without a gate
        dict(name="norm_odd_f32", op="norm", grad=True, dtype="f32", res="f32", rows=1021, F=1001,
             post=False, gates=0, scale=1.0),
        # a decoding step of four sequences, everything in bf16
        dict(name="norm_token", op="norm", grad=False, dtype="bf16", res="bf16", rows=4, F=1536,
             post=True, gates=1, scale=0.7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "f32"])
    op = rng.choice(["conv", "conv", "conv_step", "scan", "scan", "scan_step", "ssd_step", "ssd_step",
                     "norm", "norm"])
    flip = lambda: rng.random() < 0.5  # noqa: E731
    if op == "conv":
        # up to the listed training size; one in two with channels that fill no vector
        C = _log(rng, 24, 4096) if flip() else 8 * _log(rng, 4, 512)
        T = _log(rng, 1, 8192)
        B = max(1, min(_log(rng, 1, 16), (4 * 4096 * 1792) // (T * C)))
        return dict(op=op, grad=flip(), dtype=dtype, B=B, T=T, C=C, K=rng.choice([2, 3, 4, 4]),
                    silu=rng.random() < 0.8, bias=flip(), init=flip(), ragged=flip())
    if op == "conv_step":
        B = _log(rng, 1, 256)
        return dict(op=op, dtype=dtype, B=B, C=_log(rng, 24, 8192), K=rng.choice([2, 3, 4, 4]), silu=True,
                    bias=flip(), slots=B + rng.randrange(0, 64))
    if op == "scan":
        grad = flip()
        N = rng.choice([4, 8, 16, 16, 16, 24, 32, 64])
        G = rng.choice([1, 1, 2, 3])
        D = G * _log(rng, 16, 2048 // G)
        T = _log(rng, 1, 4096 if grad else 16384)
        B = max(1, min(_log(rng, 1, 8), (4 * 4096 * 1536 * 16) // (T * D * N)))
        return dict(op=op, grad=grad, dtype=dtype, B=B, T=T, D=D, N=N, G=G, z=flip(), init=flip(),
                    ragged=flip())
    if op == "scan_step":
        B, G = _log(rng, 1, 256), rng.choice([1, 1, 2, 3])
        return dict(op=op, dtype=dtype, B=B, D=G * _log(rng, 16, 4096 // G),
                    N=rng.choice([4, 8, 16, 16, 24, 32, 64]), G=G, z=flip(), slots=B + rng.randrange(0, 64))
    if op == "ssd_step":
        B, G = _log(rng, 1, 256), rng.choice([1, 1, 2, 8])
        return dict(op=op, dtype=dtype, B=B, H=G * rng.choice([2, 3, 5, 8]),
                    P=rng.choice([16, 40, 64, 64, 128]), N=rng.choice([16, 33, 64, 128, 128]), G=G,
                    slots=B + rng.randrange(0, 32))
    F = _log(rng, 64, 8192) if flip() else 8 * _log(rng, 8, 1024)
    rows = min(_log(rng, 1, 16384), (16384 * 4096) // F)
    gates = rng.choice([0, 1, 2, 4])
    if gates:
        rows = max(1, rows // gates) * gates
    return dict(op="norm", grad=flip(), dtype=dtype, res="f32" if dtype == "f32" else rng.choice(["f32", "bf16"]),
                rows=rows, F=F, post=flip(), gates=gates, scale=rng.choice([1.0, 0.5, 0.22]))


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "conv":
        n, C, K = case["B"] * case["T"] * case["C"], case["C"], case["K"]
        by = 2 * n * e + (K + 1) * C * 4 + 2 * case["B"] * (K - 1) * C * e
        fl = n * (2 * K + 6)
        if case["grad"]:
            by += 3 * n * e + 2 * (K + 1) * C * 4
            fl += n * (6 * K + 10)
        return {"bytes": by, "flops": fl}
    if op == "conv_step":
        n, K = case["B"] * case["C"], case["K"]
        return {"bytes": n * e * (2 + 2 * (K - 1)) + (K + 1) * case["C"] * 4, "flops": n * (2 * K + 6)}
    if op == "scan":
        B, T, D, N, G = (case[k] for k in "BTDNG")
        td, st = B * T * D, B * D * N
        by = td * e * (4 if case["z"] else 3) + 2 * B * T * G * N * e + (st + D * N) * 4
        fl = td * N * 8 + td * 20
        if case["grad"]:
            by += td * e * (7 if case["z"] else 5) + 2 * B * T * G * N * (e + 4) + (st + 2 * D * N) * 4
            fl += td * N * 24 + td * 40
        return {"bytes": by, "flops": fl}
    if op == "scan_step":
        B, D, N, G = (case[k] for k in "BDNG")
        return {"bytes": 2 * B * D * N * 4 + D * N * 4 + B * D * e * (4 if case["z"] else 3)
                + 2 * B * G * N * e, "flops": B * D * (8 * N + 20)}
    if op == "ssd_step":
        B, H, P, N, G = (case[k] for k in "BHPNG")
        return {"bytes": 2 * B * H * P * N * 4 + 2 * B * H * P * e + B * H * e + 2 * B * G * N * e,
                "flops": B * H * P * (6 * N + 4)}
    n, r = case["rows"] * case["F"], 2 if case["res"] == "bf16" else 4
    by, fl = n * (2 * r + 2 * e), n * 12
    if case["grad"]:
        by, fl = by + n * (3 * r + 3 * e), fl + n * 30
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


def _dt(r, bias, *shape):
    """dt such that softplus(dt + bias) is log-uniform on [1e-3, 1e-1]."""
    u = torch.exp(r.uniform(math.log(1e-3), math.log(1e-1), *shape))
    return torch.log(torch.expm1(u)) - bias


def _lengths(r, case):
    if not case["ragged"]:
        return None
    n = r.ints(0, case["T"] + 1, case["B"])
    n[0] = case["T"]
    if case["B"] > 1:
        n[-1] = 0 if case["B"] > 2 else 1
    return n


def _cache(s, t):
    """The state cache, and behind its last slot a spare one that the plain forms
    write empty rows to (so they need no host round trip to leave them out)."""
    s["cache"], s["state"] = t, t[:-1]


def prepare(case, seed):
    r = _Rng(seed)
    td = _TD[case["dtype"]]
    op, s = case["op"], {"case": case}
    if op in ("conv", "conv_step"):
        C, K, B = case["C"], case["K"], case["B"]
        s["w"] = r.uniform(-K ** -0.5, K ** -0.5, C, K)
        s["bias"] = r.uniform(-0.5, 0.5, C) if case["bias"] else None
        if op == "conv_step":
            s["x"] = r.normal(B, C, dtype=td)
            _cache(s, r.normal(case["slots"] + 1, K - 1, C, dtype=td))
            s["slots"] = r.slots(B, case["slots"])
            return s
        s["x"] = r.normal(B, case["T"], C, dtype=td)
        s["init"] = r.normal(B, K - 1, C, dtype=td) if case["init"] else None
        s["lengths"] = _lengths(r, case)
        if case["grad"]:
            s["dy"] = r.normal(B, case["T"], C, dtype=td)
        return s
    if op in ("scan", "scan_step"):
        B, D, N, G = (case[k] for k in "BDNG")
        lead = (B, case["T"]) if op == "scan" else (B,)
        s["dt_bias"] = _dt(r, 0.0, D)
        s["A"] = -torch.arange(1, N + 1, device="cuda", dtype=_F) * torch.exp(r.uniform(-0.3, 0.3, D, N))
        s["D"] = r.uniform(0.0, 1.0, D)
        s["x"] = r.normal(*lead, D, dtype=td)
        s["dt"] = _dt(r, s["dt_bias"], *lead, D).to(td)
        s["B"] = r.normal(*lead, G, N, dtype=td)
        s["C"] = r.normal(*lead, G, N, dtype=td)
        s["z"] = r.normal(*lead, D, dtype=td) if case["z"] else None
        if op == "scan_step":
            _cache(s, r.normal(case["slots"] + 1, D, N, std=0.3))
            s["slots"] = r.slots(B, case["slots"])
            return s
        s["init"] = r.normal(B, D, N, std=0.3) if case["init"] else None
        s["lengths"] = _lengths(r, case)
        if case["grad"]:
            s["dout"] = r.normal(*lead, D, dtype=td)
        return s
    if op == "ssd_step":
        B, H, P, N, G = (case[k] for k in "BHPNG")
        s["dt_bias"] = _dt(r, 0.0, H)
        s["A"] = -torch.exp(r.uniform(0.0, math.log(16.0), H))
        s["D"] = r.uniform(0.0, 1.0, H)
        s["x"] = r.normal(B, H, P, dtype=td)
        s["dt"] = _dt(r, s["dt_bias"], B, H).to(td)
        s["B"] = r.normal(B, G, N, dtype=td)
        s["C"] = r.normal(B, G, N, dtype=td)
        _cache(s, r.normal(case["slots"] + 1, H, P, N, std=0.3))
        s["slots"] = r.slots(B, case["slots"])
        return s
    rows, F, rd = case["rows"], case["F"], _TD[case["res"]]
    s["r"] = r.normal(rows, F, dtype=rd)
    s["o"] = r.normal(rows, F, dtype=td, std=0.5)
    s["w_pre"] = 1.0 + r.normal(F, std=0.1)
    s["w_post"] = 1.0 + r.normal(F, std=0.1) if case["post"] else None
    s["gate"] = r.normal(case["gates"], F) if case["gates"] else None
    if case["grad"]:
        s["dh"] = r.normal(rows, F, dtype=td)
        s["dr"] = r.normal(rows, F, dtype=rd)
    return s


# -------------------------------------------------------------- plain forms

def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _softplus(v):
    return torch.where(v > 20.0, v, torch.log1p(torch.exp(torch.minimum(v, torch.full_like(v, 20.0)))))


def _inside(T, lengths):
    """(B, T, 1) truth values: positions before each row's length."""
    return (torch.arange(T, device="cuda")[None, :] < lengths[:, None])[:, :, None]


def _plain_conv(s):
    c = s["case"]
    T, K, td = c["T"], c["K"], s["x"].dtype
    w = s["w"]
    x = s["x"].to(_F)
    pre = s["init"].to(_F) if s["init"] is not None else x.new_zeros(c["B"], K - 1, c["C"])
    xp = torch.cat([pre, x], 1)
    u = xp[:, :T] * w[:, 0]
    for k in range(1, K):
        u = u + xp[:, k:k + T] * w[:, k]
    if s["bias"] is not None:
        u = u + s["bias"]
    sg = _sigmoid(u) if c["silu"] else None
    y = u * sg if c["silu"] else u
    ln = s["lengths"]
    if ln is not None:
        ok = _inside(T, ln)
        y = torch.where(ok, y, torch.zeros_like(y))
    at = torch.full((c["B"],), T, device="cuda") if ln is None else ln
    rows = at[:, None] + torch.arange(K - 1, device="cuda")[None, :]  # of xp, which starts K-1 early
    final = torch.gather(xp, 1, rows[:, :, None].expand(-1, -1, c["C"]).long())
    out = [y.to(td), final.to(td)]
    if c["grad"]:
        du = s["dy"].to(_F)
        if c["silu"]:
            du = du * sg * (1.0 + u * (1.0 - sg))
        if ln is not None:
            du = torch.where(ok, du, torch.zeros_like(du))
        dxp = torch.zeros_like(xp)
        for k in range(K):
            dxp[:, k:k + T] += du * w[:, k]
        dw = torch.stack([(du * xp[:, k:k + T]).sum((0, 1)) for k in range(K)], 1)
        out += [dxp[:, K - 1:].to(td), dw]
        if s["bias"] is not None:
            out.append(du.sum((0, 1)))
        if s["init"] is not None:
            out.append(dxp[:, :K - 1].to(td))
    return out


def _rows(s):
    """Which rows of the batch are in use, and every row's slot (the spare one
    for the others)."""
    sl = s["slots"].long()
    live = sl >= 0
    return live, torch.where(live, sl, torch.full_like(sl, s["state"].shape[0]))


def _plain_conv_step(s):
    c = s["case"]
    live, at = _rows(s)
    win = torch.cat([s["cache"][at], s["x"][:, None]], 1)  # (B, K, C)
    u = win[:, 0].to(_F) * s["w"][:, 0]
    for k in range(1, c["K"]):
        u = u + win[:, k].to(_F) * s["w"][:, k]
    if s["bias"] is not None:
        u = u + s["bias"]
    y = u * _sigmoid(u) if c["silu"] else u
    y = torch.where(live[:, None], y, torch.zeros_like(y))
    s["cache"][at] = win[:, 1:]
    return [y.to(s["x"].dtype), s["state"]]


_CHUNK = 256  # positions whose decays the plain scan forms at a time


def _by_channel(m, D):
    """(..., G, N) of a group of channels -> (..., D, N)."""
    return m.to(_F).repeat_interleave(D // m.shape[-2], dim=-2)


def _plain_scan(s):
    c = s["case"]
    B, T, D, N, G = (c[k] for k in "BTDNG")
    td, A = s["x"].dtype, s["A"]
    v = s["dt"].to(_F) + s["dt_bias"]
    delta = _softplus(v)
    x = s["x"].to(_F)
    ok = None
    if s["lengths"] is not None:
        ok = _inside(T, s["lengths"])
        delta = torch.where(ok, delta, torch.zeros_like(delta))
    h = s["init"].clone() if s["init"] is not None else x.new_zeros(B, D, N)
    keep = c["grad"]
    y = torch.empty_like(x)
    if keep:
        hs, dec = x.new_empty(T + 1, B, D, N), x.new_empty(T, B, D, N)
        hs[0] = h
    for t0 in range(0, T, _CHUNK):
        sl = slice(t0, min(T, t0 + _CHUNK))
        n = sl.stop - t0
        dl = delta[:, sl].transpose(0, 1)[..., None]                  # (n, B, D, 1)
        a = dec[sl] if keep else x.new_empty(n, B, D, N)
        torch.exp(dl * A, out=a)
        b = (dl * x[:, sl].transpose(0, 1)[..., None]) * _by_channel(s["B"][:, sl].transpose(0, 1), D)
        hc = hs[t0 + 1:t0 + 1 + n] if keep else torch.empty_like(a)
        for a_t, b_t, h_t in zip(a.unbind(0), b.unbind(0), hc.unbind(0)):
            torch.addcmul(b_t, a_t, h, out=h_t)
            h = h_t
        y[:, sl] = (hc * _by_channel(s["C"][:, sl].transpose(0, 1), D)).sum(-1).transpose(0, 1)
    h = h.clone()
    y = y + s["D"] * x
    out = y
    if s["z"] is not None:
        z = s["z"].to(_F)
        sg = _sigmoid(z)
        out = y * (z * sg)
    if ok is not None:
        out = torch.where(ok, out, torch.zeros_like(out))
    res = [out.to(td), h]
    if not c["grad"]:
        return res
    dy = s["dout"].to(_F)
    if ok is not None:
        dy = torch.where(ok, dy, torch.zeros_like(dy))
    if s["z"] is not None:
        dz = dy * y * sg * (1.0 + z * (1.0 - sg))
        dy = dy * (z * sg)
    g = x.new_zeros(B, D, N)
    ddel, dxs = torch.empty_like(x), torch.empty_like(x)
    dA, dBs, dCs = torch.zeros_like(A), x.new_empty(B, T, G, N), x.new_empty(B, T, G, N)
    nch = (T + _CHUNK - 1) // _CHUNK
    for ci in range(nch - 1, -1, -1):
        sl = slice(ci * _CHUNK, min(T, (ci + 1) * _CHUNK))
        n = sl.stop - sl.start
        dyt = dy[:, sl].transpose(0, 1)[..., None]
        cd = dyt * _by_channel(s["C"][:, sl].transpose(0, 1), D)
        gs = torch.empty_like(cd)
        a = dec[sl]
        for i in range(n - 1, -1, -1):
            torch.add(cd[i], g, out=gs[i])
            g = gs[i] * a[i]
        w = gs * a * hs[sl]                                            # g a h_prev
        dl, xt = delta[:, sl].transpose(0, 1)[..., None], x[:, sl].transpose(0, 1)[..., None]
        gb = (gs * _by_channel(s["B"][:, sl].transpose(0, 1), D)).sum(-1)
        ddel[:, sl] = ((w * A).sum(-1) + gb * xt[..., 0]).transpose(0, 1)
        dxs[:, sl] = (gb * dl[..., 0]).transpose(0, 1)
        dA += (w * dl).sum((0, 1))
        dBs[:, sl] = (gs * (dl * xt)).view(n, B, G, D // G, N).sum(3).transpose(0, 1)
        dCs[:, sl] = (hs[sl.start + 1:sl.stop + 1] * dyt).view(n, B, G, D // G, N).sum(3).transpose(0, 1)
    dv = ddel * _sigmoid(v)
    if ok is not None:
        dv = torch.where(ok, dv, torch.zeros_like(dv))
    res += [(dxs + s["D"] * dy).to(td), dv.to(td), dA, dBs, dCs, (dy * x).sum((0, 1)), dv.sum((0, 1))]
    if s["z"] is not None:
        res.append(dz.to(td))
    if s["init"] is not None:
        res.append(g)
    return res


def _plain_scan_step(s):
    D = s["case"]["D"]
    live, at = _rows(s)
    delta = _softplus(s["dt"].to(_F) + s["dt_bias"])[..., None]
    x = s["x"].to(_F)
    h = torch.exp(delta * s["A"]) * s["cache"][at] + delta * x[..., None] * _by_channel(s["B"], D)
    y = (h * _by_channel(s["C"], D)).sum(-1) + s["D"] * x
    if s["z"] is not None:
        z = s["z"].to(_F)
        y = y * (z * _sigmoid(z))
    y = torch.where(live[:, None], y, torch.zeros_like(y))
    s["cache"][at] = h
    return [y.to(s["x"].dtype), s["state"]]


def _plain_ssd_step(s):
    H = s["case"]["H"]
    live, at = _rows(s)
    delta = _softplus(s["dt"].to(_F) + s["dt_bias"])[:, :, None, None]  # (B, H, 1, 1)
    x = s["x"].to(_F)
    h = torch.exp(delta * s["A"][:, None, None]) * s["cache"][at] \
        + (delta * x[..., None]) * _by_channel(s["B"], H)[:, :, None, :]
    y = (h * _by_channel(s["C"], H)[:, :, None, :]).sum(-1) + s["D"][:, None] * x
    y = torch.where(live[:, None, None], y, torch.zeros_like(y))
    s["cache"][at] = h
    return [y.to(s["x"].dtype), s["state"]]


_EPS = 1e-5


def _rstd(v):
    return 1.0 / torch.sqrt((v * v).mean(-1, keepdim=True) + _EPS)


def _plain_norm(s):
    c = s["case"]
    rows, F, ng = c["rows"], c["F"], c["gates"]
    o, r = s["o"].to(_F), s["r"].to(_F)
    ro = _rstd(o) if c["post"] else None
    oh = o * ro if c["post"] else o
    t = oh * s["w_post"] if c["post"] else oh
    gate = None
    if ng:
        gate = s["gate"][:, None].expand(ng, rows // ng, F).reshape(rows, F)
    rn = r + c["scale"] * (gate * t if ng else t)
    rr = _rstd(rn)
    rh = rn * rr
    out = [rn.to(s["r"].dtype), (rh * s["w_pre"]).to(s["o"].dtype)]
    if c["grad"]:
        dh = s["dh"].to(_F)
        gx = dh * s["w_pre"]
        dr = s["dr"].to(_F) + rr * (gx - rh * (gx * rh).mean(-1, keepdim=True))
        dt = dr * c["scale"]
        dgate = (dt * t).view(ng, rows // ng, F).sum(1) if ng else None
        if ng:
            dt = dt * gate
        do, dw_post = dt, None
        if c["post"]:
            dw_post = (dt * oh).sum(0)
            gy = dt * s["w_post"]
            do = ro * (gy - oh * (gy * oh).mean(-1, keepdim=True))
        out += [dr.to(s["r"].dtype), do.to(s["o"].dtype), (dh * rh).sum(0)]
        out += [v for v in (dw_post, dgate) if v is not None]
    return out


# ----------------------------------------------------------- this package

def _own(s):
    import state_space_model_sm_gb300 as ssd
    c = s["case"]
    op = c["op"]
    if op == "conv":
        y, final = ssd.causal_conv_fwd(s["x"], s["w"], s["bias"], init_state=s["init"],
                                       lengths=s["lengths"], silu=c["silu"])
        out = [y, final]
        if c["grad"]:
            g = ssd.causal_conv_bwd(s["x"], s["w"], s["bias"], s["dy"], init_state=s["init"],
                                    lengths=s["lengths"], silu=c["silu"])
            out += [g["dx"], g["dw"]]
            out += [g[k] for k, v in (("dbias", s["bias"]), ("dinit_state", s["init"])) if v is not None]
        return out
    if op == "conv_step":
        y = ssd.causal_conv_step(s["x"], s["state"], s["w"], s["bias"], slots=s["slots"], silu=c["silu"])
        return [y, s["state"]]
    if op == "scan":
        args = (s["x"], s["dt"], s["dt_bias"], s["A"], s["B"], s["C"], s["D"], s["z"])
        out = list(ssd.selective_scan_fwd(*args, init_states=s["init"], lengths=s["lengths"]))
        if c["grad"]:
            g = ssd.selective_scan_bwd(*args, s["dout"], init_states=s["init"], lengths=s["lengths"])
            out += [g[k] for k in ("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias")]
            out += [g[k] for k, v in (("dz", s["z"]), ("dinit_states", s["init"])) if v is not None]
        return out
    if op == "scan_step":
        y = ssd.selective_step(s["x"], s["dt"], s["dt_bias"], s["A"], s["B"], s["C"], s["state"], s["D"],
                               s["z"], slots=s["slots"])
        return [y, s["state"]]
    if op == "ssd_step":
        y = ssd.ssd_step(s["x"], s["dt"], s["dt_bias"], s["A"], s["B"], s["C"], s["state"], s["D"],
                         slots=s["slots"])
        return [y, s["state"]]
    args = (s["r"], s["o"], s["w_pre"], s["w_post"], s["gate"])
    out = list(ssd.block_norm_fwd(*args, scale=c["scale"], eps=_EPS))
    if c["grad"]:
        g = ssd.block_norm_bwd(*args, s["dh"], s["dr"], scale=c["scale"], eps=_EPS)
        out += [g["dresidual"], g["do"], g["dw_pre"]]
        out += [g[k] for k, v in (("dw_post", s["w_post"]), ("dgate", s["gate"])) if v is not None]
    return out


_PLAIN = {"conv": _plain_conv, "conv_step": _plain_conv_step, "scan": _plain_scan,
          "scan_step": _plain_scan_step, "ssd_step": _plain_ssd_step, "norm": _plain_norm}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------- float64, by definition
# Gradients by automatic differentiation of the definition, convolutions and
# sums in another form than above.

def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    grad = case.get("grad", False)
    if grad:
        for k, v in d.items():
            if torch.is_tensor(v) and v.is_floating_point():
                v.requires_grad_(k not in ("dy", "dout", "dh", "dr"))
    with torch.set_grad_enabled(grad):
        out = _EXACT[case["op"]](case, d)
    return [v.detach() for v in out]


def _exact_conv(c, d):
    B, T, C, K = (c[k] for k in "BTCK")
    pre = d["init"] if c["init"] else torch.zeros(B, K - 1, C, device="cuda", dtype=torch.float64)
    xp = torch.cat([pre, d["x"]], 1)
    u = torch.einsum("btck,ck->btc", xp.unfold(1, K, 1), d["w"])
    if c["bias"]:
        u = u + d["bias"]
    y = torch.nn.functional.silu(u) if c["silu"] else u
    n = [T] * B if d["lengths"] is None else d["lengths"].tolist()
    y = torch.stack([torch.cat([y[b, :n[b]], y.new_zeros(T - n[b], C)]) for b in range(B)])
    final = torch.stack([xp[b, n[b]:n[b] + K - 1] for b in range(B)])
    out = [y, final]
    if c["grad"]:
        wrt = [d["x"], d["w"]] + [d[k] for k in ("bias", "init") if c[k]]
        out += torch.autograd.grad((y * d["dy"]).sum(), wrt)
    return out


def _exact_conv_step(c, d):
    y = d["x"].new_zeros(c["B"], c["C"])
    state = d["state"].clone()
    for b, k in enumerate(d["slots"].tolist()):
        if k >= 0:
            win = torch.cat([d["state"][k], d["x"][b:b + 1]])
            u = (win.t() * d["w"]).sum(1) + (d["bias"] if c["bias"] else 0.0)
            y[b] = torch.nn.functional.silu(u) if c["silu"] else u
            state[k] = win[1:]
    return [y, state]


def _exact_scan(c, d):
    B, T, D, N, G = (c[k] for k in "BTDNG")
    h = d["init"] if c["init"] else torch.zeros(B, D, N, device="cuda", dtype=torch.float64)
    delta = torch.nn.functional.softplus(d["dt"] + d["dt_bias"], threshold=50.0)
    live = None
    if d["lengths"] is not None:
        live = torch.arange(T, device="cuda")[None, :] < d["lengths"][:, None]
        delta = delta * live[:, :, None]
    de, xs, Bs, Cs = delta.unbind(1), d["x"].unbind(1), d["B"].unbind(1), d["C"].unbind(1)
    A, ys = d["A"].view(G, D // G, N), []
    h = h.view(B, G, D // G, N)
    for t in range(T):
        dl = de[t].view(B, G, D // G, 1)
        h = torch.exp(dl * A) * h + dl * xs[t].view(B, G, D // G, 1) * Bs[t][:, :, None, :]
        ys.append(torch.einsum("bgdn,bgn->bgd", h, Cs[t]).reshape(B, D))
    y = torch.stack(ys, 1) + d["D"] * d["x"]
    out = y * torch.nn.functional.silu(d["z"]) if c["z"] else y
    if live is not None:
        out = out * live[:, :, None]
    res = [out, h.reshape(B, D, N)]
    if c["grad"]:
        wrt = [d[k] for k in ("x", "dt", "A", "B", "C", "D", "dt_bias")]
        wrt += [d[k] for k in ("z", "init") if c[k]]
        res += torch.autograd.grad((out * d["dout"]).sum(), wrt)
    return res


def _exact_scan_step(c, d):
    out, state = d["x"].new_zeros(c["B"], c["D"]), d["state"].clone()
    g = torch.arange(c["D"], device="cuda") // (c["D"] // c["G"])
    for b, k in enumerate(d["slots"].tolist()):
        if k >= 0:
            delta = torch.nn.functional.softplus(d["dt"][b] + d["dt_bias"], threshold=50.0)
            state[k] = torch.exp(delta[:, None] * d["A"]) * d["state"][k] \
                + (delta * d["x"][b])[:, None] * d["B"][b][g]
            y = torch.einsum("dn,dn->d", state[k], d["C"][b][g]) + d["D"] * d["x"][b]
            out[b] = y * torch.nn.functional.silu(d["z"][b]) if c["z"] else y
    return [out, state]


def _exact_ssd_step(c, d):
    out, state = d["x"].new_zeros(c["B"], c["H"], c["P"]), d["state"].clone()
    g = torch.arange(c["H"], device="cuda") // (c["H"] // c["G"])
    for b, k in enumerate(d["slots"].tolist()):
        if k >= 0:
            delta = torch.nn.functional.softplus(d["dt"][b] + d["dt_bias"], threshold=50.0)
            state[k] = torch.exp(delta * d["A"])[:, None, None] * d["state"][k] \
                + torch.einsum("hp,hn->hpn", delta[:, None] * d["x"][b], d["B"][b][g])
            out[b] = torch.einsum("hpn,hn->hp", state[k], d["C"][b][g]) + d["D"][:, None] * d["x"][b]
    return [out, state]


def _exact_norm(c, d):
    rows, F = c["rows"], c["F"]
    unit = lambda v: v / torch.sqrt(v.square().sum(-1, keepdim=True) / F + _EPS)  # noqa: E731
    t = unit(d["o"]) * d["w_post"] if c["post"] else d["o"]
    if c["gates"]:
        t = t * d["gate"].repeat_interleave(rows // c["gates"], 0)
    rn = d["r"] + c["scale"] * t
    h = unit(rn) * d["w_pre"]
    out = [rn, h]
    if c["grad"]:
        wrt = [d["r"], d["o"], d["w_pre"]] + [d[k] for k, on in (("w_post", c["post"]), ("gate", c["gates"])) if on]
        out += torch.autograd.grad((h * d["dh"]).sum() + (rn * d["dr"]).sum(), wrt)
    return out


_EXACT = {"conv": _exact_conv, "conv_step": _exact_conv_step, "scan": _exact_scan,
          "scan_step": _exact_scan_step, "ssd_step": _exact_ssd_step, "norm": _exact_norm}
