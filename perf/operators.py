"""Cases of the head-decay linear attention and of the block norm, for timing and comparing.

Two families of operators, each with its backward pass or its single-token form:

* ``lindecay``: linear attention with one constant decay per head,
  S_t = g_h S_{t-1} + k_t v_t^T,  o_t = S_t^T q_t  with g_h = exp(log_a[h]):
  ``fwd`` (prompts, ragged batches, segments that carry a state), ``bwd`` (training) and
  ``step`` (one token over the states).
* ``blocknorm``: the norms around a block, x' = x + scale * act(gate) * norm_g(y) w_post and
  h = norm(x') w_pre: ``fwd`` and ``bwd``.

``run`` computes a case in plain torch operations (``own`` false) or through the library's
public calls (``own`` true); ``exact`` computes it in 64 bits, written from the recurrence.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ---------------------------------------------------------------------------------
def _lin(name, op, B, T, H, hpg, dk, dv, dtype="bf16", ragged=False, state=False):
    return {"name": name, "op": op, "B": B, "T": T, "H": H, "hpg": hpg, "dk": dk, "dv": dv, "dtype": dtype,
            "ragged": ragged, "state": state}


def _norm(name, op, rows, D, group, dtype="bf16", residual=True, gate=True, pre=True):
    return {"name": name, "op": op, "rows": rows, "D": D, "group": group, "dtype": dtype, "residual": residual,
            "gate": gate, "pre": pre}


def listed():
    return [
        # a chat turn: one short prompt, where the launches' latency is what counts
        _lin("fwd short prompt", "fwd", 1, 77, 16, 1, 64, 64, state=True),
        # the repository's own prompt workload: 48 heads in 24 q/k groups, state 128, head dim 64
        _lin("fwd prompts", "fwd", 4, 8192, 48, 2, 128, 64, state=True),
        # a long document read on from a carried state, odd length, few heads
        _lin("fwd long document", "fwd", 1, 100003, 16, 1, 128, 128, state=True),
        # a padded batch of unequal requests in fp32 (evaluation, small models)
        _lin("fwd ragged f32", "fwd", 3, 1501, 8, 1, 128, 64, dtype="f32", ragged=True, state=True),
        # a fine-tuning step of a small model: short rows
        _lin("bwd short rows", "bwd", 2, 500, 8, 1, 64, 64),
        # a training step at the repository's own shape, q and k shared by two heads
        _lin("bwd training", "bwd", 2, 8192, 48, 2, 128, 64),
        # one user generating: the smallest call there is
        _lin("step one user", "step", 1, 1, 48, 2, 128, 64),
        # the repository's decode batch: 64 users generating together
        _lin("step batch", "step", 64, 1, 48, 2, 128, 64),
        # the joint between two blocks while one token is generated
        _norm("norm fwd token", "norm_fwd", 1, 2048, 2048),
        # the same joint over the tokens of a batch of prompts
        _norm("norm fwd prompts", "norm_fwd", 32768, 4096, 4096),
        # the gated norm of each head's output, before the output projection, in an fp32 run
        _norm("norm bwd heads f32", "norm_bwd", 1000, 2048, 64, dtype="f32", residual=False, pre=False),
        # the joint in a training step
        _norm("norm bwd training", "norm_bwd", 16384, 4096, 4096),
    ]


def _log_int(rng, lo, hi):
    n = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n + 1 if n == 3072 else n


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "step", "norm_fwd", "norm_bwd"])
    if op.startswith("norm"):
        dtype = rng.choice(["bf16", "bf16", "f32"])
        group = rng.choice([0, 0, 32, 64, 128])
        D = _log_int(rng, 64, 8192)
        if group:
            D = max(1, D // group) * group
        elif rng.random() < 0.7:
            D = max(8, D // 8 * 8)
        D += (group or 8) * (D == 3072)
        rows = _log_int(rng, 1, max(1, min(65536, (1 << 26) // D)))
        residual = group == 0 or rng.random() < 0.3
        return {"op": op, "rows": rows, "D": D, "group": group or D, "dtype": dtype, "residual": residual,
                "gate": rng.random() < 0.7, "pre": residual and rng.random() < 0.7}
    dims = rng.choice([(128, 64), (64, 64), (128, 128), (64, 128), (32, 64), (40, 96), (80, 80), (128, 32)])
    hpg = rng.choice([1, 1, 2, 4])
    G = _log_int(rng, 1, 32)
    H = hpg * G
    B = _log_int(rng, 1, 256 if op == "step" else 8)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "step":
        while B * H > 4096:
            B = max(1, B // 2)
        return {"op": op, "B": B, "T": 1, "H": H, "hpg": hpg, "dk": dims[0], "dv": dims[1], "dtype": dtype,
                "ragged": False, "state": True}
    # token-heads: at most those of the largest listed case of the direction, fewer in fp32
    most = (1 << 17) if dtype == "f32" else (1 << 19) if op == "bwd" else (1 << 20)
    T = _log_int(rng, 1, max(2, min(100000, most // (B * H))))
    return {"op": op, "B": B, "T": T, "H": H, "hpg": hpg, "dk": dims[0], "dv": dims[1], "dtype": dtype,
            "ragged": rng.random() < 0.3, "state": rng.random() < 0.5}


# ---- inputs --------------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def randn(*shape, mul=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device=DEV) * mul).to(dtype)

    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"].startswith("norm"):
        R, D = case["rows"], case["D"]
        s["y"] = randn(R, D, dtype=dt)
        s["x"] = randn(R, D, mul=2.0, dtype=dt) if case["residual"] else None
        s["gate"] = randn(R, D, dtype=dt) if case["gate"] else None
        s["w_post"] = 1.0 + randn(D, mul=0.1)
        s["scale"] = 0.5 + randn(D, mul=0.1) if case["residual"] else None
        s["w_pre"] = 1.0 + randn(D, mul=0.1) if case["pre"] else None
        if case["op"] == "norm_bwd":
            s["dx_new"] = randn(R, D, dtype=dt)
            s["dh"] = randn(R, D, dtype=dt) if case["pre"] else None
            # x' as the forward left it (only the norm of x' reads it)
            s["x_new"] = randn(R, D, mul=2.0, dtype=dt) if case["pre"] else None
        return s
    B, T, H, dk, dv = case["B"], case["T"], case["H"], case["dk"], case["dv"]
    G, m = H // case["hpg"], dk ** -0.5
    # a geometric range of decays over the heads, from about exp(-1) to about exp(-1/256) a token
    h = torch.arange(1, H + 1, device=DEV, dtype=torch.float32)
    s["log_a"] = -torch.exp2(-8.0 * h / H) * (0.5 + torch.rand(H, generator=g, device=DEV))
    lead = (B,) if case["op"] == "step" else (B, T)
    s["q"], s["k"] = randn(*lead, G, dk, mul=m, dtype=dt), randn(*lead, G, dk, mul=m, dtype=dt)
    s["v"] = randn(*lead, H, dv, mul=m, dtype=dt)
    if case["op"] == "step":
        s["states"] = randn(B, H, dk, dv, mul=m)
        return s
    s["lengths"] = None
    if case["ragged"]:
        n = torch.randint(0, T + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
        n[0] = T  # the batch is padded to its longest request
        s["lengths"] = n
    s["state_in"] = randn(B, H, dk, dv, mul=m) if case["state"] else None
    if case["op"] == "bwd":
        s["dO"] = randn(B, T, H, dv, dtype=dt)
        s["dstate_out"] = randn(B, H, dk, dv) if case["state"] else None
    return s


# ---- the plain forms -----------------------------------------------------------------------
def _valid(s, T):
    """(B or 1, T, 1, 1) float mask of the tokens before each row's length, and the lengths."""
    t = torch.arange(T, device=DEV)
    if s["lengths"] is None:
        return torch.ones((1, T, 1, 1), device=DEV), torch.full((1,), T, device=DEV)
    n = s["lengths"].long()
    return (t < n[:, None]).float()[:, :, None, None], n


def _pairs(X, Y, Z, la):
    """sum over s <= t of exp(la (t - s)) (X_t . Y_s) Z_s for (B, T, H, .) in fp32, by chunks."""
    B, T, H, a = X.shape
    C = 128 if T <= 16384 else 512
    N = -(-T // C)
    pad = lambda x: torch.nn.functional.pad(x, (0, 0, 0, 0, 0, N * C - T)).reshape(B, N, C, H, -1).permute(0, 3, 1, 2, 4)  # noqa: E731
    X, Y, Z = pad(X), pad(Y), pad(Z)  # (B, H, N, C, .)
    i = torch.arange(C, device=DEV, dtype=torch.float32)
    lag = i[:, None] - i[None, :]
    la = la[:, None, None]
    D = torch.exp(la * lag.clamp(min=0)) * (lag >= 0)  # (H, C, C)
    out = torch.matmul(torch.matmul(X, Y.transpose(-1, -2)) * D[:, None], Z)
    if N > 1:
        U = torch.matmul((Y * torch.exp(la * (C - 1 - i)[:, None])[:, None]).transpose(-1, -2), Z)
        c = torch.arange(N, device=DEV, dtype=torch.float32)
        before = c[:, None] - 1 - c[None, :]
        M = torch.exp(la * C * before.clamp(min=0)) * (before >= 0)  # (H, N, N)
        P = torch.matmul(M, U.reshape(B, H, N, -1)).reshape(U.shape)
        out = out + torch.matmul(X * torch.exp(la * (i + 1)[:, None])[:, None], P)
    return out.permute(0, 2, 3, 1, 4).reshape(B, N * C, H, -1)[:, :T]


def _heads(x, H):
    return x.float().repeat_interleave(H // x.shape[-2], -2)


def _powers(la, e):
    """exp(la_h e) as (B, T, H, 1) for exponents e (B, T), 0 where e < 0."""
    return (torch.exp(la * e.clamp(min=0).float()[..., None]) * (e >= 0)[..., None])[..., None]


def _plain_fwd(s):
    q, k, v, la = s["q"], s["k"], s["v"].float(), s["log_a"]
    B, T, H, _ = v.shape
    ok, n = _valid(s, T)
    q, k, v = _heads(q, H) * ok, _heads(k, H) * ok, v * ok
    t = torch.arange(T, device=DEV)
    o = _pairs(q, k, v, la)
    left = (n[:, None] - 1 - t[None, :])  # (B or 1, T)
    st = torch.einsum("bthi,bthj->bhij", k * _powers(la, left), v)
    if s["state_in"] is not None:
        o = o + torch.einsum("bthi,bhij->bthj", q * _powers(la, (t + 1)[None, :]), s["state_in"])
        st = st + torch.exp(la[None, :] * n[:, None].float())[..., None, None] * s["state_in"]
    return (o * ok).to(s["v"].dtype), st


def _plain_bwd(s):
    q, k, v, la, dO = s["q"], s["k"], s["v"].float(), s["log_a"], s["dO"].float()
    B, T, H, _ = v.shape
    G = q.shape[2]
    ok, n = _valid(s, T)
    q, k, v, dO = _heads(q, H) * ok, _heads(k, H) * ok, v * ok, dO * ok
    t = torch.arange(T, device=DEV)
    left, since = n[:, None] - 1 - t[None, :], (t + 1)[None, :]
    back = lambda X, Y, Z: _pairs(X.flip(1), Y.flip(1), Z.flip(1), la).flip(1)  # noqa: E731
    dq, dk, dv = _pairs(dO, v, k, la), back(v, dO, q), back(k, q, dO)
    grads = []
    if s["state_in"] is not None:
        dq = dq + torch.einsum("bthj,bhij->bthi", dO * _powers(la, since), s["state_in"])
        dS = s["dstate_out"]
        dk = dk + torch.einsum("bthj,bhij->bthi", v * _powers(la, left), dS)
        dv = dv + torch.einsum("bthi,bhij->bthj", k * _powers(la, left), dS)
        dS0 = torch.einsum("bthi,bthj->bhij", q * _powers(la, since), dO)
        grads = [dS0 + torch.exp(la[None, :] * n[:, None].float())[..., None, None] * dS]
    dq, dk = ((x * ok).reshape(B, T, G, H // G, -1).sum(3).to(s["q"].dtype) for x in (dq, dk))
    return [dq, dk, (dv * ok).to(s["v"].dtype)] + grads


def _plain_step(s):
    H = s["v"].shape[1]
    q, k, v = _heads(s["q"], H), _heads(s["k"], H), s["v"].float()
    s["states"].mul_(torch.exp(s["log_a"])[None, :, None, None]).add_(k[..., None] * v[..., None, :])
    return (q[..., None] * s["states"]).sum(-2).to(s["v"].dtype), s["states"]


EPS = 1e-6


def _groups(x, group):
    return x.reshape(x.shape[0], -1, group)


def _plain_norm_fwd(s):
    group = s["case"]["group"]
    y = _groups(s["y"].float(), group)
    m = (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)).reshape(s["y"].shape) * s["w_post"]
    if s["gate"] is not None:
        gate = s["gate"].float()
        m = m * (gate * torch.sigmoid(gate))
    if s["x"] is not None:
        m = s["x"].float() + s["scale"] * m
    out = [m.to(s["y"].dtype)]
    if s["w_pre"] is not None:
        out.append((m * torch.rsqrt(m.square().mean(-1, keepdim=True) + EPS) * s["w_pre"]).to(s["y"].dtype))
    return out


def _plain_norm_bwd(s):
    group, dt = s["case"]["group"], s["y"].dtype
    dx, out = s["dx_new"].float(), {}
    if s["w_pre"] is not None:
        xn, dh = s["x_new"].float(), s["dh"].float()
        r = torch.rsqrt(xn.square().mean(-1, keepdim=True) + EPS)
        u = dh * s["w_pre"]
        out["dw_pre"] = (dh * xn * r).sum(0)
        dx = dx + r * (u - xn * r * r * (u * xn).mean(-1, keepdim=True))
    y = _groups(s["y"].float(), group)
    r = torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
    yn = (y * r).reshape(dx.shape)
    n = yn * s["w_post"]
    dm, act = dx, None
    if s["gate"] is not None:
        gate = s["gate"].float()
        sig = torch.sigmoid(gate)
        act = gate * sig
    if s["scale"] is not None:
        out["dx"] = dx.to(dt)
        out["dscale"] = (dx * (n if act is None else n * act)).sum(0)
        dm = dx * s["scale"]
    if act is not None:
        out["dgate"] = (dm * n * (sig * (1 + gate * (1 - sig)))).to(dt)
        dm = dm * act
    out["dw_post"] = (dm * yn).sum(0)
    u = _groups(dm * s["w_post"], group)
    out["dy"] = (r * (u - y * r * r * (u * y).mean(-1, keepdim=True))).reshape(dx.shape).to(dt)
    return out


# ---- the library's calls -------------------------------------------------------------------
def _own(s):
    import structured_mask_linear_gb300 as sml

    op = s["case"]["op"]
    if op == "fwd":
        B, _, H, dv = s["v"].shape
        st = torch.empty((B, H, s["q"].shape[3], dv), device=DEV)
        o = sml.lindecay_fwd(s["q"], s["k"], s["v"], s["log_a"], lengths=s["lengths"], state_in=s["state_in"],
                             state_out=st)
        return o, st
    if op == "bwd":
        ds = None if s["state_in"] is None else torch.empty_like(s["state_in"])
        grads = sml.lindecay_bwd(s["q"], s["k"], s["v"], s["log_a"], s["dO"], lengths=s["lengths"],
                                 state_in=s["state_in"], dstate_out=s["dstate_out"], dstate_in=ds)
        return list(grads) + ([] if ds is None else [ds])
    if op == "step":
        o = sml.lindecay_decode_step(s["q"], s["k"], s["v"], s["log_a"], s["states"])
        return o, s["states"]
    group = s["case"]["group"]
    if op == "norm_fwd":
        x_new, h = sml.blocknorm_fwd(s["y"], s["w_post"], x=s["x"], gate=s["gate"], scale=s["scale"],
                                     w_pre=s["w_pre"], group=group, eps=EPS)
        return [x_new] if h is None else [x_new, h]
    got = sml.blocknorm_bwd(s["dx_new"], s["y"], s["w_post"], dh=s["dh"], x_new=s["x_new"], gate=s["gate"],
                            scale=s["scale"], w_pre=s["w_pre"], group=group, eps=EPS)
    return {name: g for name, g in got._asdict().items() if g is not None}


def run(state):
    if own:
        return _own(state)
    return {"fwd": _plain_fwd, "bwd": _plain_bwd, "step": _plain_step, "norm_fwd": _plain_norm_fwd,
            "norm_bwd": _plain_norm_bwd}[state["case"]["op"]](state)


# ---- work ----------------------------------------------------------------------------------
def work(case):
    """Each input read once and each output written once; the operations of the recurrence."""
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("norm"):
        R, D = case["rows"], case["D"]
        vecs = 1 + case["residual"] + case["pre"]
        if case["op"] == "norm_fwd":
            acts = 2 + case["residual"] + case["gate"] + case["pre"]
            return {"bytes": acts * R * D * e + 4 * vecs * D, "flops": 12 * R * D}
        acts = 3 + case["residual"] + 2 * case["gate"] + 2 * case["pre"]
        return {"bytes": acts * R * D * e + 8 * vecs * D, "flops": 30 * R * D}
    B, T, H, dk, dv = case["B"], case["T"], case["H"], case["dk"], case["dv"]
    G, n = H // case["hpg"], B * T
    qk, vo, st = n * G * dk * e, n * H * dv * e, 4 * B * H * dk * dv
    if case["op"] == "step":
        return {"bytes": 2 * qk + 2 * vo + 2 * st + 4 * H, "flops": 5 * B * H * dk * dv}
    if case["op"] == "fwd":
        return {"bytes": 2 * qk + 2 * vo + st * (1 + case["state"]) + 4 * H, "flops": 4 * n * H * dk * dv}
    return {"bytes": 4 * qk + 3 * vo + st * 3 * case["state"] + 4 * H, "flops": 10 * n * H * dk * dv}


# ---- 64 bits, from the recurrence ----------------------------------------------------------
def _scan64(X, Y, Z, a, S, order):
    """X_t . S_t along `order` (lists of token positions, processed in turn), where S_t =
    a S + Y_t Z_t^T; X, Y, Z (T, ., .) one batch row, S (H, i, j), a (H,) the log-decay."""
    out = torch.zeros((X.shape[0], X.shape[1], Z.shape[2]), dtype=torch.float64, device=DEV)
    for idx in order:
        c = len(idx)
        i = torch.arange(c, device=DEV, dtype=torch.float64)
        x, y, z = (w[idx].transpose(0, 1) for w in (X, Y, Z))  # (H, c, .)
        lag = i[:, None] - i[None, :]
        D = torch.where(lag >= 0, torch.exp(a[:, None, None] * lag.clamp(min=0)), 0.0)
        o = (x @ y.transpose(1, 2) * D) @ z + torch.exp(a[:, None] * (i + 1))[..., None] * (x @ S)
        out[idx] = o.transpose(0, 1)
        S = torch.exp(a * c)[:, None, None] * S + (y * torch.exp(a[:, None] * (c - 1 - i))[..., None]).transpose(1, 2) @ z
    return out, S


def _order(n, back=False):
    t = torch.arange(n, device=DEV)
    return list((t.flip(0) if back else t).split(64)) if n else []


def _exact_lin(case, s):
    H, dt, a = case["H"], torch.float64, s["log_a"].double()
    wide = lambda x: x.double().repeat_interleave(H // x.shape[-2], -2)  # noqa: E731
    q, k, v = wide(s["q"]), wide(s["k"]), s["v"].double()
    B, T = q.shape[:2]
    G = s["q"].shape[2]
    n = [T] * B if s["lengths"] is None else s["lengths"].tolist()
    zero = torch.zeros((H, case["dk"], case["dv"]), dtype=dt, device=DEV)
    S0 = [zero] * B if s["state_in"] is None else list(s["state_in"].double())
    if case["op"] == "fwd":
        got = [_scan64(q[b], k[b], v[b], a, S0[b], _order(n[b])) for b in range(B)]
        return torch.stack([g[0] for g in got]), torch.stack([g[1] for g in got])
    dO = s["dO"].double()
    dS = [zero] * B if s["dstate_out"] is None else list(s["dstate_out"].double())
    # the state's gradient before token t's own term: dS_out has not decayed past the last token
    dS = [x / torch.exp(a)[:, None, None] for x in dS]
    outs = [[], [], [], []]
    for b in range(B):
        fwd, bwd = _order(n[b]), _order(n[b], True)
        outs[0].append(_scan64(dO[b], v[b], k[b], a, S0[b].transpose(1, 2), fwd)[0])
        outs[1].append(_scan64(v[b], dO[b], q[b], a, dS[b].transpose(1, 2), bwd)[0])
        dv, d0 = _scan64(k[b], q[b], dO[b], a, dS[b], bwd)
        outs[2].append(dv)
        outs[3].append(d0 * torch.exp(a)[:, None, None])
    dq, dk, dv, dS0 = (torch.stack(o) for o in outs)
    dq, dk = (x.reshape(B, T, G, H // G, -1).sum(3) for x in (dq, dk))
    return [dq, dk, dv] + ([] if s["state_in"] is None else [dS0])


def _exact_norm(case, s):
    """Forward in 64 bits; the backward by differentiating it."""
    d = {name: (x.double() if isinstance(x, torch.Tensor) else x) for name, x in s.items()}

    def rms(x, group):
        z = x.reshape(x.shape[0], -1, group)
        return (z / torch.sqrt(z.square().mean(-1, keepdim=True) + EPS)).reshape(x.shape)

    def block(y, gate, w_post, scale):
        m = rms(y, case["group"]) * w_post
        if gate is not None:
            m = m * gate / (1 + torch.exp(-gate))
        return m if scale is None else scale * m

    if case["op"] == "norm_fwd":
        m = block(d["y"], d["gate"], d["w_post"], d["scale"])
        x = m if d["x"] is None else d["x"] + m
        return [x] + ([rms(x, case["D"]) * d["w_pre"]] if d["w_pre"] is not None else [])
    need = {n: d[n].requires_grad_() for n in ("y", "gate", "w_post", "scale", "w_pre", "x_new") if d[n] is not None}
    dx, out = d["dx_new"], {}
    if case["pre"]:
        h = rms(d["x_new"], case["D"]) * d["w_pre"]
        gx, out["dw_pre"] = torch.autograd.grad(h, [need["x_new"], need["w_pre"]], d["dh"])
        dx = dx + gx
    names = [n for n in ("y", "gate", "w_post", "scale") if n in need]
    m = block(d["y"], d["gate"], d["w_post"], d["scale"])
    out.update({"d" + n: x for n, x in zip(names, torch.autograd.grad(m, [need[n] for n in names], dx))})
    if case["residual"]:
        out["dx"] = dx
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(case, s)
    if case["op"] == "step":
        H = case["H"]
        q, k = (s[n].double().repeat_interleave(case["hpg"], 1) for n in ("q", "k"))
        S = torch.exp(s["log_a"].double())[None, :, None, None] * s["states"].double()
        S = S + torch.einsum("bhi,bhj->bhij", k, s["v"].double())
        return torch.einsum("bhi,bhij->bhj", q.reshape(-1, H, case["dk"]), S), S
    return _exact_lin(case, s)
