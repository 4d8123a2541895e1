"""Cases of the gated delta rule (prefill, backward, decode step) and of the gated norm (forward, backward).

Gated delta rule, per batch row and value head, state S (headdim x dstate):

    Delta = softplus(dt + dt_bias),  a = exp(Delta A),  beta = sigmoid(beta_raw)
    S <- a S;  u = beta (v - S k);  S <- S + u k^T;  y = scale S q

with k and q scaled to unit length (x / sqrt(|x|^2 + 1e-6)) and shared by groups of value heads.

Gated norm, per row and group: h = residual + residual_scale x (or x), y = RMSNorm(h silu(z)) w
("first") or RMSNorm(h) w silu(z) ("last"), or no gate.
"""
import math

import torch

own = False

CHUNK = 64
QK_EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- the cases --

def _delta(op, name, B, L, H, Hk, P, N, dtype="bf16", h0=False, last=True):
    c = {"op": op, "B": B, "L": L, "H": H, "Hk": Hk, "P": P, "N": N, "dtype": dtype, "h0": h0,
         "last": last}
    if name:
        c["name"] = name
    return c


def _norm(op, name, rows, dim, groups=1, dtype="bf16", gate="none", residual="none"):
    c = {"op": op, "rows": rows, "dim": dim, "groups": groups, "dtype": dtype, "gate": gate,
         "residual": residual}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # a short prompt continued from a carried state, ragged against any chunk length
        _delta("delta_fwd", "delta_fwd_short", 1, 100, 16, 8, 64, 64, h0=True),
        # the prefill of one long prompt: few heads in all, so the sequence is the long axis
        _delta("delta_fwd", "delta_fwd_prompt", 1, 8192, 32, 16, 128, 128),
        # a training-sized layer of 64 heads of 64, d_state 128, 4 x 4096 tokens
        _delta("delta_fwd", "delta_fwd_layer", 4, 4096, 64, 16, 64, 128),
        # fp32 io, an odd head width and length (a numerics check of a small model)
        _delta("delta_fwd", "delta_fwd_fp32", 2, 333, 6, 2, 40, 64, dtype="fp32", h0=True),
        # truncated backpropagation through a short ragged window, with a carried state
        _delta("delta_bwd", "delta_bwd_window", 2, 203, 8, 4, 64, 64, h0=True),
        # the backward pass of a training layer
        _delta("delta_bwd", "delta_bwd_layer", 2, 2048, 32, 16, 128, 128, last=False),
        # one decode step of one sequence: latency
        _delta("delta_update", "delta_update_b1", 1, 1, 32, 16, 128, 128, h0=True),
        # one decode step of 64 sequences of 64 heads of 64, d_state 128
        _delta("delta_update", "delta_update_b64", 64, 1, 64, 16, 64, 128, h0=True),
        # the gated output norm of a decode step, 128 sequences of a 4096-wide layer, 8 groups
        _norm("norm_fwd", "norm_fwd_decode", 128, 4096, 8, gate="first"),
        # the norm before a block with the residual stream in fp32, 4 x 4096 tokens of 4096
        _norm("norm_fwd", "norm_fwd_residual", 16384, 4096, residual="fp32"),
        # the gated norm of every head of a layer in training: rows of one head's width
        _norm("norm_bwd", "norm_bwd_heads", 2 * 2048 * 32, 128, gate="last"),
        # the norm before a block, backward, fp32, an odd width
        _norm("norm_bwd", "norm_bwd_fp32", 1000, 1537, dtype="fp32", residual="fp32"),
    ]


def _cost(c):
    return work(c)["bytes"]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["delta_fwd", "delta_fwd", "delta_bwd", "delta_update", "norm_fwd", "norm_bwd"])
    if op.startswith("delta"):
        Hk = rng.choice([1, 2, 4, 8, 16])
        H = Hk * rng.choice([1, 2, 4])
        if op == "delta_bwd":
            c = _delta(op, None, rng.randint(1, 4), log(1, 2048), H, Hk,
                       16 * rng.randint(1, 8), rng.choice([64, 128]), h0=rng.random() < 0.5,
                       last=rng.random() < 0.5)
            most = 2 * 2048 * 32 * 128 * 128
        elif op == "delta_update":
            c = _delta(op, None, log(1, 256), 1, H, Hk, rng.randint(8, 128),
                       rng.choice([32, 64, 128, 256]), rng.choice(["bf16", "bf16", "fp32"]), h0=True)
            most = 64 * 64 * 64 * 128
        else:
            dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
            if rng.random() < 0.3:  # any head width and state, on any length up to 1024
                c = _delta(op, None, rng.randint(1, 4), log(1, 1024), H, Hk, rng.randint(8, 128),
                           rng.choice([32, 64, 128, 256]), dtype, rng.random() < 0.5)
            else:
                c = _delta(op, None, rng.randint(1, 4), log(1, 8192 if dtype == "bf16" else 1024), H,
                           Hk, 16 * rng.randint(1, 8), rng.choice([64, 128]), dtype,
                           rng.random() < 0.5)
            most = 4 * 4096 * 64 * 64 * 128
        while c["B"] * c["L"] * c["H"] * c["P"] * c["N"] > most:
            if c["L"] > 1:
                c["L"] = (c["L"] + 1) // 2
            else:
                c["B"] = (c["B"] + 1) // 2
        return c
    groups = rng.choice([1, 1, 2, 4, 8])
    c = _norm(op, None, log(1, 16384), groups * log(16, 8192 // groups), groups,
              rng.choice(["bf16", "bf16", "fp32"]), rng.choice(["none", "first", "last"]),
              rng.choice(["none", "io", "fp32"]))
    while c["rows"] * c["dim"] > 16384 * 4096 // (1 if op == "norm_fwd" else 4):
        c["rows"] = (c["rows"] + 1) // 2
    return c


def work(case):
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    if c["op"].startswith("delta"):
        B, L, H, Hk, P, N = (c[k] for k in ("B", "L", "H", "Hk", "P", "N"))
        qk, v, gate, state = 2 * B * L * Hk * N, B * L * H * P, 2 * B * L * H, B * H * P * N
        if c["op"] == "delta_bwd":
            # q, k, v, dt, beta, dy in; dq, dk, dv, ddt, dbeta out; h0, dh_last in and dh0 out
            moved = es * (2 * qk + 3 * v + 2 * gate) + 4 * state * (3 if c["h0"] else 0)
            # S k, u k^T again, then dy q^T, dS k, dr k^T, S^T dy, dS^T u, S^T dr, <dS, S>
            return {"bytes": moved, "flops": 18 * B * L * H * P * N}
        moved = es * (qk + 2 * v + gate) + 4 * state * ((1 if c["h0"] else 0) + (1 if c["last"] else 0))
        return {"bytes": moved, "flops": 6 * B * L * H * P * N}
    n = c["rows"] * c["dim"]
    rs = {"none": 0, "io": es, "fp32": 4}[c["residual"]]
    z = es if c["gate"] != "none" else 0
    if c["op"] == "norm_fwd":
        return {"bytes": n * (2 * es + 2 * rs + z), "flops": 8 * n}
    # h, dy (and dh, z) in; dx (and dresidual, dz) out
    return {"bytes": n * (2 * es + (rs or es) + 2 * rs + 2 * z), "flops": 20 * n}


# --------------------------------------------------------------- the inputs --

def prepare(case, seed):
    c, dev = case, "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    ty = TYPES[c["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def uniform(lo, hi, *shape):
        return lo + (hi - lo) * torch.rand(shape, generator=gen, device=dev)

    s = {"case": dict(c)}
    if c["op"].startswith("delta"):
        B, L, H, Hk, P, N = (c[k] for k in ("B", "L", "H", "Hk", "P", "N"))
        bl = (B,) if c["op"] == "delta_update" else (B, L)
        # q, k and v as the causal convolution and its SiLU leave them
        for name, shape in (("q", (Hk, N)), ("k", (Hk, N)), ("v", (H, P))):
            x = normal(*bl, *shape)
            s[name] = (x * torch.sigmoid(x)).to(ty)
        s["dt"] = (0.5 * normal(*bl, H)).to(ty)
        s["beta"] = normal(*bl, H).to(ty)
        s["A"] = -uniform(1.0, 16.0, H)
        step = torch.exp(uniform(math.log(1e-3), math.log(0.1), H))
        s["dt_bias"] = torch.log(torch.expm1(step))
        s["h0"] = 0.5 * normal(B, H, P, N) if c["h0"] else None
        if c["op"] == "delta_bwd":
            s["dy"] = normal(B, L, H, P).to(ty)
            s["dh_last"] = 0.1 * normal(B, H, P, N) if c["h0"] else None
        return s
    rows, dim = c["rows"], c["dim"]
    rt = {"none": ty, "io": ty, "fp32": torch.float32}[c["residual"]]
    s["w"] = 1.0 + 0.1 * normal(dim)
    s["z"] = normal(rows, dim).to(ty) if c["gate"] != "none" else None
    s["scale"] = 0.7 if c["residual"] != "none" else 1.0
    if c["op"] == "norm_fwd":
        s["x"] = normal(rows, dim).to(ty)
        s["residual"] = (3.0 * normal(rows, dim)).to(rt) if c["residual"] != "none" else None
    else:
        s["h"] = (2.0 * normal(rows, dim)).to(rt)
        s["dy"] = normal(rows, dim).to(ty)
        s["dh"] = normal(rows, dim).to(rt) if c["residual"] != "none" else None
    return s


# -------------------------------------------------- the framework's own calls --

def _own(s):
    import selective_state_space_39_b200 as ssm
    c = s["case"]
    if c["op"] == "delta_fwd":
        y, h_last = ssm.ssm_gated_delta_fwd(s["q"], s["k"], s["v"], s["dt"], s["A"], s["beta"],
                                            dt_bias=s["dt_bias"], h0=s["h0"],
                                            return_last_state=c["last"])
        return {"y": y, "h_last": h_last}
    if c["op"] == "delta_update":
        y = ssm.ssm_gated_delta_update(s["h0"], s["q"], s["k"], s["v"], s["dt"], s["A"], s["beta"],
                                       dt_bias=s["dt_bias"])
        return {"y": y, "state": s["h0"]}
    if c["op"] == "delta_bwd":
        return ssm.ssm_gated_delta_bwd(s["q"], s["k"], s["v"], s["dt"], s["A"], s["beta"], s["dy"],
                                       dt_bias=s["dt_bias"], h0=s["h0"], dh_last=s["dh_last"],
                                       want_dh0=c["h0"])
    before = c["gate"] == "last"
    if c["op"] == "norm_fwd":
        y, h = ssm.ssm_gated_norm_fwd(s["x"], s["w"], z=s["z"], norm_before_gate=before,
                                      residual=s["residual"], residual_scale=s["scale"],
                                      groups=c["groups"])
        return {"y": y, "h": h if c["residual"] != "none" else None}
    return ssm.ssm_gated_norm_bwd(s["h"], s["w"], s["dy"], z=s["z"], norm_before_gate=before,
                                  dh=s["dh"], residual=c["residual"] != "none",
                                  residual_scale=s["scale"], groups=c["groups"])


# ---------------------------------------------------------- the plain forms --

def _gates(s):
    """Delta (fp32), the log decay (fp64: its sums are differences of far positions) and beta."""
    raw = s["dt"].double() + s["dt_bias"].double()
    delta = torch.where(raw > 20.0, raw, torch.log1p(torch.exp(raw)))
    return raw, delta, delta * s["A"].double(), torch.sigmoid(s["beta"].float())


def _unit(x):
    x = x.float()
    r = torch.rsqrt((x * x).sum(-1, keepdim=True) + QK_EPS)
    return x * r, r


def _chunked(x, n):
    """(B, L, H, ...) -> (B, H, n, CHUNK, ...), zeros past L."""
    B, L, H = x.shape[:3]
    pad = x.new_zeros((B, n * CHUNK, H) + tuple(x.shape[3:]))
    pad[:, :L] = x
    pad = pad.reshape((B, n, CHUNK, H) + tuple(x.shape[3:]))
    return pad.movedim(3, 1).contiguous()


def _flat(x, L):
    """(B, H, n, CHUNK, ...) -> (B, L, H, ...)."""
    B, H, n, C = x.shape[:4]
    return x.movedim(1, 3).reshape((B, n * C, H) + tuple(x.shape[4:]))[:, :L]


def _chunk_terms(s):
    """The chunks' operands. With G the running log decay inside a chunk, M_ij = k_i.k_j e^(G_i - G_j)
    below the diagonal and P_ij = q_i.k_j e^(G_i - G_j) on and below it; T = (I + M diag(beta))^-1."""
    c = s["case"]
    L, rep = c["L"], c["H"] // c["Hk"]
    n = (L + CHUNK - 1) // CHUNK
    raw, delta, g, beta = _gates(s)
    kn, kr = _unit(s["k"])
    qn, qr = _unit(s["q"])
    scale = c["N"] ** -0.5
    t = {"n": n, "raw": raw, "delta": delta, "beta_flat": beta, "kn": kn, "kr": kr, "qn": qn, "qr": qr,
         "scale": scale}
    K = _chunked(kn.repeat_interleave(rep, 2), n)
    Q = _chunked((qn * scale).repeat_interleave(rep, 2), n)
    V = _chunked(s["v"].float(), n)
    G = _chunked(g, n).cumsum(-1)
    beta = _chunked(beta, n)
    gamma = torch.exp((G[..., :, None] - G[..., None, :]).clamp(max=0.0)).float()
    keep = torch.ones(CHUNK, CHUNK, device=K.device).tril()
    M = (K @ K.transpose(-1, -2)) * gamma * keep.tril(-1)
    low = M * beta[..., None, :]
    T = torch.eye(CHUNK, device=K.device).expand(low.shape).contiguous()
    for i in range(1, CHUNK):  # forward substitution, all chunks at once
        T[..., i, :i] = -(low[..., i:i + 1, :i] @ T[..., :i, :i]).squeeze(-2)
    t |= {"K": K, "Q": Q, "V": V, "beta": beta, "gamma": gamma * keep, "M": M, "T": T,
          "W": (Q @ K.transpose(-1, -2)) * gamma * keep, "D": torch.exp(G).float(),
          "E": torch.exp(G[..., -1:] - G).float()}
    return t


def _forward(s, t, keep=False):
    c = s["case"]
    S = s["h0"].clone() if s["h0"] is not None else torch.zeros(
        (c["B"], c["H"], c["P"], c["N"]), device=t["K"].device)
    out, starts, rs = [], [], []
    for i in range(t["n"]):  # the state passes from chunk to chunk
        K, Q, D = t["K"][:, :, i], t["Q"][:, :, i], t["D"][:, :, i, :, None]
        r = t["T"][:, :, i] @ (t["V"][:, :, i] - D * (K @ S.transpose(-1, -2)))
        u = t["beta"][:, :, i, :, None] * r
        out.append(D * (Q @ S.transpose(-1, -2)) + t["W"][:, :, i] @ u)
        if keep:
            starts.append(S)
            rs.append(r)
        S = D[:, :, -1:] * S + u.transpose(-1, -2) @ (t["E"][:, :, i, :, None] * K)
    y = torch.stack(out, 2)
    return (y, S, starts, rs) if keep else (y, S)


def _delta_fwd(s):
    c = s["case"]
    t = _chunk_terms(s)
    y, S = _forward(s, t)
    return {"y": _flat(y, c["L"]).to(TYPES[c["dtype"]]), "h_last": S if c["last"] else None}


def _delta_bwd(s):
    c = s["case"]
    L, H, Hk, ty = c["L"], c["H"], c["Hk"], TYPES[c["dtype"]]
    t = _chunk_terms(s)
    y, S_end, starts, rs = _forward(s, t, keep=True)
    dO = _chunked(s["dy"].float(), t["n"])
    dS = s["dh_last"].clone() if s["dh_last"] is not None else torch.zeros_like(S_end)
    grads = [None] * t["n"]
    S_next = S_end
    for i in reversed(range(t["n"])):
        K, Q, V, W, M, T, gamma = (t[k][:, :, i] for k in ("K", "Q", "V", "W", "M", "T", "gamma"))
        D, E, beta = (t[k][:, :, i, :, None] for k in ("D", "E", "beta"))
        do, S, r = dO[:, :, i], starts[i], rs[i]
        u = beta * r
        dU = W.transpose(-1, -2) @ do + E * (K @ dS.transpose(-1, -2))
        dR = T.transpose(-1, -2) @ (beta * dU)
        X = (dR @ r.transpose(-1, -2)) * gamma.tril(-1)
        dbeta = (dU * r).sum(-1) - (X * (K @ K.transpose(-1, -2))).sum(-2)
        Nij = -X * beta.transpose(-1, -2)
        dW = (do @ u.transpose(-1, -2)) * gamma
        dQ = D * (do @ S) + dW @ K
        dK = E * (u @ dS) - D * (dR @ S) + dW.transpose(-1, -2) @ Q + Nij @ K + Nij.transpose(-1, -2) @ K
        # the log decays: d/dG_i = dy_i.y_i - dv_i.v_i, and <S, dS> at the chunk's end
        dG = (do * y[:, :, i]).sum(-1) - (dR * V).sum(-1)
        dg = dG.flip(-1).cumsum(-1).flip(-1) + (S_next * dS).sum((-1, -2))[..., None]
        dS = D[:, :, -1:] * dS + (D * do).transpose(-1, -2) @ Q - dR.transpose(-1, -2) @ (D * K)
        grads[i] = (dQ, dK, dR, dbeta, dg)
        S_next = S
    dQ, dK, dV, dbeta, dg = (_flat(torch.stack([g[j] for g in grads], 2), L) for j in range(5))

    def shared(d, xn, xr, scale):  # sum over the group's heads, then through x / |x|
        d = d.reshape(d.shape[0], L, Hk, H // Hk, d.shape[-1]).sum(3) * scale
        return (xr * (d - xn * (xn * d).sum(-1, keepdim=True))).to(ty)

    draw_ = dg * s["A"] * torch.sigmoid(t["raw"].float()).where(t["raw"] <= 20.0, torch.ones_like(dg))
    b = t["beta_flat"]
    return {"dq": shared(dQ, t["qn"], t["qr"], t["scale"]), "dk": shared(dK, t["kn"], t["kr"], 1.0),
            "dv": dV.to(ty), "ddt": draw_.to(ty), "dbeta": (dbeta * b * (1 - b)).to(ty),
            "dA": (dg * t["delta"]).sum((0, 1)).float(), "ddt_bias": draw_.sum((0, 1)),
            "dh0": dS if c["h0"] else None}


def _delta_update(s):
    c = s["case"]
    rep = c["H"] // c["Hk"]
    _, _, g, beta = _gates(s)
    k = _unit(s["k"])[0].repeat_interleave(rep, 1)
    q = _unit(s["q"])[0].repeat_interleave(rep, 1) * c["N"] ** -0.5
    S = torch.exp(g).float()[..., None, None] * s["h0"]
    u = beta[..., None] * (s["v"].float() - (S * k[:, :, None, :]).sum(-1))
    S = S + u[..., None] * k[:, :, None, :]
    s["h0"].copy_(S)
    return {"y": (S * q[:, :, None, :]).sum(-1).to(TYPES[c["dtype"]]), "state": s["h0"]}


def _norm_fwd(s):
    c = s["case"]
    ty, g = TYPES[c["dtype"]], c["groups"]
    h = s["x"].float()
    if c["residual"] != "none":
        h = s["residual"].float() + s["scale"] * h
    gate = s["z"].float() * torch.sigmoid(s["z"].float()) if c["gate"] != "none" else None
    u = (h * gate if c["gate"] == "first" else h).reshape(c["rows"], g, -1)
    y = (u * torch.rsqrt((u * u).mean(-1, keepdim=True) + 1e-5)).reshape(c["rows"], -1) * s["w"]
    if c["gate"] == "last":
        y = y * gate
    return {"y": y.to(ty), "h": h.to(s["residual"].dtype) if c["residual"] != "none" else None}


def _norm_bwd(s):
    c = s["case"]
    ty, g, rows = TYPES[c["dtype"]], c["groups"], c["rows"]
    h, dy, w = s["h"].float(), s["dy"].float(), s["w"]
    z = s["z"].float() if c["gate"] != "none" else None
    sig = torch.sigmoid(z) if z is not None else None
    u = h * z * sig if c["gate"] == "first" else h
    r = torch.rsqrt((u * u).reshape(rows, g, -1).mean(-1, keepdim=True) + 1e-5)
    n = (u.reshape(rows, g, -1) * r).reshape(rows, -1)
    dgate, dn = None, dy
    if c["gate"] == "last":
        dgate, dn = dy * n * w, dy * z * sig
    dw = (dn * n).sum(0)
    d = (dn * w).reshape(rows, g, -1)
    n3 = n.reshape(rows, g, -1)
    du = (r * (d - n3 * (d * n3).mean(-1, keepdim=True))).reshape(rows, -1)
    dh = du
    if c["gate"] == "first":
        dgate, dh = du * h, du * z * sig
    if s["dh"] is not None:
        dh = dh + s["dh"].float()
    return {"dx": (s["scale"] * dh).to(ty), "dz": (dgate * sig * (1 + z * (1 - sig))).to(ty) if z is not None else None,
            "dresidual": dh.to(s["h"].dtype) if c["residual"] != "none" else None, "dw": dw}


def run(state):
    if own:
        return _own(state)
    return {"delta_fwd": _delta_fwd, "delta_bwd": _delta_bwd, "delta_update": _delta_update,
            "norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd}[state["case"]["op"]](state)


# ------------------------------------------------------------- in 64 bits ----

def _token(S, x, at):
    """One token of the recurrence, in 64 bits; x holds (B, L, ...) operands."""
    a = torch.exp(x["g"][:, at])[..., None, None]
    k, q = x["k"][:, at, :, None, :], x["q"][:, at, :, None, :]
    S = a * S
    u = x["b"][:, at, :, None] * (x["v"][:, at] - (S * k).sum(-1))
    S = S + u[..., None] * k
    return S, (S * q).sum(-1)


def _operands(leaf, c):
    rep = c["H"] // c["Hk"]
    v = leaf["dt"] + leaf["dt_bias"]
    soft = torch.where(v > 20.0, v, torch.log1p(torch.exp(v.clamp(max=20.0))))

    def unit(x):
        return (x / torch.sqrt((x ** 2).sum(-1, keepdim=True) + QK_EPS)).repeat_interleave(rep, -2)

    return {"g": soft * leaf["A"], "b": 1 / (1 + torch.exp(-leaf["beta"])), "v": leaf["v"],
            "k": unit(leaf["k"]), "q": unit(leaf["q"]) / math.sqrt(c["N"])}


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if not c["op"].startswith("delta"):
        return _exact_norm(s, c)
    leaf = {k: s[k].double() for k in ("q", "k", "v", "dt", "beta", "A", "dt_bias")}
    S = s["h0"].double() if s["h0"] is not None else torch.zeros(
        (c["B"], c["H"], c["P"], c["N"]), dtype=torch.float64, device="cuda")
    if c["op"] == "delta_update":
        leaf = {k: (v[:, None] if v.dim() > 1 else v) for k, v in leaf.items()}
        S, y = _token(S, _operands(leaf, c), 0)
        return {"y": y, "state": S}
    if c["op"] == "delta_fwd":
        x, ys = _operands(leaf, c), []
        for i in range(c["L"]):
            S, y = _token(S, x, i)
            ys.append(y)
        return {"y": torch.stack(ys, 1), "h_last": S if c["last"] else None}
    # the backward pass by automatic differentiation, 32 tokens at a time from saved states
    step, starts = 32, []
    with torch.no_grad():
        x = _operands(leaf, c)
        S0 = S
        for i in range(c["L"]):
            if i % step == 0:
                starts.append(S)
            S, _ = _token(S, x, i)
    dS = s["dh_last"].double() if s["dh_last"] is not None else torch.zeros_like(S0)
    dx = {k: torch.zeros_like(v) for k, v in x.items()}
    for j in reversed(range(len(starts))):
        lo, hi = j * step, min(c["L"], (j + 1) * step)
        part = {k: v[:, lo:hi].detach().requires_grad_() for k, v in x.items()}
        start = starts[j].detach().requires_grad_()
        Sj, ys = start, []
        for i in range(hi - lo):
            Sj, y = _token(Sj, part, i)
            ys.append(y)
        loss = (torch.stack(ys, 1) * s["dy"][:, lo:hi].double()).sum() + (Sj * dS).sum()
        names = list(part)
        got = torch.autograd.grad(loss, [part[k] for k in names] + [start])
        for k, v in zip(names, got):
            dx[k][:, lo:hi] = v
        dS = got[-1]
    for v in leaf.values():
        v.requires_grad_()
    x = _operands(leaf, c)
    names = ["q", "k", "v", "dt", "beta", "A", "dt_bias"]
    got = torch.autograd.grad(sum((x[k] * dx[k]).sum() for k in x), [leaf[k] for k in names])
    return {"d" + k: v for k, v in zip(names, got)} | {"dh0": dS if c["h0"] else None}


def _exact_norm(s, c):
    def forward(h, w, z):
        gate = z / (1 + torch.exp(-z)) if z is not None else 1.0
        u = (h * gate if c["gate"] == "first" else h).reshape(c["rows"], c["groups"], -1)
        y = (u / torch.sqrt((u ** 2).mean(-1, keepdim=True) + 1e-5)).reshape(c["rows"], -1) * w
        return y * gate if c["gate"] == "last" else y

    w, z = s["w"].double(), s["z"].double() if s["z"] is not None else None
    if c["op"] == "norm_fwd":
        h = s["x"].double()
        if s["residual"] is not None:
            h = s["residual"].double() + s["scale"] * h
        return {"y": forward(h, w, z), "h": h if s["residual"] is not None else None}
    h = s["h"].double()
    ins = [t.requires_grad_() for t in (h, w, z) if t is not None]
    got = torch.autograd.grad((forward(h, w, z) * s["dy"].double()).sum(), ins)
    dh = got[0] + s["dh"].double() if s["dh"] is not None else got[0]
    return {"dx": s["scale"] * dh, "dz": got[2] if z is not None else None,
            "dresidual": dh if c["residual"] != "none" else None, "dw": got[1]}
