"""The gated delta rule and the gated norm in 64 bits, token by token from
their formulas (torch float64 on the CPU; gradients by differentiation), and
inputs for their tests."""
import torch

F64 = torch.float64


def bf16(t):
    return t.to(torch.bfloat16)


def make_delta(B, L, H, Hk, P, N, dtype, seed, h0=True, dt_scale=0.5):
    """Inputs of one call on the CPU: q, k, v after a SiLU, dt ~ N(0, dt_scale^2)
    with a bias of 0.001 .. 0.1 steps, A in [-16, -1], raw beta ~ N(0, 1)."""
    g = torch.Generator().manual_seed(seed)

    def n(*s):
        return torch.randn(s, generator=g)

    def silu(x):
        return x * torch.sigmoid(x)

    d = {"q": silu(n(B, L, Hk, N)).to(dtype), "k": silu(n(B, L, Hk, N)).to(dtype),
         "v": silu(n(B, L, H, P)).to(dtype), "dt": (dt_scale * n(B, L, H)).to(dtype),
         "A": -(1 + 15 * torch.rand(H, generator=g)), "beta": n(B, L, H).to(dtype),
         "dt_bias": torch.log(torch.expm1(0.001 + 0.099 * torch.rand(H, generator=g)))}
    d["h0"] = 0.5 * n(B, H, P, N) if h0 else None
    d["dy"] = n(B, L, H, P).to(dtype)
    d["dh_last"] = 0.1 * n(B, H, P, N) if h0 else None
    return d


def delta(q, k, v, dt, A, beta, dt_bias=None, softplus=True, beta_sigmoid=True, qk_norm=True,
          scale=None, h0=None):
    """(y, h_last) in float64; differentiable."""
    q, k, v, dt, A, beta = (t.to(F64) for t in (q, k, v, dt, A, beta))
    B, L, H, P = v.shape
    Hk, N = q.shape[2], q.shape[3]
    step = dt + (dt_bias.to(F64) if dt_bias is not None else 0)
    if softplus:
        step = torch.where(step > 20, step, torch.log1p(torch.exp(step.clamp(max=20))))
    a = torch.exp(step * A)
    b = torch.sigmoid(beta) if beta_sigmoid else beta
    if qk_norm:
        q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + 1e-6)
        k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + 1e-6)
    q = q * (N ** -0.5 if scale is None else scale)
    S = h0.to(F64) if h0 is not None else torch.zeros(B, H, P, N, dtype=F64)
    ys = []
    head = torch.arange(H) // (H // Hk)
    for t in range(L):
        kt, qt = k[:, t][:, head], q[:, t][:, head]
        S = a[:, t, :, None, None] * S
        u = b[:, t, :, None] * (v[:, t] - torch.einsum("bhpn,bhn->bhp", S, kt))
        S = S + u[..., None] * kt[:, :, None, :]
        ys.append(torch.einsum("bhpn,bhn->bhp", S, qt))
    y = torch.stack(ys, 1) if L else torch.zeros(B, 0, H, P, dtype=F64)
    return y, S


def delta_grads(d, **kw):
    """Gradients of sum(dy y) + sum(dh_last h_last) with respect to every input."""
    names = ["q", "k", "v", "dt", "beta", "A"] + [n for n in ("dt_bias", "h0") if d.get(n) is not None]
    leaf = {n: d[n].to(F64).requires_grad_() for n in names}
    y, S = delta(**{n: leaf[n] for n in ("q", "k", "v", "dt", "A", "beta")},
                 dt_bias=leaf.get("dt_bias"), h0=leaf.get("h0"), **kw)
    loss = (y * d["dy"].to(F64)).sum()
    if d.get("dh_last") is not None:
        loss = loss + (S * d["dh_last"].to(F64)).sum()
    got = torch.autograd.grad(loss, [leaf[n] for n in names])
    return {("ddt_bias" if n == "dt_bias" else "d" + n): g for n, g in zip(names, got)}


def delta_loss(d, **kw):
    y, S = delta(d["q"], d["k"], d["v"], d["dt"], d["A"], d["beta"], dt_bias=d.get("dt_bias"),
                 h0=d.get("h0"), **kw)
    loss = (y * d["dy"].to(F64)).sum()
    return loss + (S * d["dh_last"].to(F64)).sum() if d.get("dh_last") is not None else loss


def norm(x, w, z=None, norm_before_gate=False, residual=None, residual_scale=1.0, groups=1,
         eps=1e-5):
    """(y, h) in float64; differentiable."""
    h = x.to(F64)
    if residual is not None:
        h = residual.to(F64) + residual_scale * h
    gate = None if z is None else z.to(F64) * torch.sigmoid(z.to(F64))
    u = h * gate if gate is not None and not norm_before_gate else h
    g = u.reshape(u.shape[:-1] + (groups, -1))
    n = (g / torch.sqrt((g * g).mean(-1, keepdim=True) + eps)).reshape(u.shape)
    y = n * w.to(F64)
    return (y * gate if gate is not None and norm_before_gate else y), h


def dist(got, ref):
    """(2-norm of the difference over the 2-norm, largest difference over the largest value)."""
    got, ref = got.detach().to("cpu", F64), ref.detach().to(F64)
    d = got - ref
    n2, nm = ref.norm().item(), ref.abs().max().item() if ref.numel() else 0.0
    if not ref.numel():
        return 0.0, 0.0
    return ((d.norm().item() / n2) if n2 else d.norm().item(),
            (d.abs().max().item() / nm) if nm else d.abs().max().item())
