"""The gated norm, forward and backward, against the float64 formula of
tests/delta_ref.py.

Tolerances, as (2-norm, largest over the largest): a bf16 output carries its
final rounding (2^-8 of a value, 2.3e-3 in the 2-norm) and fp32 arithmetic
with MUFU sigmoids (2^-21): 2.6e-3, 4.5e-3. An fp32 output carries sums of at
most 16384 terms taken by at most 64 fp32 steps per thread and 10 across
threads (74 * 2^-24 = 4.4e-6): 5e-6, 1e-5. dw sums the rows in fp32 too, in up
to 300 steps of random sign: 1e-5, 2e-5."""
import pytest
import torch

from tests import delta_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TOL = {BF: (2.6e-3, 4.5e-3), F32: (5e-6, 1e-5)}
DW = (1e-5, 2e-5)


def make(shape, dtype, rtype, gate, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    d = {"x": n(*shape).to(dtype), "w": 1 + 0.1 * n(shape[-1]), "dy": n(*shape).to(dtype),
         "z": n(*shape).to(dtype) if gate else None,
         "residual": (2 * n(*shape)).to(rtype) if rtype else None,
         "dh": n(*shape).to(rtype) if rtype else None}
    return d


def cu(t):
    return None if t is None else t.cuda()


def near(got, ref, tol, what, slack=None):
    assert torch.isfinite(got.float()).all(), what
    if slack is not None:  # differences within the slack count as none
        d = got.detach().double().cpu() - ref
        got = ref + torch.sign(d) * (d.abs() - slack).clamp(min=0)
    a, b = R.dist(got, ref)
    assert a <= tol[0] and b <= tol[1], (what, a, b)


def check(shape, dtype, rtype=None, gate=None, groups=1, seed=0, scale=0.7, eps=1e-5, d=None):
    from selective_state_space_39_b200 import ssm_gated_norm_bwd, ssm_gated_norm_fwd
    d = d or make(shape, dtype, rtype, gate, seed)
    before = gate == "last"
    s = scale if rtype else 1.0
    y, h = ssm_gated_norm_fwd(cu(d["x"]), cu(d["w"]), z=cu(d["z"]), norm_before_gate=before,
                              residual=cu(d["residual"]), residual_scale=s, groups=groups, eps=eps)
    yr, hr = R.norm(d["x"], d["w"], d["z"], before, d["residual"], s, groups, eps)
    near(y, yr, TOL[dtype], "y")
    if rtype:
        near(h, hr, TOL[rtype], "h")
    # gradients, from the h the forward call left
    hin = h.cpu().double().requires_grad_()
    w = d["w"].double().requires_grad_()
    z = d["z"].double().requires_grad_() if d["z"] is not None else None
    out, _ = R.norm(hin, w, z, before, groups=groups, eps=eps)
    ins = [t for t in (hin, w, z) if t is not None]
    got = torch.autograd.grad((out * d["dy"].double()).sum(), ins)
    dh = got[0] + (d["dh"].double() if rtype else 0)
    g = ssm_gated_norm_bwd(h, cu(d["w"]), cu(d["dy"]), z=cu(d["z"]), norm_before_gate=before,
                           dh=cu(d["dh"]), residual=rtype is not None, residual_scale=s,
                           groups=groups, eps=eps)
    # the slack of the difference (see above), through the gate where it comes first
    hd, sig = hin.detach(), (torch.sigmoid(d["z"].double()) if gate else None)
    silu = d["z"].double() * sig if gate else 1.0
    u = hd * silu if gate == "first" else hd
    t = d["dy"].double() * d["w"].double() * (silu if gate == "last" else 1.0)
    grp = lambda a: a.reshape(a.shape[:-1] + (groups, -1))  # noqa: E731
    inv = 1 / torch.sqrt((grp(u) ** 2).mean(-1, keepdim=True) + eps)
    n = grp(u) * inv
    slack = 16 * 2.0 ** -24 * inv * (grp(t).abs() + n.abs() * (grp(t) * n).abs().mean(-1, keepdim=True))
    slack = slack.reshape(u.shape)
    sh = slack * abs(silu) if gate == "first" else slack
    near(g["dx"], s * dh, TOL[dtype], "dx", s * sh)
    near(g["dw"], got[1], DW, "dw")
    if rtype:
        near(g["dresidual"], dh, TOL[rtype], "dresidual", sh)
    if gate:
        dsilu = sig * (1 + d["z"].double() * (1 - sig))
        near(g["dz"], got[2], TOL[dtype], "dz", slack * (hd * dsilu).abs() if gate == "first" else None)


@pytest.mark.parametrize("gate", [None, "first", "last"])
@pytest.mark.parametrize("dtype,rtype", [(BF, None), (BF, BF), (BF, F32), (F32, None), (F32, F32)],
                         ids=["bf16", "bf16_bf16", "bf16_fp32", "fp32", "fp32_fp32"])
@pytest.mark.parametrize("shape,groups", [((37, 128), 1), ((2, 5, 1024), 8), ((9, 1537), 1),
                                          ((3, 40), 5)], ids=str)
def test_types_gates_groups(shape, groups, dtype, rtype, gate):
    check(shape, dtype, rtype, gate, groups, seed=len(shape) * 100 + groups)


@pytest.mark.parametrize("dim", [1, 2, 7, 8, 16, 63, 64, 96, 256, 520, 2048, 4096, 8192, 16384, 16392,
                                 30000])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_widths(dim, dtype):
    """One element to rows longer than a block's registers; whole units and not."""
    check((6, dim), dtype, F32, "first", seed=dim)


@pytest.mark.parametrize("rows", [1, 2, 3, 17, 1000, 5003])
def test_rows(rows):
    """Fewer rows than a block takes, several slices of rows for dw."""
    check((rows, 64), BF, None, "last", seed=rows)


def test_zero_rows_and_large_values():
    """A zero row (only eps under the root), rows of 1e4 and gates at +-60."""
    d = make((12, 256), F32, None, "last", 4)
    d["x"][3] = 0
    d["x"][5] *= 1e4
    d["z"][:, ::7] = 60
    d["z"][:, 1::7] = -60
    check((12, 256), F32, None, "last", d=d)
    d["z"][:, ::7] = 3
    check((12, 256), F32, None, "first", d=d)


def test_empty_and_in_place():
    from selective_state_space_39_b200 import ssm_gated_norm_bwd, ssm_gated_norm_fwd
    w = torch.ones(64, device="cuda")
    y, h = ssm_gated_norm_fwd(torch.empty(0, 64, device="cuda"), w)
    assert y.shape == (0, 64)
    g = ssm_gated_norm_bwd(torch.empty(0, 64, device="cuda"), w, torch.empty(0, 64, device="cuda"))
    assert not g["dw"].any()
    d = make((10, 64), BF, F32, None, 5)  # the residual stream updated in place
    res = cu(d["residual"])
    y, h = ssm_gated_norm_fwd(cu(d["x"]), cu(d["w"]), residual=res, h=res)
    yr, hr = R.norm(d["x"], d["w"], None, False, d["residual"])
    assert h is res
    near(res, hr, TOL[F32], "h")
    near(y, yr, TOL[BF], "y")


def test_repeatable_and_captured():
    from selective_state_space_39_b200 import ssm_gated_norm_bwd
    d = {k: cu(v) for k, v in make((4000, 128), BF, None, "last", 6).items()}

    def call():
        return ssm_gated_norm_bwd(d["x"], d["w"], d["dy"], z=d["z"], norm_before_gate=True)

    a = call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b = call()
    graph.replay()
    for k in ("dx", "dz", "dw"):
        assert torch.equal(a[k], b[k])


def test_against_differences():
    from selective_state_space_39_b200 import ssm_gated_norm_bwd
    for gate in ("first", "last"):
        d = make((4, 48), F32, None, gate, 8)
        g = ssm_gated_norm_bwd(cu(d["x"]), cu(d["w"]), cu(d["dy"]), z=cu(d["z"]),
                               norm_before_gate=gate == "last", groups=2)
        for name, out in (("x", "dx"), ("z", "dz"), ("w", "dw")):
            v = torch.randn(d[name].shape, generator=torch.Generator().manual_seed(3), dtype=torch.float64)
            loss = lambda e: (R.norm(**{k: (d[k].double() + e * v if k == name else d[k].double())  # noqa: E731
                                        for k in ("x", "w", "z")}, norm_before_gate=gate == "last",
                                     groups=2)[0] * d["dy"].double()).sum()
            want = ((loss(1e-5) - loss(-1e-5)) / 2e-5).item()
            got = (g[out].double().cpu() * v).sum().item()
            assert abs(got - want) <= 1e-5 * g[out].double().norm().item() * 4, (gate, name)


def test_refusals_on_the_gpu():
    from selective_state_space_39_b200 import SsmError, ssm_gated_norm_bwd, ssm_gated_norm_fwd
    x, w = torch.zeros(4, 48, device="cuda"), torch.ones(48, device="cuda")
    with pytest.raises(SsmError):
        ssm_gated_norm_fwd(x, w, groups=5)
    with pytest.raises(SsmError):
        ssm_gated_norm_fwd(x, w, y=x)
    with pytest.raises(SsmError):
        ssm_gated_norm_fwd(x, w, residual=x.to(BF))
    with pytest.raises(ValueError):
        ssm_gated_norm_fwd(x, w, h=x)
    with pytest.raises(ValueError):
        ssm_gated_norm_bwd(x.to(BF), w, x)
    with pytest.raises(SsmError):
        ssm_gated_norm_bwd(x, w, x.clone(), workspace=torch.empty(4, dtype=torch.uint8, device="cuda"))
