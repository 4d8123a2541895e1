"""The gated delta rule (token by token, chunk by chunk, decode step, gradients)
against the float64 recurrence of tests/delta_ref.py.

Tolerances, as (2-norm, largest) relative differences:
  Y     bf16 output: the final rounding is at most 2^-8 of a value (2-norm below
        2^-8 / sqrt(3) = 2.3e-3 over a spread of mantissas); the chunk kernels
        add one fp16 rounding (2^-12) each of S, P and u, below 3 * 2^-12 =
        7.4e-4 in the 2-norm and a few times that for a single sum: 3.5e-3, 8e-3.
  S32   fp32 results of fp32 or two-piece fp16 products: operands to 2^-22,
        sums of at most 512 accumulation steps of at most 2^-23, random in sign
        (512^0.5 * 2^-23 = 2.7e-6) over a few dependent products: 2e-5, 5e-5.
  G     bf16 gradients: the final rounding (2.3e-3), and terms whose two
        operands are each rounded to bf16 (sqrt(2) * 2.3e-3 = 3.2e-3), up to
        four terms that may partly cancel (a factor 2): below 8e-3, 2e-2.
  G32   fp32 gate gradients: S32-accurate row products summed with signs: 1e-4."""
import pytest
import torch

from tests import delta_ref as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
Y, S32, G, G32 = (3.5e-3, 8e-3), (2e-5, 5e-5), (8e-3, 2e-2), (1e-4, 1e-4)
F32Y = (2e-5, 5e-5)


def cu(t):
    return None if t is None else t.cuda()


def fwd(d, **kw):
    from selective_state_space_39_b200 import ssm_gated_delta_fwd
    return ssm_gated_delta_fwd(cu(d["q"]), cu(d["k"]), cu(d["v"]), cu(d["dt"]), cu(d["A"]),
                               cu(d["beta"]), dt_bias=cu(d.get("dt_bias")), h0=cu(d.get("h0")), **kw)


def bwd(d, **kw):
    from selective_state_space_39_b200 import ssm_gated_delta_bwd
    return ssm_gated_delta_bwd(cu(d["q"]), cu(d["k"]), cu(d["v"]), cu(d["dt"]), cu(d["A"]),
                               cu(d["beta"]), cu(d["dy"]), dt_bias=cu(d.get("dt_bias")),
                               h0=cu(d.get("h0")), dh_last=cu(d.get("dh_last")), **kw)


def near(got, ref, tol, what):
    assert torch.isfinite(got.float()).all(), what
    a, b = R.dist(got, ref)
    print(f"{what}: {a:.2e} {b:.2e}")
    assert a <= tol[0] and b <= tol[1], (what, a, b)


def check_fwd(d, dtype, what, **kw):
    from selective_state_space_39_b200 import ssm_gated_delta_status
    y, S = fwd(d, **kw)
    assert ssm_gated_delta_status() == 0
    yr, Sr = R.delta(d["q"], d["k"], d["v"], d["dt"], d["A"], d["beta"], dt_bias=d.get("dt_bias"),
                     h0=d.get("h0"), **{k: v for k, v in kw.items() if k in
                                        ("softplus", "beta_sigmoid", "qk_norm", "scale")})
    near(y, yr, Y if dtype == BF else F32Y, what + " y")
    near(S, Sr, S32, what + " h_last")


@pytest.mark.parametrize("dtype", [F32, BF], ids=["fp32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 1, 32), (2, 7, 3, 1, 5, 64), (3, 31, 4, 2, 40, 128),
                                   (1, 19, 2, 2, 33, 256), (2, 65, 6, 3, 24, 32)])
def test_token_by_token(shape, dtype):
    """Any head width, one token, head counts that share keys: the step kernel."""
    d = R.make_delta(*shape, dtype, 10 + shape[1])
    check_fwd(d, dtype, f"{shape}")


@pytest.mark.parametrize("L", [32, 63, 64, 65, 127, 128, 200, 321])
@pytest.mark.parametrize("N", [64, 128])
def test_chunks_lengths(L, N):
    """Lengths around whole chunks, ragged last chunks."""
    check_fwd(R.make_delta(2, L, 4, 2, 64, N, BF, 100 + L), BF, f"L={L} N={N}")


@pytest.mark.parametrize("H,Hk,P", [(1, 1, 16), (3, 3, 48), (6, 2, 80), (8, 1, 128), (5, 1, 112),
                                    (2, 2, 160), (16, 4, 32)])
def test_chunks_heads(H, Hk, P):
    """Head widths in 16-row blocks (whole and part CTAs), heads sharing keys."""
    check_fwd(R.make_delta(1, 150, H, Hk, P, 128, BF, 7 * H + P, h0=P != 48), BF, f"{H} {Hk} {P}")


@pytest.mark.parametrize("kw", [dict(softplus=False), dict(beta_sigmoid=False), dict(qk_norm=False),
                                dict(scale=0.37), dict(softplus=False, beta_sigmoid=False)],
                         ids=str)
@pytest.mark.parametrize("P", [64, 24], ids=["chunks", "tokens"])
def test_options(kw, P):
    d = R.make_delta(2, 100, 4, 2, P, 64, BF, 5)
    if kw.get("softplus") is False:  # the steps themselves: positive and small
        d["dt"] = (d["dt"].float().abs() * 0.1).to(BF)
        d["dt_bias"] = None
    if kw.get("beta_sigmoid") is False:  # between 0 and 2, zeros among them
        d["beta"] = (2 * torch.sigmoid(d["beta"].float())).to(BF)
        d["beta"][:, ::5] = 0
    if kw.get("qk_norm") is False:  # short keys keep the recurrence stable
        d["k"] = (d["k"].float() / 12).to(BF)
    check_fwd(d, BF, str(kw), **kw)


def test_extreme_values():
    """Steps of 60 (decays of e^-60 .. e^-960) and of almost zero beside
    ordinary ones, zero keys and queries, large and small magnitudes per row."""
    d = R.make_delta(1, 200, 4, 2, 64, 128, BF, 77)
    d["dt"][:, 20:23] = 60
    d["dt"][:, 70] = 60
    d["dt"][:, 100:110] = -30
    d["k"][:, 40:50] = 0
    d["q"][:, 45:55] = 0
    d["k"][:, 120:130] *= 2.0 ** 20
    d["q"][:, 125:135] *= 2.0 ** -20
    d["v"][:, 140:150] *= 2.0 ** 12
    d["v"][:, :, :, 5] = 0
    check_fwd(d, BF, "extreme")


def test_repeated_keys():
    """Every token has the same key: T's entries do not decay along a row."""
    d = R.make_delta(1, 130, 2, 1, 32, 64, BF, 3)
    d["k"][:] = d["k"][:, :1]
    d["dt"][:] = -20
    check_fwd(d, BF, "same key")


@pytest.mark.parametrize("P", [64, 20], ids=["chunks", "tokens"])
def test_split_carries_the_state(P):
    """Two calls, the second from the first one's state (updated in place),
    against one call."""
    d = R.make_delta(1, 190, 4, 2, P, 64, BF, 21)
    yr, Sr = R.delta(**{k: d[k] for k in ("q", "k", "v", "dt", "A", "beta", "dt_bias", "h0")})
    ys, S = [], cu(d["h0"])
    for lo, hi in ((0, 77), (77, 190)):
        part = dict(d, h0=None, **{k: d[k][:, lo:hi].contiguous() for k in ("q", "k", "v", "dt", "beta")})
        part["h0"] = S
        y, S2 = fwd(part, h_last=S)
        assert S2 is S
        ys.append(y)
    near(torch.cat(ys, 1), yr, Y, "y")
    near(S, Sr, S32, "h_last")


@pytest.mark.parametrize("dtype", [F32, BF], ids=["fp32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 32), (5, 6, 2, 40, 64), (3, 4, 4, 64, 128), (2, 2, 1, 7, 256)])
def test_decode_steps(shape, dtype):
    """60 steps on a carried state: every y and the state, which stays the
    caller's tensor."""
    from selective_state_space_39_b200 import ssm_gated_delta_update
    B, H, Hk, P, N = shape
    d = R.make_delta(B, 60, H, Hk, P, N, dtype, 31)
    yr, Sr = R.delta(**{k: d[k] for k in ("q", "k", "v", "dt", "A", "beta", "dt_bias", "h0")})
    S = cu(d["h0"])
    g = {k: cu(d[k]) for k in ("q", "k", "v", "dt", "beta", "A", "dt_bias")}
    ys = [ssm_gated_delta_update(S, *(g[k][:, t].contiguous() for k in ("q", "k", "v", "dt")), g["A"],
                                 g["beta"][:, t].contiguous(), dt_bias=g["dt_bias"])
          for t in range(60)]
    near(torch.stack(ys, 1), yr, Y if dtype == BF else F32Y, "y")
    near(S, Sr, S32, "state")


def test_prefill_then_decode_in_a_graph():
    """A prefill's state continued by decode steps captured once and replayed."""
    from selective_state_space_39_b200 import ssm_gated_delta_update
    d = R.make_delta(2, 140, 4, 2, 64, 128, BF, 8, h0=False)
    yr, Sr = R.delta(**{k: d[k] for k in ("q", "k", "v", "dt", "A", "beta", "dt_bias", "h0")})
    pre = dict(d, **{k: d[k][:, :128].contiguous() for k in ("q", "k", "v", "dt", "beta")})
    y0, S = fwd(pre)
    g = {k: cu(d[k]) for k in ("q", "k", "v", "dt", "beta", "A", "dt_bias")}
    cur = {k: g[k][:, 128].clone() for k in ("q", "k", "v", "dt", "beta")}
    y = torch.empty_like(cur["v"])
    keep = S.clone()

    def step():
        ssm_gated_delta_update(S, cur["q"], cur["k"], cur["v"], cur["dt"], g["A"], cur["beta"],
                               dt_bias=g["dt_bias"], y=y)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    S.copy_(keep)
    ys = [y0]
    for t in range(128, 140):
        for k in cur:
            cur[k].copy_(g[k][:, t])
        graph.replay()
        ys.append(y.clone()[:, None])
    near(torch.cat(ys, 1), yr, Y, "y")
    near(S, Sr, S32, "state")


def check_bwd(d, what, **kw):
    from selective_state_space_39_b200 import ssm_gated_delta_status
    g = bwd(d, **kw)
    assert ssm_gated_delta_status() == 0
    ref = R.delta_grads(d, **kw)
    for name, t in ref.items():
        tol = G32 if name in ("dA", "ddt_bias") else S32 if name == "dh0" else G
        near(g[name], t, tol, f"{what} {name}")
    return g


@pytest.mark.parametrize("L", [1, 5, 63, 64, 65, 130, 200])
@pytest.mark.parametrize("N", [64, 128])
def test_bwd_lengths(L, N):
    check_bwd(R.make_delta(2, L, 4, 2, 64, N, BF, 300 + L), f"L={L} N={N}")


@pytest.mark.parametrize("H,Hk,P", [(1, 1, 16), (3, 3, 48), (6, 2, 80), (4, 1, 128)])
def test_bwd_heads(H, Hk, P):
    check_bwd(R.make_delta(1, 100, H, Hk, P, 128, BF, 40 + P, h0=P != 48), f"{H} {Hk} {P}")


@pytest.mark.parametrize("kw", [dict(softplus=False), dict(beta_sigmoid=False), dict(qk_norm=False),
                                dict(scale=0.37)], ids=str)
def test_bwd_options(kw):
    d = R.make_delta(2, 100, 4, 2, 64, 64, BF, 5)
    if kw.get("softplus") is False:
        d["dt"] = (d["dt"].float().abs() * 0.1).to(BF)
        d["dt_bias"] = None
    if kw.get("beta_sigmoid") is False:
        d["beta"] = (2 * torch.sigmoid(d["beta"].float())).to(BF)
        d["beta"][:, ::5] = 0  # a token that writes nothing has a gradient of its own
    if kw.get("qk_norm") is False:
        d["k"] = (d["k"].float() / 12).to(BF)
    check_bwd(d, str(kw), **kw)


def test_bwd_extreme_values():
    d = R.make_delta(1, 150, 4, 2, 64, 128, BF, 78)
    d["dt"][:, 20:23] = 60
    d["dt"][:, 100:110] = -30
    d["k"][:, 40:50] = 0
    d["q"][:, 45:55] = 0
    d["v"][:, :, :, 5] = 0
    d["dy"][:, 60:70] = 0
    check_bwd(d, "extreme")


def test_bwd_against_differences():
    """Directional derivatives of the float64 loss by central differences
    against the kernel's gradients (2-norm tolerance of a bf16 gradient times
    the direction's size)."""
    d = R.make_delta(1, 70, 2, 1, 32, 64, BF, 9)
    g = bwd(d)
    for name in ("q", "k", "v", "dt", "beta", "A", "dt_bias", "h0"):
        gen = torch.Generator().manual_seed(len(name))
        dirn = torch.randn(d[name].shape, generator=gen, dtype=torch.float64)
        eps = 1e-5
        hi = R.delta_loss(dict(d, **{name: d[name].double() + eps * dirn}))
        lo = R.delta_loss(dict(d, **{name: d[name].double() - eps * dirn}))
        want = ((hi - lo) / (2 * eps)).item()
        grad = g["ddt_bias" if name == "dt_bias" else "d" + name].double().cpu()
        got = (grad * dirn).sum().item()
        size = grad.norm().item() * 4  # a random direction of unit entries: |<g, d>| ~ |g|
        assert abs(got - want) <= (1e-4 if name in ("A", "dt_bias", "h0") else G[0]) * size, name


def test_bwd_is_repeatable_and_captured():
    """The same call twice and from a captured graph: the same bits."""
    d = R.make_delta(2, 200, 4, 2, 64, 128, BF, 55)
    a, b = bwd(d), bwd(d)
    from selective_state_space_39_b200 import ssm_gated_delta_bwd
    c = {k: cu(d[k]) for k in ("q", "k", "v", "dt", "A", "beta", "dy", "dt_bias", "h0", "dh_last")}
    args = [c.pop(k) for k in ("q", "k", "v", "dt", "A", "beta", "dy")]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        e = ssm_gated_delta_bwd(*args, **c)
    graph.replay()
    graph.replay()
    for k in a:
        assert torch.equal(a[k], b[k]) and torch.equal(a[k], e[k]), k


def test_misaligned_rows_go_token_by_token():
    """v and y two bytes off a 16-byte boundary: the same results from the step
    kernel (the chunk kernels copy whole units)."""
    d = R.make_delta(1, 80, 2, 1, 32, 64, BF, 13)
    flat = torch.zeros(d["v"].numel() + 1, dtype=BF, device="cuda")
    flat[1:] = cu(d["v"]).reshape(-1)
    y, S = fwd(dict(d, v=flat[1:].view(d["v"].shape)))
    yr, Sr = R.delta(**{k: d[k] for k in ("q", "k", "v", "dt", "A", "beta", "dt_bias", "h0")})
    near(y, yr, Y, "y")
    near(S, Sr, S32, "h_last")


def test_empty_sequences():
    d = R.make_delta(2, 0, 4, 2, 32, 64, BF, 1)
    y, S = fwd(d)
    assert y.shape == (2, 0, 4, 32) and torch.equal(S.cpu(), d["h0"])
    y, S = fwd(dict(d, h0=None))
    assert not S.any()
    g = bwd(d)
    assert torch.equal(g["dh0"].cpu(), d["dh_last"]) and not g["dA"].any() and not g["ddt_bias"].any()


def test_other_stream_and_given_outputs():
    """On a side stream, with outputs and workspace of the caller's; bytes
    behind them stay as they were."""
    from selective_state_space_39_b200 import gated_delta_workspace_bytes, ssm_gated_delta_fwd
    d = R.make_delta(2, 100, 4, 2, 48, 64, BF, 14)
    g = {k: cu(d[k]) for k in ("q", "k", "v", "dt", "A", "beta", "dt_bias", "h0")}
    n = d["v"].numel()
    buf = torch.full((n + 64,), 7.0, dtype=BF, device="cuda")
    need = gated_delta_workspace_bytes(2, 100, 4, 2, 48, 64)
    ws = torch.full((need + 256,), 5, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, S = ssm_gated_delta_fwd(g["q"], g["k"], g["v"], g["dt"], g["A"], g["beta"],
                               dt_bias=g["dt_bias"], h0=g["h0"], y=buf[:n].view(d["v"].shape),
                               workspace=ws[:need], stream=side)
    side.synchronize()
    yr, Sr = R.delta(**{k: d[k] for k in ("q", "k", "v", "dt", "A", "beta", "dt_bias", "h0")})
    near(y, yr, Y, "y")
    near(S, Sr, S32, "h_last")
    assert (buf[n:] == 7).all() and (ws[need:] == 5).all()


def test_wait_that_runs_out_is_reported(monkeypatch):
    from selective_state_space_39_b200 import ssm_gated_delta_status
    d = R.make_delta(1, 300, 2, 1, 64, 64, BF, 2)
    assert ssm_gated_delta_status() == 0
    monkeypatch.setenv("SSM_DELTA_TEST_STALL", "1")
    monkeypatch.setenv("SSM_SCAN_WAIT_LIMIT_NS", "20000000")
    fwd(d)
    assert ssm_gated_delta_status() == -5
    monkeypatch.delenv("SSM_DELTA_TEST_STALL")
    monkeypatch.delenv("SSM_SCAN_WAIT_LIMIT_NS")
    assert ssm_gated_delta_status() == 0
    check_fwd(d, BF, "after")


def test_refusals_on_the_gpu():
    from selective_state_space_39_b200 import SsmError, ssm_gated_delta_fwd, ssm_gated_delta_bwd
    d = {k: cu(v) for k, v in R.make_delta(1, 64, 4, 2, 32, 64, BF, 1).items()}
    args = [d[k] for k in ("q", "k", "v", "dt", "A", "beta")]
    with pytest.raises(SsmError):
        ssm_gated_delta_fwd(*args, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        ssm_gated_delta_fwd(d["q"].transpose(1, 2), *args[1:])
    with pytest.raises(TypeError):
        ssm_gated_delta_fwd(args[0].float(), *args[1:])
    with pytest.raises(TypeError):
        ssm_gated_delta_fwd(*[a.half() for a in args])
    with pytest.raises(ValueError):
        ssm_gated_delta_fwd(*args, h0=d["h0"][:, :2])
    with pytest.raises(ValueError):
        ssm_gated_delta_fwd(args[0], args[1].cpu(), *args[2:])
    with pytest.raises(SsmError):
        ssm_gated_delta_fwd(*args, y=d["v"])
    with pytest.raises(SsmError):  # fp32 gradients are not built
        ssm_gated_delta_bwd(*[a.float() for a in args], d["dy"].float())
    with pytest.raises(SsmError):  # 4 heads cannot share 3 keys
        ssm_gated_delta_fwd(*[torch.zeros(1, 64, 3, 64, dtype=BF, device="cuda")] * 2, *args[2:])
