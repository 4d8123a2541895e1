"""The gated delta rule and the gated norm as a layer uses them, after the
convolution, and the wide CTAs, streams and edges that the operators' own tests
do not reach, against the float64 formulas of tests/delta_ref.py.

Tolerances, as (2-norm, largest) relative differences, where a rounding to bf16
counts 2^-8 of a value (2-norm below 2.3e-3):
  LAYER  an output behind a chain of bf16 tensors, each rounded where the
         float64 chain is not: the convolution's output (three tensors, into q,
         k and v: two of them meet in every product), the rule's y, and the
         norm's output, with the 3.5e-3 of the rule itself: the root of the sum
         of squares is below 2.3e-3 * 5^0.5 + 3.5e-3 = 8.7e-3, twice that where
         k, scaled to unit length, meets itself (k k^T in the state's own
         correction): 1.8e-2; single values may be ten times the mean: 0.1.
  STATE  the fp32 state behind the rounded q, k, v: the same roundings without
         the last two: 1.5e-2, 0.1.
  GRAD   gradients through the chain: every tensor on the way forward and back
         is rounded (conv, y, dy of the norm, dq / dk / dv): 2 * LAYER.
The rest as in test_gpu_gated_delta.py."""
import pytest
import torch

from tests import delta_ref as R
from tests.test_gpu_gated_delta import BF, bwd, check_bwd, check_fwd, cu, fwd, near

pytestmark = pytest.mark.gpu
LAYER, STATE, GRAD = (1.8e-2, 0.1), (1.5e-2, 0.1), (3.6e-2, 0.2)
H, HK, P, N, W = 4, 2, 64, 64, 4


def layer_inputs(B, L, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    wide = 2 * HK * N + H * P
    return {"x": n(B, L, wide).to(BF), "w": 0.5 * n(wide, W), "bias": 0.1 * n(wide),
            "dt": (0.5 * n(B, L, H)).to(BF), "beta": n(B, L, H).to(BF),
            "A": -(1 + 15 * torch.rand(H, generator=g)),
            "dt_bias": torch.log(torch.expm1(0.001 + 0.099 * torch.rand(H, generator=g))),
            "z": n(B, L, H, P).to(BF), "nw": 1 + 0.1 * n(P), "res": n(B, L, H * P),
            "rw": 1 + 0.1 * n(H * P), "dout": n(B, L, H * P).to(BF)}


def split(c):
    B, L = c.shape[:2]
    q, k, v = c.split([HK * N, HK * N, H * P], dim=-1)
    return q.reshape(B, L, HK, N), k.reshape(B, L, HK, N), v.reshape(B, L, H, P)


def layer64(d):
    """(out, residual, state) in float64: causal convolution and SiLU, the delta rule,
    the gated norm of each head, then the residual sum and its norm."""
    x = d["x"].double()
    B, L = x.shape[:2]
    pad = torch.cat([torch.zeros(B, W - 1, x.shape[2], dtype=torch.float64), x], 1)
    c = d["bias"].double() + sum(d["w"].double()[:, j] * pad[:, j:j + L] for j in range(W))
    q, k, v = split(c * torch.sigmoid(c))
    y, S = R.delta(q, k, v, d["dt"], d["A"], d["beta"], dt_bias=d["dt_bias"])
    o, _ = R.norm(y, d["nw"], d["z"], True)
    out, h = R.norm(o.reshape(B, L, H * P), d["rw"], residual=d["res"])
    return out, h, S


def test_layer_prefill_then_decode():
    """Convolution, rule, gated norm, residual norm: 100 tokens at once, then 8
    one by one on the convolution's window and the state."""
    from selective_state_space_39_b200 import (ssm_conv1d_silu_fwd, ssm_conv1d_silu_update,
                                               ssm_gated_delta_fwd, ssm_gated_delta_update,
                                               ssm_gated_norm_fwd)
    B, L, L0 = 2, 108, 100
    d = layer_inputs(B, L, 3)
    g = {k: cu(t) for k, t in d.items()}

    def tail(y, z, res):
        o, _ = ssm_gated_norm_fwd(y, g["nw"], z=z, norm_before_gate=True)
        return ssm_gated_norm_fwd(o.view(res.shape), g["rw"], residual=res)

    pre = {k: g[k][:, :L0].contiguous() for k in ("x", "dt", "beta", "z", "res")}
    q, k, v = (t.contiguous() for t in split(ssm_conv1d_silu_fwd(pre["x"], g["w"], g["bias"])))
    y, S = ssm_gated_delta_fwd(q, k, v, pre["dt"], g["A"], pre["beta"], dt_bias=g["dt_bias"])
    outs, hs = ([t] for t in tail(y, pre["z"], pre["res"]))
    window = g["x"][:, L0 - W + 1:L0].transpose(1, 2).contiguous()
    for t in range(L0, L):
        c = ssm_conv1d_silu_update(window, g["x"][:, t].contiguous(), g["w"], g["bias"])
        q, k, v = (u[:, 0].contiguous() for u in split(c[:, None]))
        y = ssm_gated_delta_update(S, q, k, v, g["dt"][:, t].contiguous(), g["A"],
                                   g["beta"][:, t].contiguous(), dt_bias=g["dt_bias"])
        o, h = tail(y, g["z"][:, t].contiguous(), g["res"][:, t].contiguous())
        outs.append(o[:, None])
        hs.append(h[:, None])
    out, h, state = layer64(d)
    near(torch.cat(outs, 1), out, LAYER, "out")
    near(torch.cat(hs, 1), h, LAYER, "residual")
    near(S, state, STATE, "state")


def test_layer_gradients():
    """The backward calls in reverse order, against float64 differentiation."""
    from selective_state_space_39_b200 import (ssm_conv1d_silu_bwd, ssm_conv1d_silu_fwd,
                                               ssm_gated_delta_bwd, ssm_gated_delta_fwd,
                                               ssm_gated_norm_bwd, ssm_gated_norm_fwd)
    B, L = 2, 90
    d = layer_inputs(B, L, 5)
    g = {k: cu(t) for k, t in d.items()}
    c = ssm_conv1d_silu_fwd(g["x"], g["w"], g["bias"])
    q, k, v = (t.contiguous() for t in split(c))
    y, _ = ssm_gated_delta_fwd(q, k, v, g["dt"], g["A"], g["beta"], dt_bias=g["dt_bias"])
    o, _ = ssm_gated_norm_fwd(y, g["nw"], z=g["z"], norm_before_gate=True)
    out, h = ssm_gated_norm_fwd(o.view(B, L, H * P), g["rw"], residual=g["res"])
    b2 = ssm_gated_norm_bwd(h, g["rw"], g["dout"], residual=True)
    b1 = ssm_gated_norm_bwd(y, g["nw"], b2["dx"].view(B, L, H, P), z=g["z"], norm_before_gate=True)
    bd = ssm_gated_delta_bwd(q, k, v, g["dt"], g["A"], g["beta"], b1["dx"], dt_bias=g["dt_bias"])
    dc = torch.cat([bd[n].reshape(B, L, -1) for n in ("dq", "dk", "dv")], -1)
    bc = ssm_conv1d_silu_bwd(g["x"], g["w"], dc, g["bias"])
    got = {"x": bc["dx"], "w": bc["dw"], "bias": bc["dbias"], "dt": bd["ddt"], "beta": bd["dbeta"],
           "A": bd["dA"], "dt_bias": bd["ddt_bias"], "z": b1["dz"], "nw": b1["dw"], "rw": b2["dw"],
           "res": b2["dresidual"]}
    leaf = {n: d[n].double().requires_grad_() for n in got}
    ref = torch.autograd.grad((layer64({**d, **leaf})[0] * d["dout"].double()).sum(),
                              [leaf[n] for n in got])
    for n, r in zip(got, ref):
        near(got[n], r, GRAD, n)


# More groups of row blocks than SMs: the CTAs of eight blocks (one warp each), of one head,
# of two, and with a part of the last CTA empty; the backward walks then take four.
@pytest.mark.parametrize("shape", [(5, 70, 16, 16, 128, 128), (5, 130, 32, 16, 64, 64),
                                   (5, 70, 16, 16, 112, 64), (4, 70, 32, 16, 80, 128),
                                   (10, 33, 16, 16, 144, 64)], ids=str)
def test_wide_ctas(shape):
    check_fwd(R.make_delta(*shape, BF, 60 + shape[4]), BF, str(shape))


@pytest.mark.parametrize("shape", [(5, 70, 16, 16, 64, 128), (5, 70, 32, 16, 32, 64),
                                   (5, 66, 16, 16, 48, 64), (5, 65, 16, 16, 128, 64)], ids=str)
def test_wide_ctas_bwd(shape):
    check_bwd(R.make_delta(*shape, BF, 70 + shape[4]), str(shape))


@pytest.mark.parametrize("L", [7, 12, 20, 31])
def test_short_sequences_of_many_rows(L):
    """Short sequences over a state that fills the GPU."""
    check_fwd(R.make_delta(4, L, 64, 16, 64, 64, BF, L), BF, f"L={L}")


def test_first_token_without_a_state():
    """A first decay that has nothing to act on has no gradient: exactly zero."""
    d = R.make_delta(3, 1, 4, 2, 64, 128, BF, 4, h0=False)
    g = bwd(d)
    assert not g["ddt"].any() and not g["dA"].any() and not g["ddt_bias"].any()
    d = R.make_delta(3, 70, 4, 2, 64, 128, BF, 4, h0=False)
    g = bwd(d)
    assert not g["ddt"][:, 0].any() and g["ddt"][:, 1:].any()


def test_no_rows():
    """headdim 0: there is nothing to learn from, and the gradients say so."""
    d = R.make_delta(2, 40, 4, 2, 0, 64, BF, 1)
    g = bwd(d)
    for n in ("dq", "dk", "ddt", "dbeta", "dA", "ddt_bias"):
        assert not g[n].any(), n


def test_two_streams_at_once():
    """Two calls in flight with a workspace each: the bits of the calls alone."""
    a, b = R.make_delta(2, 500, 8, 4, 64, 128, BF, 1), R.make_delta(2, 300, 8, 2, 128, 64, BF, 2)
    alone = [fwd(a), fwd(b)]
    grads = [bwd(a), bwd(b)]
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got, back = [], []
    for _ in range(3):
        for d, st in ((a, s[0]), (b, s[1])):
            with torch.cuda.stream(st):
                got.append(fwd(d))
                back.append(bwd(d))
    torch.cuda.synchronize()
    for i in range(6):
        for x, y in zip(got[i], alone[i % 2]):
            assert torch.equal(x, y)
        for n in back[i]:
            assert torch.equal(back[i][n], grads[i % 2][n]), n


def test_a_call_on_a_given_stream_keeps_its_memory():
    """Results and workspace belong to the stream of the call: what the current
    stream allocates meanwhile is other memory."""
    from selective_state_space_39_b200 import ssm_gated_delta_fwd, ssm_gated_norm_fwd
    d = R.make_delta(2, 600, 8, 4, 64, 128, BF, 6)
    g = {k: cu(d[k]) for k in ("q", "k", "v", "dt", "A", "beta", "dt_bias", "h0")}
    want, S = fwd(d)
    w = torch.ones(64, device="cuda")
    normed, _ = ssm_gated_norm_fwd(want, w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        y, S2 = ssm_gated_delta_fwd(g["q"], g["k"], g["v"], g["dt"], g["A"], g["beta"],
                                    dt_bias=g["dt_bias"], h0=g["h0"], stream=side)
        n, _ = ssm_gated_norm_fwd(y, w, stream=side)
        junk = [torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
        side.synchronize()
        assert torch.equal(y, want) and torch.equal(S2, S) and torch.equal(n, normed)
        del junk


def test_shared_workspace_of_two_graphs():
    """Two graphs captured over one workspace, replayed in turn on one stream."""
    from selective_state_space_39_b200 import gated_delta_workspace_bytes, ssm_gated_delta_fwd
    ds = [R.make_delta(1, L, 4, 2, 64, 64, BF, L) for L in (200, 90)]
    ws = torch.empty(gated_delta_workspace_bytes(1, 200, 4, 2, 64, 64), dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for d in ds:
        g = {k: cu(d[k]) for k in ("q", "k", "v", "dt", "A", "beta", "dt_bias", "h0")}
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(ssm_gated_delta_fwd(g["q"], g["k"], g["v"], g["dt"], g["A"], g["beta"],
                                            dt_bias=g["dt_bias"], h0=g["h0"], workspace=ws))
        graphs.append((graph, g))
    want = [fwd(d) for d in ds]
    for i in (0, 1, 1, 0):
        graphs[i][0].replay()
        assert torch.equal(outs[i][0], want[i][0]) and torch.equal(outs[i][1], want[i][1])


def test_decays_above_one():
    """Growing states (A > 0, and steps of either sign without softplus)."""
    d = R.make_delta(1, 150, 4, 2, 64, 128, BF, 12)
    d["A"] = d["A"].abs() * 0.02
    check_fwd(d, BF, "A > 0")
    check_bwd(d, "A > 0")
    d = R.make_delta(1, 150, 4, 2, 64, 64, BF, 13)
    d["dt"] = (d["dt"].float() * 0.1).to(BF)
    d["A"], d["dt_bias"] = d["A"] * 0.1, None
    check_fwd(d, BF, "signed steps", softplus=False)


def big(B, L, Hh, Hk, Pp, Nn, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=BF)  # noqa: E731
    return {"q": n(B, L, Hk, Nn), "k": n(B, L, Hk, Nn), "v": n(B, L, Hh, Pp),
            "dt": n(B, L, Hh) - 3, "A": -1 - torch.arange(Hh, device="cuda") / 8.0,
            "beta": n(B, L, Hh), "dt_bias": torch.zeros(Hh, device="cuda"), "h0": None}


def row(d, b, lo, hi):
    return {n: (t[b:b + 1, lo:hi].contiguous() if t is not None and t.dim() > 1 else t)
            for n, t in d.items()}


def test_offsets_past_32_bits():
    """More than 2^31 elements of v: the last batch row is that row's own call,
    and its first tokens are the reference's."""
    d = big(2, 131136, 64, 16, 128, 64, 1)
    assert d["v"].numel() > 2 ** 31
    y, S = fwd(d)
    y1, S1 = fwd(row(d, 1, 0, 131136))
    assert torch.equal(y[1], y1[0]) and torch.equal(S[1], S1[0])
    c = {n: (t.cpu() if t is not None else None) for n, t in row(d, 1, 0, 70).items()}
    yr, _ = R.delta(c["q"], c["k"], c["v"], c["dt"], c["A"], c["beta"], dt_bias=c["dt_bias"])
    near(y[1:2, :70], yr, (3.5e-3, 8e-3), "y")


def test_bwd_offsets_past_32_bits():
    """More than 2^31 elements of states between the walks: the last batch row's
    gradients are those of the row's own call."""
    d = big(2, 65600, 64, 16, 128, 128, 2)
    g = torch.Generator(device="cuda").manual_seed(3)
    d["dy"] = torch.randn(d["v"].shape, generator=g, device="cuda", dtype=BF)
    assert 2 * 65600 // 64 * 64 * 128 * 128 > 2 ** 31
    a = bwd(d)
    b = bwd(row(d, 1, 0, 65600))
    for n in ("dq", "dk", "dv", "ddt", "dbeta", "dh0"):
        assert torch.isfinite(a[n][1].float()).all() and torch.equal(a[n][1], b[n][0]), n
