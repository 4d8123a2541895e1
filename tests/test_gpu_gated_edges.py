"""The gated delta rule and the gated norm where single tokens or heads differ
from the rest by many orders of magnitude, and at the edges of their dispatch,
against the float64 formulas of tests/delta_ref.py.

Tolerances as in test_gpu_gated_delta.py, on the tokens, rows or heads named."""
import pytest
import torch

from tests import delta_ref as R
from tests.test_gpu_gated_delta import BF, G, G32, S32, Y, bwd, check_fwd, cu, fwd, near

pytestmark = pytest.mark.gpu


# ------------------------------------------------ the gates' gradients -------
# Per head, of the root of the sum of squares of the tokens' parts. A decay's
# gradient is about e^g of the row products that suffix sums take it from
# (fp32, 64 terms: 8 * 2^-24 of a term, e^5 * 10 times that of the value), or a
# sum over pairs of two bf16 pieces each (2^-16): below 1e-3. With a state
# before or after the call, one token per sequence end meets it as bf16 (two
# roundings of 2^-9, the token up to all of the sum): 4e-3.
@pytest.mark.parametrize("states", [False, True], ids=["bare", "states"])
@pytest.mark.parametrize("L", [64, 130, 300])
@pytest.mark.parametrize("logs", [(0.5, 2.0, 3.0, 4.0), (4.4, 5.7, 8.0, 10.0), (12.0, 16.0, 19.0, 24.0)],
                         ids=str)
def test_gates_of_heads_that_decay_at_every_token(logs, L, states):
    d = R.make_delta(1, L, 4, 2, 64, 128, BF, 91, h0=states)
    d["A"] = -torch.tensor(logs)
    steps = torch.tensor([0.875, 1.0, 1.125]).repeat(L)[:L]
    d["dt"] = steps.to(BF).reshape(1, L, 1).repeat(1, 1, 4)
    d["dt_bias"] = None
    g = bwd(d, softplus=False)
    ref = R.delta_grads(d, softplus=False)
    for h in range(4):
        near(g["ddt"][:, :, h], ref["ddt"][:, :, h], G, f"ddt e^-{logs[h]}")
        part = ref["ddt"][0, :, h] / d["A"][h].double()  # each token's part of dA / step
        scale = (part * steps.double()).norm().item()
        off = abs(g["dA"][h].item() - ref["dA"][h].item()) / scale
        print(f"dA e^-{logs[h]}: {off:.2e}")
        assert off <= (4e-3 if states else 1e-3), (logs[h], off)


@pytest.mark.parametrize("P,N,H,Hk", [(16, 64, 2, 1), (128, 64, 2, 2), (80, 128, 3, 1), (128, 128, 2, 1)])
def test_gates_of_single_strong_decays(P, N, H, Hk):
    """A few tokens with decays of e^-4.5 .. e^-40 among weak ones, at every place
    of a chunk and of its blocks of 16: each token's gradient for itself, of the
    products (of a value with two bf16 roundings, G) that make it."""
    L = 200
    d = R.make_delta(2, L, H, Hk, P, N, BF, 92)
    d["A"] = -torch.ones(H)
    d["dt"] = torch.full((2, L, H), 0.0625, dtype=BF)
    at = [0, 1, 15, 16, 17, 31, 40, 63, 64, 65, 100, 127, 128, 150, 191, 192, 199]
    for i, t in enumerate(at):
        d["dt"][:, t] = (4.5, 7.0, 11.0, 16.0, 22.0, 40.0)[i % 6]
    d["dt_bias"] = None
    g = bwd(d, softplus=False)
    ref = R.delta_grads(d, softplus=False)
    got, want = g["ddt"].double().cpu(), ref["ddt"]
    for i in range(6):  # the tokens of one strength together
        near(got[:, at[i::6]], want[:, at[i::6]], (2 * G[0], 2 * G[1]), f"strength {i}")
    weak = [t for t in range(L) if t not in at]
    near(got[:, weak], want[:, weak], G, "weak")


@pytest.mark.parametrize("raw", [None, 5.0, -12.0, -40.0])
def test_beta_gradient_of_repeated_keys(raw):
    """Equal keys and hardly any decay: a token's write is undone by the next
    ones, and its gradient is the small difference."""
    d = R.make_delta(1, 130, 2, 1, 32, 64, BF, 3)
    d["k"][:] = d["k"][:, :1]
    d["dt"][:] = -20
    if raw is not None:
        d["beta"][:] = raw
    g = bwd(d)
    ref = R.delta_grads(d)
    for n in ("dbeta", "dv", "dk", "dq"):
        near(g[n], ref[n], G, f"{n} raw {raw}")


def test_beta_gradient_beside_tokens_that_write_nothing():
    """Raw weights of 0, 1e-12 and 1e-3 beside 1: the gradient does not depend
    on the weight itself, a token's dv does."""
    d = R.make_delta(1, 100, 4, 2, 64, 64, BF, 6)
    d["beta"] = torch.ones_like(d["beta"])
    for i, b in enumerate((0.0, 1e-12, 1e-3, -1e-12)):
        d["beta"][:, i::5] = b
    g = bwd(d, beta_sigmoid=False)
    ref = R.delta_grads(d, beta_sigmoid=False)
    for i in range(5):
        near(g["dbeta"][:, i::5], ref["dbeta"][:, i::5], G, f"dbeta {i}")
        near(g["dv"][:, i::5], ref["dv"][:, i::5], G, f"dv {i}")
    assert not g["dv"][:, 0::5].any()


# ------------------------------------------ values far above the others ------
SHAPES = [(1, 130, 4, 2, 64, 128), (5, 70, 32, 16, 64, 64), (1, 130, 2, 1, 48, 64)]


def refer(d, **kw):
    return R.delta(**{k: d[k] for k in ("q", "k", "v", "dt", "A", "beta", "dt_bias", "h0")}, **kw)


def near_where_finite(got, ref, tol, what):
    """Finite exactly where the reference is, and near it there."""
    ok = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(got.float().cpu()), ok), what
    near(got.cpu()[ok], ref[ok], tol, what)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")], ids=str)
def test_an_infinite_value_reaches_only_later_tokens(shape, value):
    d = R.make_delta(*shape, BF, 21)
    d["v"][0, 40, 1, 5] = value
    y, S = fwd(d)
    yr, Sr = refer(d)
    near_where_finite(y, yr, Y, "y")
    near_where_finite(S, Sr, S32, "h_last")


@pytest.mark.parametrize("name", ["k", "dt", "beta", "q"])
def test_a_nan_of_a_token_reaches_only_later_tokens(name):
    d = R.make_delta(1, 130, 4, 2, 64, 128, BF, 22)
    d[name][0, 37, 1] = float("nan")
    y, S = fwd(d)
    yr, Sr = refer(d)
    near_where_finite(y, yr, Y, "y")
    near_where_finite(S, Sr, S32, "h_last")


@pytest.mark.parametrize("L0", [36, 50, 64, 100])
def test_padding_that_holds_anything(L0):
    """Tokens behind a sequence's last one, of NaN in every tensor: the ones
    before them are the call without padding."""
    d = R.make_delta(2, 130, 4, 2, 64, 64, BF, 23)
    cut = {k: (d[k][:, :L0].contiguous() if k in ("q", "k", "v", "dt", "beta") else d[k])
           for k in ("q", "k", "v", "dt", "A", "beta", "dt_bias", "h0")}
    yr, _ = refer(cut)
    for k in ("q", "k", "v", "dt", "beta"):
        d[k][:, L0:] = float("nan")
    y, S = fwd(d)
    near(y[:, :L0], yr, Y, "y")
    assert torch.isnan(S).all() and torch.isnan(y[:, L0:].float()).all()


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("value", [float("inf"), float("nan")], ids=str)
def test_a_state_that_is_not_finite(shape, value):
    """In one row of one head: that row only."""
    d = R.make_delta(*shape, BF, 24)
    d["h0"][0, 1, 7, 3] = value
    y, S = fwd(d)
    yr, Sr = refer(d)
    near_where_finite(y, yr, Y, "y")
    near_where_finite(S, Sr, S32, "h_last")


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("power", [20, 24, 30, 36, 60, 100])
@pytest.mark.parametrize("late", [False, True], ids=["token", "from"])
def test_a_large_value_leaves_earlier_tokens_alone(shape, power, late):
    """One token's v (or every one from it on) 2^power times the others'."""
    d = R.make_delta(*shape, BF, 25)
    if late:
        d["v"][:, 40:] *= 2.0 ** power
    else:
        d["v"][:, 40] *= 2.0 ** power
    y, S = fwd(d)
    yr, Sr = refer(d)
    near(y[:, :40], yr[:, :40], Y, "before")
    near(y[:, 40:], yr[:, 40:], Y, "behind")
    near(S, Sr, S32, "h_last")


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("power", [20, 24, 30, 36, 60])
def test_a_large_value_that_is_forgotten(shape, power):
    """A decay of e^-60 or more behind a large token, in its chunk: what follows
    does not remember it."""
    d = R.make_delta(*shape, BF, 26)
    d["v"][:, 20] *= 2.0 ** power
    d["dt"][:, 30] = 60
    y, S = fwd(d)
    yr, Sr = refer(d)
    near(y[:, :20], yr[:, :20], Y, "before")
    near(y[:, 30:], yr[:, 30:], Y, "behind")
    near(S, Sr, S32, "h_last")


@pytest.mark.parametrize("what", ["v", "dy"])
@pytest.mark.parametrize("value", [2.0 ** 24, 2.0 ** 36, float("inf"), float("nan")], ids=str)
@pytest.mark.parametrize("strong", [False, True], ids=["", "strong"])
def test_gradients_beside_a_large_value(what, value, strong):
    """A token's v reaches the gradients of no earlier token but through y, which
    dy does not see; a token's dy reaches those of no later token."""
    L, at = 130, 40
    d = R.make_delta(1, L, 4, 2, 64, 128, BF, 27)
    if strong:  # decays of e^-5 .. e^-40 on either side
        d["dt"][:, 30:32] = 2.5
        d["dt"][:, 50:53] = 2.5
    if value > 1 and value < float("inf"):
        d[what][:, at] *= value
    else:
        d[what][0, at, :, 5] = value
    g = bwd(d)
    ref = R.delta_grads(d)
    if what == "v":
        near(g["dv"], ref["dv"], G, "dv")
        near(g["dh0"], ref["dh0"], S32, "dh0")
        for n, end in (("dq", at), ("dk", at), ("dbeta", at), ("ddt", at + 1)):
            near(g[n][:, :end], ref[n][:, :end], G, n + " before")
    else:
        for n in ("dq", "dk", "dv", "dbeta", "ddt"):
            near(g[n][:, at + 1:], ref[n][:, at + 1:], G, n + " behind")
    for n in ("dq", "dk", "dv", "dbeta", "ddt"):  # nothing that is not finite turns finite
        bad = ~torch.isfinite(ref[n])
        assert not torch.isfinite(g[n].float().cpu()[bad]).any(), n


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("value", [float("inf"), float("nan")], ids=str)
def test_an_adjoint_that_is_not_finite(shape, value):
    """dh_last in one row of one head: no other row's dv and dh0, and no dq."""
    d = R.make_delta(*shape, BF, 28)
    d["dh_last"][0, 1, 7, 3] = value
    g = bwd(d)
    ref = R.delta_grads(d)
    near(g["dq"], ref["dq"], G, "dq")
    near_where_finite(g["dv"], ref["dv"], G, "dv")
    near_where_finite(g["dh0"], ref["dh0"], S32, "dh0")


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("power", [20, 28, 36, 60])
def test_a_large_gradient_leaves_later_tokens_alone(shape, power):
    """The tokens up to 30 with a dy of 2^power times the others'."""
    d = R.make_delta(*shape, BF, 29)
    d["dy"][:, :30] *= 2.0 ** power
    g = bwd(d)
    ref = R.delta_grads(d)
    for n in ("dq", "dk", "dv", "dbeta", "ddt"):
        near(g[n][:, 30:], ref[n][:, 30:], G, n + " behind")
        near(g[n][:, :30], ref[n][:, :30], G, n + " before")
    near(g["dh0"], ref["dh0"], S32, "dh0")


@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("power", [8, 12, 14, 16, 18, 20, 30, 60])
@pytest.mark.parametrize("late", [False, True], ids=["token", "from"])
def test_gates_before_a_large_value(N, power, late):
    """The decays' gradients of the tokens before it, and the heads' sums, which
    the large ones make up (suffix sums of fp32 row products: G32)."""
    d = R.make_delta(1, 130, 4, 2, 64, N, BF, 25)
    if late:
        d["v"][:, 40:] *= 2.0 ** power
    else:
        d["v"][:, 40] *= 2.0 ** power
    g = bwd(d)
    ref = R.delta_grads(d)
    near(g["ddt"][:, :41], ref["ddt"][:, :41], G, "before")
    near(g["ddt"][:, 41:], ref["ddt"][:, 41:], G, "behind")
    for n in ("dA", "ddt_bias"):
        near(g[n], ref[n], G32, n)


def test_gates_around_tokens_of_zeros():
    """Sequences that begin, pause and end with tokens of zeros (padding): their
    decays act on the state alone, or on nothing."""
    d = R.make_delta(1, 200, 4, 2, 64, 64, BF, 32, h0=False)
    for k in ("q", "k", "v", "dy"):
        d[k][:, :80] = 0
        d[k][:, 110:125] = 0
        d[k][:, 180:] = 0
    g = bwd(d)
    ref = R.delta_grads(d)
    assert not g["ddt"][:, :81].any() and not g["ddt"][:, 180:].any()
    for n in ("dq", "dk", "dv", "dbeta", "ddt"):
        near(g[n], ref[n], G, n)
    near(g["ddt"][:, 110:125], ref["ddt"][:, 110:125], G, "ddt of the pause")
    for n in ("dA", "ddt_bias"):
        near(g[n], ref[n], G32, n)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("power", [12, 18, 24, 40, 100])
@pytest.mark.parametrize("at", [0, 40, 63])
def test_a_long_key(shape, power, at):
    """Keys as they are (qk_norm off), one 2^power times the others: at a token
    that writes nothing (no state yet, v = 0) it changes nothing; at a later one
    the tokens before it."""
    d = R.make_delta(*shape, BF, 33, h0=at > 0)
    d["k"] = (d["k"].float() / 12).to(BF)
    d["k"][:, at] *= 2.0 ** power
    if at == 0:
        d["v"][:, 0] = 0
    d["dh_last"] = None
    y, S = fwd(d, qk_norm=False)
    g = bwd(d, qk_norm=False)
    yr, Sr = refer(d, qk_norm=False)
    ref = R.delta_grads(d, qk_norm=False)
    if at == 0:
        near(y, yr, Y, "y")
        near(S, Sr, S32, "h_last")
        for n in ("dq", "dv", "dbeta", "ddt"):
            near(g[n], ref[n], G, n)
        near(g["dk"][:, 1:], ref["dk"][:, 1:], G, "dk")
    else:
        near(y[:, :at], yr[:, :at], Y, "y before")
        near(g["dq"][:, :at], ref["dq"][:, :at], G, "dq before")


@pytest.mark.parametrize("power", [9, 20, 40])
@pytest.mark.parametrize("at", [0, 30, 63])
def test_a_large_write_strength(power, at):
    """beta as it is, one 2^power: nothing before it changes (and nothing at all
    where there is nothing to write)."""
    d = R.make_delta(1, 130, 4, 2, 64, 64, BF, 34, h0=at > 0)
    d["beta"] = torch.sigmoid(d["beta"].float()).to(BF)
    d["beta"][:, at] = 2.0 ** power
    if at == 0:
        d["v"][:, 0] = 0
    d["dh_last"] = None
    y, S = fwd(d, beta_sigmoid=False)
    yr, Sr = refer(d, beta_sigmoid=False)
    if at == 0:
        near(y, yr, Y, "y")
        near(S, Sr, S32, "h_last")
    else:
        near(y[:, :at], yr[:, :at], Y, "y before")


def test_a_recurrence_that_grows():
    """Steps beyond 2 / |k|^2: every write overshoots, the state grows by a factor
    of two a token for a while, then falls. y's products take one fp16 piece
    each of the state, u and P (2^-12, three of them), so a token's y is off by
    that of the largest y that its sum went through, beside its rounding."""
    d = R.make_delta(1, 100, 2, 1, 32, 64, BF, 35, h0=False)
    d["k"][:] = d["k"][:, :1]
    d["dt"][:] = -20
    d["beta"] = torch.full_like(d["beta"], 0.5)
    d["beta"][:, 20:34] = 3.0
    y, S = fwd(d, beta_sigmoid=False)
    yr, Sr = refer(d, beta_sigmoid=False)
    y = y.double().cpu()
    for t in range(100):
        off, most = (y[:, t] - yr[:, t]).norm(), yr[:, :t + 1].abs().max() * yr[:, t].numel() ** 0.5
        assert off <= Y[0] * yr[:, t].norm() + 3 * 2.0 ** -12 * most, t
    # a rounding of the state at its peak stays where keys do not reach: fp32's 2^-24 of
    # the peak, at each of the few steps that are near it
    peak = refer(dict(d, **{k: d[k][:, :34] for k in ("q", "k", "v", "dt", "beta")}), beta_sigmoid=False)[1].norm()
    assert (S.double().cpu() - Sr).norm() <= S32[0] * Sr.norm() + 4 * 2.0 ** -24 * peak


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("power", [12, 18])
def test_state_columns_of_different_sizes(shape, power):
    """Unit keys by turns of two columns, one column's values 2^power times the
    other's: each column for itself. Two pieces see the small one to 2^-40 of the
    large one's size, 2^-22 of its own at least; y's one piece of it has 2^-12."""
    d = R.make_delta(*shape, BF, 36, h0=False)
    L = shape[1]
    d["k"].zero_()
    d["k"][:, 0::2, :, 0] = 1
    d["k"][:, 1::2, :, 1] = 1
    d["q"].zero_()
    g = torch.Generator().manual_seed(37)
    at = torch.randint(0, 2, (L,), generator=g)
    d["q"][:, torch.arange(L), :, at] = 1
    d["v"][:, 0::2] *= 2.0 ** power
    y, S = fwd(d)
    yr, Sr = refer(d)
    for c in range(2):
        near(y[:, at == c], yr[:, at == c], Y, f"y of column {c}")
        near(S[..., c], Sr[..., c], S32, f"column {c}")
    assert not S[..., 2:].any()


# ------------------------------------------------ calls from two threads -----
def test_norm_gradients_of_several_widths_from_several_threads():
    """Rows that are read twice take shared memory for their width: a narrow
    call's limit must not stand in a wide one's way. The C calls themselves, so
    that little else is between them."""
    import threading

    from selective_state_space_39_b200 import gated_norm_bwd_workspace_bytes, lib, ssm_gated_norm_bwd
    fn, failed, keep = lib().ssm_gated_norm_bwd, [], []

    def calls(args):
        for _ in range(4000):
            rc = fn(*args)
            if rc != 0:
                failed.append((args[1], rc))
                return

    threads = []
    for width in (49152, 16384, 49151, 12416):
        h, dy = torch.randn(2, 2, width, device="cuda")
        w = torch.ones(width, device="cuda")
        dx, dw = torch.zeros_like(dy), torch.zeros_like(w)
        need = gated_norm_bwd_workspace_bytes(2, width, 1, torch.float32)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        stream = torch.cuda.Stream()
        keep.append((ssm_gated_norm_bwd(h, w, dy), dx, dw, h, dy, w, ws, stream))
        p = [t.data_ptr() for t in (h, w, dy, dx, dw, ws)]
        threads.append(threading.Thread(target=calls, args=((
            2, width, 1, 0, 0, p[0], 1.0, None, 0, p[1], 1e-5, p[2], None, p[3], None, None, p[4], p[5], need,
            stream.cuda_stream),)))
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for want, dx, dw, *_ in keep:
        assert torch.equal(dx, want["dx"]) and torch.equal(dw, want["dw"])


def test_another_library_s_stream():
    """An object that has a stream's pointer only."""
    from selective_state_space_39_b200 import ssm_gated_delta_fwd

    class Foreign:
        pass

    d = R.make_delta(1, 100, 4, 2, 64, 64, BF, 30)
    g = [cu(d[k]) for k in ("q", "k", "v", "dt", "A", "beta")]
    want, S = ssm_gated_delta_fwd(*g)
    side, f = torch.cuda.Stream(), Foreign()
    f.cuda_stream = side.cuda_stream
    side.wait_stream(torch.cuda.current_stream())
    y, S2 = ssm_gated_delta_fwd(*g, stream=f)
    side.synchronize()
    assert torch.equal(y, want) and torch.equal(S, S2)


# ------------------------------------------------ the edges of the dispatch --
# Chunks from 36 tokens on, or from 6 where tokens times state rows reach 2^17.
@pytest.mark.parametrize("shape,chunks", [((1, 35, 4, 2, 64, 64), False), ((1, 36, 4, 2, 64, 64), True),
                                          ((2, 5, 256, 16, 64, 64), False), ((2, 6, 256, 16, 64, 64), True),
                                          ((1, 7, 128, 16, 128, 128), False), ((1, 8, 128, 16, 128, 128), True),
                                          ((1, 31, 64, 16, 64, 128), False), ((1, 32, 64, 16, 64, 128), True)],
                         ids=str)
def test_both_sides_of_the_dispatch(shape, chunks):
    from selective_state_space_39_b200 import gated_delta_workspace_bytes
    assert (gated_delta_workspace_bytes(*shape) > 0) == chunks
    check_fwd(R.make_delta(*shape, BF, 31), BF, str(shape))


@pytest.mark.parametrize("which,by", [("y", 1), ("q", 4), ("k", 4), ("v", 1)])
def test_a_base_off_16_bytes_goes_token_by_token(which, by):
    """By `by` bf16 values: the results of the aligned call, to rounding, and
    nothing written beside y."""
    d = R.make_delta(1, 100, 2, 1, 32, 64, BF, 13)
    n = d["v" if which == "y" else which].numel()
    flat = torch.full((n + 2 * by,), 7.0, dtype=BF, device="cuda")
    at = flat[by:by + n].view(d["v" if which == "y" else which].shape)
    if which == "y":
        y, S = fwd(d, y=at)
        assert y is at
    else:
        at.copy_(d[which])
        y, S = fwd(dict(d, **{which: at}))
    yr, Sr = refer(d)
    near(y, yr, Y, "y")
    near(S, Sr, S32, "h_last")
    assert (flat[:by] == 7).all() and (flat[by + n:] == 7).all()

