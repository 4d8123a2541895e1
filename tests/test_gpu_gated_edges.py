"""The gated delta rule and the gated norm where single tokens or heads differ
from the rest by many orders of magnitude, and at the edges of their dispatch,
against the float64 formulas of tests/delta_ref.py.

Tolerances as in test_gpu_gated_delta.py, on the tokens, rows or heads named."""
import pytest
import torch

from tests import delta_ref as R
from tests.test_gpu_gated_delta import BF, F32Y, G, S32, Y, bwd, check_fwd, cu, fwd, near

pytestmark = pytest.mark.gpu


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
