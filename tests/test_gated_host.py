"""The gated delta rule and the gated norm on the host: refusals before
anything is enqueued, workspace sizes, the binding's checks of arguments, and
the float64 gradients of tests/delta_ref.py against differences. Every call
with fake pointers is one that the library must reject on the host; they run
only on machines without a GPU."""
import ctypes

import pytest
import torch

from selective_state_space_39_b200 import _binding as bnd
from tests import delta_ref as R

no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(),
                                 reason="fake-pointer validation tests run only without a GPU")
M = 1 << 24  # distance between fake buffers


@pytest.fixture(scope="module")
def L():
    from selective_state_space_39_b200 import build
    build.build()
    return bnd.lib()


def at(i):
    return (i + 1) * M


def fwd(L, **kw):
    a = dict(batch=2, seqlen=100, nheads=4, nkheads=2, headdim=64, dstate=64, io=1, q=at(0), k=at(1),
             v=at(2), dt=at(3), A=at(4), beta=at(5), bias=None, sp=1, sg=1, qn=1, scale=0.125,
             h0=None, y=at(6), h_last=at(7), ws=None, ws_bytes=0, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return L.ssm_gated_delta_fwd(*a.values())


def upd(L, **kw):
    a = dict(batch=2, nheads=4, nkheads=2, headdim=64, dstate=64, io=1, state=at(8), q=at(0), k=at(1),
             v=at(2), dt=at(3), A=at(4), beta=at(5), bias=None, sp=1, sg=1, qn=1, scale=0.125,
             y=at(6), stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return L.ssm_gated_delta_update(*a.values())


def bwd(L, **kw):
    a = dict(batch=2, seqlen=100, nheads=4, nkheads=2, headdim=64, dstate=64, io=1, q=at(0), k=at(1),
             v=at(2), dt=at(3), A=at(4), beta=at(5), bias=None, sp=1, sg=1, qn=1, scale=0.125,
             h0=None, dy=at(6), dh_last=None, dq=at(7), dk=at(8), dv=at(9), ddt=at(10), dbeta=at(11),
             dA=at(12), dbias=at(13), dh0=at(14), ws=None, ws_bytes=0, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return L.ssm_gated_delta_bwd(*a.values())


@no_gpu_only
def test_delta_forward_refusals(L):
    assert fwd(L) == -3                                   # a chunked call needs a workspace
    need = L.ssm_gated_delta_workspace_bytes(2, 100, 4, 2, 64, 64, 1)
    assert fwd(L, ws=at(20), ws_bytes=need - 1) == -3
    assert fwd(L, ws=at(20) + 8, ws_bytes=need) == -3     # not 16-byte aligned
    assert fwd(L, ws=at(6), ws_bytes=need) == -1          # over y
    for name in ("q", "k", "v", "dt", "A", "beta"):
        assert fwd(L, **{name: None}) == -1, name
    assert fwd(L, y=None, h_last=None) == -1
    assert fwd(L, q=at(0) + 2) == -1 and fwd(L, k=at(1) + 4) == -1   # four bf16 at a time
    assert fwd(L, h0=at(9) + 8) == -1 and fwd(L, h_last=at(7) + 4) == -1
    assert fwd(L, y=at(2)) == -1 and fwd(L, h_last=at(0)) == -1 and fwd(L, y=at(7) + 64) == -1
    assert fwd(L, h0=at(9), h_last=at(9) + 16) == -1      # part of h0
    assert fwd(L, nkheads=3) == -1 and fwd(L, nkheads=0) == -1
    assert fwd(L, dstate=48) == -2 and fwd(L, dstate=512) == -2 and fwd(L, io=5) == -2
    assert fwd(L, seqlen=-1) == -1 and fwd(L, batch=70000) == -2
    assert fwd(L, batch=0) == 0 and fwd(L, headdim=0) == 0
    assert fwd(L, batch=60000, nheads=32768, nkheads=1, headdim=4096) == -2


@no_gpu_only
def test_delta_update_refusals(L):
    assert upd(L, state=None) == -1 and upd(L, y=None) == -1 and upd(L, q=None) == -1
    assert upd(L, state=at(8) + 8) == -1
    assert upd(L, y=at(8)) == -1 and upd(L, y=at(2)) == -1
    assert upd(L, state=at(0)) == -1                      # the state over q
    assert upd(L, dstate=16) == -2 and upd(L, nheads=3) == -1
    assert upd(L, batch=0) == 0


@no_gpu_only
def test_delta_backward_refusals(L):
    assert bwd(L) == -3
    need = L.ssm_gated_delta_bwd_workspace_bytes(2, 100, 4, 2, 64, 64, 1)
    assert bwd(L, ws=at(20), ws_bytes=need - 1) == -3
    assert bwd(L, ws=at(9), ws_bytes=need) == -1
    for name in ("q", "k", "v", "dt", "A", "beta", "dy", "dq", "dk", "dv", "ddt", "dbeta"):
        assert bwd(L, **{name: None}) == -1, name
    assert bwd(L, dq=at(8)) == -1                         # two outputs in one buffer
    assert bwd(L, dv=at(6)) == -1 and bwd(L, dh0=at(0)) == -1
    assert bwd(L, dy=at(6) + 2) == -1 and bwd(L, dA=at(12) + 2) == -1
    assert bwd(L, io=0) == -2 and bwd(L, dstate=32) == -2 and bwd(L, dstate=256) == -2
    assert bwd(L, headdim=40) == -2 and bwd(L, headdim=256) == -2
    assert bwd(L, nheads=0, nkheads=0) == 0


@no_gpu_only
def test_norm_refusals(L):
    def f(**kw):
        a = dict(rows=8, dim=64, groups=2, io=1, rd=1, x=at(0), res=None, scale=1.0, z=None, before=0,
                 w=at(2), eps=1e-5, y=at(3), h=None, stream=None)
        assert set(kw) <= set(a)
        a.update(kw)
        return L.ssm_gated_norm_fwd(*a.values())

    def b(**kw):
        a = dict(rows=8, dim=64, groups=2, io=1, hd=1, h=at(0), scale=1.0, z=None, before=0, w=at(2),
                 eps=1e-5, dy=at(3), dh=None, dx=at(4), dres=None, dz=None, dw=at(5), ws=None, wsb=0,
                 stream=None)
        assert set(kw) <= set(a)
        a.update(kw)
        return L.ssm_gated_norm_bwd(*a.values())

    assert f(x=None) == -1 and f(w=None) == -1 and f(y=None) == -1
    assert f(groups=3) == -1 and f(groups=0) == -1 and f(rows=-1) == -1
    assert f(res=at(6)) == -1                             # a residual without its sum
    assert f(h=at(6)) == -1                               # a sum without a residual
    assert f(y=at(0)) == -1 and f(res=at(6), h=at(0)) == -1 and f(res=at(6), h=at(6) + 64) == -1
    assert f(io=0, rd=1, res=at(6), h=at(7)) == -2 and f(io=9) == -2
    assert f(x=at(0) + 1) == -1 and f(w=at(2) + 2) == -1
    assert f(dim=49153, groups=1) == -2 and f(rows=1 << 31, groups=2) == -2
    assert f(rows=0) == 0 and f(dim=0) == 0
    assert b() == -3                                      # dw needs a workspace
    need = L.ssm_gated_norm_bwd_workspace_bytes(8, 64, 2, 1)
    assert need > 0 and b(ws=at(9), wsb=need - 1) == -3
    assert b(ws=at(4), wsb=need) == -1
    assert b(h=None) == -1 and b(dy=None) == -1 and b(dx=None) == -1
    assert b(z=at(6)) == -1 and b(dz=at(6)) == -1         # a gate and its gradient go together
    assert b(dx=at(0)) == -1 and b(dw=at(2)) == -1 and b(dx=at(5)) == -1


def test_workspace_sizes(L):
    w = L.ssm_gated_delta_workspace_bytes
    assert w(2, 31, 4, 2, 64, 64, 1) == 0                 # token by token
    assert w(2, 100, 4, 2, 40, 64, 1) == 0 and w(2, 100, 4, 2, 64, 32, 1) == 0
    assert w(2, 100, 4, 2, 64, 64, 0) == 0                # fp32 io
    # two chunks: k and q tiles of the key heads, a block per head
    assert w(2, 100, 4, 2, 64, 64, 1) == 2 * 2 * (2 * 2 * 64 * 64 * 2 + 4 * (7 * 256 + 3 * 5120))
    assert w(2, 100, 3, 2, 64, 64, 1) == 0
    assert L.ssm_gated_delta_bwd_workspace_bytes(2, 100, 4, 2, 64, 64, 0) == 0


def test_binding_refuses_wrong_tensors():
    d = R.make_delta(1, 40, 4, 2, 16, 64, torch.bfloat16, 1)
    args = [d[k] for k in ("q", "k", "v", "dt", "A", "beta")]
    with pytest.raises(ValueError):
        bnd.ssm_gated_delta_fwd(*args)                    # CPU tensors
    with pytest.raises(ValueError):
        bnd.ssm_gated_delta_fwd(args[0][0], *args[1:])    # three axes
    with pytest.raises(ValueError):
        bnd.ssm_gated_delta_update(d["h0"], *args)        # a sequence in a decode step
    with pytest.raises(ValueError):
        bnd.ssm_gated_norm_fwd(torch.zeros(2, 8), torch.ones(8))
    with pytest.raises(ValueError):
        bnd.ssm_gated_norm_bwd(torch.zeros(2, 8), torch.ones(8), torch.zeros(2, 8), residual_scale=2.0)


@pytest.mark.parametrize("name", ["q", "k", "v", "dt", "beta", "A", "dt_bias", "h0"])
def test_reference_gradients_against_differences(name):
    d = {k: v.double() for k, v in R.make_delta(1, 9, 2, 1, 3, 4, torch.float64, 2).items()}
    g = R.delta_grads(d)["ddt_bias" if name == "dt_bias" else "d" + name]
    v = torch.randn(d[name].shape, generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    hi, lo = (R.delta_loss(dict(d, **{name: d[name] + e * v})) for e in (1e-5, -1e-5))
    want = ((hi - lo) / 2e-5).item()
    assert abs((g * v).sum().item() - want) <= 1e-7 * max(1.0, abs(want))


def test_header_argument_counts(L):
    """The binding passes as many arguments as the header declares."""
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                             "ssm_scan.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    for name in ("ssm_gated_delta_fwd", "ssm_gated_delta_bwd", "ssm_gated_delta_update",
                 "ssm_gated_norm_fwd", "ssm_gated_norm_bwd", "ssm_gated_delta_workspace_bytes",
                 "ssm_gated_delta_bwd_workspace_bytes", "ssm_gated_norm_bwd_workspace_bytes"):
        args = re.search(name + r"\((.*?)\);", text, flags=re.S).group(1)
        assert len(args.split(",")) == len(getattr(L, name).argtypes), name
        assert isinstance(getattr(L, name), ctypes._CFuncPtr)
