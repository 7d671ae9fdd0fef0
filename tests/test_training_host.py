"""Host-side checks of the training operators: the oracle against automatic
differentiation and differences, and the refusals of the C ABI and the
binding, all of which come before anything touches a device."""

import ctypes

import numpy as np
import pytest
import torch

import oracle
from efficient_attention_transformer_gb300 import binding as bd
from efficient_attention_transformer_gb300 import build as buildmod

EPS = 1e-5
KINDS = ["none", "layer", "scale"]


@pytest.fixture(scope="module")
def L():
    buildmod.build()
    return bd.lib()


# ---- the oracle --------------------------------------------------------------
def _case(post, norm, gate, scale, seed, M=5, d=7):
    rng = np.random.default_rng(seed)
    par = lambda kind: ((None, None) if kind == "none" else  # noqa: E731
                        (rng.normal(1, 0.2, d), rng.normal(0, 0.2, d)) if kind == "layer" else
                        (rng.normal(2, 0.2, 1), None))
    pg, pb = par(post)
    ng, nb = par(norm)
    return dict(post=post, post_g=pg, post_b=pb, norm=norm, norm_g=ng, norm_b=nb,
                gate=rng.normal(size=(M, d)) if gate else None,
                scale=rng.normal(size=d) if scale else None, eps=EPS), rng


@pytest.mark.parametrize("post", KINDS)
@pytest.mark.parametrize("norm", KINDS)
@pytest.mark.parametrize("gate,scale", [(True, True), (False, False)])
def test_oracle_residual_norm_against_autograd_and_differences(post, norm, gate, scale):
    o, rng = _case(post, norm, gate, scale, 3)
    M, d = 5, 7
    h, y, dr, dn = (rng.normal(size=(M, d)) for _ in range(4))
    r, n = oracle.residual_norm(h, y, **o)
    T = lambda a: None if a is None else torch.tensor(a, requires_grad=True)  # noqa: E731
    th, ty = T(h), T(y)
    tp = {k: T(o[k]) for k in ("post_g", "post_b", "norm_g", "norm_b", "gate", "scale")}

    def tnorm(x, kind, g, b):
        if kind == "none":
            return x
        if kind == "layer":
            return torch.nn.functional.layer_norm(x, (d,), g, b, EPS)
        return torch.nn.functional.normalize(x, dim=1, eps=EPS) * g

    add = tnorm(ty, post, tp["post_g"], tp["post_b"])
    add = add if tp["gate"] is None else add * tp["gate"]
    add = add if tp["scale"] is None else add * tp["scale"]
    tr = th + add
    tn = tnorm(tr, norm, tp["norm_g"], tp["norm_b"])
    np.testing.assert_allclose(r, tr.detach().numpy(), rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(n, tn.detach().numpy(), rtol=1e-12, atol=1e-12)
    ((tr * torch.tensor(dr)).sum() + (tn * torch.tensor(dn)).sum()).backward()
    g = oracle.residual_norm_grad(dr, dn if norm != "none" else None, r, y, **o)
    if norm == "none":  # n is r: its gradient comes in dr
        g = oracle.residual_norm_grad(dr + dn, None, r, y, **o)
    want = {"dh": th, "dy": ty, "dgate": tp["gate"], "dscale": tp["scale"],
            "dpost_g": tp["post_g"], "dpost_b": tp["post_b"], "dnorm_g": tp["norm_g"],
            "dnorm_b": tp["norm_b"]}
    for k, t in want.items():
        if t is None:
            assert g[k] is None
        else:
            np.testing.assert_allclose(g[k], t.grad.numpy(), rtol=1e-9, atol=1e-10, err_msg=k)

    def f(h_):
        r_, n_ = oracle.residual_norm(h_, y, **o)
        return (dr * r_).sum() + (dn * n_).sum()

    step = rng.normal(size=h.shape)
    diff = (f(h + 1e-6 * step) - f(h - 1e-6 * step)) / 2e-6
    assert abs(diff - (g["dh"] * step).sum()) <= 1e-6 * (1 + abs(diff))


def test_oracle_scale_norm_of_short_rows():
    """Below eps the ScaleNorm divides by eps: linear, no projection."""
    x = np.array([[1e-6, -2e-6], [0.0, 0.0]])
    g = oracle.residual_norm_grad(None, np.ones((2, 2)), x, None, "none", None, None, None, None,
                                  "scale", np.array([3.0]), None, EPS)
    np.testing.assert_allclose(g["dh"], np.full((2, 2), 3.0 / EPS), rtol=1e-12)


def test_oracle_adamw_against_torch():
    rng = np.random.default_rng(5)
    p = torch.tensor(rng.normal(size=50), requires_grad=True)
    opt = torch.optim.AdamW([p], lr=1e-2, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1)
    q, m, v = p.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    for t in range(1, 5):
        g = rng.normal(size=50)
        p.grad = torch.tensor(g)
        opt.step()
        q, m, v = oracle.adamw(q, g, m, v, 1e-2, 0.8, 0.95, 1e-6, 0.1, t)
        np.testing.assert_allclose(q, p.detach().numpy(), rtol=1e-12)


def test_oracle_codes():
    """Codes meet a block's largest value, keep zeros and nonzero seconds, and
    are off by at most half a step: with |x| = s c^2, half a step of c is
    s (c + 1/4) of x, and fp32 rounding adds less than 1e-4 of a step."""
    rng = np.random.default_rng(6)
    x = (rng.normal(size=600) * np.exp(rng.normal(size=600) * 3)).astype(np.float32)
    x[7] = 0.0
    for top, a in ((127, x), (255, np.abs(x))):
        c, s = oracle.encode_moments(a, top)
        full = np.repeat(s, 256)[:600].astype(np.float64)
        got = full * c.astype(np.float64) * np.abs(c.astype(np.float64))
        # the fourth of a step: (c + 1/2)^2 - c^2 = c + 1/4; a value that is
        # raised to code 1 is off by less than one
        bound = full * (np.abs(c.astype(np.float64)) + 0.2501 + 1e-4)
        raised = (c == 1) & (top == 255)
        assert np.all(np.abs(got - a) <= np.where(raised, full * 1.2502, bound))
        assert c[7] == 0 and np.all(c[a != 0] != 0) if top == 255 else c[7] == 0
        for k in range(3):
            b = slice(256 * k, min(256 * k + 256, 600))
            assert np.abs(c[b].astype(int)).max() == top
    c, s = oracle.encode_moments(np.full(256, 2.0 ** -61, np.float32), 255)
    assert not c.any() and s[0] == 0


# ---- refusals of the C ABI -----------------------------------------------------
A, B, C, D, E_, F_ = (1 << 32, 2 << 32, 3 << 32, 4 << 32, 5 << 32, 6 << 32)  # fake arrays


def _residual(**kw):
    o = dict(post=bd.NORM_NONE, norm=bd.NORM_LAYER, post_g=None, post_b=None, norm_g=64,
             norm_b=None, scale=None, gate=None, eps=EPS)
    o.update(kw)
    return bd.Residual(*(o[k] for k, _ in bd.Residual._fields_))


@pytest.mark.parametrize("opts,args,code", [
    (dict(), dict(h=None), bd.EINVAL),
    (dict(), dict(M=0), bd.EINVAL),
    (dict(), dict(d=0), bd.EINVAL),
    (dict(), dict(d=8193), bd.ENOTSUP),
    (dict(), dict(dtype=2), bd.EINVAL),
    (dict(norm=3), dict(), bd.EINVAL),
    (dict(post=-1), dict(), bd.EINVAL),
    (dict(norm_g=None), dict(), bd.EINVAL),
    (dict(eps=0.0), dict(), bd.EINVAL),
    (dict(eps=float("nan")), dict(), bd.EINVAL),
    (dict(eps=1e-40), dict(), bd.EINVAL),
    (dict(), dict(n=None), bd.EINVAL),                   # a norm and no place for it
    (dict(norm=bd.NORM_NONE), dict(), bd.EINVAL),        # a place and no norm
    (dict(norm=bd.NORM_NONE), dict(n=None, r=None), bd.EINVAL),
    (dict(scale=64), dict(y=None), bd.EINVAL),           # a scale of nothing
    (dict(post=bd.NORM_SCALE, post_g=64), dict(y=None), bd.EINVAL),
    (dict(), dict(r=A + 4), bd.EINVAL),                  # overlaps h
    (dict(), dict(n=C), bd.EINVAL),                      # n is r
    (dict(), dict(h=A + 1), bd.EINVAL),                  # odd address
    (dict(scale=C + 8), dict(), bd.EINVAL),              # the scale inside r
])
def test_residual_norm_refuses(L, opts, args, code):
    a = dict(h=A, y=B, M=10, d=64, dtype=bd.BF16, r=C, n=D)
    a.update(args)
    o = _residual(**opts)
    assert L.flash_gau_residual_norm(a["h"], a["y"], ctypes.byref(o), a["M"], a["d"], a["dtype"],
                                     a["r"], a["n"], None) == code
    assert L.flash_gau_residual_norm(a["h"], a["y"], None, a["M"], a["d"], a["dtype"], a["r"],
                                     a["n"], None) == bd.EINVAL


@pytest.mark.parametrize("opts,args,code", [
    (dict(), dict(dh=None), bd.EINVAL),
    (dict(), dict(dn=None), bd.EINVAL),
    (dict(), dict(r=None), bd.EINVAL),
    (dict(norm=bd.NORM_NONE), dict(dn=None, dr=None), bd.EINVAL),
    (dict(norm=bd.NORM_NONE), dict(), bd.EINVAL),               # dn without a norm
    (dict(scale=64), dict(y=None), bd.EINVAL),
    (dict(scale=64), dict(dy=None), bd.EINVAL),
    (dict(), dict(dgate=F_), bd.EINVAL),                        # no gate
    (dict(), dict(dscale=F_), bd.EINVAL),
    (dict(), dict(dpost_g=F_), bd.EINVAL),
    (dict(norm=bd.NORM_SCALE), dict(dnorm_b=F_), bd.EINVAL),
    (dict(), dict(dh=A + 2), bd.EINVAL),                        # overlaps dr
    (dict(), dict(dy=E_), bd.EINVAL),                           # dy is dh
    (dict(), dict(dnorm_g=64), bd.EINVAL),                      # the parameter itself
    (dict(), dict(dnorm_g=C), bd.EINVAL),                       # inside r
    (dict(), dict(ws=1 << 40 | 8), bd.EWORKSPACE),
    (dict(), dict(wsb=100), bd.EWORKSPACE),
    (dict(), dict(ws=E_), bd.EINVAL),                           # the workspace is dh
    (dict(), dict(d=9000), bd.ENOTSUP),
])
def test_residual_norm_backward_refuses(L, opts, args, code):
    a = dict(dr=A, dn=B, r=C, y=D, M=10, d=64, dtype=bd.BF16, dh=E_, dy=7 << 32, ws=1 << 40,
             wsb=1 << 30, dgate=None, dscale=None, dpost_g=None, dpost_b=None, dnorm_g=None,
             dnorm_b=None)
    a.update(args)
    o = _residual(**opts)
    g = bd.ResidualGrads(*(a[k] for k, _ in bd.ResidualGrads._fields_))
    assert L.flash_gau_residual_norm_backward(
        a["dr"], a["dn"], a["r"], a["y"], ctypes.byref(o), a["M"], a["d"], a["dtype"],
        ctypes.byref(g), a["ws"], a["wsb"], None) == code


def test_residual_norm_arrays_that_only_look_like_rows(L):
    """One fp32 row is as long as a parameter, and a row array may be as long
    as the workspace: neither may stand in for the other."""
    o = _residual(norm_g=A, scale=B)
    for r, n in ((A, D), (C, A), (B, D), (C, B)):
        assert L.flash_gau_residual_norm(E_, F_, ctypes.byref(o), 1, 64, bd.FP32, r, n,
                                         None) == bd.EINVAL
    W = 1 << 40

    def back(M, d, ws, **kw):
        a = dict(dh=E_, dy=7 << 32)
        a.update(kw)
        g = bd.ResidualGrads(*(a.get(k) for k, _ in bd.ResidualGrads._fields_))
        return L.flash_gau_residual_norm_backward(W, C, D, 8 << 32, ctypes.byref(o), M, d, bd.FP32,
                                                  ctypes.byref(g), ws, 1 << 30, None)

    assert back(1, 64, 1 << 41, dh=A) == bd.EINVAL
    assert back(1, 64, 1 << 41, dy=B) == bd.EINVAL
    f = L.flash_gau_residual_norm_backward_workspace_bytes
    M, d = next((M, d) for M in range(1, 40000) for d in (64, 128, 256, 512, 1024)
                if f(M, d) == M * d * 4)
    assert back(M, d, W) == bd.EINVAL                           # the workspace is dr


def test_residual_norm_backward_workspace(L):
    f = L.flash_gau_residual_norm_backward_workspace_bytes
    assert f(0, 64) == 0 and f(4, 0) == 0 and f(4, 8193) == 0
    assert f(1, 1) >= 20 and f(1 << 30, 4096) <= 608 * (5 * 4096 + 32) * 4


def _tensor(**kw):
    t = dict(p=A, copy=None, g=B, m=C, v=D, m_scale=None, v_scale=None, n=1000, g_dtype=bd.FP32,
             weight_decay=0.0)
    t.update(kw)
    return bd.AdamWTensor(*(t[k] for k, _ in bd.AdamWTensor._fields_))


def _hyper(**kw):
    h = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1, state_bits=32, grad_scale=None)
    h.update(kw)
    return bd.AdamWHyper(*(h[k] for k, _ in bd.AdamWHyper._fields_))


@pytest.mark.parametrize("tensor,hyper", [
    (dict(p=None), {}), (dict(g=None), {}), (dict(m=None), {}), (dict(n=-1), {}),
    (dict(g_dtype=5), {}), (dict(weight_decay=-0.1), {}), (dict(weight_decay=float("nan")), {}),
    (dict(p=A + 2), {}), (dict(g=B + 1), {}), (dict(v=C + 100), {}), (dict(copy=A + 16), {}),
    (dict(g=A), {}),                                            # the gradient is the parameter
    ({}, dict(lr=-1.0)), ({}, dict(lr=float("inf"))), ({}, dict(beta1=1.0)),
    ({}, dict(beta2=-0.5)), ({}, dict(beta1=float("nan"))), ({}, dict(eps=0.0)),
    ({}, dict(step=0)), ({}, dict(state_bits=16)), ({}, dict(grad_scale=3)),
    ({}, dict(state_bits=8)),                                   # no scales
    (dict(m_scale=E_, v_scale=E_ + 8), dict(state_bits=8)),     # scales overlap
])
def test_adamw_refuses(L, tensor, hyper):
    t, h = _tensor(**tensor), _hyper(**hyper)
    assert L.flash_gau_adamw_step(ctypes.byref(t), 1, ctypes.byref(h), None) == bd.EINVAL
    assert L.flash_gau_adamw_step(ctypes.byref(t), 1, None, None) == bd.EINVAL
    assert L.flash_gau_adamw_step(None, 1, ctypes.byref(_hyper()), None) == bd.EINVAL
    assert L.flash_gau_adamw_step(None, -1, ctypes.byref(_hyper()), None) == bd.EINVAL


@pytest.mark.parametrize("hyper", [dict(eps=1e-39), dict(eps=1e39), dict(lr=1e39),
                                   dict(lr=1e38, beta1=0.999), dict(lr=float("nan"))])
def test_adamw_refuses_what_fp32_cannot_hold(L, hyper):
    assert L.flash_gau_adamw_step(ctypes.byref(_tensor()), 1, ctypes.byref(_hyper(**hyper)),
                                  None) == bd.EINVAL


def test_adamw_moments_refuses_overlaps(L):
    P = ctypes.c_void_p
    t = _tensor(m_scale=E_, v_scale=F_)
    far = 7 << 32
    for m, v in ((far, far + 400), (C, far), (far, D + 500), (far, E_), (F_ + 8, far)):
        assert L.flash_gau_adamw_moments(ctypes.byref(t), 1, (P * 1)(m), (P * 1)(v),
                                         None) == bd.EINVAL


def test_adamw_moments_refuses(L):
    P = ctypes.c_void_p
    t = _tensor(m_scale=E_, v_scale=F_)
    for m, v in ((None, 8), (8, None), (9, 8)):
        assert L.flash_gau_adamw_moments(ctypes.byref(t), 1, (P * 1)(m), (P * 1)(v),
                                         None) == bd.EINVAL
    assert L.flash_gau_adamw_moments(ctypes.byref(_tensor()), 1, (P * 1)(8), (P * 1)(8),
                                     None) == bd.EINVAL
    assert L.flash_gau_adamw_moments(ctypes.byref(t), 1, None, (P * 1)(8), None) == bd.EINVAL


def test_binding_refuses_host_tensors(L):
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        bd.residual_norm(x, x, norm=bd.NORM_NONE)
    with pytest.raises(ValueError):
        bd.residual_norm_backward(x, None, x, x, norm=bd.NORM_NONE)
    with pytest.raises(ValueError):
        bd.AdamW([x])
    with pytest.raises(TypeError):
        bd.residual_norm(x.half(), None)
    with pytest.raises(ValueError):
        bd.AdamW([x], state_bits=4)


# ---- cross entropy ------------------------------------------------------------
@pytest.mark.parametrize("reduction", ["mean", "sum"])
def test_oracle_xent_against_autograd(reduction):
    rng = np.random.default_rng(8)
    X, W = rng.normal(size=(9, 6)), rng.normal(size=(11, 6))
    labels = np.array([0, 10, 3, -1, 5, 11, 7, 7, -100])
    X[3] = np.nan
    x, w = torch.tensor(np.nan_to_num(X), requires_grad=True), torch.tensor(W, requires_grad=True)
    keep = (labels >= 0) & (labels < 11)
    t = torch.tensor(np.where(keep, labels, -100))
    loss = torch.nn.functional.cross_entropy(x @ w.t(), t, reduction=reduction) * 0.5
    loss.backward()
    got = oracle.xent(X, W, labels, reduction, 0.5)
    assert abs(got["total"] - float(loss.detach())) < 1e-12
    np.testing.assert_allclose(got["dX"], x.grad.numpy(), rtol=1e-10, atol=1e-13)
    np.testing.assert_allclose(got["dW"], w.grad.numpy(), rtol=1e-10, atol=1e-13)
    assert not got["dX"][~keep].any() and not got["loss"][~keep].any()
    none = oracle.xent(X, W, np.full(9, -1), reduction)
    assert none["total"] == 0 and not none["dW"].any()


@pytest.mark.parametrize("args,out,code", [
    (dict(X=None), {}, bd.EINVAL), (dict(W=None), {}, bd.EINVAL), (dict(labels=None), {}, bd.EINVAL),
    (dict(N=0), {}, bd.EINVAL), (dict(d=0), {}, bd.EINVAL), (dict(V=-1), {}, bd.EINVAL),
    (dict(dtype=9), {}, bd.EINVAL), (dict(reduction=2), {}, bd.EINVAL),
    (dict(scale=float("inf")), {}, bd.EINVAL),
    (dict(d=60), {}, bd.ENOTSUP), (dict(V=(1 << 22) + 1), {}, bd.ENOTSUP),
    (dict(d=65544), {}, bd.ENOTSUP),
    (dict(X=A + 8), {}, bd.EINVAL), (dict(labels=C + 2), {}, bd.EINVAL),
    ({}, dict(total=None), bd.EINVAL), ({}, dict(loss=None), bd.EINVAL),
    ({}, dict(dX=A), bd.EINVAL), ({}, dict(dW=B + 160), bd.EINVAL), ({}, dict(dW=9 << 32 | 2), bd.EINVAL),
    ({}, dict(lse=F_), bd.EINVAL),                       # the losses
    (dict(ws=1 << 44 | 64), {}, bd.EWORKSPACE), (dict(wsb=1000), {}, bd.EWORKSPACE),
    (dict(ws=A), {}, bd.EINVAL),
])
def test_xent_refuses(L, args, out, code):
    a = dict(X=A, W=B, labels=C, N=40, d=64, V=500, dtype=bd.BF16, reduction=bd.MEAN, scale=1.0,
             ws=1 << 44, wsb=1 << 30)
    a.update(args)
    o = dict(total=D, loss=F_, lse=None, dX=7 << 32, dW=8 << 32)
    o.update(out)
    x = bd.XentOut(*(o[k] for k, _ in bd.XentOut._fields_))
    assert L.flash_gau_xent(a["X"], a["W"], a["labels"], a["N"], a["d"], a["V"], a["dtype"],
                            a["reduction"], a["scale"], ctypes.byref(x), a["ws"], a["wsb"],
                            None) == code


def test_xent_workspace(L):
    f = L.flash_gau_xent_workspace_bytes
    assert f(0, 64, 10, bd.BF16, 1) == 0 and f(4, 64, 10, 7, 1) == 0 and f(4, 4, 10, bd.BF16, 1) == 0
    assert f(4, 4, 10, bd.FP32, 1) > 0
    # a piece's [tokens, V] never passes 2 GiB however many tokens there are;
    # a token itself takes three words
    for N in (1, 1000, 16384, 1 << 20, 1 << 30):
        assert 0 < f(N, 768, 50257, bd.BF16, 1) < (3 << 30) + 12 * N
        assert 0 < f(N, 768, 50257, bd.BF16, 0) < (3 << 30) + 12 * N
        assert 0 < f(N, 768, 50257, bd.FP32, 1) < (3 << 30) + 12 * N


def test_xent_binding_refuses_host_tensors(L):
    with pytest.raises(ValueError):
        bd.xent(torch.zeros(4, 8), torch.zeros(5, 8), torch.zeros(4, dtype=torch.int32))


def test_a_stream_of_another_device_is_refused():
    class Stream:
        device = torch.device("cuda", 1)

    with pytest.raises(ValueError):
        bd._scope(torch.device("cuda", 0), Stream())
