"""GPU checks of the residual stream operators against the float64 oracle on
the same io-typed inputs.

Bounds, element by element, with u = 2^-24 and the io rounding of half a step
(2^-8 of the value for bf16, u for fp32).  A row sum of the kernel is at most
d / 32 additions in a lane (fewer in a tree) and 5 shuffles behind one
another: its error is under (d / 32 + 32) u =: k u of the sum of magnitudes,
and so is that of what is formed from a few of them.  With s = 1 / spread of
a row, a normalised value u_j is off by at most
k u (|u_j| + s (|x_j| + mean|x|)) =: e_j.  What a gradient is formed of enters
with the same k u of its terms' magnitudes and with e_j where it reads u_j.
Column sums add rows one after another in a thread (rows / 608 of them, and a
tile of up to 64), then a 32nd of the threads' parts behind one another: 608
blocks of 128 / (d / 4) threads a column, one where d is wider."""

import itertools

import numpy as np
import pytest
import torch

import oracle
from efficient_attention_transformer_gb300 import binding as bd

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
KIND = {"none": bd.NORM_NONE, "layer": bd.NORM_LAYER, "scale": bd.NORM_SCALE}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from efficient_attention_transformer_gb300.build import build
    build()


def f64(t):
    return None if t is None else t.double().cpu().numpy()


class Problem:
    def __init__(self, M, d, dtype, post, norm, gate, scale, seed, offset=0, mean=0.0):
        g = torch.Generator().manual_seed(seed)
        self.io = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.half = 2.0 ** -8 if dtype == "bf16" else U
        self.M, self.d, self.post, self.norm = M, d, post, norm

        def dev(x, dt=torch.float32):
            # `offset` elements behind an aligned address
            flat = torch.empty(x.numel() + offset, dtype=dt, device="cuda")[offset:]
            flat.copy_(x.reshape(-1))
            return flat.view(x.shape)

        rows = lambda sd=1.0, m=0.0: dev(torch.randn(M, d, generator=g) * sd + m, self.io)  # noqa: E731
        vec = lambda m, sd=0.3: dev(torch.randn(d, generator=g) * sd + m)  # noqa: E731

        def params(kind):
            if kind == "layer":
                return vec(1.0), vec(0.0)
            if kind == "scale":
                return torch.full((1,), float(np.sqrt(d)) * 0.9, device="cuda"), None
            return None, None

        self.kw = dict(zip(("post_g", "post_b"), params(post)))
        self.kw.update(zip(("norm_g", "norm_b"), params(norm)))
        self.kw.update(gate=rows() if gate else None, scale=vec(0.7) if scale else None, eps=1e-5)
        self.h, self.y = rows(1.5, mean), rows(2.0, -mean)
        self.dr, self.dn = rows(), rows()
        self.ref = {k: f64(v) if torch.is_tensor(v) else v for k, v in self.kw.items()}
        self.ref.update(post=post, norm=norm)
        self.call = dict(self.kw, post_norm=KIND[post], norm=KIND[norm])


def unit_error(x, kind, eps):
    """e: the bound on the error of the normalised rows; and u itself, s."""
    u, s, _ = oracle.norm_rows(x, kind, 1.0, None, eps)
    if kind == "none":
        return np.zeros_like(u), u, s
    return (x.shape[1] / 32 + 32) * U * (np.abs(u) + s * (np.abs(x) + np.abs(x).mean(1, keepdims=True))), u, s


def within(name, got, want, bound):
    got = f64(got)
    assert got.shape == want.shape, name
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (name, int(bad.sum()), float(np.max(np.abs(got - want) / bound)))


def one(v):
    return 1.0 if v is None else np.abs(v)


def check_forward(p):
    r, n = bd.residual_norm(p.h, p.y, **p.call)
    torch.cuda.synchronize()
    h, y, q = f64(p.h), f64(p.y), p.ref
    wr, wn = oracle.residual_norm(h, y, **q)
    e, uy, _ = unit_error(y, p.post, q["eps"])
    k = one(q["gate"]) * one(q["scale"])
    pg, pb = one(q["post_g"]), 0.0 if q["post_b"] is None else np.abs(q["post_b"])
    er = k * (pg * e + 8 * U * (np.abs(uy) * pg + pb)) + 4 * U * np.abs(h)
    within("r", r, wr, er + p.half * (np.abs(wr) + er))
    if p.norm == "none":
        assert n is None
        return
    # n is a smooth function of r: s (er + mean er) more on its normalised row,
    # and as much along it
    e, un, s = unit_error(wr, p.norm, q["eps"])
    e = e + s * (er + er.mean(1, keepdims=True)) * (1 + np.abs(un))
    if p.norm == "layer":
        e = e + np.abs(un) * s * (np.abs(un) * er).mean(1, keepdims=True)
    else:
        e = e + np.abs(un) * s * (np.abs(un) * er).sum(1, keepdims=True)
    ng, nb = one(q["norm_g"]), 0.0 if q["norm_b"] is None else np.abs(q["norm_b"])
    en = ng * e + 8 * U * (ng * np.abs(un) + nb)
    within("n", n, wn, en + p.half * (np.abs(wn) + en))


def grad_error(x, kind, g, dout, edout, eps):
    """Bounds of (dx, dg terms) for an output gradient known to edout."""
    if kind == "none":
        return edout, None
    e, u, s = unit_error(x, kind, eps)
    w, ew = np.abs(dout * g), edout * np.abs(g)
    mean = (lambda a: a.mean(1, keepdims=True)) if kind == "layer" else (
        lambda a: a.sum(1, keepdims=True))
    au = np.abs(u)
    base = w + au * mean(w * au) + (mean(w) if kind == "layer" else 0.0)
    err = ew + mean(ew) * (kind == "layer") + au * mean(ew * au + w * e) + e * mean(w * au)
    # the sums', the products' and s's own roundings: 2 k u of the terms
    return s * (2 * (x.shape[1] / 32 + 32) * U * base + err), edout * au + np.abs(dout) * (e + 4 * U * au)


def check_backward(p):
    out = bd.residual_norm_backward(p.dr, p.dn if p.norm != "none" else None, p.h, p.y, **p.call)
    torch.cuda.synchronize()
    q = p.ref
    dr, r, y = f64(p.dr), f64(p.h), f64(p.y)
    dn = f64(p.dn) if p.norm != "none" else None
    want = oracle.residual_norm_grad(dr, dn, r, y, **q)
    adds = min(p.M, p.M / 608 + 64 + 608 / 32 * max(1, 128 // -(-p.d // 4))) + 40
    col = lambda terms, err: err.sum(0) + adds * U * np.abs(terms).sum(0)  # noqa: E731
    edh = 4 * U * np.abs(dr)
    if p.norm != "none":
        ex, eg = grad_error(r, p.norm, q["norm_g"], dn, np.zeros_like(dn), q["eps"])
        edh = edh + ex + 2 * U * np.abs(want["dh"])
        un = oracle.norm_rows(r, p.norm, 1.0, None, q["eps"])[0]
        bound = col(dn * un, eg)
        if p.norm == "scale":
            bound = bound.sum().reshape(1) + 64 * U * np.abs(dn * un).sum()
        within("dnorm_g", out["dnorm_g"], want["dnorm_g"], bound)
        if p.norm == "layer":
            within("dnorm_b", out["dnorm_b"], want["dnorm_b"], col(dn, 0 * dn))
    within("dh", out["dh"], want["dh"], edh + p.half * (np.abs(want["dh"]) + edh))
    e, uy, _ = unit_error(y, p.post, q["eps"])
    post = oracle.norm_rows(y, p.post, q["post_g"], q["post_b"], q["eps"])[2]
    pg, pb = one(q["post_g"]), 0.0 if q["post_b"] is None else np.abs(q["post_b"])
    ep = pg * e + 8 * U * (pg * np.abs(uy) + pb)
    adh = np.abs(want["dh"])
    gate, scale = one(q["gate"]), one(q["scale"])
    eprod = edh * np.abs(post) + adh * ep + 4 * U * adh * np.abs(post)
    if q["gate"] is not None:
        b = eprod * scale
        within("dgate", out["dgate"], want["dgate"], b + p.half * (np.abs(want["dgate"]) + b))
    if q["scale"] is not None:
        within("dscale", out["dscale"], want["dscale"], col(adh * post * gate, eprod * gate))
    dp = want["dh"] * (1.0 if q["gate"] is None else q["gate"]) * (
        1.0 if q["scale"] is None else q["scale"])
    edp = edh * gate * scale + 4 * U * np.abs(dp)
    ey, eg = grad_error(y, p.post, q["post_g"], dp, edp, q["eps"])
    within("dy", out["dy"], want["dy"], ey + p.half * (np.abs(want["dy"]) + ey))
    if p.post != "none":
        bound = col(dp * uy, eg)
        if p.post == "scale":
            bound = bound.sum().reshape(1) + 64 * U * np.abs(dp * uy).sum()
        within("dpost_g", out["dpost_g"], want["dpost_g"], bound)
    if p.post == "layer":
        within("dpost_b", out["dpost_b"], want["dpost_b"], col(dp, edp))
    for k, v in want.items():
        assert (out[k] is None) == (v is None), k


SIZES = [(1, 768), (2, 1), (3, 5), (7, 31), (64, 64), (5, 257), (130, 768), (33, 1001), (9, 1032),
         (3, 2048), (2, 4096), (2, 4095), (1300, 40), (700, 3), (40, 2056), (17, 8192), (9, 8191),
         (5, 6000), (400, 1536)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("M,d", SIZES)
def test_sizes(M, d, dtype):
    p = Problem(M, d, dtype, "layer", "layer", True, True, M + d)
    check_forward(p)
    check_backward(p)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("post,norm", list(itertools.product(KIND, KIND)))
@pytest.mark.parametrize("gate,scale", [(False, False), (True, False), (False, True)])
def test_options(post, norm, gate, scale, dtype):
    p = Problem(37, 200, dtype, post, norm, gate, scale, 11)
    check_forward(p)
    check_backward(p)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_unaligned_arrays(dtype):
    p = Problem(19, 128, dtype, "scale", "layer", True, True, 5, offset=1)
    assert p.h.data_ptr() % 16
    check_forward(p)
    check_backward(p)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("M,d,offset", [(300, 1501, 0), (9, 8191, 0), (6, 8192, 0), (70, 4104, 0),
                                        (70, 4104, 3), (5, 250, 1), (1300, 255, 0), (40, 2052, 0)])
def test_wide_and_odd_rows(M, d, offset, dtype):
    """Forms of eight columns a thread, tiles that start anywhere in memory."""
    for post, norm in (("layer", "scale"), ("scale", "layer")):
        p = Problem(M, d, dtype, post, norm, True, True, 17, offset=offset)
        check_forward(p)
        check_backward(p)
    r, n = bd.residual_norm(p.h, p.y, **p.call)
    h, y = p.h.clone(), p.y.clone()
    bd.residual_norm(h, y, out_r=h, out_n=y, **p.call)
    assert torch.equal(h, r) and torch.equal(y, n)


def test_rows_far_from_zero():
    """Means 1000 spreads away from zero: the squares around the mean are
    taken after it, so nothing is lost but the inputs' own digits."""
    p = Problem(50, 768, "fp32", "layer", "layer", False, True, 6, mean=1000.0)
    check_forward(p)
    check_backward(p)


def test_zero_rows_and_one_large_column():
    p = Problem(8, 96, "fp32", "scale", "scale", False, False, 7)
    for t in (p.h, p.y):
        t[1:3] = 0.0
        t[4, 17] = 1e4
    out = bd.residual_norm_backward(p.dr, p.dn, p.h, p.y, **p.call)
    want = oracle.residual_norm_grad(f64(p.dr), f64(p.dn), f64(p.h), f64(p.y), **p.ref)
    for k in ("dh", "dy"):
        got = f64(out[k])
        # zero rows: dn g / eps + dr, exactly linear; others as in the bounds
        assert np.all(np.abs(got - want[k]) <= 1e-5 * np.abs(want[k]).max(1, keepdims=True))
    r, n = bd.residual_norm(p.h, p.y, **p.call)
    assert torch.equal(r[1:3], torch.zeros_like(r[1:3])) and not n[1:3].any()


def test_large_problem_and_repeat():
    """The widths of the layer's long workload, more rows than blocks hold at
    once; twice the same bits."""
    p = Problem(16384, 768, "bf16", "scale", "layer", True, True, 8)
    check_forward(p)
    check_backward(p)
    a = bd.residual_norm_backward(p.dr, p.dn, p.h, p.y, **p.call)
    b = bd.residual_norm_backward(p.dr, p.dn, p.h, p.y, **p.call)
    assert all(a[k] is None or torch.equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_without_y_in_place_and_optional(dtype):
    p = Problem(40, 72, dtype, "none", "layer", False, False, 9)
    n0 = bd.residual_norm(p.h, None, norm=bd.NORM_LAYER, norm_g=p.kw["norm_g"],
                          norm_b=p.kw["norm_b"])
    assert n0[0] is p.h
    np.testing.assert_array_equal(
        f64(n0[1]), f64(bd.residual_norm(p.h, torch.zeros_like(p.y), **p.call)[1]))
    r, n = bd.residual_norm(p.h, p.y, **p.call)
    h, y = p.h.clone(), p.y.clone()
    r1, n1 = bd.residual_norm(h, y, out_r=h, out_n=y, **p.call)
    assert r1 is h and torch.equal(r1, r) and torch.equal(n1, n)
    g = bd.residual_norm_backward(p.dr, p.dn, r, p.y, **p.call)
    dr, dn = p.dr.clone(), p.dn.clone()
    g1 = bd.residual_norm_backward(dr, dn, r, p.y, out=dict(dh=dr, dy=dn), **p.call)
    assert all(g[k] is None or torch.equal(g[k], g1[k]) for k in g) and g1["dh"] is dr
    # nothing else reads the stream: dr left out is a dr of zeros
    a = bd.residual_norm_backward(None, p.dn, r, p.y, **p.call)
    b = bd.residual_norm_backward(torch.zeros_like(p.dr), p.dn, r, p.y, **p.call)
    assert all(a[k] is None or torch.equal(a[k], b[k]) for k in a)


def test_nan_stays_in_its_row():
    p = Problem(6, 768, "bf16", "layer", "layer", True, True, 10)
    r0, n0 = bd.residual_norm(p.h, p.y, **p.call)
    p.y[2, 5] = float("nan")
    p.h[4, 0] = float("inf")
    r, n = bd.residual_norm(p.h, p.y, **p.call)
    keep = [0, 1, 3, 5]
    assert torch.equal(r[keep], r0[keep]) and torch.equal(n[keep], n0[keep])
    assert n[2].isnan().all() and n[4].isnan().any()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("d", [768, 767, 2304])
def test_nan_takes_its_whole_row_of_a_scale_norm(d, dtype):
    """A length that is not a number is not one below eps."""
    p = Problem(6, d, dtype, "scale", "scale", True, True, 11)
    r0, n0 = bd.residual_norm(p.h, p.y, **p.call)
    g0 = bd.residual_norm_backward(p.dr, p.dn, p.h, p.y, **p.call)
    p.y[2, 5] = float("nan")
    p.h[4, 0] = float("nan")
    r, n = bd.residual_norm(p.h, p.y, **p.call)
    g = bd.residual_norm_backward(p.dr, p.dn, p.h, p.y, **p.call)
    keep = [0, 1, 3, 5]
    assert r[2].isnan().all() and n[[2, 4]].isnan().all()
    assert g["dy"][[2, 4]].isnan().all() and g["dh"][4].isnan().all()
    assert g["dpost_g"].isnan().all() and g["dnorm_g"].isnan().all()
    for a, b in ((r, r0), (n, n0), (g["dh"], g0["dh"]), (g["dy"], g0["dy"])):
        assert torch.equal(a[keep], b[keep])


def test_other_stream_and_captured():
    p = Problem(300, 768, "bf16", "scale", "layer", True, True, 12)
    r, n = bd.residual_norm(p.h, p.y, **p.call)
    g = bd.residual_norm_backward(p.dr, p.dn, p.h, p.y, **p.call)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    r1, n1 = bd.residual_norm(p.h, p.y, stream=s, **p.call)
    g1 = bd.residual_norm_backward(p.dr, p.dn, p.h, p.y, stream=s, **p.call)
    s.synchronize()
    assert torch.equal(r, r1) and torch.equal(n, n1)
    assert all(g[k] is None or torch.equal(g[k], g1[k]) for k in g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r2, n2 = bd.residual_norm(p.h, p.y, **p.call)
        g2 = bd.residual_norm_backward(p.dr, p.dn, r2, p.y, **p.call)
    p.h.mul_(-0.5)
    graph.replay()
    r3, n3 = bd.residual_norm(p.h, p.y, **p.call)
    g3 = bd.residual_norm_backward(p.dr, p.dn, r3, p.y, **p.call)
    torch.cuda.synchronize()
    assert torch.equal(r2, r3) and torch.equal(n2, n3)
    assert all(g2[k] is None or torch.equal(g2[k], g3[k]) for k in g2)


def test_refusals():
    p = Problem(4, 16, "bf16", "none", "layer", False, False, 13)
    with pytest.raises(ValueError):
        bd.residual_norm(p.h, p.y.float(), **p.call)
    with pytest.raises(ValueError):
        bd.residual_norm(p.h, p.y[:2], **p.call)
    with pytest.raises(ValueError):
        bd.residual_norm(p.h.t(), p.y.t(), **p.call)
    with pytest.raises(ValueError):
        bd.residual_norm(p.h, p.y, norm_g=torch.ones(15, device="cuda"))
    with pytest.raises(bd.FlashGauError):
        bd.residual_norm(p.h, p.y, norm_g=None)
    with pytest.raises(bd.FlashGauError):
        bd.residual_norm(p.h, p.y, out_r=p.h, out_n=p.h, norm_g=p.kw["norm_g"])
    with pytest.raises(bd.FlashGauError):
        wide = torch.zeros(1, 8200, dtype=torch.bfloat16, device="cuda")
        bd.residual_norm(wide, None, norm=bd.NORM_SCALE, norm_g=torch.ones(1, device="cuda"))
    with pytest.raises(bd.FlashGauError):
        empty = torch.zeros(0, 16, dtype=torch.bfloat16, device="cuda")
        bd.residual_norm(empty, None, norm=bd.NORM_SCALE, norm_g=torch.ones(1, device="cuda"))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("M,d", [(9, 200), (9, 768), (5, 2048), (7, 513), (3, 4096), (3, 5000)])
@pytest.mark.parametrize("norm", ["none", "layer"])
def test_gradient_of_y_without_a_norm_does_not_read_y(M, d, norm, dtype):
    """dy = dh scale gate, whatever y holds: infinities and NaN reach the
    gradients that are formed of y, at their own places."""
    p = Problem(M, d, dtype, "none", norm, True, True, 21)
    dn = p.dn if norm != "none" else None
    clean = bd.residual_norm_backward(p.dr, dn, p.h, p.y, **p.call)
    p.y[0, 3], p.y[1, d - 1], p.y[2, 0] = float("inf"), float("nan"), -float("inf")
    got = bd.residual_norm_backward(p.dr, dn, p.h, p.y, **p.call)
    for k in ("dh", "dy"):
        assert torch.equal(got[k], clean[k]), k
    bad = ~torch.isfinite(p.y)
    assert not torch.isfinite(got["dgate"][bad]).any()
    assert torch.equal(got["dgate"][~bad], clean["dgate"][~bad])
    cols = bad.any(0)
    assert not torch.isfinite(got["dscale"][cols]).any()
    assert torch.equal(got["dscale"][~cols], clean["dscale"][~cols])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("post,norm", list(itertools.product(KIND, KIND)))
@pytest.mark.parametrize("gate,scale", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("d", [512, 768, 1024, 1536])
def test_options_of_several_warps_a_row(d, post, norm, gate, scale, dtype):
    """The row form at the widths that two and four warps share, few rows."""
    p = Problem(37, d, dtype, post, norm, gate, scale, 12)
    check_forward(p)
    check_backward(p)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("post,norm", list(itertools.product(KIND, KIND)))
@pytest.mark.parametrize("M,d,on", [(1301, 512, True), (1301, 1024, False), (701, 1536, True),
                                    (2500, 256, False)])
def test_options_of_more_rows_than_blocks(M, d, on, post, norm, dtype):
    p = Problem(M, d, dtype, post, norm, on, on, 13)
    check_forward(p)
    check_backward(p)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("M,d", [(5, 264), (130, 512), (9, 776), (700, 1024), (3, 1280), (6, 256),
                                 (4, 1288)])
def test_aligned_widths(M, d, dtype):
    p = Problem(M, d, dtype, "layer", "layer", True, True, M + d)
    check_forward(p)
    check_backward(p)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,d", [(1, 64), (50, 255), (700, 1024)])
def test_infinite_sums_of_a_scale_norms_g(M, d, dtype):
    """An infinity of dn makes norm_g's gradient infinite and one of dr post_g's,
    two of unlike signs make it no number."""
    gen = torch.Generator().manual_seed(d)
    rows = lambda: (torch.rand(M, d, generator=gen) + torch.linspace(-3, 3, d)).to(dtype).cuda()  # noqa: E731
    r, y, g = rows(), rows(), torch.ones(1, device="cuda")
    inf, m = float("inf"), M // 2
    for values, want in (({d - 1: inf}, inf), ({d - 1: -inf}, -inf), ({0: inf}, -inf),
                         ({0: inf, d - 1: inf}, None), ({0: float("nan")}, None)):
        grad = torch.randn(M, d, generator=gen).to(dtype).cuda()
        for k, v in values.items():
            grad[m, k] = v
        a = bd.residual_norm_backward(None, grad, r, None, norm=bd.NORM_SCALE, norm_g=g)["dnorm_g"]
        b = bd.residual_norm_backward(grad, None, None, y, post_norm=bd.NORM_SCALE, post_g=g,
                                      norm=bd.NORM_NONE)["dpost_g"]
        for x in (a, b):
            assert bool(torch.isnan(x)) if want is None else float(x) == want
