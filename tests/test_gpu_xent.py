"""GPU checks of the cross entropy over a vocabulary against float64.

Bounds, element by element.  S is the largest sum of |x_k w_k| of a row, u
the unit of fp32 arithmetic, 2^-24.  A logit of the tensor cores is a sum of
d / 16 steps, each within 2^-22 of the magnitudes that it adds, so it is off
by at most el = (d / 16 + 8) 2^-22 S, and so is the label's.  With fp32 io
there are five more passes whose terms are below 2^-8 of S together, and what
they leave out is below 2^-22 S: el = (1.05 d / 16 + 9) 2^-22 S.  (The dot
products of few tokens add d / 32 terms and 5 shuffles within u each: less.)
An exponential is off by twice that, its argument's rounding (2 u |l| log2 e
each for the product and the difference, 2^-22 for the function), a row's sum
by the additions behind one another; together the relative error ep of a
probability, and the error of a loss up to 1 where the loss is below.  With
bf16 io the exponentials, their factors and the results are rounded to bf16:
2^-8 each at most."""

import numpy as np
import pytest
import torch

import oracle
from efficient_attention_transformer_gb300 import binding as bd

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from efficient_attention_transformer_gb300.build import build
    build()


def f64(t):
    return t.double().cpu().numpy()


def make(N, d, V, dtype, seed, ignored=0.2, pull=0.2, size=1.0):
    g = torch.Generator().manual_seed(seed)
    io = torch.bfloat16 if dtype == "bf16" else torch.float32
    W = torch.randn(V, d, generator=g) * (size / d ** 0.5)
    y = (V * torch.rand(N, generator=g) ** 2).long().clamp(max=V - 1)
    X = torch.randn(N, d, generator=g)
    X += pull * d ** 0.5 * torch.rand(N, 1, generator=g) * W[y] / size
    y = torch.where(torch.rand(N, generator=g) < ignored, torch.full_like(y, -1), y)
    return X.to(io).cuda(), W.to(io).cuda(), y.to(torch.int32).cuda()


def check(X, W, y, reduction="mean", scale=1.0, got=None):
    io = X.dtype
    bf16 = io == torch.bfloat16
    if got is None:
        got = bd.xent(X, W, y, reduction=bd.MEAN if reduction == "mean" else bd.SUM, scale=scale)
    torch.cuda.synchronize()
    x, w, lab = np.nan_to_num(f64(X)), f64(W), y.cpu().numpy()
    N, d, V = len(x), x.shape[1], len(w)
    want = oracle.xent(x, w, lab, reduction, scale)
    live = (lab >= 0) & (lab < V)
    x[~live] = 0.0
    S = (np.abs(x) @ np.abs(w).T).max(1)
    top = np.abs(x @ w.T).max(1)
    steps = (lambda k: k / 16 + 8) if bf16 else (lambda k: 1.05 * k / 16 + 9)  # noqa: E731
    el = steps(d) * 2.0 ** -22 * S
    adds = 40 + V / 256
    ep = 2 * el + 4 * U * 1.4427 * top + 2.0 ** -21 + adds * U
    # loss = log(1 + r): its error is at most r / (1 + r) of r's
    r = np.expm1(np.minimum(want["loss"], 700.0))
    eloss = 2 * ep * r / (1 + r) + 8 * U * want["loss"]
    assert np.all(np.abs(f64(got["loss"]) - want["loss"]) <= eloss), "loss"
    elo = eloss + el + 8 * U * np.abs(want["lse"]) + 4 * U * top
    assert np.all(np.abs(f64(got["lse"]) - want["lse"]) <= elo), "lse"
    n = max(int(live.sum()), 1) if reduction == "mean" else 1
    f = abs(scale) / n
    et = f * (eloss.sum() + (N / 1024 + 16) * U * want["loss"].sum()) + 4 * U * abs(want["total"])
    assert abs(float(got["total"]) - want["total"]) <= et, "total"
    if got["dX"] is None:
        return
    # |softmax - onehot| times the factor, and its relative error
    at = np.where(live, lab, 0)
    P = np.exp(x @ w.T - want["lse"][:, None])
    P[np.arange(N), at] = 0.0
    P[np.arange(N), at] = P.sum(1)
    P *= (f * live)[:, None]
    io_half = 2.0 ** -8 if bf16 else U
    rel = (2 * ep + 8 * U)[:, None] + (2.0 ** -8 if bf16 else 0.0)
    acc = steps(V) * 2.0 ** -22
    bound = ((P * rel) @ np.abs(w)) * 1.01 + acc * (P @ np.abs(w))
    err = np.abs(f64(got["dX"]) - want["dX"])
    lim = bound + io_half * (np.abs(want["dX"]) + bound) + 1e-38
    assert np.all(err <= lim), ("dX", float(np.max(err / lim)))
    if bf16:
        rel = rel + 2.0 ** -8 * 1.01                       # the scaled rows of X
    acc = steps(N) * 2.0 ** -22
    bound = ((P * rel).T @ np.abs(x)) * 1.01 + acc * (P.T @ np.abs(x))
    err = np.abs(f64(got["dW"]) - want["dW"])
    # a factor below the normal numbers of bf16 keeps no relative precision
    lim = bound + io_half * (np.abs(want["dW"]) + bound) + 1e-38
    assert np.all(err <= lim), ("dW", float(np.max(err / lim)))


SIZES = [(1, 8, 1), (1, 64, 2), (2, 72, 63), (3, 128, 127), (5, 64, 128), (31, 136, 129),
         (33, 200, 255), (255, 64, 256), (256, 256, 257), (257, 264, 383), (129, 768, 385),
         (700, 520, 1003), (300, 768, 5003), (40, 1032, 20011)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N,d,V", SIZES)
def test_sizes(N, d, V, dtype):
    check(*make(N, d, V, dtype, N + V))


@pytest.mark.parametrize("N,d,V", [(3, 1, 5), (17, 7, 33), (130, 33, 131), (200, 65, 1001),
                                   (9, 770, 640), (600, 514, 2050)])
def test_fp32_odd_widths(N, d, V):
    check(*make(N, d, V, "fp32", N))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 7, 8, 9])
@pytest.mark.parametrize("d,V", [(8, 1), (64, 5), (72, 33), (768, 1000), (264, 20011), (4104, 70)])
def test_few_tokens(N, d, V, dtype):
    """Without gradients: a form of its own for at most 8 tokens."""
    X, W, y = make(N, d, V, dtype, N + V, ignored=0.3)
    check(X, W, y, got=bd.xent(X, W, y, grad=False))
    check(X, W, y, reduction="sum", scale=-2.0,
          got=bd.xent(X, W, y, reduction=bd.SUM, scale=-2.0, grad=False))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_few_tokens_sure_far_and_left_out(dtype):
    X, W, y = make(8, 64, 300, dtype, 14, ignored=0.0, size=30.0, pull=0.0)
    y[5] = -1
    y[6] = 300
    X[5] = float("nan")
    W[:, 0] = 0
    W[17, 0] = 1.0
    X[:4, 1:] = 0
    X[:4, 0] = torch.tensor([0.0, 20.0, 50.0, -50.0], device="cuda").to(X.dtype)
    y[:4] = 17
    got = bd.xent(X, W, y, grad=False)
    check(X, W, y, got=got)
    assert 0 < float(got["loss"][2]) < 1e-15 and float(got["loss"][3]) > 50
    keep = [0, 1, 2, 3, 4, 7]
    X[1, 2] = float("inf")
    bad = bd.xent(X, W, y, grad=False)
    assert not torch.isfinite(bad["loss"][1])
    keep.remove(1)
    assert torch.equal(bad["loss"][keep], got["loss"][keep])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N", [2, 4])
def test_few_tokens_keep_to_themselves(N, dtype):
    """A token that is not a number, a sure one and one without a label beside
    an ordinary one; the status word of a workspace that held anything."""
    X, W, y = make(N, 96, 1234, dtype, 15, ignored=0.0)
    ws = torch.full((bd.xent_workspace_bytes(N, 96, 1234, bd.BF16 if dtype == "bf16" else bd.FP32,
                                             False),), 255, dtype=torch.uint8, device="cuda")
    got = bd.xent(X, W, y, grad=False, workspace=ws)
    check(X, W, y, got=got)
    assert bd.workspace_status(ws) == 0
    X[0, 95] = float("nan")
    if N == 4:
        y[2] = -7
        X[2] = float("inf")
        X[3] = W[int(y[3])] * 64
    bad = bd.xent(X, W, y, grad=False, workspace=ws)
    assert bool(bad["loss"][0].isnan()) and torch.equal(bad["loss"][1], got["loss"][1])
    if N == 4:
        assert float(bad["loss"][2]) == 0.0 and float(bad["lse"][2]) == 0.0
        one = bd.xent(X[3:], W, y[3:], grad=False)
        check(X[3:], W, y[3:], got=one)
        check(X[1:2], W, y[1:2], got=bd.xent(X[1:2], W, y[1:2], grad=False))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_loss_only_gives_the_same_loss(dtype):
    X, W, y = make(500, 128, 3001, dtype, 1)
    a, b = bd.xent(X, W, y), bd.xent(X, W, y, grad=False)
    assert b["dX"] is None and b["dW"] is None
    for k in ("loss", "lse", "total"):
        assert torch.equal(a[k], b[k])
    check(X, W, y, got=b)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("reduction,scale", [("sum", 1.0), ("mean", 1024.0), ("sum", -0.25),
                                             ("mean", 0.0)])
def test_reductions(reduction, scale, dtype):
    check(*make(100, 64, 500, dtype, 2), reduction=reduction, scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_left_out_tokens(dtype):
    """Rows without a label are not looked at, labels behind the vocabulary
    count as none, and none at all gives zeros."""
    X, W, y = make(300, 72, 700, dtype, 3, ignored=0.5)
    clean = bd.xent(X, W, y)
    y2 = y.clone()
    out = torch.nonzero(y < 0)[:, 0]
    y2[out[::2]] = 700
    y2[out[1::3]] = 2 ** 31 - 1
    X2 = X.clone()
    X2[out] = float("nan")
    X2[out[::3]] = float("inf")
    dirty = bd.xent(X2, W, y2)
    assert all(torch.equal(clean[k], dirty[k]) for k in clean)
    check(X, W, y, got=dirty)
    none = bd.xent(torch.full_like(X, float("nan")), W, torch.full_like(y, -1))
    assert all(not none[k].any() for k in none)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_sure_predictions_keep_their_digits(dtype):
    """Logits far below the label's: losses down to 1e-30, whose gradients are
    minus the small probability of all the others."""
    X, W, y = make(64, 64, 300, dtype, 4, ignored=0.0)
    y.fill_(17)
    W[:, 0] = 0
    W[17, 0] = 1.0
    X[:, 0] = torch.linspace(1.0, 64.0, 64, device="cuda").to(X.dtype)
    got = bd.xent(X, W, y)
    assert float(got["loss"].min()) < 1e-20 and float(got["loss"].min()) > 0
    check(X, W, y, got=got)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_labels_far_below_the_largest_logit(dtype):
    """Logits from -200 to 200: most rows take other references than their
    label's, some in a few of their parts only."""
    X, W, y = make(300, 64, 1500, dtype, 5, size=40.0, pull=0.0)
    l = f64(X) @ f64(W).T
    far = l.max(1) - l[np.arange(300), y.clamp(min=0).long().cpu().numpy()]
    assert (far > 60).mean() > 0.5
    check(X, W, y)
    # one word far above all others, in one part of 128
    X, W, y = make(300, 64, 1500, dtype, 6)
    W[777] = 0
    W[777, 3] = 60.0
    X[:, 3] = torch.linspace(-2.0, 2.0, 300, device="cuda").to(X.dtype)
    check(X, W, y)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_labels_far_below_in_many_parts(dtype):
    """Rows of E that are rescaled by the whole block, in more than one step."""
    check(*make(70, 64, 9001, dtype, 16, size=40.0, pull=0.0))


def test_infinite_and_nan_rows():
    X, W, y = make(64, 64, 300, "bf16", 7, ignored=0.0)
    clean = bd.xent(X, W, y)
    X[5, 3] = float("nan")
    got = bd.xent(X, W, y, grad=False)
    keep = torch.arange(64, device="cuda") != 5
    assert got["loss"][5].isnan() and torch.equal(got["loss"][keep], clean["loss"][keep])
    assert got["total"].isnan()


def reference(X, W, y, rows=2048):
    """total, loss, dX, dW in float64 on the GPU, a few rows at a time."""
    W64, N = W.double(), len(X)
    n = int((y >= 0).sum())
    loss = torch.zeros(N, dtype=torch.float64, device="cuda")
    dX, dW = torch.zeros(X.shape, dtype=torch.float64, device="cuda"), torch.zeros_like(W64)
    for a in range(0, N, rows):
        x, t = X[a:a + rows].double(), y[a:a + rows].long()
        live = (t >= 0).double()[:, None]
        l = torch.log_softmax(x @ W64.t(), 1)
        at = t.clamp(min=0)[:, None]
        loss[a:a + rows] = -l.gather(1, at)[:, 0] * live[:, 0]
        p = l.exp_()
        p.scatter_add_(1, at, -torch.ones_like(p[:, :1]))
        p *= live / n
        dX[a:a + rows], dW = p @ W64, dW + p.t() @ x
    return loss.sum() / n, loss, dX, dW


def near(got, want, tol):
    """In the 2-norm: the elementwise bounds above add up to the same share of
    the magnitudes, of which roundings in both directions leave less."""
    d = (got.double() - want).norm() / want.norm()
    assert float(d) <= tol, float(d)


@pytest.mark.parametrize("dtype,N,d,V", [("bf16", 4096, 768, 50257), ("bf16", 20000, 64, 65537),
                                         ("fp32", 9000, 32, 70001)])
def test_large_and_in_pieces(dtype, N, d, V):
    """The second and third take more than one piece of tokens."""
    X, W, y = make(N, d, V, dtype, 8, ignored=0.1)
    assert (N * V * X.element_size() > 2 << 30) == (N > 4096)
    got = bd.xent(X, W, y)
    total, loss, dX, dW = reference(X, W, y)
    e = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -18
    assert float((got["loss"] - loss).abs().max()) <= 1e-4
    assert abs(float(got["total"] - total)) <= 1e-5 * float(total)
    near(got["dX"], dX, 2 * e)
    near(got["dW"], dW, 3 * e)
    again = bd.xent(X, W, y)
    assert all(torch.equal(got[k], again[k]) for k in got)


def test_gradient_against_differences():
    """total along a direction, by differences of float64 losses of nearby
    inputs, against the gradients' products with it."""
    X, W, y = make(200, 64, 700, "fp32", 9)
    got = bd.xent(X, W, y)
    g = torch.Generator(device="cuda").manual_seed(1)
    a, b = (torch.randn(t.shape, generator=g, device="cuda") for t in (X, W))
    h = 1e-4
    lo, hi = (oracle.xent(f64(X) + s * h * f64(a), f64(W) + s * h * f64(b), y.cpu().numpy())["total"]
              for s in (-1, 1))
    along = float((got["dX"].double() * a).sum() + (got["dW"].double() * b).sum())
    assert abs((hi - lo) / (2 * h) - along) <= 1e-5 * (1 + abs(along))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_streams_graphs_and_given_outputs(dtype):
    X, W, y = make(130, 64, 1000, dtype, 10)
    X = X.view(2, 65, 64)
    y = y.view(2, 65)
    want = bd.xent(X, W, y)
    assert want["dX"].shape == X.shape and want["loss"].shape == y.shape
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = bd.xent(X, W, y, stream=s)
    s.synchronize()
    assert all(torch.equal(want[k], got[k]) for k in want)
    out = {k: torch.full_like(v, 7) for k, v in want.items()}
    ws = torch.empty(bd.xent_workspace_bytes(130, 64, 1000, bd.dtype_code(X.dtype)),
                     dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    bd.xent(X, W, y, out=out, workspace=ws)
    with torch.cuda.graph(graph):
        bd.xent(X, W, y, out=out, workspace=ws)
    X.mul_(0.5)
    graph.replay()
    want = bd.xent(X, W, y)
    torch.cuda.synchronize()
    assert all(torch.equal(want[k], out[k]) for k in want)
    assert bd.workspace_status(ws) == 0


def test_one_gradient_only():
    X, W, y = make(130, 64, 1000, "bf16", 11)
    want = bd.xent(X, W, y)
    import ctypes
    for name in ("dX", "dW"):
        got = torch.empty_like(want[name])
        total, loss = torch.empty(1, device="cuda"), torch.empty(130, device="cuda")
        ws = torch.empty(bd.xent_workspace_bytes(130, 64, 1000, bd.BF16), dtype=torch.uint8,
                         device="cuda")
        o = bd.XentOut(total.data_ptr(), loss.data_ptr(), None, None, None)
        setattr(o, name, got.data_ptr())
        st = bd.lib().flash_gau_xent(X.data_ptr(), W.data_ptr(), y.data_ptr(), 130, 64, 1000,
                                     bd.BF16, bd.MEAN, 1.0, ctypes.byref(o), ws.data_ptr(),
                                     ws.numel(), torch.cuda.current_stream().cuda_stream)
        assert st == bd.OK
        torch.cuda.synchronize()
        assert torch.equal(got, want[name])


def test_refusals():
    X, W, y = make(10, 64, 100, "bf16", 12)
    with pytest.raises(ValueError):
        bd.xent(X, W, y.long())
    with pytest.raises(ValueError):
        bd.xent(X, W.float(), y)
    with pytest.raises(ValueError):
        bd.xent(X, W[:, :32], y)
    with pytest.raises(ValueError):
        bd.xent(X, W.t(), y)
    with pytest.raises(ValueError):
        bd.xent(X, W, y[:5])
    with pytest.raises(ValueError):
        bd.xent(X, W, y, out=dict(dX=W))
    with pytest.raises(bd.FlashGauError):
        bd.xent(X, W, y, scale=float("nan"))
    with pytest.raises(bd.FlashGauError):
        bd.xent(X[:, :60].contiguous(), W[:, :60].contiguous(), y)
    with pytest.raises(bd.FlashGauError):
        bd.xent(X, W, y, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(bd.FlashGauError):
        bd.xent(X[:0], W, y[:0])


@pytest.mark.parametrize("dtype,N,d", [("fp32", 8, 1536), ("fp32", 5, 1524), ("fp32", 8, 1540),
                                       ("fp32", 8, 2048), ("bf16", 2, 6136), ("bf16", 2, 6144),
                                       ("fp32", 2, 6144), ("bf16", 1, 12288), ("fp32", 1, 12276),
                                       ("bf16", 1, 12296), ("bf16", 1, 16384), ("bf16", 4, 4096)])
def test_few_tokens_at_every_width(dtype, N, d):
    """The tokens fill shared memory up to and past what a kernel may have
    without asking for it, beside what it keeps there itself."""
    X, W, y = make(N, d, 70, dtype, N + d, ignored=0.0)
    check(X, W, y, got=bd.xent(X, W, y, grad=False))


@pytest.mark.parametrize("N", [3, 20])
def test_lse_beside_a_label_at_minus_infinity(N):
    """The label's own logit at minus infinity: an infinite loss, and the
    normaliser is the other words'."""
    X, W, y = make(N, 64, 300, "bf16", 17, ignored=0.0)
    X[:, 0] = 1.0
    y.fill_(17)
    W[17, 0] = -float("inf")
    want = torch.logsumexp((X.double() @ W.double().t()), 1)
    got = bd.xent(X, W, y, grad=False)
    assert bool((got["loss"] == float("inf")).all())
    # sums of 300 terms and logits below 10 of 64 products each
    assert float((got["lse"] - want).abs().max()) <= 1e-4


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("d", [4096, 8192, 32768])
def test_fp32_logits_of_wide_rows(d, grad):
    """Positive terms, whose running sum a tensor core cuts off at each of its
    d / 16 steps, against a label whose logit is zero exactly: what the others'
    logits l lose shows in the losses.  In works of n steps that add up in fp32 a
    step loses under 2^-23 of a sum that grows evenly, (n + 1) / 2 of them for a
    work's share: 16.5 2^-23 l with the eight k-blocks of four steps each.  The
    d / 512 works add with roundings of 2^-24 of a sum that grows too, d / 1024
    2^-24 l in all; the five small products before them are under 2^-8 of l
    together, and lose 5 d / 32 2^-23 of that.  Then 2^-21 for an exponential,
    4 u l log2 e for its argument, and (40 + V / 256) u for the sum."""
    g = torch.Generator().manual_seed(d)
    N, V = 40, 300
    X = (torch.rand(N, d, generator=g) / 2 + 0.5).cuda()
    W = (torch.rand(V, d, generator=g) / 2 + 0.5).mul_(40.0 / d).cuda()
    W[17] = 0.0
    y = torch.full((N,), 17, dtype=torch.int32, device="cuda")
    got = bd.xent(X, W, y, grad=grad)
    l = X.double() @ W.double().t()
    err = float((got["loss"] - torch.logsumexp(l, 1)).abs().max())
    top = float(l.max())
    lost = (16.5 * 2 + d / 1024 + 5 * d / 16 * 2.0 ** -8) * U
    limit = lost * top + 2.0 ** -21 + 4 * U * 1.4427 * top + (40 + V / 256) * U + 2 * U * top
    assert err <= limit, (err, limit)


def test_outputs_of_other_names_are_refused():
    X, W, y = make(10, 64, 100, "bf16", 19)
    with pytest.raises(ValueError):
        bd.xent(X, W, y, out=dict(dx=torch.empty_like(X)))
    with pytest.raises(ValueError):
        bd.xent(X, W, y, grad=False, out=dict(losses=torch.empty(10, device="cuda")))


@pytest.mark.parametrize("N,d,V,size", [(64, 64, 500, 8.0), (1001, 520, 8003, 1.0)])
def test_fp32_gradients_take_all_six_products(N, d, V, size):
    """Relative errors in the 2-norm.  With all six products there is what the
    sums cut off (under 5e-7 for eight k-blocks) and roundings to fp32 of about
    2e-7.  Without any one of them it is 2.4e-6 or more in a gradient's product
    at either size, and without one in the logits' (whose errors the first
    size's large logits show) 4e-6: each by arithmetic in 64 bits on the split
    values."""
    X, W, y = make(N, d, V, "fp32", 18, ignored=0.1, pull=0.0 if size > 1 else 0.2, size=size)
    got = bd.xent(X, W, y)
    _, _, dX, dW = reference(X, W, y)
    near(got["dX"], dX, 1.5e-6)
    near(got["dW"], dW, 1.5e-6)


@pytest.mark.parametrize("N,d,V", [(2225, 8, 554), (391, 8, 3), (300, 16, 7), (1000, 64, 20)])
def test_few_other_words_count(N, d, V):
    """Rows whose gradient is the label's word against one or two others: what
    the label's term loses to its rounding is not theirs to bear."""
    X, W, y = make(N, d, V, "bf16", 20, ignored=0.0, size=8.0)
    W *= (torch.arange(V, device="cuda") % 4 + 1)[:, None].to(W.dtype)
    check(X, W, y)
    check(*make(N, d, V, "bf16", 21, ignored=0.1, size=8.0, pull=0.0))


@pytest.mark.parametrize("N,d,V,size", [(6, 8, 5085, 40.0), (92, 24, 3143, 40.0), (29, 32, 812, 8.0)])
def test_words_that_one_token_reaches(N, d, V, size):
    """dW where no sum evens roundings out: a word that is not its token's label
    takes E's rounding, the scaled row's, that of the label's E, which the row's
    factor carries in dW, and the result's, 2^-8 each."""
    X, W, y = make(N, d, V, "bf16", 22, ignored=0.0, size=size, pull=0.0)
    got = bd.xent(X, W, y)
    x, w, lab = f64(X), f64(W), y.cpu().numpy()
    want = oracle.xent(x, w, lab)
    P = np.exp(x @ w.T - want["lse"][:, None])
    P[np.arange(N), lab] = 0.0
    P[np.arange(N), lab] = P.sum(1)
    S = (np.abs(x) @ np.abs(w).T).max(1)
    el = (d / 16 + 8) * 2.0 ** -22 * S + 8 * U * np.abs(x @ w.T).max(1)
    h = 2.0 ** -8
    rel = ((1 + h) ** 3 - 1 + 4 * el + 2.0 ** -20 + V * U / 8)[:, None] + (N / 16 + 8) * 2.0 ** -22
    bound = (P * rel / N).T @ np.abs(x)
    lim = bound + h * (np.abs(want["dW"]) + bound) + 1e-33
    err = np.abs(f64(got["dW"]) - want["dW"])
    assert np.all(err <= lim), float(np.max(err / lim))
