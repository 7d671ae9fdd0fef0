"""GPU checks of sampling against the float64 oracle.

Tokens and counts are equal to the oracle's.  Both turn on sums of w, which
the kernel knows to 2^-40 of w and half a unit of 2^-44: of the rows here (some
thousand with up to 140000 words) one in a hundred thousand could differ.  logp
is one rounding of its value, and 2^-40 and V / 2 units of 2^-44 of the mass."""

import ctypes

import numpy as np
import pytest
import torch

import oracle
from efficient_attention_transformer_gb300 import binding as bd

pytestmark = pytest.mark.gpu
MODES = ["none", "top_k", "top_p", "min_p", "all"]
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from efficient_attention_transformer_gb300.build import build
    build()


def settings(mode, N, rng, V):
    kw = dict(temperature=torch.tensor(rng.uniform(0.5, 1.5, N), dtype=torch.float32))
    if mode in ("top_k", "all"):
        kw["top_k"] = torch.tensor(rng.integers(0, min(V, 200) + 2, N), dtype=torch.int32)
    if mode in ("top_p", "all"):
        kw["top_p"] = torch.tensor(rng.uniform(0.1, 0.999, N), dtype=torch.float32)
    if mode in ("min_p", "all"):
        kw["min_p"] = torch.tensor(rng.uniform(0.0, 0.2, N), dtype=torch.float32)
    return kw


def check(logits, u, kw, rows=None):
    """logits, u and the settings (host or device tensors) against the oracle."""
    dev = {k: v.cuda() for k, v in kw.items()}
    logits, u = logits.cuda(), u.cuda()
    token, logp, kept = bd.sample(logits, u, **dev)
    torch.cuda.synchronize()
    l, V = logits.double().cpu().numpy(), logits.shape[1]
    got = [t.cpu().numpy() for t in (token, logp, kept)]
    args = [None if kw.get(k) is None else kw[k].double().cpu().numpy()
            for k in ("temperature", "top_k", "top_p", "min_p")]
    for i in range(len(l)) if rows is None else rows:
        t, k, p, m = (d if a is None else a[i] for a, d in zip(args, (1.0, 0, 1.0, 0.0)))
        want = oracle.sample_row(l[i], float(u[i]), t, k, p, m)
        assert (got[0][i], got[2][i]) == (want[0], want[2]), (i, want, [g[i] for g in got])
        if want[0] < 0:
            assert np.isnan(got[1][i])
        else:
            assert abs(got[1][i] - want[1]) <= abs(want[1]) * 2.0 ** -24 + 2.0 ** -40 + V * 2.0 ** -45
    return token, logp, kept


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("N,V", [(3, 1), (4, 2), (5, 31), (5, 33), (4, 257), (40, 1000), (3, 1025),
                                 (160, 2049), (6, 4097), (8, 8003), (4, 32000), (3, 50257)])
def test_sizes(N, V, mode, dtype):
    rng = np.random.default_rng(V + len(mode))
    logits = torch.tensor(rng.normal(size=(N, V)) * 3).to(dtype)
    check(logits, torch.tensor(rng.random(N), dtype=torch.float32), settings(mode, N, rng, V))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("values", [1, 2, 7, 100])
@pytest.mark.parametrize("V", [300, 5000, 20000])
def test_equal_words(V, values, mode, dtype):
    """Rows of a few values: places inside long runs of equal words."""
    rng = np.random.default_rng(V + values)
    logits = torch.tensor(rng.integers(0, values, (6, V)) * 0.37 - 1).to(dtype)
    kw = settings(mode, 6, rng, V)
    if "top_k" in kw:
        kw["top_k"] = torch.tensor(rng.integers(1, V, 6), dtype=torch.int32)
    check(logits, torch.tensor(rng.random(6), dtype=torch.float32), kw)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("spread", [1e-6, 1e-3, 0.02, 300.0])
def test_words_close_together_and_far_apart(spread, mode):
    """All of a row in one bin of the first search (keys decide), or most of
    it below any weight."""
    rng = np.random.default_rng(5)
    logits = torch.tensor(20 + rng.normal(size=(5, 9000)) * spread, dtype=torch.float32)
    check(logits, torch.tensor(rng.random(5), dtype=torch.float32), settings(mode, 5, rng, 9000))
    logits = torch.tensor(rng.normal(size=(5, 9000)) * spread, dtype=torch.float32)  # around zero
    check(logits, torch.tensor(rng.random(5), dtype=torch.float32), settings(mode, 5, rng, 9000))


def test_exact_shares():
    """Shares that equal words meet exactly: the word that reaches p is the last."""
    V = 64
    logits = torch.zeros(5, V)
    p = torch.tensor([0.5, 0.25, 0.015625, 1.0, 0.0])
    u = torch.tensor([0.0, 0.5, 0.99, 0.75, 0.3])
    token, _, kept = check(logits, u, dict(top_p=p))
    assert kept.tolist() == [32, 16, 1, 64, 1] and token.tolist() == [0, 8, 0, 48, 0]


def test_settings_at_their_ends():
    rng = np.random.default_rng(3)
    N, V = 24, 700
    logits = torch.tensor(rng.normal(size=(N, V)) * 2, dtype=torch.float32)
    u = torch.tensor(rng.random(N), dtype=torch.float32)
    u[0], u[1], u[2], u[3] = 0.0, 1 - 2.0 ** -24, 1.0, 5.0
    T = torch.ones(N)
    T[4], T[5], T[6], T[7], T[8], T[9] = 0.0, 1e-31, 1e-29, 1e4, 1e30, INF
    T[10], T[11] = -1.0, NAN
    k = torch.zeros(N, dtype=torch.int32)
    k[12], k[13], k[14], k[15], k[16] = 1, V, V + 1, -3, V - 1
    p = torch.ones(N)
    p[17], p[18], p[19] = 0.0, -1.0, NAN
    m = torch.zeros(N)
    m[20], m[21], m[22] = 1.0, 2.0, NAN
    u[23] = NAN
    check(logits, u, dict(temperature=T, top_k=k, top_p=p, min_p=m))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("mode", MODES)
def test_masked_and_unusable_rows(mode, dtype):
    rng = np.random.default_rng(9)
    N, V = 12, 3001
    l = rng.normal(size=(N, V)) * 2
    l[0] = -INF
    l[1, 1:] = -INF
    l[2, :-1] = -INF
    l[3, 5] = NAN
    l[4, 3000] = INF
    l[5, ::2] = -INF
    l[6] = -3.0e38
    l[7, :100] = 3.0e38
    l[8] = np.where(rng.random(V) < 0.5, -0.0, 0.0)
    l[9] = rng.choice([1e-40, -1e-40, 0.0], V)
    l[10, 0], l[10, 1:] = 3.0e38, -3.0e38
    l[11, :] = -INF
    l[11, 0], l[11, 2999] = NAN, 1.0
    kw = settings(mode, N, rng, V)
    check(torch.tensor(l).to(dtype), torch.tensor(rng.random(N), dtype=torch.float32), kw)


# Long rows of fp32, few enough that several blocks take each.
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("N,V", [(1, 16384), (14, 16385), (1, 131072), (15, 20480), (33, 20483),
                                 (34, 28672), (76, 28675), (77, 28672), (2, 300001)])
def test_long_rows(N, V, mode):
    rng = np.random.default_rng(V + N)
    logits = torch.tensor(rng.normal(size=(N, V)) * 3, dtype=torch.float32)
    logits[torch.tensor(rng.random((N, V)) < 0.1)] = -float("inf")
    check(logits, torch.tensor(rng.random(N), dtype=torch.float32), settings(mode, N, rng, V),
          rows=sorted({0, N // 2, N - 1}))


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("N", [3, 20, 40])
@pytest.mark.parametrize("kind", ["few values", "close together", "one word", "last words"])
def test_long_rows_of_a_kind(kind, N, mode):
    V = 30011
    rng = np.random.default_rng(N)
    if kind == "few values":
        x = rng.integers(0, 3, (N, V)) * 0.37 - 1
    elif kind == "close together":
        x = 20 + rng.normal(size=(N, V)) * 1e-3
    else:
        x = np.full((N, V), -np.inf)
        if kind == "one word":
            x[np.arange(N), rng.integers(0, V, N)] = rng.normal(size=N)
        else:
            x[:, V - 5:] = rng.normal(size=(N, 5))
    kw = settings(mode, N, rng, V)
    if "top_k" in kw:
        kw["top_k"] = torch.tensor(rng.integers(1, V, N), dtype=torch.int32)
    check(torch.tensor(x, dtype=torch.float32), torch.tensor(rng.random(N), dtype=torch.float32),
          kw, rows=sorted({0, 1, N - 1}))


@pytest.mark.parametrize("N", [8, 24, 60])
def test_long_rows_of_every_outcome_at_once(N):
    """Greedy rows, rows without a distribution and unusable settings beside
    ordinary ones: each leaves by a way of its own."""
    V, rng = 30000, np.random.default_rng(N)
    logits = torch.tensor(rng.normal(size=(N, V)), dtype=torch.float32)
    kw = settings("all", N, rng, V)
    logits[0] = -float("inf")
    logits[1, 29999] = float("nan")
    logits[2, 7] = float("inf")
    kw["temperature"][3] = 0.0
    kw["temperature"][4] = -1.0
    kw["top_p"][5] = float("nan")
    kw["top_k"][6] = 1
    token, _, _ = check(logits, torch.tensor(rng.random(N), dtype=torch.float32), kw)
    assert (token[[0, 1, 2, 4, 5]] == -1).all()


def test_long_rows_do_not_depend_on_their_number():
    """One block a row, or a cluster of two, four or eight: the same bits, on
    replays of a captured call too."""
    V, rng = 33001, np.random.default_rng(8)
    rows = torch.tensor(rng.normal(size=(100, V)) * 2, dtype=torch.float32).cuda()
    u = torch.tensor(rng.random(100), dtype=torch.float32).cuda()
    kw = dict(top_k=1000, top_p=0.9, min_p=0.001, temperature=0.8)
    want = [x.clone() for x in bd.sample(rows, u, **kw)]
    for n in (1, 14, 33, 76):
        got = bd.sample(rows[:n], u[:n], **kw)
        assert all(torch.equal(g, w[:n]) for g, w in zip(got, want)), n
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            again = bd.sample(rows[:n], u[:n], **kw)
        for _ in range(3):
            for x in again:
                x.fill_(-7)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(g, w[:n]) for g, w in zip(again, want)), n


@pytest.mark.parametrize("N,offset,ld", [(5, 1, 20001), (16, 3, 24007), (40, 2, 30002)])
def test_long_rows_further_apart_and_odd_addresses(N, offset, ld):
    V, rng = ld - 9, np.random.default_rng(ld)
    flat = torch.tensor(rng.normal(size=N * ld + offset), dtype=torch.float32).cuda()
    logits = flat[offset:].view(N, ld)[:, :V]
    u = torch.tensor(rng.random(N), dtype=torch.float32)
    check(logits, u, settings("all", N, rng, V), rows=[0, N - 1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset,ld", [(1, 1001), (3, 1016), (0, 1004), (5, 2001)])
def test_rows_further_apart_and_odd_addresses(dtype, offset, ld):
    rng = np.random.default_rng(7)
    N, V = 9, 1000
    flat = torch.full((N * ld + offset,), NAN, dtype=dtype, device="cuda")
    rows = flat[offset:].view(N, ld)[:, :V]
    rows.copy_(torch.tensor(rng.normal(size=(N, V)) * 2))
    kw = settings("all", N, rng, V)
    u = torch.tensor(rng.random(N), dtype=torch.float32)
    a = check(rows, u, kw)
    b = bd.sample(rows.contiguous(), u.cuda(), **{k: v.cuda() for k, v in kw.items()})
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_most_words(dtype):
    """The largest vocabulary, in smaller units."""
    g = torch.Generator(device="cuda").manual_seed(0)
    logits = torch.randn(2, 1 << 22, generator=g, device="cuda").mul_(2).to(dtype)
    u = torch.tensor([0.37, 0.93])
    check(logits, u, {})
    check(logits, u, dict(top_p=torch.tensor([0.9, 0.5])))
    check(logits, u, dict(top_k=torch.tensor([100, 2000000], dtype=torch.int32)))


@pytest.mark.parametrize("mode", MODES)
def test_bf16_rows_of_every_value(mode):
    """bf16 rows are counted by value where all words lie between 2^-40 and 2^8
    in magnitude (or are zero or minus infinity): rows at those borders, rows
    with words just outside, many equal words, and every value there is."""
    rng = np.random.default_rng(12)
    V = 140001
    l = rng.normal(size=(8, V))
    l[0, :70000] = 1.5
    l[1] = np.where(rng.random(V) < 0.5, -0.0, 0.0)
    l[1, ::1000] = 1.0
    l[2] = 0.25
    bits = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    bits = bits[torch.isfinite(bits)].double()
    l[3] = rng.choice(bits[bits.abs() < 1000].numpy(), V)
    l[4] = rng.choice(bits[(bits.abs() < 256) & ((bits.abs() >= 2.0 ** -40) | (bits == 0))].numpy(), V)
    l[5, 77] = 255.0
    l[6, 77] = 256.0
    l[7] = -np.abs(l[7]) - 0.1
    l[7, 1000], l[7, 2000] = -2.0 ** -40, -2.0 ** -41
    kw = settings(mode, 8, rng, V)
    kw["temperature"][3:5] = 100.0
    kw["temperature"][5:7] = 60.0
    check(torch.tensor(l).to(torch.bfloat16), torch.tensor(rng.random(8), dtype=torch.float32), kw)
    l = torch.tensor(rng.normal(size=(3, 500)) * 20).to(torch.bfloat16)
    check(l, torch.tensor([0.1, 0.5, 0.9]), dict(min_p=torch.tensor([1e-30, 1e-16, 1e-12])))
    l = -torch.rand(4, 3000, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16) - 2 ** -9
    check(l, torch.tensor([0.1, 0.5, 0.9, 0.99]), settings(mode, 4, rng, 3000))


def test_draws_follow_the_distribution():
    """4096 even steps of u: each word as often as its probability says, to one
    step at each of its ends."""
    logits = torch.tensor([0.5, -1.0, 2.0, 0.5, -INF, 1.0], device="cuda").expand(4096, 6)
    u = (torch.arange(4096, device="cuda") + 0.5) / 4096
    token, logp, kept = bd.sample(logits.contiguous(), u, temperature=0.8)
    p = torch.softmax(logits[0].double() / 0.8, 0)
    n = torch.bincount(token.long(), minlength=6).double()
    assert bool(((n - 4096 * p).abs() <= 1 + 1e-6).all()) and bool((kept == 5).all())
    assert torch.allclose(logp.double(), p.log()[token.long()], atol=1e-6)


def test_single_values_and_leading_shapes():
    g = torch.Generator(device="cuda").manual_seed(1)
    logits = torch.randn(2, 3, 500, generator=g, device="cuda")
    u = torch.rand(2, 3, generator=g, device="cuda")
    a = bd.sample(logits, u, temperature=0.7, top_k=20, top_p=0.9, min_p=0.01)
    full = lambda v, dt=torch.float32: torch.full((6,), v, dtype=dt, device="cuda")  # noqa: E731
    b = bd.sample(logits.view(6, 500), u.view(6), temperature=full(0.7),
                  top_k=full(20, torch.int32), top_p=full(0.9), min_p=full(0.01))
    assert a[0].shape == (2, 3) and all(torch.equal(x.view(6), y) for x, y in zip(a, b))
    one = bd.sample(logits[0, 0], u[0, 0], temperature=0.7, top_k=20, top_p=0.9, min_p=0.01)
    assert one[0].shape == () and one[0] == a[0][0, 0]


def test_rows_do_not_depend_on_one_another():
    """Any subset of rows, on other streams and replayed, gives the same."""
    rng = np.random.default_rng(4)
    N, V = 200, 3000
    logits = torch.tensor(rng.normal(size=(N, V)) * 2, dtype=torch.bfloat16, device="cuda")
    u = torch.tensor(rng.random(N), dtype=torch.float32, device="cuda")
    kw = {k: v.cuda() for k, v in settings("all", N, rng, V).items()}
    want = bd.sample(logits, u, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    part = bd.sample(logits[50:57], u[50:57], stream=s, **{k: v[50:57] for k, v in kw.items()})
    s.synchronize()
    assert all(torch.equal(a, b[50:57]) for a, b in zip(part, want))
    outs = [torch.full((N + 2,), 7, dtype=t.dtype, device="cuda") for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bd.sample(logits, u, out_token=outs[0][1:-1], out_logp=outs[1][1:-1],
                  out_kept=outs[2][1:-1], **kw)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a[1:-1], b) and a[0] == 7 and a[-1] == 7
    u.copy_(1 - u)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a[1:-1], b) for a, b in zip(outs, bd.sample(logits, u, **kw)))


def test_only_the_token():
    logits = torch.randn(5, 100, device="cuda")
    u = torch.rand(5, device="cuda")
    token = torch.empty(5, dtype=torch.int32, device="cuda")
    s = bd.Sampling(None, None, None, None)
    bd._check(bd.lib().flash_gau_sample(logits.data_ptr(), 100, 5, 100, bd.FP32, u.data_ptr(),
                                        ctypes.byref(s), token.data_ptr(), None, None,
                                        torch.cuda.current_stream().cuda_stream))
    assert torch.equal(token, bd.sample(logits, u)[0])


def test_binding_refuses():
    l, u = torch.randn(4, 10, device="cuda"), torch.rand(4, device="cuda")
    for kw in (dict(temperature=u[:3]), dict(top_k=u), dict(top_p=u.double()), dict(min_p=u.cpu()),
               dict(out_token=u)):
        with pytest.raises(ValueError):
            bd.sample(l, u, **kw)
    with pytest.raises(ValueError):
        bd.sample(l.t(), torch.rand(10, device="cuda"))
    with pytest.raises(ValueError):
        bd.sample(l, u.double())
    with pytest.raises(bd.FlashGauError):
        bd.sample(l[:0], u[:0])
    with pytest.raises(bd.FlashGauError):
        bd.sample(l[:, :0], u)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,V", [(6, 3), (6, 5000), (6, 40000), (40, 30000)])
def test_min_p_above_one_keeps_the_first_word(N, V, dtype):
    """Rows whose largest word has equals, with the other filters on and off: at
    min_p 1 all of them are kept, above it the first one alone."""
    rng = np.random.default_rng(V)
    logits = torch.tensor(rng.normal(size=(N, V))).clamp(max=1.0)
    logits[:, 1:3] = 1.0
    m = torch.tensor(np.resize([1.0, 1.0 + 2.0 ** -23, 2.0, INF], N), dtype=torch.float32)
    u = torch.full((N,), 0.9)
    for kw in (dict(), dict(top_p=torch.full((N,), 0.95)),
               dict(top_k=torch.full((N,), 3, dtype=torch.int32))):
        _, _, kept = check(logits.to(dtype), u, dict(min_p=m, **kw), rows=range(min(N, 8)))
        assert (kept[m.cuda() > 1] == 1).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("N,V", [(9, 7), (9, 3000), (9, 30000)])
def test_logits_and_temperatures_of_every_size(N, V, mode, dtype):
    """Differences of finite logits that fp32 does not hold, temperatures at
    which those have a weight, and the same in other sizes."""
    rng = np.random.default_rng(V)
    most = 3.3e38
    l, kw = rng.uniform(-1, 1, (N, V)), settings(mode, N, rng, V)
    T = kw["temperature"]
    for i, (size, t) in enumerate([(most, 1e38), (most, 3e37), (most, INF), (most, 1.0),
                                   (1e36, 2.5e35), (2.0 ** 63, 2.0 ** 64), (1e20, 1.8e19),
                                   (1e-30, 1e-30), (1e-38, 3.4e38)]):
        l[i] *= size
        T[i] = t
    l[:3, 0], l[:3, 1] = most, -most
    u = torch.tensor(rng.random(N), dtype=torch.float32)
    u[0] = 1 - 2.0 ** -24  # the last word, which weighs e^-6.6 here
    check(torch.tensor(l).to(dtype), u, kw)
    if mode == "none":
        x = torch.tensor([[3e38, -3e38]], dtype=dtype)
        assert check(x, u[:1], dict(temperature=torch.tensor([1e38])))[0].tolist() == [1]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [2, 3000, 30000])
def test_min_p_that_lets_every_finite_logit_through(V, dtype):
    """top + T ln(min_p) below the lowest finite number, and where it is not."""
    rng = np.random.default_rng(V)
    l = rng.uniform(-3.3e38, -3e38, (6, V))
    T = torch.tensor([1e38, 1e38, 1e37, INF, 3.4e38, 1e30])
    m = torch.tensor([0.1, 2.0 ** -140, 0.01, 0.999, 0.5, 0.9])
    u = torch.tensor(rng.random(6), dtype=torch.float32)
    _, _, kept = check(torch.tensor(l).to(dtype), u, dict(temperature=T, min_p=m))
    assert (kept[:5] == V).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [5, 3000, 30000])
def test_zeros_of_either_sign(V, dtype):
    """u, T, top_p and min_p at minus zero are at zero."""
    rng = np.random.default_rng(V)
    logits = torch.tensor(rng.normal(size=(6, V))).to(dtype)
    zero = torch.zeros(6)
    zero[1::2] = -0.0
    logits[1::2] = logits[::2]
    settings = [dict(), dict(top_p=torch.full((6,), 0.9)), dict(min_p=zero),
                dict(top_k=torch.full((6,), 3, dtype=torch.int32)), dict(top_p=zero),
                dict(temperature=zero)]
    for kw in settings:
        got = check(logits, zero, kw)
        assert all(torch.equal(x[::2], x[1::2]) for x in got)
        assert torch.equal(got[0], check(logits, torch.zeros(6), dict(temperature=torch.zeros(6)))[0])
