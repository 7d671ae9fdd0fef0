"""GPU checks of the 8-bit activation checkpoints against the float64 oracle.

r, codes, scales and the restored stream follow from their definition to the
last bit: r is one rounding of h + y, a code the nearest whole number to an
exact quotient, a value the fp32 product of code and scale (rounded to bf16
once more).  Norms and gradients get the bounds of the residual stream's own
tests, which count the same sums; column sums here add M / 608 rows of a warp
(of a fourth of them where four warps share a row), 4 warps and 608 blocks'
parts in eighths behind one another."""

import ctypes

import numpy as np
import pytest
import torch

import oracle
from efficient_attention_transformer_gb300 import binding as bd
from test_gpu_residual_norm import KIND, U, f64, grad_error, one, unit_error, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from efficient_attention_transformer_gb300.build import build
    build()


class Problem:
    def __init__(self, M, d, dtype, norm, seed=0, offset=0, with_y=True):
        g = torch.Generator().manual_seed(seed)
        self.io = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.half = 2.0 ** -8 if dtype == "bf16" else U
        self.M, self.d, self.norm = M, d, norm

        def dev(x, dt=torch.float32):
            flat = torch.empty(x.numel() + offset, dtype=dt, device="cuda")[offset:]
            return flat.copy_(x.reshape(-1)).view(x.shape)

        rows = lambda sd=1.0, m=0.0: dev(torch.randn(M, d, generator=g) * sd + m, self.io)  # noqa: E731
        # a few loud channels
        loud = 1 + 20 * (torch.rand(d, generator=g) < 0.02).float()
        self.h = dev((torch.randn(M, d, generator=g) * 1.5 + 0.2) * loud, self.io)
        self.y = rows(2.0) if with_y else None
        self.dr, self.dn = rows(), rows()
        self.kw = dict(norm=KIND[norm], norm_g=None, norm_b=None, eps=1e-5)
        if norm == "layer":
            self.kw.update(norm_g=dev(torch.randn(d, generator=g) * 0.3 + 1),
                           norm_b=dev(torch.randn(d, generator=g) * 0.3))
        elif norm == "scale":
            self.kw.update(norm_g=dev(torch.full((1,), 0.9 * d ** 0.5)))
        # memory of every array behind `offset` elements
        self.out = bd.Checkpoint(dev(torch.zeros(M, d), torch.int8),
                                 dev(torch.zeros(M, -(-d // 128))))

    def params(self):
        return f64(self.kw["norm_g"]), f64(self.kw["norm_b"])


def check_norm(name, n, x, p, e_in=0.0):
    """n = norm(x), x known to e_in."""
    g, b = p.params()
    want = oracle.norm_rows(x, p.norm, g, b, 1e-5)[2]
    e, u, s = unit_error(x, p.norm, 1e-5)
    e_in = np.broadcast_to(e_in, x.shape)
    e = e + s * (e_in + e_in.mean(1, keepdims=True)) * (1 + np.abs(u))
    tot = (np.abs(u) * e_in).mean(1, keepdims=True) if p.norm == "layer" else (
        np.abs(u) * e_in).sum(1, keepdims=True)
    e = e + np.abs(u) * s * tot
    ag, ab = one(g), 0.0 if b is None else np.abs(b)
    en = ag * e + 8 * U * (ag * np.abs(u) + ab)
    within(name, n, want, en + p.half * (np.abs(want) + en))


def check(p):
    packed, r, n = bd.checkpoint_pack(p.h, p.y, out=p.out, **p.kw)
    x, xn = bd.checkpoint_restore(packed, p.io, **p.kw)
    torch.cuda.synchronize()
    if p.y is None:
        assert r is p.h
        exact = f64(p.h)
    else:
        assert torch.equal(r, (p.h.float() + p.y.float()).to(p.io))
        exact = f64(p.h) + f64(p.y)
    codes, scales = oracle.checkpoint_codes(f64(r))
    assert np.array_equal(packed.scales.cpu().numpy(), scales)
    assert np.array_equal(packed.codes.cpu().numpy(), codes)
    v = oracle.checkpoint_values(codes, scales)
    assert torch.equal(x, torch.tensor(v, device="cuda").float().to(p.io))
    if p.norm == "none":
        assert n is None and xn is None
        return
    check_norm("n", n, exact, p, 2 * U * np.abs(exact))
    check_norm("xn", xn, v, p)
    check_grad(p, packed, v)


def check_grad(p, packed, v, dr=True):
    out = bd.checkpoint_backward(p.dr if dr else None, p.dn, packed, **p.kw)
    torch.cuda.synchronize()
    g, b = p.params()
    d0, dn = f64(p.dr) * dr, f64(p.dn)
    want = oracle.residual_norm_grad(d0, dn, v, None, "none", None, None, None, None, p.norm, g, b,
                                     1e-5)
    ex, eg = grad_error(v, p.norm, g, dn, np.zeros_like(dn), 1e-5)
    e = 4 * U * np.abs(d0) + ex + 2 * U * np.abs(want["dh"])
    within("dh", out["dh"], want["dh"], e + p.half * (np.abs(want["dh"]) + e))
    adds = min(p.M, p.M / 608 + 4 + 608 / 8 + 8) + 40
    col = lambda terms, err: err.sum(0) + adds * U * np.abs(terms).sum(0)  # noqa: E731
    un = oracle.norm_rows(v, p.norm, 1.0, None, 1e-5)[0]
    bound = col(dn * un, eg)
    if p.norm == "scale":
        bound = bound.sum().reshape(1) + 64 * U * np.abs(dn * un).sum()
        assert out["dnorm_b"] is None
    else:
        within("dnorm_b", out["dnorm_b"], want["dnorm_b"], col(dn, 0 * dn))
    within("dnorm_g", out["dnorm_g"], want["dnorm_g"], bound)
    return out


SIZES = [(1, 768), (2, 1), (3, 5), (7, 31), (64, 64), (5, 127), (5, 128), (5, 129), (5, 257),
         (130, 768), (33, 1001), (9, 1024), (9, 1032), (3, 2048), (2, 4096), (2, 4095), (1300, 40),
         (700, 3), (40, 2056), (17, 8192), (9, 8191), (5, 6000), (400, 1536), (3000, 200)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("M,d", SIZES)
def test_sizes(M, d, dtype):
    check(Problem(M, d, dtype, "layer", M + d))


# Widths on both sides of what a row's threads span with up to seven columns in
# front, and enough rows that each of a LayerNorm's warps has several.
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("norm", ["layer", "scale"])
@pytest.mark.parametrize("M,d", [(2600, 249), (2500, 250), (2500, 511), (3001, 761), (1999, 762),
                                 (1500, 767), (1300, 1017), (1301, 1018), (700, 1501), (333, 2041),
                                 (334, 2042), (320, 4089), (317, 4090), (200, 6001), (170, 8185),
                                 (170, 8186), (4001, 12), (5000, 7)])
def test_rows_that_are_not_whole_vectors(M, d, norm, dtype):
    check(Problem(M, d, dtype, norm, 5))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,d", [(1, 5), (3, 129), (5, 767), (9, 1500), (3, 4099), (4, 256)])
def test_nothing_beside_the_arrays_is_written(M, d, dtype):
    """codes, scales and r in the middle of larger buffers; the others' neighbours
    are the rows before and behind, whose values every test compares."""
    groups, g = -(-d // 128), torch.Generator().manual_seed(3)
    codes = torch.full((16 + M * d + 16,), 77, dtype=torch.int8, device="cuda")
    scales = torch.full((16 + M * groups + 16,), 7.0, device="cuda")
    h = torch.full((16 + M * d + 16,), 3.0, dtype=dtype, device="cuda")
    inner = lambda x, n: x[16:16 + n]  # noqa: E731
    rows = inner(h, M * d).view(M, d)
    rows.copy_(torch.randn(M, d, generator=g))
    packed = bd.Checkpoint(inner(codes, M * d).view(M, d),
                           inner(scales, M * groups).view(M, groups))
    want = oracle.checkpoint_codes(f64(rows) * 2)
    bd.checkpoint_pack(rows, rows.clone(), out=packed, out_r=rows)
    for x, v in ((codes, 77), (scales, 7.0), (h, 3.0)):
        assert (x[:16] == v).all() and (x[-16:] == v).all()
    assert (packed.codes.cpu().numpy() == want[0]).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("norm", ["none", "layer", "scale"])
@pytest.mark.parametrize("with_y", [True, False])
@pytest.mark.parametrize("d,offset", [(200, 0), (384, 1), (384, 8), (1100, 3), (2048, 4)])
def test_options_and_addresses(d, offset, norm, dtype, with_y):
    check(Problem(37, d, dtype, norm, 11, offset, with_y))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_no_gradient_from_the_stream(dtype):
    p = Problem(50, 320, dtype, "layer", 3)
    packed = bd.checkpoint_pack(p.h)[0]
    check_grad(p, packed, oracle.checkpoint_values(*(t.cpu().numpy() for t in packed)), dr=False)


def test_codes_of_every_kind():
    """Quotients at and next to halves, in both directions, and all sizes of
    scale down to the least."""
    g = torch.Generator().manual_seed(8)
    n = torch.randint(-126, 127, (2000, 128), generator=g).float() + 0.5
    scale = torch.exp2(torch.randint(-90, 90, (2000, 1), generator=g).float())
    scale = scale * (1 + torch.rand(2000, 1, generator=g))
    x = n * scale
    k = torch.randint(-2, 3, x.shape, generator=g, dtype=torch.int32)
    x = (x.view(torch.int32) + k).view(torch.float32)  # some last places off
    x[:, 0] = 127.0 * scale[:, 0]
    x[::3] = x[::3].to(torch.bfloat16).float()
    for io in (torch.float32, torch.bfloat16):
        h = x.to(io).cuda()
        packed = bd.checkpoint_pack(h)[0]
        codes, scales = oracle.checkpoint_codes(f64(h))
        assert np.array_equal(packed.codes.cpu().numpy(), codes)
        assert np.array_equal(packed.scales.cpu().numpy(), scales)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_special_values(dtype):
    inf, nan = float("inf"), float("nan")
    h = torch.zeros(8, 300)
    h[1, 5], h[2, 290], h[3, 130], h[3, 131] = inf, nan, -inf, nan
    h[4, 7] = 2.0 ** -101
    h[5, 7] = 2.0 ** -100
    h[6, ::3] = 3e38
    h[7, 0], h[7, 299] = -nan, 1.0
    h = h.to(dtype).cuda()
    packed = bd.checkpoint_pack(h)[0]
    codes, scales = oracle.checkpoint_codes(f64(h))
    assert np.array_equal(packed.scales.cpu().numpy(), scales, equal_nan=True)
    assert np.array_equal(packed.codes.cpu().numpy(), codes)
    x = bd.checkpoint_restore(packed, dtype)[0]
    v = torch.tensor(oracle.checkpoint_values(codes, scales), device="cuda").float().to(dtype)
    assert torch.equal(torch.isnan(x), torch.isnan(v))
    assert torch.equal(x.nan_to_num(), v.nan_to_num())
    # a row that is not finite has no norm; the others are not touched by it
    g = torch.ones(300, device="cuda")
    n = bd.checkpoint_restore(packed, dtype, norm=bd.NORM_LAYER, norm_g=g)[1]
    assert [bool(torch.isnan(r).all()) for r in n] == [False, True, True, True, False, False,
                                                        bool(torch.isnan(n[6]).all()), True]


@pytest.mark.parametrize("norm", ["layer", "scale"])
def test_zero_rows_and_constant_rows(norm):
    p = Problem(6, 256, "fp32", norm, 4)
    p.h[0] = 0
    p.y[0] = 0
    p.h[1] = 1.0
    p.y[1] = 2.0
    check(p)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("d", [768, 513, 3000])
def test_rows_in_their_inputs_place(dtype, d):
    p = Problem(45, d, dtype, "layer", 9)
    packed, r, n = bd.checkpoint_pack(p.h, p.y, **p.kw)
    a, b = p.h.clone(), p.y.clone()
    bd.checkpoint_pack(a, b, out_r=a, out_n=b, **p.kw)
    assert torch.equal(a, r) and torch.equal(b, n)
    a, b = p.h.clone(), p.y.clone()
    again = bd.checkpoint_pack(a, b, out_r=b, out_n=a, **p.kw)[0]
    assert torch.equal(b, r) and torch.equal(a, n) and torch.equal(again.codes, packed.codes)
    want = bd.checkpoint_backward(p.dr, p.dn, packed, **p.kw)
    for k in ("dr", "dn"):
        t = dict(dr=p.dr.clone(), dn=p.dn.clone())
        got = bd.checkpoint_backward(t["dr"], t["dn"], packed, out=dict(dh=t[k]), **p.kw)
        assert got["dh"] is t[k]
        assert all(torch.equal(got[x], want[x]) for x in want)


def test_same_as_the_residual_stream():
    """r and n are residual_norm's, and the gradients residual_norm_backward's
    at the restored stream (fp32: the same numbers up to the order of sums)."""
    p = Problem(200, 640, "fp32", "layer", 13)
    packed, r, n = bd.checkpoint_pack(p.h, p.y, **p.kw)
    r2, n2 = bd.residual_norm(p.h, p.y, **p.kw)
    assert torch.equal(r, r2)
    torch.testing.assert_close(n, n2, rtol=1e-5, atol=1e-5)
    x, _ = bd.checkpoint_restore(packed, torch.float32)
    a = bd.checkpoint_backward(p.dr, p.dn, packed, **p.kw)
    b = bd.residual_norm_backward(p.dr, p.dn, x, p.y, **p.kw)
    for k in ("dh", "dnorm_g", "dnorm_b"):
        torch.testing.assert_close(a[k], b[k], rtol=1e-4, atol=1e-4)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("norm", ["layer", "scale"])
def test_repeats_streams_and_replays(dtype, norm):
    p = Problem(2500, 392, dtype, norm, 21)

    def once():
        packed, r, n = bd.checkpoint_pack(p.h, p.y, **p.kw)
        x, xn = bd.checkpoint_restore(packed, p.io, **p.kw)
        g = bd.checkpoint_backward(p.dr, p.dn, packed, **p.kw)
        return [packed.codes, packed.scales, r, n, x, xn] + [t for t in g.values() if t is not None]

    want = once()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(once())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        captured = once()
    graph.replay()
    torch.cuda.synchronize()
    for g in got + [captured]:
        assert all(torch.equal(a, b) for a, b in zip(g, want))
    p.h.add_(1.0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(captured, once()))


def test_only_what_is_asked_for():
    """Through the C ABI: no r, one of the parameters' gradients, rows behind
    the last left alone, a workspace full of NaN."""
    p = Problem(10, 256, "bf16", "layer", 2)
    L, at = bd.lib(), torch.cuda.current_stream().cuda_stream
    o = bd.Residual(0, bd.NORM_LAYER, None, None, p.kw["norm_g"].data_ptr(),
                    p.kw["norm_b"].data_ptr(), None, None, 1e-5)
    packed, r, n = bd.checkpoint_pack(p.h, p.y, **p.kw)
    n2 = torch.full((12, 256), 7.0, dtype=p.io, device="cuda")
    c2 = torch.full((12, 256), 7, dtype=torch.int8, device="cuda")
    s2 = torch.full((12, 2), 7.0, device="cuda")
    bd._check(L.flash_gau_checkpoint_pack(p.h.data_ptr(), p.y.data_ptr(), ctypes.byref(o), 10, 256,
                                          bd.BF16, None, n2.data_ptr(), c2.data_ptr(),
                                          s2.data_ptr(), at))
    assert torch.equal(n2[:10], n) and torch.equal(c2[:10], packed.codes)
    assert torch.equal(s2[:10], packed.scales)
    assert all(bool((t[10:] == 7).all()) for t in (n2, c2, s2))
    want = bd.checkpoint_backward(p.dr, p.dn, packed, **p.kw)
    nw = L.flash_gau_checkpoint_backward_workspace_bytes(10, 256)
    for name in ("dnorm_g", "dnorm_b", None):
        ws = torch.full((nw // 4,), float("nan"), device="cuda")
        dh = torch.full((12, 256), 7.0, dtype=p.io, device="cuda")
        g = bd.ResidualGrads(dh=dh.data_ptr())
        t = torch.full((256,), 7.0, device="cuda")
        if name:
            setattr(g, name, t.data_ptr())
        bd._check(L.flash_gau_checkpoint_backward(
            p.dr.data_ptr(), p.dn.data_ptr(), packed.codes.data_ptr(), packed.scales.data_ptr(),
            ctypes.byref(o), 10, 256, bd.BF16, ctypes.byref(g), ws.data_ptr(), nw, at))
        torch.cuda.synchronize()
        assert torch.equal(dh[:10], want["dh"]) and bool((dh[10:] == 7).all())
        assert torch.equal(t, want[name]) if name else bool((t == 7).all())


def test_binding_refuses():
    p = Problem(4, 256, "bf16", "layer", 2)
    packed = bd.checkpoint_pack(p.h)[0]
    bad = [lambda: bd.checkpoint_pack(p.h, p.y[:3]), lambda: bd.checkpoint_pack(p.h, p.y.float()),
           lambda: bd.checkpoint_pack(p.h, out=bd.Checkpoint(packed.codes, packed.scales[:, :1])),
           lambda: bd.checkpoint_pack(p.h, out=bd.Checkpoint(packed.codes.view(torch.uint8),
                                                             packed.scales)),
           lambda: bd.checkpoint_pack(p.h.t()), lambda: bd.checkpoint_restore((packed.codes, None),
                                                                              p.io),
           lambda: bd.checkpoint_pack(p.h, norm=bd.NORM_LAYER, norm_g=p.kw["norm_g"][:5]),
           lambda: bd.checkpoint_backward(p.dr, p.dn, packed, out=dict(dy=p.dr), **p.kw),
           lambda: bd.checkpoint_backward(p.dr, p.dn, packed, norm=bd.NORM_SCALE,
                                          norm_g=p.kw["norm_g"][:1],
                                          out=dict(dnorm_b=p.kw["norm_b"])),
           lambda: bd.checkpoint_backward(p.dr.float(), p.dn, packed, **p.kw)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: bd.checkpoint_pack(p.h, norm=bd.NORM_LAYER),
              lambda: bd.checkpoint_restore(packed, p.io, want_x=False),
              lambda: bd.checkpoint_backward(p.dr, p.dn, packed, norm=bd.NORM_NONE),
              lambda: bd.checkpoint_pack(p.h[:0])):
        with pytest.raises(bd.FlashGauError):
            f()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("norm", ["layer", "scale"])
@pytest.mark.parametrize("M,d", [(1, 64), (50, 256), (50, 255), (700, 1501)])
def test_infinite_sums(M, d, norm, dtype):
    """An infinity of dn makes the parameters' sums it enters infinite, two of
    unlike signs make them no number, and nothing else does."""
    gen = torch.Generator().manual_seed(d)
    h = (torch.rand(M, d, generator=gen) + torch.linspace(-3, 3, d)).to(dtype).cuda()
    dn = torch.randn(M, d, generator=gen).to(dtype).cuda()
    g = torch.ones(d if norm == "layer" else 1, device="cuda")
    packed = bd.checkpoint_pack(h)[0]
    x = oracle.checkpoint_values(*(t.cpu().numpy() for t in packed))
    inf = float("inf")
    m, c = M // 2, d - 1
    for values in ({c: inf}, {c: -inf}, {0: inf}, {0: inf, c: inf}, {0: float("nan")}):
        dirty = dn.clone()
        for k, v in values.items():
            dirty[m, k] = v
        got = bd.checkpoint_backward(None, dirty, packed, norm=KIND[norm], norm_g=g)
        with np.errstate(invalid="ignore"):
            u = oracle.norm_rows(x, norm, f64(g), None, 1e-5)[0]
            terms = f64(dirty) * u
            want = dict(dnorm_g=terms.sum(0) if norm == "layer" else terms.sum().reshape(1),
                        dnorm_b=f64(dirty).sum(0) if norm == "layer" else None)
        for name, w in want.items():
            if w is None:
                assert got[name] is None
                continue
            a = f64(got[name])
            assert np.array_equal(np.isnan(a), np.isnan(w)), (values, name)
            assert np.array_equal(np.where(np.isinf(a), a, 0), np.where(np.isinf(w), w, 0))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("norm", ["none", "layer", "scale"])
@pytest.mark.parametrize("M,d", [(1, 5), (3, 129), (5, 767), (9, 1500), (3, 4099), (4, 256),
                                 (1, 8191), (350, 767), (333, 2041), (2, 1)])
@pytest.mark.parametrize("offset", [16, 17])
def test_nothing_beside_any_output_is_written(M, d, norm, dtype, offset):
    """Every output of the three calls in the middle of a larger buffer, on a
    vector's boundary and one element behind it: what stands before and behind
    is left, and the outputs are those of arrays of their own."""
    gen = torch.Generator().manual_seed(M + d)
    rows = lambda: torch.randn(M, d, generator=gen).to(dtype).cuda()  # noqa: E731
    groups, held = -(-d // 128), []

    def inner(shape, dt=dtype):
        n = int(np.prod(shape))
        flat = torch.full((offset + n + 16,), 7, dtype=dt, device="cuda")
        held.append((flat, n))
        return flat[offset:offset + n].view(shape)

    h, y, dr, dn = rows(), rows(), rows(), rows()
    kw = dict(norm=KIND[norm], norm_g=None, norm_b=None)
    if norm == "layer":
        kw.update(norm_g=torch.randn(d, generator=gen).cuda(),
                  norm_b=torch.randn(d, generator=gen).cuda())
    elif norm == "scale":
        kw.update(norm_g=torch.ones(1, device="cuda"))
    packed, r, n = bd.checkpoint_pack(h, y, **kw)
    x, xn = bd.checkpoint_restore(packed, dtype, **kw)
    want = [packed.codes, packed.scales, r, n, x, xn]
    out = bd.Checkpoint(inner((M, d), torch.int8), inner((M, groups), torch.float32))
    a, b = inner((M, d)), None if norm == "none" else inner((M, d))
    bd.checkpoint_pack(h, y, out=out, out_r=a, out_n=b, **kw)
    e, f = inner((M, d)), None if norm == "none" else inner((M, d))
    bd.checkpoint_restore(packed, dtype, out_x=e, out_n=f, **kw)
    got = [out.codes, out.scales, a, b, e, f]
    if norm != "none":
        grads = bd.checkpoint_backward(dr, dn, packed, **kw)
        to = dict(dh=inner((M, d)), dnorm_g=inner(kw["norm_g"].shape, torch.float32))
        if norm == "layer":
            to["dnorm_b"] = inner((d,), torch.float32)
        bd.checkpoint_backward(dr, dn, packed, out=to, **kw)
        # element by element the sums are added up in another order
        exact = [("dh", dtype)] if offset == 16 else []
        want += [grads[k] for k, _ in exact]
        got += [to[k] for k, _ in exact]
        for k, t in to.items():
            torch.testing.assert_close(t, grads[k], rtol=1e-2, atol=1e-2)
    torch.cuda.synchronize()
    for flat, size in held:
        assert bool((flat[:offset] == 7).all()) and bool((flat[offset + size:] == 7).all())
    for k, (p, q) in enumerate(zip(got, want)):
        if p is not None and (offset == 16 or k in (0, 1, 2, 4)):
            assert torch.equal(p, q), k


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_whose_statistics_fp32_does_not_hold(dtype):
    """A hundred values of 3e38 add up to infinity in fp32, which is the norm's
    word for a row above 1e19 in length: no number of a LayerNorm, as of the
    residual stream's, zero of a ScaleNorm, and the rows beside it as ever."""
    h = torch.zeros(3, 300)
    h[1, ::3] = 3e38
    h[::2] = torch.randn(2, 300, generator=torch.Generator().manual_seed(6))
    h = h.to(dtype).cuda()
    packed = bd.checkpoint_pack(h)[0]
    for kind, g in (("layer", torch.ones(300)), ("scale", torch.ones(1))):
        kw = dict(norm=KIND[kind], norm_g=g.cuda())
        x, n = bd.checkpoint_restore(packed, dtype, **kw)
        other = bd.residual_norm(x, **kw)[1]
        for t in (n, other):
            assert bool((torch.isnan(t[1]) if kind == "layer" else t[1] == 0).all())
            assert bool(torch.isfinite(t[::2]).all())
