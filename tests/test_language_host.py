"""Host-side checks of the operators of a language model on the layer: the
oracle against other statements of the same definitions, and the refusals of
the C ABI and the binding, all of which come before anything touches a device."""

import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
from efficient_attention_transformer_gb300 import binding as bd
from efficient_attention_transformer_gb300 import build as buildmod

EPS = 1e-5


@pytest.fixture(scope="module")
def L():
    buildmod.build()
    return bd.lib()


# ---- the oracle: buckets -------------------------------------------------------
@pytest.mark.parametrize("C,buckets,far,causal", [
    (300, 32, 128, True), (300, 32, 128, False), (64, 8, 20, False), (512, 33, 200, True),
    (10, 2, 2, True), (40, 4, 3, False), (100, 64, 4096, False), (435 + 5, 42, 1006, False)])
def test_oracle_buckets_against_logarithms(C, buckets, far, causal):
    """The formula in floating point, wherever it is not next to a border."""
    got = oracle.buckets_of_offsets(C, buckets, far, causal)
    n = buckets if causal else buckets // 2
    near = n // 2
    for o in range(-(C - 1), C):
        t = max(-o, 0) if causal else abs(o)
        b = n if o > 0 and not causal else 0
        if t < near:
            assert got[o + C - 1] == b + t
            continue
        x = math.log(t / near) / math.log(far / near) * (n - near)
        if abs(x - round(x)) > 1e-9:
            assert got[o + C - 1] == b + min(n - 1, near + int(x)), o


def test_oracle_buckets_on_borders():
    """n = 32, near 16, far 256: borders at 16 * 2^(j / 4), whole at j = 4, 8,
    12, whose distances open their bucket."""
    b = oracle.buckets_of_offsets(400, 32, 256, True)[::-1][399:]
    assert [b[t] for t in (15, 16, 31, 32, 63, 64, 127, 128, 255, 256, 399)] == [
        15, 16, 19, 20, 23, 24, 27, 28, 31, 31, 31]


def test_oracle_bucket_gradient_is_the_transpose():
    rng = np.random.default_rng(0)
    table, d = rng.normal(size=(3, 12)), rng.normal(size=(2, 3, 41))
    for causal in (True, False):
        a = (oracle.bucket_bias(table, 21, 30, causal) * d.sum(0)).sum()
        b = (table * oracle.bucket_bias_grad(d, 12, 30, causal)).sum()
        assert abs(a - b) <= 1e-12 * abs(a) + 1e-12
    # as differences give it
    step = np.zeros_like(table)
    step[1, 3] = 1.0
    g = oracle.bucket_bias_grad(d, 12, 30, False)
    diff = ((oracle.bucket_bias(table + step, 21, 30, False) -
             oracle.bucket_bias(table, 21, 30, False)) * d.sum(0)).sum()
    assert abs(diff - g[1, 3]) <= 1e-12 * (1 + abs(diff))


# ---- the oracle: checkpoints -----------------------------------------------------
def test_oracle_codes_are_nearest():
    rng = np.random.default_rng(1)
    x = (rng.normal(size=(6, 300)) * np.exp(rng.normal(size=(6, 1)) * 5)).astype(np.float32)
    c, s = oracle.checkpoint_codes(x)
    per = np.repeat(s, 128, axis=1)[:, :300].astype(np.float64)
    assert np.all(np.abs(x - c * per) <= 0.5 * per * (1 + 1e-6))
    for k, g in enumerate((slice(0, 128), slice(128, 256), slice(256, 300))):
        assert np.all(np.abs(c[:, g]).max(axis=1) == 127)
        assert np.array_equal(s[:, k], np.abs(x[:, g]).max(axis=1) * np.float32(1 / 127))


def test_oracle_codes_special_values():
    x = np.zeros((5, 130), np.float32)
    x[1, 3] = np.inf
    x[2, 129] = np.nan
    x[3, 0] = 2.0 ** -101
    # a scale of one: quotients of n + 1/2 go to the even neighbour
    x[4, :4] = [127.0, 0.5, 1.5, -2.5]
    c, s = oracle.checkpoint_codes(x)
    v = oracle.checkpoint_values(c, s)
    assert not v[0].any() and not v[3].any() and s[3, 0] == 0
    assert np.isnan(v[1, :128]).all() and not v[1, 128:].any()
    assert np.isnan(v[2, 128:]).all() and not v[2, :128].any()
    assert list(c[4, :4]) == [127, 0, 2, -2]


# ---- the oracle: sampling ---------------------------------------------------------
def _by_probabilities(l, u, T, k, p, m):
    """The same through probabilities that are renormalised after each filter."""
    l = np.asarray(l, float)
    order = np.argsort(-l, kind="stable")
    q = np.exp((l[order] - l.max()) / T)
    q /= q.sum()
    if k > 0:
        q[k:] = 0
        q /= q.sum()
    keep = q > 0
    if p < 1:
        keep &= np.concatenate([[True], np.cumsum(q)[:-1] < p])
    if m > 0:
        keep &= (q >= m * q.max()) | (np.arange(len(q)) == 0)
    q = np.where(keep, q, 0)
    q /= q.sum()
    j = int(np.searchsorted(np.cumsum(q), u, side="right"))
    return int(order[j]), math.log(q[j]), int(keep.sum())


def test_oracle_sampling_against_probabilities():
    rng = np.random.default_rng(2)
    for _ in range(300):
        V = int(rng.integers(1, 60))
        l = np.round(rng.normal(size=V) * 3, 1)  # with ties
        args = (rng.random(), rng.uniform(0.3, 2), int(rng.integers(0, V + 3)),
                rng.choice([1.0, rng.uniform(0.01, 1)]), rng.choice([0.0, rng.uniform(0, 0.5)]))
        a, b = oracle.sample_row(l, *args), _by_probabilities(l, *args)
        assert a[0] == b[0] and a[2] == b[2] and abs(a[1] - b[1]) < 1e-9


def test_oracle_sampling_follows_the_distribution():
    """Even steps of u meet each word as often as its probability says."""
    l = np.array([0.3, -1.0, 2.0, 0.3])
    n = 20000
    got = np.bincount([oracle.sample_row(l, (i + 0.5) / n, 0.7)[0] for i in range(n)], minlength=4)
    p = np.exp(l / 0.7)
    assert np.all(np.abs(got / n - p / p.sum()) <= 1.0 / n + 1e-12)


def test_oracle_sampling_special_rows():
    inf, nan = np.inf, np.nan
    assert oracle.sample_row([-inf, -inf], 0.5)[0] == -1
    assert oracle.sample_row([1.0, nan], 0.5)[0] == -1
    assert oracle.sample_row([1.0, inf], 0.5)[0] == -1
    assert oracle.sample_row([1.0, 2.0], -0.1)[0] == -1
    assert oracle.sample_row([1.0, 2.0], 0.1, temperature=-1.0)[0] == -1
    assert oracle.sample_row([-inf, 1.0, 1.0], 0.9, temperature=0.0) == (1, 0.0, 1)
    assert oracle.sample_row([-inf, 1.0, 1.0], 0.9)[0] == 2
    assert oracle.sample_row([3.0, 1.0], 0.99, top_p=0.0) == (0, 0.0, 1)
    assert oracle.sample_row([1.0, 1.0, 1.0, 1.0], 0.0, top_p=0.5)[2] == 2


def test_oracle_min_p_above_one_keeps_the_first_word():
    """No word's share reaches it, those that tie with the largest neither."""
    for m in (1.0000001, 2.0, np.inf):
        assert oracle.sample_row([1.0, 1.0, 0.0], 0.9, min_p=m) == (0, 0.0, 1)
    assert oracle.sample_row([1.0, 1.0, 0.0], 0.9, min_p=1.0)[::2] == (1, 2)


# ---- refusals of the C ABI -----------------------------------------------------
A, B, C, D, E_, F_ = (1 << 32, 2 << 32, 3 << 32, 4 << 32, 5 << 32, 6 << 32)  # fake arrays


@pytest.mark.parametrize("args,code", [
    (dict(table=None), bd.EINVAL),
    (dict(relpos=None), bd.EINVAL),
    (dict(H=0), bd.EINVAL),
    (dict(H=65536), bd.EINVAL),
    (dict(C=0), bd.EINVAL),
    (dict(C=4097), bd.EINVAL),
    (dict(buckets=1), bd.EINVAL),
    (dict(buckets=257), bd.EINVAL),
    (dict(buckets=258, causal=0), bd.EINVAL),
    (dict(buckets=2, causal=0), bd.EINVAL),
    (dict(buckets=33, causal=0), bd.EINVAL),
    (dict(far=16), bd.EINVAL),                 # near is 16
    (dict(far=8, causal=0), bd.EINVAL),
    (dict(far=(1 << 20) + 1), bd.EINVAL),
    (dict(table=A + 2), bd.EINVAL),
    (dict(relpos=B + 1), bd.EINVAL),
    (dict(relpos=A + 64), bd.EINVAL),          # overlaps the table
    (dict(R=0), bd.EINVAL),
])
def test_bucket_bias_refuses(L, args, code):
    a = dict(table=A, relpos=B, H=2, buckets=32, far=128, C=64, causal=1, R=1)
    a.update(args)
    if a["R"] > 0:
        assert L.flash_gau_bucket_bias(a["table"], a["H"], a["buckets"], a["far"], a["C"],
                                       a["causal"], a["relpos"], None) == code
    assert L.flash_gau_bucket_bias_backward(a["relpos"], a["R"], a["H"], a["buckets"], a["far"],
                                            a["C"], a["causal"], a["table"], None) == code


@pytest.mark.parametrize("R", [(1 << 20) + 1, (1 << 31) - 8, (1 << 31) - 1])
def test_bucket_bias_backward_refuses_more_tables_than_it_sums(L, R):
    assert L.flash_gau_bucket_bias_backward(B, R, 1, 32, 128, 1, 1, A, None) == bd.EINVAL


def _norm(**kw):
    o = dict(post=bd.NORM_NONE, norm=bd.NORM_LAYER, post_g=None, post_b=None, norm_g=64,
             norm_b=None, scale=None, gate=None, eps=EPS)
    o.update(kw)
    return bd.Residual(*(o[k] for k, _ in bd.Residual._fields_))


# what all three calls refuse of the options and sizes
COMMON = [
    (dict(), dict(M=0), bd.EINVAL),
    (dict(), dict(d=0), bd.EINVAL),
    (dict(), dict(d=8193), bd.ENOTSUP),
    (dict(), dict(M=(1 << 32) + 1), bd.ENOTSUP),
    (dict(), dict(dtype=2), bd.EINVAL),
    (dict(norm=3), dict(), bd.EINVAL),
    (dict(norm=-1), dict(), bd.EINVAL),
    (dict(norm_g=None), dict(), bd.EINVAL),
    (dict(norm_g=66), dict(), bd.EINVAL),
    (dict(eps=0.0), dict(), bd.EINVAL),
    (dict(eps=float("inf")), dict(), bd.EINVAL),
    (dict(eps=1e-40), dict(), bd.EINVAL),
    (dict(post=bd.NORM_SCALE, post_g=64), dict(), bd.EINVAL),
    (dict(post_g=64), dict(), bd.EINVAL),
    (dict(post_b=64), dict(), bd.EINVAL),
    (dict(scale=64), dict(), bd.EINVAL),
    (dict(gate=F_), dict(), bd.EINVAL),
    (dict(), dict(codes=None), bd.EINVAL),
    (dict(), dict(scales=None), bd.EINVAL),
    (dict(), dict(scales=F_ + 2), bd.EINVAL),
]


@pytest.mark.parametrize("opts,args,code", COMMON + [
    (dict(), dict(h=None), bd.EINVAL),
    (dict(), dict(n=None), bd.EINVAL),                   # a norm and no place for it
    (dict(norm=bd.NORM_NONE), dict(), bd.EINVAL),        # a place and no norm
    (dict(), dict(r=A + 4), bd.EINVAL),                  # overlaps h
    (dict(), dict(n=C), bd.EINVAL),                      # n is r
    (dict(), dict(h=A + 1), bd.EINVAL),
    (dict(), dict(n=D + 1), bd.EINVAL),
    (dict(), dict(codes=A + 64), bd.EINVAL),             # inside h
    (dict(), dict(codes=C + 64), bd.EINVAL),             # inside r
    (dict(), dict(scales=E_ + 64), bd.EINVAL),           # inside the codes
    (dict(norm_g=C + 8), dict(), bd.EINVAL),
    (dict(norm_g=E_ + 8), dict(), bd.EINVAL),
    (dict(norm_b=F_ + 8), dict(), bd.EINVAL),
])
def test_checkpoint_pack_refuses(L, opts, args, code):
    a = dict(h=A, y=B, M=10, d=64, dtype=bd.BF16, r=C, n=D, codes=E_, scales=F_)
    a.update(args)
    o = _norm(**opts)
    assert L.flash_gau_checkpoint_pack(a["h"], a["y"], ctypes.byref(o), a["M"], a["d"], a["dtype"],
                                       a["r"], a["n"], a["codes"], a["scales"], None) == code
    assert L.flash_gau_checkpoint_pack(a["h"], a["y"], None, a["M"], a["d"], a["dtype"], a["r"],
                                       a["n"], a["codes"], a["scales"], None) == bd.EINVAL


@pytest.mark.parametrize("opts,args,code", COMMON + [
    (dict(), dict(n=None), bd.EINVAL),
    (dict(norm=bd.NORM_NONE), dict(), bd.EINVAL),
    (dict(norm=bd.NORM_NONE), dict(n=None, x=None), bd.EINVAL),
    (dict(), dict(x=C + 1), bd.EINVAL),
    (dict(), dict(n=C + 2), bd.EINVAL),
    (dict(), dict(x=E_), bd.EINVAL),
    (dict(), dict(n=F_), bd.EINVAL),
    (dict(norm_g=D), dict(), bd.EINVAL),
])
def test_checkpoint_restore_refuses(L, opts, args, code):
    a = dict(M=10, d=64, dtype=bd.BF16, x=C, n=D, codes=E_, scales=F_)
    a.update(args)
    o = _norm(**opts)
    assert L.flash_gau_checkpoint_restore(a["codes"], a["scales"], ctypes.byref(o), a["M"], a["d"],
                                          a["dtype"], a["x"], a["n"], None) == code


@pytest.mark.parametrize("opts,args,code", COMMON + [
    (dict(norm=bd.NORM_NONE), dict(), bd.EINVAL),
    (dict(), dict(dn=None), bd.EINVAL),
    (dict(), dict(dh=None), bd.EINVAL),
    (dict(), dict(ws=None), bd.EINVAL),
    (dict(), dict(dy=F_ + (1 << 20)), bd.EINVAL),
    (dict(), dict(dscale=F_ + (1 << 20)), bd.EINVAL),
    (dict(norm=bd.NORM_SCALE), dict(dnorm_b=7 << 32), bd.EINVAL),
    (dict(), dict(dh=A + 2), bd.EINVAL),                 # overlaps dr
    (dict(), dict(dh=E_), bd.EINVAL),
    (dict(), dict(dnorm_g=64), bd.EINVAL),               # the parameter itself
    (dict(), dict(dnorm_g=A + 64), bd.EINVAL),
    (dict(), dict(dnorm_g=7 << 32, dnorm_b=7 << 32), bd.EINVAL),
    (dict(), dict(ws=1 << 40 | 8), bd.EWORKSPACE),
    (dict(), dict(wsb=100), bd.EWORKSPACE),
    (dict(), dict(ws=A), bd.EINVAL),
    (dict(), dict(ws=C), bd.EINVAL),
])
def test_checkpoint_backward_refuses(L, opts, args, code):
    a = dict(dr=A, dn=B, M=10, d=64, dtype=bd.BF16, dh=C, codes=E_, scales=F_, ws=1 << 40,
             wsb=1 << 30, dy=None, dgate=None, dscale=None, dpost_g=None, dpost_b=None,
             dnorm_g=None, dnorm_b=None)
    a.update(args)
    o = _norm(**opts)
    g = bd.ResidualGrads(*(a[k] for k, _ in bd.ResidualGrads._fields_))
    assert L.flash_gau_checkpoint_backward(a["dr"], a["dn"], a["codes"], a["scales"],
                                           ctypes.byref(o), a["M"], a["d"], a["dtype"],
                                           ctypes.byref(g), a["ws"], a["wsb"], None) == code
    assert L.flash_gau_checkpoint_backward(a["dr"], a["dn"], a["codes"], a["scales"],
                                           ctypes.byref(o), a["M"], a["d"], a["dtype"], None,
                                           a["ws"], a["wsb"], None) != bd.OK


def test_checkpoint_workspace_bytes(L):
    f = L.flash_gau_checkpoint_backward_workspace_bytes
    assert f(0, 64) == f(5, 0) == f(5, 8193) == f((1 << 32) + 1, 64) == 0
    assert f(1, 1) > 0 and f(1 << 32, 8192) % 256 == 0


@pytest.mark.parametrize("args,code", [
    (dict(logits=None), bd.EINVAL),
    (dict(u=None), bd.EINVAL),
    (dict(token=None), bd.EINVAL),
    (dict(N=0), bd.EINVAL),
    (dict(V=0), bd.EINVAL),
    (dict(ld=99), bd.EINVAL),
    (dict(dtype=5), bd.EINVAL),
    (dict(V=(1 << 22) + 1, ld=1 << 23), bd.ENOTSUP),
    (dict(N=(1 << 30) + 1), bd.ENOTSUP),
    (dict(ld=(1 << 32) + 1), bd.ENOTSUP),
    (dict(logits=A + 1), bd.EINVAL),
    (dict(u=B + 2), bd.EINVAL),
    (dict(temperature=F_ + 1), bd.EINVAL),
    (dict(kept=E_ + 3), bd.EINVAL),
    (dict(token=A + 4 * 100), bd.EINVAL),       # inside the logits
    (dict(logp=C), bd.EINVAL),                  # the tokens' place
    (dict(kept=B), bd.EINVAL),                  # u's place
    (dict(top_k=C), bd.EINVAL),
])
def test_sample_refuses(L, args, code):
    a = dict(logits=A, ld=100, N=4, V=100, dtype=bd.BF16, u=B, temperature=None, top_k=None,
             top_p=None, min_p=None, token=C, logp=D, kept=E_)
    a.update(args)
    s = bd.Sampling(a["temperature"], a["top_k"], a["top_p"], a["min_p"])
    rest = (a["token"], a["logp"], a["kept"], None)
    assert L.flash_gau_sample(a["logits"], a["ld"], a["N"], a["V"], a["dtype"], a["u"],
                              ctypes.byref(s), *rest) == code
    assert L.flash_gau_sample(a["logits"], a["ld"], a["N"], a["V"], a["dtype"], a["u"], None,
                              *rest) == bd.EINVAL


# ---- refusals of the binding ------------------------------------------------------
def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 128)
    packed = bd.Checkpoint.empty((4, 128), "cpu")
    assert packed.codes.shape == (4, 128) and packed.scales.shape == (4, 1)
    for f in (lambda: bd.bucket_bias(x, 8, True), lambda: bd.bucket_bias_backward(x, 8, True),
              lambda: bd.checkpoint_pack(x), lambda: bd.checkpoint_restore(packed, torch.float32),
              lambda: bd.checkpoint_backward(x, x, packed), lambda: bd.sample(x, x[:, 0])):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        bd.sample(x.double(), x[:, 0])
    with pytest.raises(TypeError):
        bd.checkpoint_pack(x.half())
    with pytest.raises(ValueError):
        bd.sample(x, x[:3, 0])
    assert bd.Checkpoint.empty((3, 129), "cpu").scales.shape == (3, 2)
