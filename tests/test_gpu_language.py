"""The operators of a language model on the layer together, as they are used: a
stack of two causal layers that share one table of values by buckets is
trained for a step with its residual stream kept in 8 bits, then decoded and
sampled.  The float64 oracles' chain takes the same restored streams in its
backward pass, so what is left between the two is rounding: the bounds are
those of the training step's test (ten times the layer's own fp32 bar, five
times its bf16 one, of a result's maximum)."""

import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import oracle
from efficient_attention_transformer_gb300 import binding as bd
from efficient_attention_transformer_gb300.synthetic import make_inputs

pytestmark = pytest.mark.gpu

TOL = {"fp32": 1e-3, "bf16": 1e-1}
SHAPES = {"fp32": dict(B=2, T=128, d=64, e=128, s=32, C=64),
          "bf16": dict(B=2, T=256, d=128, e=256, s=128, C=128)}
LAYERS, V, BUCKETS, FAR, LR = 2, 500, 16, 48, 1e-2


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from efficient_attention_transformer_gb300.build import build
    build()


def f64(t):
    return t.double().cpu().numpy()


class Model:
    def __init__(self, dtype):
        self.S, self.io = SHAPES[dtype], torch.float32 if dtype == "fp32" else torch.bfloat16
        S, f32 = self.S, torch.float32
        rng = np.random.default_rng(7)
        dev = lambda a, dt=f32: torch.tensor(np.asarray(a), dtype=dt, device="cuda")  # noqa: E731
        self.table = dev(rng.normal(0, 0.2, (1, BUCKETS)))
        self.relpos = torch.empty(1, 2 * S["C"] - 1, device="cuda")
        self.layers, self.norms = [], []
        for k in range(LAYERS):
            i = make_inputs(S["B"], S["T"], S["d"], S["e"], S["s"], S["C"], dtype, seed=k)
            W = np.concatenate([i["W_u"], i["W_v"], i["W_z"]], axis=1)
            self.layers.append(bd.GauWeights(
                dev(W, self.io), dev(i["W_o"], self.io), dev(i["gamma"]), dev(i["beta"]),
                self.relpos[0], S["d"], S["e"], S["s"], 1.0 / S["C"]))
        for k in range(LAYERS + 1):
            self.norms.append(dict(norm=bd.NORM_LAYER, norm_g=dev(rng.normal(1, 0.1, S["d"])),
                                   norm_b=dev(rng.normal(0, 0.1, S["d"]))))
        self.head = dev(rng.normal(0, S["d"] ** -0.5, (V, S["d"])), self.io)

    def fill(self):
        bd.bucket_bias(self.table, self.S["C"], True, max_distance=FAR, out=self.relpos)

    def step(self, h, labels):
        """Gradients of the table, of the norms and of h; the packed streams."""
        S = self.S
        self.fill()
        packed = []
        p, r, n = bd.checkpoint_pack(h, **self.norms[0])
        packed.append(p)
        for k, w in enumerate(self.layers):
            p, r, n = bd.checkpoint_pack(r, bd.forward(n, w, S["C"], True), **self.norms[k + 1])
            packed.append(p)
        loss = bd.xent(n, self.head, labels)
        dr, dn, norms, rel = None, loss["dX"], [], []
        for k in range(LAYERS, -1, -1):
            g = bd.checkpoint_backward(dr, dn, packed[k], **self.norms[k])
            norms.append((g["dnorm_g"], g["dnorm_b"]))
            dr = g["dh"]
            if k:
                x = bd.checkpoint_restore(packed[k - 1], self.io, want_x=False,
                                          **self.norms[k - 1])[1]
                lg = bd.backward(x, dr, self.layers[k - 1], S["C"], True)
                rel.append(lg["drelpos"])
                dn = lg["dX"]
        dtable = bd.bucket_bias_backward(torch.stack(rel)[:, None], BUCKETS, True, max_distance=FAR)
        return dict(loss=loss["total"], dh=dr, dtable=dtable, norms=norms[::-1], packed=packed)

    def reference(self, h, labels, packed):
        S = self.S
        shape, d, e = (S["B"], S["T"], S["d"]), S["d"], S["e"]
        rel = oracle.bucket_bias(f64(self.table), S["C"], FAR, True)[0]
        layer = []
        for w in self.layers:
            W = f64(w.W_uvz)
            layer.append(dict(W_u=W[:, :e], W_v=W[:, e:2 * e], W_z=W[:, 2 * e:], W_o=f64(w.W_o),
                              gamma=f64(w.gamma), beta=f64(w.beta), relpos=rel, C=S["C"],
                              causal=True, lin_scale=1.0 / S["C"]))
        par = [(f64(n["norm_g"]), f64(n["norm_b"])) for n in self.norms]
        r = f64(h).reshape(-1, d)
        n = oracle.norm_rows(r, "layer", *par[0], 1e-5)[2]
        for k in range(LAYERS):
            y, _ = oracle.flash_gau(n.reshape(shape), **layer[k])
            r = r + y.reshape(-1, d)
            n = oracle.norm_rows(r, "layer", *par[k + 1], 1e-5)[2]
        loss = oracle.xent(n, f64(self.head), labels.cpu().numpy().reshape(-1))
        xs = [oracle.checkpoint_values(p.codes.cpu().numpy().reshape(-1, d),
                                       p.scales.cpu().numpy().reshape(S["B"] * S["T"], -1))
              for p in packed]
        dr, dn, norms, drel = None, loss["dX"], [], []
        for k in range(LAYERS, -1, -1):
            g = oracle.residual_norm_grad(dr, dn, xs[k], None, "none", None, None, None, None,
                                          "layer", *par[k], 1e-5)
            norms.append((g["dnorm_g"], g["dnorm_b"]))
            dr = g["dh"]
            if k:
                x = oracle.norm_rows(xs[k - 1], "layer", *par[k - 1], 1e-5)[2]
                lg = oracle.flash_gau_backward(x.reshape(shape), dO=dr.reshape(shape),
                                               **layer[k - 1])
                drel.append(lg["drelpos"])
                dn = lg["dX"].reshape(-1, d)
        dtable = oracle.bucket_bias_grad(np.stack(drel)[:, None], BUCKETS, FAR, True)
        return dict(loss=loss["total"], dh=dr, dtable=dtable, norms=norms[::-1])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_training_step_then_decoding(dtype):
    m = Model(dtype)
    S, g = m.S, torch.Generator().manual_seed(3)
    h = torch.randn((S["B"], S["T"], S["d"]), generator=g).to(m.io).cuda()
    labels = torch.randint(-20, V, (S["B"], S["T"]), generator=g, dtype=torch.int32).cuda()
    got = m.step(h, labels)
    torch.cuda.synchronize()
    want = m.reference(h, labels, got["packed"])
    assert abs(float(got["loss"]) - want["loss"]) <= TOL[dtype] * abs(want["loss"])
    pairs = [("dh", got["dh"], want["dh"]), ("dtable", got["dtable"], want["dtable"])]
    for k, (a, b) in enumerate(zip(got["norms"], want["norms"])):
        pairs += [("norm_g%d" % k, a[0], b[0]), ("norm_b%d" % k, a[1], b[1])]
    for name, a, b in pairs:
        err = np.abs(f64(a).reshape(b.shape) - b).max() / np.abs(b).max()
        assert err <= TOL[dtype], (name, err)
    # the table's step, and the new table in every layer at once
    before = f64(m.table)
    bd.AdamW([m.table]).step([got["dtable"]], lr=LR)
    assert np.abs(f64(m.table) - before).max() > 0.5 * LR
    m.fill()
    at = oracle.buckets_of_offsets(S["C"], BUCKETS, FAR, True)
    assert np.array_equal(f64(m.relpos)[0], f64(m.table)[0][at])
    # decode with it: each token's logits sampled, the draw embedded as the next
    decoders = [bd.Decoder(w, S["B"], S["C"]) for w in m.layers]
    x = h[:, 0].contiguous()
    for t in range(S["C"] + 3):
        r, n = bd.residual_norm(x, None, **m.norms[0])
        for k, dec in enumerate(decoders):
            r, n = bd.residual_norm(r, dec.step(n), **m.norms[k + 1])
        logits = n @ m.head.t()
        u = torch.rand(S["B"], generator=g).cuda()
        token, logp, kept = bd.sample(logits, u, temperature=0.8, top_k=50, top_p=0.9)
        l = f64(logits)
        for i in range(S["B"]):
            ref = oracle.sample_row(l[i], float(u[i]), float(np.float32(0.8)), 50,
                                    float(np.float32(0.9)))
            assert (int(token[i]), int(kept[i])) == (ref[0], ref[2]), t
        x = m.head[token.long()].contiguous()


FIRST = """
import torch
from efficient_attention_transformer_gb300 import binding as bd
torch.manual_seed(0)
h, y, dr, dn = (torch.randn(40, 5000, device="cuda") for _ in range(4))
g = torch.ones(5000, device="cuda")
table, drel = torch.randn(3, 16, device="cuda"), torch.randn(2, 3, 511, device="cuda")
logits, u = torch.randn(9, 5000, device="cuda"), torch.rand(9, device="cuda")

def step():
    packed, r, n = bd.checkpoint_pack(h, y, norm=bd.NORM_LAYER, norm_g=g)
    x, xn = bd.checkpoint_restore(packed, h.dtype, norm=bd.NORM_LAYER, norm_g=g)
    back = bd.checkpoint_backward(dr, dn, packed, norm_g=g)
    return [*packed, r, n, x, xn, back["dh"], back["dnorm_g"], back["dnorm_b"],
            bd.bucket_bias(table, 256, True), bd.bucket_bias_backward(drel, 16, True),
            *bd.sample(logits, u, temperature=0.9, top_p=0.9)]

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
want = step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want))
print("same")
"""


def test_first_calls_captured():
    r = subprocess.run([sys.executable, "-c", FIRST], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_streams_and_threads_at_once(dtype):
    """Four threads, a stream each, all operators over and over: the results
    are those of one call at a time."""
    torch.manual_seed(1)
    jobs = []
    for k in range(4):
        N, d = 100 + 70 * k, 128 + 601 * k
        h, y = (torch.randn(N, d, device="cuda").to(dtype) for _ in range(2))
        jobs.append((h, y, torch.rand(d, device="cuda") + 0.5, torch.rand(N, device="cuda"),
                     torch.randn(2 + k, 16, device="cuda")))

    def once(job):
        h, y, g, u, table = job
        packed, r, n = bd.checkpoint_pack(h, y, norm=bd.NORM_LAYER, norm_g=g)
        x, xn = bd.checkpoint_restore(packed, dtype, norm=bd.NORM_LAYER, norm_g=g)
        back = bd.checkpoint_backward(n, h, packed, norm_g=g)
        rel = bd.bucket_bias(table, 100, False)
        return [*packed, r, n, x, xn, back["dh"], back["dnorm_g"], rel,
                bd.bucket_bias_backward(rel, 16, False), *bd.sample(r, u, top_p=0.8)]

    want = [once(j) for j in jobs]
    torch.cuda.synchronize()
    wrong = []

    def work(k):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(10):
                got = once(jobs[k])
                s.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[k])):
                    wrong.append(k)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_whole_numbers_that_the_library_does_not_take():
    """Refused, not taken without their upper 32 bits: sizes as arguments, and
    those of tensors of that many elements."""
    more = 1 << 32
    t, d = torch.randn(3, 32, device="cuda"), torch.randn(1, 3, 39, device="cuda")
    h = torch.zeros(4, 64, device="cuda")
    g = torch.ones(1, device="cuda")
    packed = bd.checkpoint_pack(h)[0]
    long = torch.empty(1, more + 128, dtype=torch.bfloat16, device="cuda")
    bytes_ = long.view(torch.int8)[:, :more + 128]
    many = torch.empty(more + 1, 1, 1, device="cuda")
    u = torch.rand(1, device="cuda")
    calls = [lambda: bd.bucket_bias(t, 20, True, max_distance=more + 128),
             lambda: bd.bucket_bias(t, more + 20, True),
             lambda: bd.bucket_bias(t, 20 - more, True),
             lambda: bd.bucket_bias(many.view(1, -1), 20, True),
             lambda: bd.bucket_bias_backward(d, more + 32, True),
             lambda: bd.bucket_bias_backward(d, 32, True, max_distance=more + 128),
             lambda: bd.bucket_bias_backward(many, 32, True),
             lambda: bd.checkpoint_pack(long),
             lambda: bd.checkpoint_pack(h, norm=more + bd.NORM_SCALE, norm_g=g),
             lambda: bd.checkpoint_restore((bytes_, u), torch.float32),
             lambda: bd.checkpoint_backward(None, long, (bytes_, u)),
             lambda: bd.checkpoint_backward(None, h, packed, norm=more + bd.NORM_SCALE, norm_g=g),
             lambda: bd.sample(long, u)]
    for call in calls:
        with pytest.raises(bd.FlashGauError):
            call()


@pytest.mark.parametrize("d", [2048, 2047])
def test_checkpoints_of_more_than_31_bits_of_elements(d):
    """The last rows come out as those of a call of their own."""
    M, last, io = 1_100_000, 16, torch.bfloat16
    gen = torch.Generator(device="cuda").manual_seed(d)
    h = torch.empty(M, d, dtype=io, device="cuda").normal_(generator=gen)
    for kind, g in ((bd.NORM_LAYER, torch.rand(d, generator=gen, device="cuda")),
                    (bd.NORM_SCALE, torch.ones(1, device="cuda"))):
        kw = dict(norm=kind, norm_g=g)
        packed, _, n = bd.checkpoint_pack(h, **kw)
        x, xn = bd.checkpoint_restore(packed, io, **kw)
        dh = bd.checkpoint_backward(x, h, packed, **kw)["dh"]
        few = h[-last:].clone()
        p, _, fn = bd.checkpoint_pack(few, **kw)
        fx, fxn = bd.checkpoint_restore(p, io, **kw)
        want = [p.codes, p.scales, fn, fx, fxn, bd.checkpoint_backward(fx, few, p, **kw)["dh"]]
        got = [packed.codes, packed.scales, n, x, xn, dh]
        assert all(torch.equal(a[-last:], b) for a, b in zip(got, want))
        del packed, n, x, xn, dh, got


def test_logits_of_more_than_31_bits_of_elements():
    N, V = 40_000, 60_001
    gen = torch.Generator(device="cuda").manual_seed(2)
    logits = torch.empty(N, V, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    u = torch.rand(N, generator=gen, device="cuda")
    kw = dict(temperature=0.8, top_k=500, top_p=0.9)
    got = bd.sample(logits, u, **kw)
    want = bd.sample(logits[-9:].clone(), u[-9:].clone(), **kw)
    assert all(torch.equal(a[-9:], b) for a, b in zip(got, want))


def test_bias_gradients_of_more_than_31_bits_of_elements():
    """Whole numbers: an offset's sum, 700000 at most and so below 2^24, is
    exact, and a bucket's where it is below 2^24 too; above, a lane adds up to
    32 offsets, then there are 5 shuffles and 8 blocks, and each addition is off
    by 2^-24 of the bucket's sum at most."""
    R, H, C = 70_000, 10, 1700
    d = torch.empty(R, H, 2 * C - 1, device="cuda")
    d.copy_(torch.arange(1.0, H + 1, device="cuda")[:, None])
    got = bd.bucket_bias_backward(d, 32, False)
    size = np.bincount(oracle.buckets_of_offsets(C, 32, 128, False), minlength=32)
    want = size * R * np.arange(1, H + 1)[:, None]
    err = np.abs(f64(got) - want)
    assert np.all(err <= (32 + 5 + 8) * 2.0 ** -24 * want) and not err[want < 2 ** 24].any()
