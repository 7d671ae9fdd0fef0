"""A training step of a small language model from the library's operators
together: embedded tokens, two GAU layers with the residual stream's norms,
gates and scales between them, the vocabulary's cross entropy, the backward
pass through all of it, and AdamW on every parameter.  Gradients are compared
with the float64 oracles' chain at the same weights, the update with the
oracle's on the same gradients.

The layer's own tests hold it to 1e-4 (fp32 io) and 2e-2 (bf16 io) of an
output's or gradient's maximum.  The chain passes four of them and six
smaller stages one after another, so it gets ten times the fp32 bar and five
times the bf16 one."""

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
V, LAYERS, LR = 500, 2, 1e-3


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from efficient_attention_transformer_gb300.build import build
    build()


def f64(t):
    return t.double().cpu().numpy()


class Model:
    """Weights in the io type (bf16: beside fp32 masters), the rest fp32."""

    def __init__(self, dtype, bits):
        self.dtype, self.S = dtype, SHAPES[dtype]
        S, self.io = self.S, torch.float32 if dtype == "fp32" else torch.bfloat16
        rng = np.random.default_rng(4)
        self.names, self.params, self.copies = [], [], []

        def add(name, a, weight):
            p = torch.tensor(np.asarray(a), dtype=torch.float32, device="cuda")
            if weight and dtype == "bf16":
                p = p.to(self.io).float()
            self.names.append(name)
            self.params.append(p)
            self.copies.append(p.to(self.io) if weight and dtype == "bf16" else None)
            return p if self.copies[-1] is None else self.copies[-1]

        self.layers, self.norms = [], []
        d = S["d"]
        for k in range(LAYERS):
            i = make_inputs(S["B"], S["T"], d, S["e"], S["s"], S["C"], dtype, seed=k)
            W = np.concatenate([i["W_u"], i["W_v"], i["W_z"]], axis=1)
            args = [add("%s%d" % (n, k), a, n in ("W_uvz", "W_o")) for n, a in (
                ("W_uvz", W), ("W_o", i["W_o"]), ("gamma", i["gamma"]), ("beta", i["beta"]),
                ("relpos", i["relpos"]))]
            self.layers.append(bd.GauWeights(*args, d, S["e"], S["s"], 1.0 / S["C"]))
        for k in range(LAYERS + 1):
            n = {"norm_g": add("norm_g%d" % k, rng.normal(1, 0.1, d), False),
                 "norm_b": add("norm_b%d" % k, rng.normal(0, 0.1, d), False)}
            if k:
                n["post_g"] = add("post_g%d" % k, [d ** 0.5], False)
                n["scale"] = add("scale%d" % k, rng.normal(0.5, 0.1, d), False)
            self.norms.append(n)
        self.head = add("head", rng.normal(0, d ** -0.5, (V, d)), True)
        self.opt = bd.AdamW(self.params, copies=self.copies, weight_decay=0.01, state_bits=bits)

    def step(self, h, gates, labels):
        """Gradients by name, the loss, and the gradient of h."""
        S = self.S
        kw = [dict(post_norm=bd.NORM_SCALE if k else bd.NORM_NONE, gate=gates[k - 1] if k else None,
                   **self.norms[k]) for k in range(LAYERS + 1)]
        r, n = bd.residual_norm(h, None, norm_g=kw[0]["norm_g"], norm_b=kw[0]["norm_b"])
        rs, ns, ys = [r], [n], [None]
        for k, w in enumerate(self.layers):
            ys.append(bd.forward(ns[k], w, S["C"], True))
            r, n = bd.residual_norm(rs[k], ys[-1], **kw[k + 1])
            rs.append(r)
            ns.append(n)
        loss = bd.xent(ns[-1], self.head, labels)
        grads, dr, dn, dgates = {"head": loss["dW"]}, None, loss["dX"], []
        for k in range(LAYERS, 0, -1):
            g = bd.residual_norm_backward(dr, dn, rs[k], ys[k], **kw[k])
            for name in self.norms[k]:
                grads["%s%d" % (name, k)] = g["d" + name]
            dgates.append(g["dgate"])
            lg = bd.backward(ns[k - 1], g["dy"], self.layers[k - 1], S["C"], True)
            for name in ("W_uvz", "W_o", "gamma", "beta", "relpos"):
                grads["%s%d" % (name, k - 1)] = lg["d" + name]
            dr, dn = g["dh"], lg["dX"]
        g = bd.residual_norm_backward(dr, dn, rs[0], None, norm_g=kw[0]["norm_g"],
                                      norm_b=kw[0]["norm_b"])
        grads["norm_g0"], grads["norm_b0"] = g["dnorm_g"], g["dnorm_b"]
        return grads, loss["total"], g["dh"], dgates[::-1]

    def reference(self, h, gates, labels):
        S, d = self.S, self.S["d"]
        par = {n: f64(p if c is None else c) for n, p, c in zip(self.names, self.params, self.copies)}
        flat = lambda x: x.reshape(-1, d)  # noqa: E731
        kw = [dict(post="scale" if k else "none", post_g=par.get("post_g%d" % k), post_b=None,
                   gate=flat(f64(gates[k - 1])) if k else None, scale=par.get("scale%d" % k),
                   norm="layer", norm_g=par["norm_g%d" % k], norm_b=par["norm_b%d" % k], eps=1e-5)
              for k in range(LAYERS + 1)]
        e = S["e"]
        layer = [dict(W_u=par["W_uvz%d" % k][:, :e], W_v=par["W_uvz%d" % k][:, e:2 * e],
                      W_z=par["W_uvz%d" % k][:, 2 * e:], W_o=par["W_o%d" % k],
                      gamma=par["gamma%d" % k], beta=par["beta%d" % k], relpos=par["relpos%d" % k],
                      C=S["C"], causal=True, lin_scale=1.0 / S["C"]) for k in range(LAYERS)]
        r, n = oracle.residual_norm(flat(f64(h)), None, **kw[0])
        rs, ns, ys = [r], [n], [None]
        for k in range(LAYERS):
            y, _ = oracle.flash_gau(ns[k].reshape(S["B"], S["T"], d), **layer[k])
            ys.append(flat(y))
            r, n = oracle.residual_norm(rs[k], ys[-1], **kw[k + 1])
            rs.append(r)
            ns.append(n)
        loss = oracle.xent(ns[-1], par["head"], labels.cpu().numpy().reshape(-1))
        grads, dr, dn, dgates = {"head": loss["dW"]}, None, loss["dX"], []
        for k in range(LAYERS, 0, -1):
            g = oracle.residual_norm_grad(dr, dn, rs[k], ys[k], **kw[k])
            for name in self.norms[k]:
                grads["%s%d" % (name, k)] = g["d" + name]
            dgates.append(g["dgate"])
            shape = (S["B"], S["T"], d)
            lg = oracle.flash_gau_backward(ns[k - 1].reshape(shape), dO=g["dy"].reshape(shape),
                                           **layer[k - 1])
            grads["W_uvz%d" % (k - 1)] = np.concatenate([lg["dW_u"], lg["dW_v"], lg["dW_z"]], axis=1)
            for name in ("W_o", "gamma", "beta", "relpos"):
                grads["%s%d" % (name, k - 1)] = lg["d" + name]
            dr, dn = g["dh"], flat(lg["dX"])
        g = oracle.residual_norm_grad(dr, dn, rs[0], None, **kw[0])
        grads["norm_g0"], grads["norm_b0"] = g["dnorm_g"], g["dnorm_b"]
        return grads, loss["total"], g["dh"], dgates[::-1]


@pytest.mark.parametrize("dtype,bits", [("fp32", 32), ("bf16", 32), ("bf16", 8)])
def test_training_steps(dtype, bits):
    m = Model(dtype, bits)
    S, g = m.S, torch.Generator().manual_seed(1)
    shape = (S["B"], S["T"], S["d"])
    for step in (1, 2):
        h = torch.randn(shape, generator=g).to(m.io).cuda()
        gates = [torch.randn(shape, generator=g).to(m.io).cuda() for _ in range(LAYERS)]
        labels = torch.randint(-50, V, shape[:2], generator=g, dtype=torch.int32).cuda()
        grads, total, dh, dgates = m.step(h, gates, labels)
        torch.cuda.synchronize()
        want, wtotal, wdh, wdgates = m.reference(h, gates, labels)
        assert abs(float(total) - wtotal) <= TOL[dtype] * abs(wtotal)
        pairs = [(n, grads[n], want[n]) for n in m.names] + [("h", dh, wdh)]
        pairs += [("gate%d" % k, a, b) for k, (a, b) in enumerate(zip(dgates, wdgates))]
        for name, got, ref in pairs:
            err = np.abs(f64(got).reshape(ref.shape) - ref).max() / np.abs(ref).max()
            assert err <= TOL[dtype], (name, err)
        # the update, from the gradients as they are
        before = [f64(p) for p in m.params]
        mv = [(f64(a), f64(b)) for a, b in zip(*m.opt.moments())]
        m.opt.step([grads[n] for n in m.names], lr=LR)
        torch.cuda.synchronize()
        for name, p, p0, (m0, v0), c in zip(m.names, m.params, before, mv, m.copies):
            gr = f64(grads[name]).reshape(p0.shape)
            want_p, wm, wv = oracle.adamw(p0, gr, m0, v0, LR, 0.9, 0.999, 1e-8, 0.01, step)
            up = LR / (1 - 0.9 ** step) / (np.sqrt(wv / (1 - 0.999 ** step)) + 1e-8)
            # 16 roundings of the update's terms, 5 of the parameter's own
            bound = 2.0 ** -24 * (5 * np.abs(p0) + up * 16 * (0.9 * np.abs(m0) + 0.1 * np.abs(gr)))
            assert np.all(np.abs(f64(p) - want_p) <= bound + 1e-12), name
            assert c is None or torch.equal(c, p.to(torch.bfloat16)), name
    assert m.opt.steps == 2
