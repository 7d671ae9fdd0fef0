"""The training operators where a program may call them in an unusual place:
captured as a process's first call, on several streams and from several
threads at once, and replayed beside eager calls."""

import subprocess
import sys
import threading

import pytest
import torch

from efficient_attention_transformer_gb300 import binding as bd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from efficient_attention_transformer_gb300.build import build
    build()


FIRST = """
import torch
from efficient_attention_transformer_gb300 import binding as bd
torch.manual_seed(0)
io = torch.bfloat16
h, y, dr, dn = (torch.randn(40, 256, device="cuda").to(io) for _ in range(4))
g, b = torch.ones(256, device="cuda"), torch.zeros(256, device="cuda")
W = torch.randn(300, 256, device="cuda").to(io)
labels = torch.randint(0, 300, (40,), device="cuda", dtype=torch.int32)
p, grad = torch.randn(5000, device="cuda"), torch.randn(5000, device="cuda")

def step(opts):
    r, n = bd.residual_norm(h, y, norm_g=g, norm_b=b)
    out = bd.residual_norm_backward(dr, dn, r, y, norm_g=g, norm_b=b)
    x = bd.xent(n, W, labels)
    few = bd.xent(n[:3], W, labels[:3], grad=False)
    for o in opts:
        o.step([grad], lr=1e-3, step=1)
    return [r, n, out["dh"], out["dnorm_g"], x["total"], x["dX"], x["dW"], few["loss"]]

opts = [bd.AdamW([p.clone()], state_bits=k) for k in (32, 8)]
twins = [bd.AdamW([p.clone()], state_bits=k) for k in (32, 8)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step(opts)
graph.replay()
want = step(twins)
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want))
assert all(torch.equal(a.params[0], b.params[0]) for a, b in zip(opts, twins))
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
        N, d, V = 100 + 70 * k, 128 + 64 * k, 900 + 333 * k
        h, y = (torch.randn(N, d, device="cuda").to(dtype) for _ in range(2))
        g = torch.rand(d, device="cuda") + 0.5
        W = torch.randn(V, d, device="cuda").to(dtype)
        labels = torch.randint(-9, V, (N,), device="cuda", dtype=torch.int32)
        jobs.append((h, y, g, W, labels))

    def once(job):
        h, y, g, W, labels = job
        r, n = bd.residual_norm(h, y, norm_g=g)
        back = bd.residual_norm_backward(n, h, r, y, norm_g=g)
        x = bd.xent(n, W, labels)
        few = bd.xent(n[:5], W, labels[:5], grad=False)
        p = g.clone()
        bd.AdamW([p], state_bits=8).step([back["dnorm_g"]], lr=1e-2)
        return [r, n, back["dh"], back["dnorm_g"], x["loss"], x["dX"], x["dW"], few["loss"], p]

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


def test_wide_rows_of_many_column_tiles():
    """More column tiles than CTA pairs: pairs take several of them."""
    torch.manual_seed(2)
    N, d, V = 20, 20480, 300
    X = torch.randn(N, d, device="cuda").to(torch.bfloat16)
    W = (torch.randn(V, d, device="cuda") * d ** -0.5).to(torch.bfloat16)
    labels = torch.randint(0, V, (N,), device="cuda", dtype=torch.int32)
    got = bd.xent(X, W, labels)
    x, w = X.double().requires_grad_(), W.double().requires_grad_()
    loss = torch.nn.functional.cross_entropy(x @ w.t(), labels.long())
    loss.backward()
    assert abs(float(got["total"]) - loss.item()) <= 1e-4
    # three roundings to bf16 of half a step each
    for a, b in ((got["dX"], x.grad), (got["dW"], w.grad)):
        assert float((a.double() - b).norm() / b.norm()) <= 3 * 2.0 ** -8
