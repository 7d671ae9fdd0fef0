"""GPU checks of the relative position tables by buckets and their gradient.

A table's values are copies of the learned ones: equal bit for bit.  A
gradient is a sum of fp32 values, of at most 16 behind one another, R / 16 of
those, then 1024 / 32 in a lane of a warp, 5 shuffles and 8 blocks: its error
is below that many roundings of 2^-24 of the sum of magnitudes."""

import random
import time

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


def check(H, C, buckets, far, causal, R=1, seed=0, offset=0):
    g = torch.Generator().manual_seed(seed)

    def dev(*shape):
        flat = torch.empty(int(np.prod(shape)) + offset, device="cuda")[offset:]
        return flat.copy_(torch.randn(flat.numel(), generator=g)).view(shape)

    table, d = dev(H, buckets), dev(R, H, 2 * C - 1)
    rel = bd.bucket_bias(table, C, causal, max_distance=far)
    dt = bd.bucket_bias_backward(d, buckets, causal, max_distance=far)
    torch.cuda.synchronize()
    want = oracle.bucket_bias(table.cpu().numpy(), C, far, causal)
    assert np.array_equal(rel.double().cpu().numpy(), want)
    d64 = d.double().cpu().numpy()
    wd = oracle.bucket_bias_grad(d64, buckets, far, causal)
    most = oracle.bucket_bias_grad(np.abs(d64), buckets, far, causal)
    adds = min(R, 16) + R / 16 + 32 + 5 + 8
    assert np.all(np.abs(dt.double().cpu().numpy() - wd) <= adds * U * most)
    return table, d, rel, dt


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,C,buckets,far,R", [
    (1, 1, 4, 3, 1), (1, 2, 4, 2, 1), (2, 3, 8, 5, 3), (12, 256, 32, 128, 1), (3, 257, 32, 128, 2),
    (5, 129, 34, 100, 17), (2, 4096, 64, 2048, 6), (1, 4095, 256, 1 << 20, 33), (70, 64, 16, 17, 1),
    (1, 440, 42, 1006, 1), (300, 5, 6, 4, 2), (1, 4096, 4, 4, 100)])
def test_sizes(H, C, buckets, far, R, causal):
    check(H, C, buckets, far if not causal else max(far, buckets // 2 + 1), causal, R)


def test_odd_buckets_and_addresses():
    for b in (2, 3, 5, 33, 255):
        check(2, 300, b, 200, True, offset=1)
    check(3, 300, 30, 200, False, R=2, offset=3)


def test_borders_that_are_whole_numbers():
    """far = near 2^k: the logarithm is whole at powers of two."""
    for far in (32, 64, 128, 256, 1024, 4096):
        check(1, 4096, 32, far, True)
        check(1, 4096, 64, far, False)


def test_many_tables():
    check(65535, 2, 4, 3, False)


def test_leading_shapes():
    t = torch.randn(8, device="cuda")
    r = bd.bucket_bias(t, 20, True, max_distance=16)
    assert r.shape == (39,) and bd.bucket_bias_backward(r, 8, True, max_distance=16).shape == (8,)
    t = torch.randn(2, 3, 8, device="cuda")
    r3 = bd.bucket_bias(t, 20, True, max_distance=16)
    assert r3.shape == (2, 3, 39)
    assert torch.equal(r3.view(6, 39), bd.bucket_bias(t.view(6, 8), 20, True, max_distance=16))
    with pytest.raises(ValueError):
        bd.bucket_bias_backward(r3.view(2, 3, 39)[:, :, :38].contiguous(), 8, True)
    with pytest.raises(ValueError):
        bd.bucket_bias(t, 20, True, out=torch.empty(2, 3, 40, device="cuda"))
    with pytest.raises(ValueError):
        bd.bucket_bias(t.transpose(0, 1), 20, True)
    with pytest.raises(bd.FlashGauError):
        bd.bucket_bias(t, 20, True, max_distance=4)
    with pytest.raises(bd.FlashGauError):
        bd.bucket_bias(t, 0, True)


def test_what_is_not_finite_stays_in_its_bucket():
    d = torch.zeros(1, 2, 101, device="cuda")
    d[0, 1, 50 + 3] = float("inf")
    d[0, 0, 50 - 7] = float("nan")
    g = bd.bucket_bias_backward(d, 32, False, max_distance=40)
    bad = ~torch.isfinite(g)
    assert bad.sum() == 2 and g[1, 16 + 3] == float("inf") and torch.isnan(g[0, 7])


def test_repeats_writes_only_its_rows_and_replays():
    table, d, rel, dt = check(4, 700, 32, 300, False, R=5)
    out = torch.full((6, 1399), 7.0, device="cuda")
    bd.bucket_bias(table, 700, False, max_distance=300, out=out[1:5])
    assert torch.equal(out[1:5], rel) and bool((out[0] == 7).all()) and bool((out[5] == 7).all())
    gout = torch.full((6, 32), 7.0, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    bd.bucket_bias_backward(d, 32, False, max_distance=300, out=gout[1:5], stream=s)
    s.synchronize()
    assert torch.equal(gout[1:5], dt) and bool((gout[0] == 7).all()) and bool((gout[5] == 7).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = bd.bucket_bias(table, 700, False, max_distance=300)
        b = bd.bucket_bias_backward(d, 32, False, max_distance=300)
    table.mul_(2.0)
    d.mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, 2 * rel) and torch.equal(b, 2 * dt)


@pytest.mark.parametrize("R,H,C", [(5000, 2, 130), (1 << 20, 1, 1), (100003, 1, 3)])
def test_many_gradients_of_a_table(R, H, C):
    """Eight gradients behind one another, then R / 8 of those sums, then a run's
    offsets and the blocks as ever."""
    g = torch.Generator().manual_seed(R)
    d = torch.randn(R, H, 2 * C - 1, generator=g).cuda()
    for causal in (True, False):
        dt = bd.bucket_bias_backward(d, 16, causal, max_distance=64)
        d64 = d.double().cpu().numpy()
        want = oracle.bucket_bias_grad(d64, 16, 64, causal)
        most = oracle.bucket_bias_grad(np.abs(d64), 16, 64, causal)
        adds = 8 + -(-R // 8) + 32 + 5 + 8
        assert np.all(np.abs(dt.double().cpu().numpy() - want) <= adds * U * most)


@pytest.mark.parametrize("seed", range(6))
def test_distances_of_every_size(seed):
    """max_distance from next to the exact buckets up to the largest, far behind
    the chunk among them, and borders that are whole numbers."""
    rng = random.Random(seed)
    for _ in range(12):
        causal = rng.random() < 0.5
        buckets = rng.randint(2, 256) if causal else 2 * rng.randint(2, 128)
        near = (buckets if causal else buckets // 2) // 2
        far = rng.choice([near + 1, rng.randint(near + 1, 4096), rng.randint(near + 1, 1 << 20),
                          near << rng.randint(1, 10), near * rng.randint(2, 40), 1 << 20])
        check(2, rng.choice([1, 2, rng.randint(3, 300), 4096]), buckets, far, causal, seed=seed)


def test_large_distances_cost_the_host_no_more():
    """A call's time on the host, the least of many: with max_distance at its
    largest within four times that of a small one."""
    table = torch.randn(1, 256, device="cuda")

    def least(far):
        best = 1.0
        for _ in range(50):
            torch.cuda.synchronize()
            start = time.perf_counter()
            bd.bucket_bias(table, 256, True, max_distance=far)
            best = min(best, time.perf_counter() - start)
        return best

    assert least(1 << 20) <= 4 * least(200)
