"""GPU checks of the AdamW step.  With 32-bit moments against float64, with
u = 2^-24: m and v are two products and a sum of rounded constants (4 u of
their terms), the update adds a square root, a product, a sum, a division and
the rounded step size (12 u of itself, and half of v's error), p two more
roundings of its own.  With 8-bit moments the codes and scales have to be
those of the fp32 definition, bit for bit."""

import numpy as np
import pytest
import torch

import oracle
from efficient_attention_transformer_gb300 import binding as bd

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HYPER = dict(betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01)
LR = 3e-4


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from efficient_attention_transformer_gb300.build import build
    build()


def f64(t):
    return t.double().cpu().numpy().reshape(-1)


def make(sizes, grad_dtype, seed, offset=0):
    g = torch.Generator().manual_seed(seed)

    def dev(x, dt=torch.float32):
        flat = torch.empty(x.numel() + offset, dtype=dt, device="cuda")[offset:]
        return flat.copy_(x)

    params = [dev(torch.randn(n, generator=g) * 0.05) for n in sizes]
    grads = [[dev(torch.randn(n, generator=g) * 10.0 ** float(torch.empty(1).uniform_(-5, 0, generator=g)),
                  grad_dtype) for n in sizes] for _ in range(3)]
    return params, grads


def check_step32(params, grads, steps, lr, betas, eps, weight_decay, scale=1.0, copies=None, opt=None):
    before = [(f64(p), f64(m), f64(v)) for p, m, v in zip(params, opt.m, opt.v)]
    opt.step(grads, lr=lr)
    torch.cuda.synchronize()
    b1, b2 = betas
    for i, (p0, m0, v0) in enumerate(before):
        g = f64(grads[i])
        wd = weight_decay[i] if isinstance(weight_decay, list) else weight_decay
        p, m, v = oracle.adamw(p0, g, m0, v0, lr, b1, b2, eps, wd, steps, scale)
        em = 4 * U * (np.abs(b1 * m0) + np.abs((1 - b1) * g * scale))
        ev = 5 * U * v
        up = lr / (1 - b1 ** steps) / (np.sqrt(v / (1 - b2 ** steps)) + eps)
        ep = 3 * U * np.abs(p0) + up * (em + 16 * U * np.abs(m)) + 2 * U * np.abs(p)
        assert np.all(np.abs(f64(opt.m[i]) - m) <= em), i
        assert np.all(np.abs(f64(opt.v[i]) - v) <= ev + 1e-45), i
        assert np.all(np.abs(f64(params[i]) - p) <= ep), i
        if copies and copies[i] is not None:
            assert torch.equal(copies[i], params[i].to(torch.bfloat16)), i


@pytest.mark.parametrize("grad_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("sizes", [[1], [255, 256, 257, 3], [2048], [100003, 5, 4096, 1000]])
def test_fp32_moments(sizes, grad_dtype, offset):
    params, grads = make(sizes, grad_dtype, 3 + offset, offset)
    copies = [p.to(torch.bfloat16) if i % 2 == 0 else None for i, p in enumerate(params)]
    opt = bd.AdamW(params, copies=copies, **HYPER)
    for t in (1, 2, 3):
        check_step32(params, grads[t - 1], t, LR, copies=copies, opt=opt, **HYPER)


def test_long_list_and_empty_tensors():
    """More tensors than one launch takes, some of them empty, decay by tensor."""
    sizes = [(k * 37) % 700 for k in range(900)]
    assert 0 in sizes
    params, grads = make(sizes, torch.float32, 9)
    decay = [0.1 if k % 3 else 0.0 for k in range(900)]
    kw = dict(HYPER, weight_decay=decay)
    opt = bd.AdamW(params, **kw)
    check_step32(params, grads[0], 1, LR, opt=opt, **kw)
    only = bd.AdamW([torch.empty(0, device="cuda")])
    only.step([torch.empty(0, device="cuda")], lr=LR)
    bd.AdamW([]).step([], lr=LR)
    torch.cuda.synchronize()


def test_grad_scale_and_step_number():
    params, grads = make([777], torch.float32, 10)
    opt = bd.AdamW(params, **HYPER)
    p0 = f64(params[0])
    scale = torch.tensor([0.25], device="cuda")
    opt.step(grads[0], lr=LR, step=1000, grad_scale=scale)
    p, m, v = oracle.adamw(p0, f64(grads[0][0]), np.zeros(777), np.zeros(777), LR, 0.9, 0.999, 1e-8,
                           0.01, 1000, 0.25)
    assert opt.steps == 1000
    up = LR / (np.sqrt(v / (1 - 0.999 ** 1000)) + 1e-8)
    assert np.all(np.abs(f64(params[0]) - p) <= 5 * U * np.abs(p0) + up * 20 * U * np.abs(m))
    opt.step(grads[1], lr=LR)
    assert opt.steps == 1001


@pytest.mark.parametrize("grad_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset", [0, 1, 2])
@pytest.mark.parametrize("sizes", [[1], [255, 256, 257, 3], [2048, 513], [100003, 5]])
def test_8bit_moments_bit_for_bit(sizes, grad_dtype, offset):
    params, grads = make(sizes, grad_dtype, 20 + offset, offset)
    opt = bd.AdamW(params, state_bits=8, **HYPER)
    if offset:  # codes behind an aligned address too
        for k in (opt.m, opt.v):
            for i, x in enumerate(k):
                k[i] = torch.zeros(x.numel() + offset, dtype=x.dtype, device="cuda")[offset:]
        opt = bd.AdamW(params, state_bits=8, m=opt.m, v=opt.v, **HYPER)
    b1, b2 = HYPER["betas"]
    scale = torch.tensor([0.5], device="cuda")
    state = [(x.cpu().numpy() for x in (opt.m[i], opt.m_scale[i], opt.v[i], opt.v_scale[i]))
             for i in range(len(sizes))]
    state = [tuple(s) for s in state]
    for t in (1, 2, 3):
        gs = scale if t == 2 else None
        p0 = [f64(p) for p in params]
        opt.step(grads[t - 1], lr=LR, grad_scale=gs)
        torch.cuda.synchronize()
        for i in range(len(sizes)):
            mc, ms, vc, vs, m1, v1 = oracle.adamw_codes(
                grads[t - 1][i].float().cpu().numpy(), *state[i], b1, b2, None if gs is None else 0.5)
            state[i] = (mc, ms, vc, vs)
            for got, want in ((opt.m[i], mc), (opt.m_scale[i], ms), (opt.v[i], vc),
                              (opt.v_scale[i], vs)):
                np.testing.assert_array_equal(got.cpu().numpy(), want)
            # the update uses the fresh moments
            c1, c2 = 1 - b1 ** t, 1 - b2 ** t
            up = LR / c1 / (np.sqrt(v1.astype(np.float64) / c2) + 1e-8)
            p = p0[i] * (1 - LR * 0.01) - up * m1
            bound = 5 * U * np.abs(p0[i]) + up * 16 * U * np.abs(m1) + 2 * U * np.abs(p)
            assert np.all(np.abs(f64(params[i]) - p) <= bound)
    m, v = opt.moments()
    for i in range(len(sizes)):
        wm, wv = oracle.decode_moments(*state[i])
        np.testing.assert_array_equal(m[i].cpu().numpy().reshape(-1), wm)
        np.testing.assert_array_equal(v[i].cpu().numpy().reshape(-1), wv)


@pytest.mark.parametrize("many", [False, True])
def test_8bit_long_list_as_its_tensors_alone(many):
    """A list long enough for the staged kernel against a step of each tensor
    by itself: ragged ends, tensors that end inside a warp's share, either
    gradient type, arrays that are not on 16 bytes."""
    sizes = [1000003, 2 ** 20, 1500000, 770, 256, 1, 2300001, 1200 * 1000, 1400000] + [300] * (10 * many)
    assert sum(sizes) >= 2 ** 23
    params, copies, m, v = [], [], [], []
    grads = [[] for _ in range(2)]
    g = torch.Generator(device="cuda").manual_seed(50)
    for k, n in enumerate(sizes):
        off = 1 if k in (2, 4) else 0
        dev = lambda dt, x=None: torch.empty(n + off, dtype=dt, device="cuda")[off:].copy_(  # noqa: E731
            x if x is not None else torch.zeros(n, device="cuda"))
        rand = lambda: torch.randn(n, generator=g, device="cuda")  # noqa: E731
        params.append(dev(torch.float32, rand() * 0.05))
        copies.append(dev(torch.bfloat16) if k % 3 else None)
        m.append(dev(torch.int8))
        v.append(dev(torch.uint8))
        for t in range(2):
            grads[t].append(dev(torch.bfloat16 if k % 2 else torch.float32, rand() * 0.01))
    clone = lambda x: None if x is None else x.clone()  # noqa: E731
    alone = [bd.AdamW([params[k].clone()], copies=[clone(copies[k])], state_bits=8, **HYPER)
             for k in range(len(sizes))]
    opt = bd.AdamW(params, copies=copies, state_bits=8, m=m, v=v, **HYPER)
    for t in range(2):
        opt.step(grads[t], lr=LR)
        for k, a in enumerate(alone):
            a.step([grads[t][k]], lr=LR)
    torch.cuda.synchronize()
    for k, a in enumerate(alone):
        for x, y in ((params[k], a.params[0]), (m[k], a.m[0]), (v[k], a.v[0]),
                     (opt.m_scale[k], a.m_scale[0]), (opt.v_scale[k], a.v_scale[0])):
            assert torch.equal(x, y), (k, sizes[k])
        assert copies[k] is None or torch.equal(copies[k], a.copies[0])


def test_8bit_stays_near_32bit():
    """Twenty steps with both kinds: a code's first moment is off by at most
    half a step of 2 c + 1 in c^2, so that what differs stays a small part of
    the way that the parameters went."""
    torch.manual_seed(0)
    p = torch.randn(4096, device="cuda") * 0.05
    a, b = p.clone(), p.clone()
    o32, o8 = bd.AdamW([a], **HYPER), bd.AdamW([b], state_bits=8, **HYPER)
    for _ in range(20):
        g = torch.randn(4096, device="cuda") * 1e-2 + 5e-3
        o32.step([g], lr=LR)
        o8.step([g], lr=LR)
    # a value near the block's top is off by under 1% each step, smaller ones
    # by more of themselves but not of the top: under a tenth of the way
    assert float((a - b).norm()) <= 0.1 * float((a - p).norm())


def test_8bit_nonfinite_gradients_show():
    p = torch.zeros(512, device="cuda")
    opt = bd.AdamW([p], state_bits=8)
    g = torch.ones(512, device="cuda")
    g[3] = float("nan")
    opt.step([g], lr=LR)
    m, v = opt.moments()
    assert p[3].isnan() and not p[256:].isnan().any()
    assert m[0][:256].isnan().any() and not m[0][256:].isnan().any()
    # tiny blocks are zeros
    opt = bd.AdamW([torch.zeros(256, device="cuda")], state_bits=8)
    opt.step([torch.full((256,), 1e-25, device="cuda")], lr=LR)
    assert not opt.m[0].any() and float(opt.m_scale[0]) == 0.0


@pytest.mark.parametrize("bits", [8, 32])
def test_captured_and_other_stream(bits):
    params, grads = make([5000, 77], torch.float32, 30)
    twin = [p.clone() for p in params]
    a, b = (bd.AdamW(x, state_bits=bits, **HYPER) for x in (params, twin))
    scale = torch.ones(1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step(grads[0], lr=LR, step=7, grad_scale=scale)
    for f in (1.0, 0.5):
        scale.fill_(f)
        graph.replay()
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        b.step(grads[0], lr=LR, step=7, grad_scale=scale, stream=s)
        s.synchronize()
    for x, y in zip(params + a.m + a.v, twin + b.m + b.v):
        assert torch.equal(x, y)


@pytest.mark.parametrize("bits", [8, 32])
def test_moments_to_lists_on_a_stream(bits):
    params, grads = make([300, 5], torch.float32, 33)
    opt = bd.AdamW(params, state_bits=bits, **HYPER)
    opt.step(grads[0], lr=LR)
    want = [[t.clone() for t in x] for x in opt.moments()]
    m, v = ([torch.full_like(p, 7.0) for p in params] for _ in range(2))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = opt.moments(m, v, stream=s)
    s.synchronize()
    assert got[0] is m and got[1] is v
    for a, b in zip(want[0] + want[1], m + v):
        assert torch.equal(a, b)
    for lists in ((m[:1], v), (m, v + v)):
        with pytest.raises(ValueError):
            opt.moments(*lists)


def test_replaced_memory_is_refused():
    held = torch.zeros(600, device="cuda")
    opt = bd.AdamW([held])
    held.data = torch.ones(600, device="cuda")
    with pytest.raises(ValueError):
        opt.step([torch.zeros(600, device="cuda")], lr=LR)
    assert opt.steps == 0 and bool((held == 1).all())


def test_large_stack():
    """The parameters of several layers at the long workload's widths."""
    sizes = [768 * 3200, 1536 * 768, 512, 512, 511] * 3
    params, grads = make(sizes, torch.float32, 40)
    copies = [p.to(torch.bfloat16) if p.numel() > 1000 else None for p in params]
    opt = bd.AdamW(params, copies=copies, **HYPER)
    check_step32(params, grads[0], 1, LR, copies=copies, opt=opt, **HYPER)


def test_refusals():
    p = torch.zeros(600, device="cuda")
    with pytest.raises(ValueError):
        bd.AdamW([p, p])                                     # the same tensor twice
    with pytest.raises(ValueError):
        bd.AdamW([p[:300], p[200:]])
    with pytest.raises(ValueError):
        bd.AdamW([p], copies=[torch.zeros(600, device="cuda")])
    with pytest.raises(ValueError):
        bd.AdamW([p], weight_decay=[0.1, 0.2])
    with pytest.raises(ValueError):
        bd.AdamW([p.view(20, 30).t()])
    with pytest.raises(ValueError):
        bd.AdamW([p.double()])
    opt = bd.AdamW([p])
    with pytest.raises(ValueError):
        opt.step([], lr=LR)
    with pytest.raises(ValueError):
        opt.step([torch.zeros(601, device="cuda")], lr=LR)
    with pytest.raises(TypeError):
        opt.step([torch.zeros(600, device="cuda", dtype=torch.float16)], lr=LR)
    with pytest.raises(ValueError):
        opt.step([torch.zeros(600)], lr=LR)
    with pytest.raises(bd.FlashGauError):
        opt.step([torch.zeros(600, device="cuda")], lr=-1.0)
    with pytest.raises(bd.FlashGauError):
        opt.step([p], lr=LR)                                 # the parameter as its gradient
    assert opt.steps == 0


@pytest.mark.parametrize("bits", [8, 32])
def test_lists_that_are_changed_keep_their_memory(bits):
    """A handle's lists are read when it is made: what is put into them later
    is not taken, and the memory of what was there stays the handle's."""
    p = torch.zeros(3 << 20, device="cuda")
    opt = bd.AdamW([p], copies=[torch.zeros(3 << 20, dtype=torch.bfloat16, device="cuda")],
                   state_bits=bits)
    kinds = ("m", "v", "copies") + (("m_scale", "v_scale") if bits == 8 else ())
    for k in kinds:
        old = getattr(opt, k)[0]
        at, like = old.data_ptr(), torch.zeros_like(old)
        if k == "v":
            old.data = like
        del old
        getattr(opt, k)[0] = like
        others = [torch.empty_like(like) for _ in range(8)]
        assert at not in [t.data_ptr() for t in others], k


def test_8bit_moments_come_whole():
    """Codes and scales of a checkpoint belong together: parts of them are
    refused (codes that are all zero need no scales), and a handle made of
    copies of all four carries on bit for bit."""
    params, grads = make([700, 3], torch.float32, 60)
    a = bd.AdamW(params, state_bits=8, **HYPER)
    a.step(grads[0], lr=LR)
    twin = [p.clone() for p in params]
    kinds = ("m", "v", "m_scale", "v_scale")
    state = {k: [t.clone() for t in getattr(a, k)] for k in kinds}
    b = bd.AdamW(twin, state_bits=8, **state, **HYPER)
    b.steps = a.steps
    a.step(grads[1], lr=LR)
    b.step(grads[1], lr=LR)
    for x, y in zip(params, twin):
        assert torch.equal(x, y)
    for k in kinds:
        for x, y in zip(getattr(a, k), getattr(b, k)):
            assert torch.equal(x, y), k
    for left_out in (("m_scale", "v_scale"), ("m", "v"), ("m",), ("v",), ("m_scale",), ("v_scale",),
                     ("v", "v_scale"), ("m", "m_scale")):
        part = {k: x for k, x in state.items() if k not in left_out}
        with pytest.raises(ValueError):
            bd.AdamW([p.clone() for p in params], state_bits=8, **part)
    full = [torch.zeros(p.shape, device="cuda") for p in params]
    for part in (dict(m=full), dict(v=full), dict(m=full, v=[t.clone() for t in full],
                                                  m_scale=state["m_scale"])):
        with pytest.raises(ValueError):
            bd.AdamW([p.clone() for p in params], **part)


def test_moments_of_32_bits_check_their_lists():
    p = torch.zeros(8, 40, device="cuda")
    opt = bd.AdamW([p])
    good = [torch.empty(8, 40, device="cuda")]
    for bad in (torch.empty(8, 40, device="cuda", dtype=torch.bfloat16), torch.empty(2, 8, 40, device="cuda"),
                torch.empty(8, 40), torch.empty(40, 8, device="cuda").t()):
        with pytest.raises(ValueError):
            opt.moments([bad], good)
        with pytest.raises(ValueError):
            opt.moments(good, [bad])
