"""The operators of a training step around the layer, as a user's program calls
them, each with a plain form in elementary torch operations:

  xent      softmax cross entropy of X W^T over a vocabulary, with the gradients
            of X and W
  norm      residual stream: r = h + scale * gate * post_norm(y), n = norm(r),
            and the gradients of all of it
  adamw     one AdamW step over a list of tensors, moments in 32 or in 8 bits

listed() holds the cases that are timed, draw() makes more of the same ranges,
prepare() makes the inputs, run() is one pass (the plain form, or the
framework's calls where `own` is set), exact() gives the outputs from the
definitions in 64 bits.
"""

import math

import torch

own = False

NONE, LAYER, SCALE = 0, 1, 2  # norms
EPS = 1e-5                    # of the norms
BLOCK = 256                   # elements that share a scale of 8-bit moments
STEP = 100                    # of the optimiser, a run some way in
LR, BETA1, BETA2, ADAM_EPS, DECAY = 3e-4, 0.9, 0.999, 1e-8, 0.01

# ------------------------------------------------------------------- cases


def listed():
    return [
        # one generated token scored against the vocabulary: latency
        dict(name="xent_score_1", op="xent", N=1, d=768, V=50257, io="bf16", grad=False,
             ignored=0.0),
        # evaluation, prompts masked out
        dict(name="xent_eval_2048", op="xent", N=2048, d=1024, V=32000, io="bf16", grad=False,
             ignored=0.5),
        # a training step of the smaller language model: 8 rows of 1024 tokens
        dict(name="xent_train_8192", op="xent", N=8192, d=768, V=50257, io="bf16", grad=True,
             ignored=0.0),
        # a training step at the larger width, rows of 8192 tokens, with padding
        dict(name="xent_train_16384", op="xent", N=16384, d=1024, V=50257, io="bf16", grad=True,
             ignored=0.1),
        # a small fp32 model with a byte-pair vocabulary, odd sizes
        dict(name="xent_fp32_1001", op="xent", N=1001, d=520, V=8003, io="fp32", grad=True,
             ignored=0.1),
        # decode: the residual and the next block's norm for 64 sequences
        dict(name="norm_decode_64", op="norm", M=64, d=768, io="bf16", post=NONE, pre=LAYER,
             gate=False, scale=False, backward=False),
        # a block's boundary at the long workload, everything on
        dict(name="norm_block_16384", op="norm", M=16384, d=768, io="bf16", post=SCALE, pre=LAYER,
             gate=True, scale=True, backward=False),
        dict(name="norm_block_grad_16384", op="norm", M=16384, d=768, io="bf16", post=SCALE,
             pre=LAYER, gate=True, scale=True, backward=True),
        # fp32 rows of an odd width
        dict(name="norm_grad_fp32_2000", op="norm", M=2000, d=513, io="fp32", post=LAYER,
             pre=SCALE, gate=False, scale=True, backward=True),
        # the parameters of one small fp32 layer: latency
        dict(name="adamw_layer_fp32", op="adamw", layers=1, d=64, e=128, s=32, C=64, V=0,
             io="fp32", bits=32),
        # twelve layers in bf16 with fp32 masters
        dict(name="adamw_stack_32", op="adamw", layers=12, d=768, e=1536, s=128, C=256, V=0,
             io="bf16", bits=32),
        # the same with the vocabulary's matrix, moments in 8 bits
        dict(name="adamw_model_8", op="adamw", layers=12, d=768, e=1536, s=128, C=256, V=50257,
             io="bf16", bits=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["xent", "norm", "adamw"])
    io = rng.choice(["bf16", "bf16", "fp32"])
    if op == "xent":
        # any number of tokens and of words; widths in steps of 8
        grad = rng.random() < 0.7
        N, d, V = _log(rng, 1, 16384), 8 * _log(rng, 8, 160), _log(rng, 300, 100000)
        most = 16384 * 1024 * 50257 if io == "bf16" else 1000 * 512 * 8000 * 16
        while N * d * V > most:
            N, V = (N + 1) // 2, (V + 1) // 2
        return dict(op=op, N=N, d=d, V=V, io=io, grad=grad, ignored=rng.choice([0.0, 0.1, 0.9]))
    if op == "norm":
        M, d = _log(rng, 1, 16384), _log(rng, 32, 2048)
        if rng.random() < 0.6:
            d = (d + 63) // 64 * 64
        while M * d > 16384 * 768:
            M = (M + 1) // 2
        return dict(op=op, M=M, d=d, io=io, post=rng.choice([NONE, LAYER, SCALE]),
                    pre=rng.choice([LAYER, SCALE]), gate=rng.random() < 0.5,
                    scale=rng.random() < 0.5, backward=rng.random() < 0.6)
    s = rng.choice([32, 64, 128])
    return dict(op=op, layers=rng.randint(1, 12), d=8 * _log(rng, 8, 128),
                e=8 * _log(rng, 8, 192), s=s, C=rng.choice([64, 128, 256]),
                V=rng.choice([0, _log(rng, 300, 50000)]), io=io, bits=rng.choice([8, 32]))


def _shapes(c):
    """The matrices (the vocabulary's first, where V is not zero; W_uvz and W_o
    of each layer) and the other parameters (gamma, beta, relpos)."""
    big = [(c["d"], 2 * c["e"] + c["s"]), (c["e"], c["d"])] * c["layers"]
    small = [(4, c["s"]), (4, c["s"]), (2 * c["C"] - 1,)] * c["layers"]
    return ([(c["V"], c["d"])] if c["V"] else []) + big, small


def work(case):
    c, io = case, 2 if case["io"] == "bf16" else 4
    if c["op"] == "xent":
        N, d, V = c["N"], c["d"], c["V"]
        # ignored tokens need no logits and have no gradient
        Nv = max(1, round(N * (1.0 - c["ignored"])))
        b = (Nv + V) * d * io + N * 4 + N * 4
        f = 2.0 * Nv * d * V
        if c["grad"]:
            b, f = b + (N + V) * d * io, 3 * f
        return {"bytes": b, "flops": f}
    if c["op"] == "norm":
        n = c["M"] * c["d"]
        if c["backward"]:  # dr, dn, r, y, gate; dh, dy, dgate
            return {"bytes": n * io * (6 + 2 * c["gate"]), "flops": 30.0 * n}
        return {"bytes": n * io * (4 + c["gate"]), "flops": 15.0 * n}
    big, n = (sum(math.prod(s) for s in x) for x in (_shapes(c)[0], sum(_shapes(c), [])))
    b = 12 * n + (2 * big if c["io"] == "bf16" else 0)  # master in and out, gradient, bf16 copy
    b -= 2 * c["V"] * c["d"] if c["io"] == "bf16" else 0  # the vocabulary's gradient is bf16
    # moments in and out; 8-bit ones also as the values they stand for
    b += 16 * n if c["bits"] == 32 else 4 * n + 16 * n // BLOCK + 8 * n
    return {"bytes": b, "flops": 15.0 * n}


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    io = torch.bfloat16 if c["io"] == "bf16" else torch.float32
    f32 = torch.float32

    def normal(*shape, dtype=f32, sd=1.0, mean=0.0):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(sd).add_(mean).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    st = {"case": c}
    if c["op"] == "xent":
        N, d, V = c["N"], c["d"], c["V"]
        W = normal(V, d, sd=d ** -0.5)
        # frequent words have low numbers; hidden states point some way to their word
        y = (V * uniform(N) ** 3).long().clamp_(max=V - 1)
        X = normal(N, d)
        X += uniform(N, 1).mul_(0.3 * d ** 0.5) * W[y]
        if c["ignored"]:
            y = torch.where(uniform(N) < c["ignored"], torch.full_like(y, -1), y)
        st.update(X=X.to(io), W=W.to(io), labels=y.to(torch.int32))
        return st
    if c["op"] == "norm":
        M, d = c["M"], c["d"]

        def params(kind):
            if kind == NONE:
                return None, None
            if kind == LAYER:
                return normal(d, sd=0.1, mean=1.0), normal(d, sd=0.1)
            return normal(1, sd=0.1, mean=1.0).mul_(d ** 0.5), None

        st["post_g"], st["post_b"] = params(c["post"])
        st["pre_g"], st["pre_b"] = params(c["pre"])
        st["scale"] = normal(d, sd=0.1, mean=0.5) if c["scale"] else None
        st["gate"] = normal(M, d, dtype=io) if c["gate"] else None
        st["y"] = normal(M, d, dtype=io, sd=2.0)
        st["h"] = normal(M, d, dtype=io, sd=1.5, mean=0.1)  # backward: the stored r
        if c["backward"]:
            st["dr"], st["dn"] = normal(M, d, dtype=io), normal(M, d, dtype=io)
        return st
    # One flat buffer of each kind, the tensors being views of it: fp32 masters,
    # gradients and moments, and for bf16 io the matrices' bf16 copies (they
    # come first).  The vocabulary's gradient comes in the io type, as xent
    # gives it.
    big, small = _shapes(c)
    n_big, n = (sum(_padded(s) for s in x) for x in (big, big + small))
    shapes = big + small
    live = torch.zeros(n, device="cuda")
    for x in _views(live, shapes):
        x.fill_(1.0)
    st["p"] = normal(n, sd=0.03) * live
    st["copy"] = st["p"][:n_big].to(io) if c["io"] == "bf16" else None
    n_vocab = _padded(big[0]) if c["V"] else 0
    st["g"] = (normal(n, sd=1e-3) * live)[n_vocab:].clone()
    st["g_vocab"] = normal(c["V"], c["d"], dtype=io, sd=1e-3) if c["V"] else None
    m = normal(n, sd=3e-4) * live
    v = normal(n, sd=1e-3).square_().add_(1e-10) * live
    if c["bits"] == 32:
        st["m"], st["v"] = m, v
    else:
        st["m"], st["m_scale"] = _encode(m, False)
        st["v"], st["v_scale"] = _encode(v.sqrt(), True)
        st["m_values"], st["v_values"] = m, v
    return st


def _padded(shape):
    return -(-math.prod(shape) // BLOCK) * BLOCK


def _views(flat, shapes):
    """The tensors of a flat buffer, each from a multiple of BLOCK on."""
    at = [0]
    for s in shapes:
        at.append(at[-1] + _padded(s))
    return [flat[a:a + math.prod(s)].view(s) for a, s in zip(at, shapes)]


# ------------------------------------------------------- 8-bit moments
# Blocks of 256 elements share an fp32 scale.  The first moment is
# scale * c |c| with c in -127..127, the square root of the second scale * c^2
# with c in 0..255, c at least 1 where the value is not zero: steps are fine
# near zero, and the largest value of a block is met.  Every line is one
# correctly rounded fp32 operation, so that an implementation that takes the
# same ones in the same order gets the same codes.


def _encode(x, root):
    """Codes and the blocks' scales of a flat buffer."""
    top = 255 if root else 127
    a = x.reshape(-1, BLOCK)
    big = a.abs().amax(1, keepdim=True)
    live = big >= 2.0 ** -60
    zero = torch.zeros_like(big)
    scale = torch.where(live, big * (1.0 / (top * top)), zero)
    inv = torch.where(live, big.reciprocal() * float(top * top), zero)
    q = torch.round(torch.sqrt(a.abs() * inv)).clamp(max=float(top))
    if root:
        q = torch.where((a > 0) & live, q.clamp(min=1.0), q)
    q = (q * torch.sign(a)).reshape(-1)
    return q.to(torch.uint8 if root else torch.int8), scale.reshape(-1)


def _decode(q, scale):
    c = q.to(torch.float32).reshape(-1, BLOCK)
    return ((c * c.abs()) * scale[:, None]).reshape(-1)


# ------------------------------------------------------------ plain forms


def _xent(st):
    X, W, y = st["X"], st["W"], st["labels"].long()
    valid = (y >= 0)[:, None]
    Xf = torch.where(valid, X.float(), torch.zeros_like(X, dtype=torch.float32))
    Wf = W.float()
    at = y.clamp(min=0)[:, None]
    l = Xf @ Wf.t()
    l -= l.amax(1, keepdim=True)
    target = l.gather(1, at)
    l.exp_()
    z = l.sum(1, keepdim=True)
    loss = torch.where(valid, z.log() - target, torch.zeros_like(z))
    share = valid.float() / valid.sum().clamp(min=1)
    out = {"loss": loss[:, 0], "total": loss.sum() / valid.sum().clamp(min=1)}
    if st["case"]["grad"]:
        # softmax minus one at the label, in which the label's own term is
        # minus the sum of the others (1 - p loses digits next to 1)
        l /= z
        l.scatter_(1, at, 0.0)
        l.scatter_(1, at, -l.sum(1, keepdim=True))
        l *= share
        out["dX"], out["dW"] = (l @ Wf).to(X.dtype), (l.t() @ Xf).to(W.dtype)
    return out


def _norm(x, kind, g, b):
    """The normalised rows, and what they are times the parameters."""
    if kind == LAYER:
        u = x - x.mean(1, keepdim=True)
        u = u / (u.square().mean(1, keepdim=True) + EPS).sqrt()
        return u, u * g + b
    if kind == SCALE:
        u = x / x.square().sum(1, keepdim=True).sqrt().clamp(min=EPS)
        return u, u * g
    return x, x


def _norm_grad(x, kind, g, dy):
    """Gradients of x, g and b (None: the norm has none)."""
    if kind == LAYER:
        u = x - x.mean(1, keepdim=True)
        s = (u.square().mean(1, keepdim=True) + EPS).rsqrt()
        u, du = u * s, dy * g
        dx = s * (du - du.mean(1, keepdim=True) - u * (du * u).mean(1, keepdim=True))
        return dx, (dy * u).sum(0), dy.sum(0)
    if kind == SCALE:
        len_ = x.square().sum(1, keepdim=True).sqrt()
        u = x / len_.clamp(min=EPS)
        along = torch.where(len_ > EPS, (dy * u).sum(1, keepdim=True), torch.zeros_like(len_))
        return (dy - u * along) * g / len_.clamp(min=EPS), (dy * u).sum().reshape(1), None
    return dy, None, None


def _residual_norm(st):
    c, io = st["case"], st["y"].dtype
    y, k = st["y"].float(), 1.0
    k = k if st["scale"] is None else st["scale"] * k
    k = k if st["gate"] is None else st["gate"].float() * k
    post = _norm(y, c["post"], st["post_g"], st["post_b"])[1]
    if not c["backward"]:
        r = st["h"].float() + k * post
        n = _norm(r, c["pre"], st["pre_g"], st["pre_b"])[1]
        return {"r": r.to(io), "n": n.to(io)}
    dx, dg, db = _norm_grad(st["h"].float(), c["pre"], st["pre_g"], st["dn"].float())
    dh = st["dr"].float() + dx
    dy, dpg, dpb = _norm_grad(y, c["post"], st["post_g"], dh * k)
    out = {"dh": dh.to(io), "dy": dy.to(io), "dnorm_g": dg, "dnorm_b": db, "dpost_g": dpg,
           "dpost_b": dpb, "dgate": None, "dscale": None}
    dk = dh * post
    if st["gate"] is not None:
        out["dgate"] = (dk if st["scale"] is None else dk * st["scale"]).to(io)
        dk = dk * st["gate"].float()
    if st["scale"] is not None:
        out["dscale"] = dk.sum(0)
    return out


def _adamw(st):
    eight = st["case"]["bits"] == 8
    p, g = st["p"], st["g"]
    if st["g_vocab"] is not None:
        front = torch.zeros(p.numel() - g.numel(), device=g.device)
        front[:st["g_vocab"].numel()] = st["g_vocab"].reshape(-1)
        g = torch.cat([front, g])
    m = _decode(st["m"], st["m_scale"]) if eight else st["m"]
    v = _decode(st["v"], st["v_scale"]).square() if eight else st["v"]
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + (g * (1.0 - BETA2)) * g
    root = v.sqrt()
    c1, c2 = 1.0 - BETA1 ** STEP, math.sqrt(1.0 - BETA2 ** STEP)
    p.mul_(1.0 - LR * DECAY).sub_((LR / c1) * m / (root / c2 + ADAM_EPS))
    if st["copy"] is not None:
        st["copy"].copy_(p[:st["copy"].numel()])
    if not eight:
        st["m"].copy_(m)
        st["v"].copy_(v)
        return p, st["copy"], st["m"], st["v"]
    for k, (q, s) in {"m": _encode(m, False), "v": _encode(root, True)}.items():
        st[k].copy_(q)
        st[k + "_scale"].copy_(s)
    return p, st["copy"], _decode(st["m"], st["m_scale"]), _decode(st["v"], st["v_scale"]).square()


# -------------------------------------------------------------------- run


def _own_adamw(st):
    from efficient_attention_transformer_gb300 import binding as bd
    c = st["case"]
    shapes = sum(_shapes(c), [])
    n_big = len(_shapes(c)[0])
    if "opt" not in st:  # a program makes its handle once
        kinds = {k: _views(st[k], shapes) for k in ("p", "m", "v")}
        copies = [None] * len(shapes)
        if st["copy"] is not None:
            copies[:n_big] = _views(st["copy"], shapes[:n_big])
        scales = None
        if c["bits"] == 8:
            at = [x.data_ptr() - st["m"].data_ptr() for x in kinds["m"]]
            scales = [[st[k][a // BLOCK:(a + math.prod(s) - 1) // BLOCK + 1]
                       for a, s in zip(at, shapes)] for k in ("m_scale", "v_scale")]
            st["values"] = [_views(st[k], shapes) for k in ("m_values", "v_values")]
        st["opt"] = bd.AdamW(kinds["p"], copies=copies, betas=(BETA1, BETA2), eps=ADAM_EPS,
                             weight_decay=DECAY, state_bits=c["bits"], m=kinds["m"], v=kinds["v"],
                             m_scale=scales and scales[0], v_scale=scales and scales[1])
        st["grads"] = ([st["g_vocab"]] if c["V"] else []) + _views(st["g"], shapes[bool(c["V"]):])
    st["opt"].step(st["grads"], lr=LR, step=STEP)
    if c["bits"] == 32:
        return st["p"], st["copy"], st["m"], st["v"]
    st["opt"].moments(*st["values"])
    return st["p"], st["copy"], st["m_values"], st["v_values"]


def run(state):
    st, c = state, state["case"]
    if c["op"] == "adamw":
        p, copy, m, v = _own_adamw(st) if own else _adamw(st)
        return {"p": p, "copy": copy, "m": m, "v": v}
    if not own:
        return _xent(st) if c["op"] == "xent" else _residual_norm(st)
    from efficient_attention_transformer_gb300 import binding as bd
    if c["op"] == "xent":
        out = bd.xent(st["X"], st["W"], st["labels"], grad=c["grad"])
        keys = ("loss", "total") + (("dX", "dW") if c["grad"] else ())
        return {k: out[k] for k in keys}
    kw = dict(post_norm=c["post"], post_g=st["post_g"], post_b=st["post_b"], gate=st["gate"],
              scale=st["scale"], norm=c["pre"], norm_g=st["pre_g"], norm_b=st["pre_b"], eps=EPS)
    if c["backward"]:
        return bd.residual_norm_backward(st["dr"], st["dn"], st["h"], st["y"], **kw)
    r, n = bd.residual_norm(st["h"], st["y"], **kw)
    return {"r": r, "n": n}


# ------------------------------------------------------------------ exact


def exact(case, seed):
    st, c = prepare(case, seed), case
    d64 = lambda x: None if x is None else x.double()  # noqa: E731
    if c["op"] == "xent":
        return _exact_xent(c, st["X"], d64(st["W"]), st["labels"].long())
    if c["op"] == "adamw":
        if c["bits"] == 8:
            # the moments as the codes say, rounded codes having no 64-bit value
            m, v = _decode(st["m"], st["m_scale"]), _decode(st["v"], st["v_scale"]).square()
        else:
            m, v = st["m"], st["v"]
        g = d64(st["g"])
        if c["V"]:
            gv = torch.zeros(_padded((c["V"], c["d"])), dtype=torch.float64, device=g.device)
            gv[:c["V"] * c["d"]] = st["g_vocab"].reshape(-1)
            g = torch.cat([gv, g])
        m, v = torch.lerp(g, d64(m), BETA1), torch.lerp(g * g, d64(v), BETA2)
        step = m / (1 - BETA1 ** STEP) / ((v / (1 - BETA2 ** STEP)).sqrt() + ADAM_EPS)
        p = d64(st["p"])
        p = p - LR * (step + DECAY * p)
        copy = None if st["copy"] is None else p[:st["copy"].numel()]
        return {"p": p, "copy": copy, "m": m if c["bits"] == 32 else None,
                "v": v if c["bits"] == 32 else None}
    # norms: the definition, and its derivatives by automatic differentiation
    names = ["h", "y", "pre_g", "pre_b", "post_g", "post_b", "gate", "scale"]
    t = {k: d64(st[k]) for k in names}
    t = {k: x if x is None else x.requires_grad_(c["backward"]) for k, x in t.items()}

    def norm(x, kind, g, b):
        if kind == LAYER:
            return torch.nn.functional.layer_norm(x, (c["d"],), g, b, EPS)
        return g * x / torch.linalg.vector_norm(x, dim=1, keepdim=True).clamp(min=EPS) if kind else x

    add = norm(t["y"], c["post"], t["post_g"], t["post_b"])
    add = add if t["scale"] is None else add * t["scale"]
    add = add if t["gate"] is None else add * t["gate"]
    if not c["backward"]:
        r = t["h"] + add
        return {"r": r, "n": norm(r, c["pre"], t["pre_g"], t["pre_b"])}
    # h holds the stored r: d(n dn) / dr plus dr is what reaches h and the sum
    (norm(t["h"], c["pre"], t["pre_g"], t["pre_b"]) * d64(st["dn"])).sum().backward()
    dh = t["h"].grad + d64(st["dr"])
    (add * dh).sum().backward()
    grad = {k: None if t[k] is None else t[k].grad for k in names}
    return {"dh": dh, "dy": grad["y"], "dnorm_g": grad["pre_g"], "dnorm_b": grad["pre_b"],
            "dpost_g": grad["post_g"], "dpost_b": grad["post_b"], "dgate": grad["gate"],
            "dscale": grad["scale"]}


def _exact_xent(c, X, W, y):
    """Row pieces of log-sum-exp and softmax - onehot."""
    n = max(1, int((y >= 0).sum()))
    loss = torch.zeros(c["N"], dtype=torch.float64, device=X.device)
    dX = torch.zeros(c["N"], c["d"], dtype=torch.float64, device=X.device)
    dW = torch.zeros_like(W)
    live = torch.nonzero(y >= 0)[:, 0]
    for rows in live.split(1024):
        x, t = X[rows].double(), y[rows]
        logits = torch.matmul(x, W.T)
        lse = torch.logsumexp(logits, 1)
        at = torch.arange(len(rows), device=X.device)
        loss[rows] = lse - logits[at, t]
        if c["grad"]:
            dl = torch.exp(logits - lse[:, None])
            dl[at, t] -= 1.0
            dX[rows] = torch.matmul(dl, W) / n
            dW += torch.matmul(dl.T, x) / n
    out = {"loss": loss, "total": loss.sum() / n}
    return dict(out, dX=dX, dW=dW) if c["grad"] else out
