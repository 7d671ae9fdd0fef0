"""Three more operators of a language model on the layer, as a user's program
calls them, each with a plain form in elementary torch operations:

  bias        the layer's relative position table from learned values by buckets
              of distance, and the gradient of those values
  checkpoint  activations kept in 8 bits between the passes: the residual stream
              packed at a block's boundary and restored with its norm, and the
              boundary's gradients taken from the packed stream
  sample      the next token of each row of logits: temperature, top-k, top-p,
              min-p, and one given random number

listed() holds the cases that are timed, draw() makes more of the same ranges,
prepare() makes the inputs, run() is one pass (the plain form, or the
framework's calls where `own` is set), exact() gives the outputs from the
definitions in 64 bits.
"""

import math

import numpy as np
import torch

own = False

NONE, LAYER, SCALE = 0, 1, 2  # norms
EPS = 1e-5                    # of the norms
GROUP = 128                   # neighbours of a row that share a scale of 8-bit codes

# ------------------------------------------------------------------- cases


def listed():
    return [
        # the tables of twelve causal layers at the default chunk, one per layer: latency
        dict(name="bias_12x256", op="bias", shared=1, tables=12, C=256, buckets=32, far=128,
             causal=True),
        # heads' tables that six layers share, both directions, the longest chunk
        dict(name="bias_64x4096", op="bias", shared=6, tables=64, C=4096, buckets=64, far=2048,
             causal=False),
        # boundary of a short batch: latency
        dict(name="checkpoint_512", op="checkpoint", M=512, d=768, io="bf16", norm=LAYER,
             backward=False),
        # a boundary of the long workload, forward and what its backward restores
        dict(name="checkpoint_16384", op="checkpoint", M=16384, d=768, io="bf16", norm=LAYER,
             backward=False),
        # a large fp32 batch of wider rows
        dict(name="checkpoint_fp32_32768", op="checkpoint", M=32768, d=1024, io="fp32",
             norm=SCALE, backward=False),
        # the gradients of the long workload's boundary from its packed stream
        dict(name="checkpoint_grad_16384", op="checkpoint", M=16384, d=768, io="bf16",
             norm=LAYER, backward=True),
        # fp32 rows of an odd width, whose last group is a single element
        dict(name="checkpoint_grad_fp32_2000", op="checkpoint", M=2000, d=513, io="fp32",
             norm=SCALE, backward=True),
        # one sequence's next token, all filters on: latency
        dict(name="sample_1x50257", op="sample", N=1, V=50257, io="bf16", filters="all",
             banned=0.0),
        # a serving batch, every request with filters of its own, some greedy
        dict(name="sample_64x32000", op="sample", N=64, V=32000, io="fp32", filters="mixed",
             banned=0.01),
        # many samples of a small vocabulary from the whole distribution
        dict(name="sample_333x8003", op="sample", N=333, V=8003, io="fp32", filters="none",
             banned=0.0),
        # the largest batch and vocabulary, nucleus sampling
        dict(name="sample_256x131072", op="sample", N=256, V=131072, io="bf16", filters="top_p",
             banned=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["bias", "checkpoint", "sample"])
    io = rng.choice(["bf16", "bf16", "fp32"])
    if op == "bias":
        causal = rng.random() < 0.5
        buckets = 2 * rng.randint(2, 64)
        exact_ones = buckets // 2 if causal else buckets // 4
        return dict(op=op, shared=_log(rng, 1, 6), tables=_log(rng, 1, 64), C=_log(rng, 2, 4096),
                    buckets=buckets, far=_log(rng, max(exact_ones, 1) + 1, 4096), causal=causal)
    if op == "checkpoint":
        M, d = _log(rng, 1, 32768), _log(rng, 32, 2048)
        if rng.random() < 0.6:
            d = (d + 63) // 64 * 64
        while M * d > 32768 * (1024 if io == "fp32" else 2048):
            M = (M + 1) // 2
        return dict(op=op, M=M, d=d, io=io, norm=rng.choice([LAYER, SCALE]),
                    backward=rng.random() < 0.5)
    N, V = _log(rng, 1, 512), _log(rng, 200, 131072)
    while N * V > (256 if io == "bf16" else 64) * 131072:
        N = (N + 1) // 2
    return dict(op=op, N=N, V=V, io=io, banned=rng.choice([0.0, 0.01, 0.5]),
                filters=rng.choice(["none", "top_k", "top_p", "min_p", "all", "mixed"]))


def work(case):
    c = case
    if c["op"] == "bias":
        rows = c["tables"] * (2 * c["C"] - 1)
        return {"bytes": 4 * (rows * (1 + c["shared"]) + 2 * c["tables"] * c["buckets"]),
                "flops": float(rows * c["shared"])}
    io = 2 if c["io"] == "bf16" else 4
    if c["op"] == "checkpoint":
        n = c["M"] * c["d"]
        packed = n + 4 * c["M"] * -(-c["d"] // GROUP)
        if c["backward"]:  # dr, dn and the packed stream; dh
            return {"bytes": 3 * n * io + packed, "flops": 20.0 * n}
        # h, y; r, n; the packed stream out and in; restored stream and norm
        return {"bytes": 6 * n * io + 2 * packed, "flops": 25.0 * n}
    n = c["N"] * c["V"]
    return {"bytes": n * io + c["N"] * (5 * 4 + 3 * 4), "flops": 20.0 * n}


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    f32 = torch.float32

    def normal(*shape, dtype=f32, sd=1.0, mean=0.0):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(sd).add_(mean).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    st = {"case": c}
    if c["op"] == "bias":
        st["table"] = normal(c["tables"], c["buckets"], sd=0.1)
        st["drelpos"] = normal(c["shared"], c["tables"], 2 * c["C"] - 1)
        if c["causal"]:  # the layer's gradient of a masked offset is zero
            st["drelpos"][:, :, c["C"]:] = 0.0
        return st
    io = torch.bfloat16 if c["io"] == "bf16" else f32
    if c["op"] == "checkpoint":
        M, d = c["M"], c["d"]
        if c["norm"] == LAYER:
            st["g"], st["b"] = normal(d, sd=0.1, mean=1.0), normal(d, sd=0.1)
        else:
            st["g"], st["b"] = normal(1, sd=0.1, mean=1.0).mul_(d ** 0.5), None
        # a stream with a few channels that stand out
        loud = torch.where(uniform(d) < 0.01, 8.0, 1.0)
        h = (normal(M, d, sd=1.5, mean=0.1) * loud).to(io)
        if not c["backward"]:
            st["h"], st["y"] = h, normal(M, d, dtype=io, sd=2.0)
            return st
        st["codes"], st["scales"] = _pack(h)
        st["dr"], st["dn"] = normal(M, d, dtype=io), normal(M, d, dtype=io)
        return st
    N, V = c["N"], c["V"]
    # a broad body, and for each row a few words that the text calls for
    logits = normal(N, V, sd=2.0)
    at = (uniform(N, 16) * V).long().clamp_(max=V - 1)
    logits.scatter_add_(1, at, 6.0 + 4.0 * uniform(N, 16) * uniform(N, 1))
    if c["banned"]:
        logits.masked_fill_(uniform(N, V) < c["banned"], float("-inf"))
    st["logits"], st["u"] = logits.to(io), uniform(N)
    kind = c["filters"]

    def setting(name, values, off):
        """One value a row where the case has this filter, None where it has not."""
        if kind not in (name, "all", "mixed"):
            return None
        return torch.where(uniform(N) < 0.5, values, off) if kind == "mixed" else values

    st["temperature"] = 0.6 + 0.8 * uniform(N)
    if kind == "mixed":  # some requests are greedy
        st["temperature"] = torch.where(uniform(N) < 0.1, torch.zeros(N, device="cuda"),
                                        st["temperature"])
    zero = torch.zeros(N, device="cuda")
    st["top_k"] = setting("top_k", 1 + (100 * uniform(N) ** 2).int(), zero.int())
    st["top_p"] = setting("top_p", 0.7 + 0.28 * uniform(N), zero + 1.0)
    st["min_p"] = setting("min_p", 0.02 + 0.1 * uniform(N), zero)
    return st


# ------------------------------------------------------------ plain forms


def _buckets(c):
    """The bucket of each offset -(C-1)..C-1 of a key from its query: distances
    below half the buckets of a direction have one each, the others share them
    by the logarithm of the distance up to `far`, the last takes all beyond."""
    o = torch.arange(1 - c["C"], c["C"], device="cuda")
    n = c["buckets"] if c["causal"] else c["buckets"] // 2
    ahead = torch.zeros_like(o) if c["causal"] else (o > 0).long() * n
    dist = (-o).clamp(min=0) if c["causal"] else o.abs()
    near = n // 2
    # floor of a logarithm: a distance that meets a border is in the upper bucket
    place = torch.log(dist.clamp(min=1).double() / near) / math.log(c["far"] / near) * (n - near)
    wide = (near + torch.floor(place + 1e-9)).clamp(max=n - 1).long()
    return ahead + torch.where(dist < near, dist, wide)


def _bias(st):
    c = st["case"]
    at = _buckets(c)
    drel = st["drelpos"].double().sum(0)
    dtable = torch.zeros(c["tables"], c["buckets"], dtype=torch.float64, device="cuda")
    dtable.index_add_(1, at, drel)
    return {"relpos": st["table"][:, at], "dtable": dtable.float()}


def _groups(x):
    M, d = x.shape
    return torch.nn.functional.pad(x, (0, -d % GROUP)).view(M, -1, GROUP)


def _pack(x):
    """Codes [M, d] int8 and scales [M, groups] fp32: each scale is the largest
    magnitude of its group / 127 in fp32, each code the whole number next to
    x / scale (ties to even); a group below 2^-100 is zero."""
    a = _groups(x.float())
    top = a.abs().amax(2)
    scale = torch.where(top >= 2.0 ** -100, top / 127.0, torch.zeros_like(top))
    by = torch.where(scale > 0, scale, torch.ones_like(scale)).double()
    codes = torch.round(a.double() / by[:, :, None]) * (scale > 0)[:, :, None]
    return codes.to(torch.int8).view(len(x), -1)[:, :x.shape[1]].contiguous(), scale


def _unpack(codes, scales):
    d = codes.shape[1]
    return (_groups(codes.float()) * scales[:, :, None]).view(len(codes), -1)[:, :d]


def _norm(x, kind, g, b):
    if kind == LAYER:
        u = x - x.mean(1, keepdim=True)
        return u / (u.square().mean(1, keepdim=True) + EPS).sqrt() * g + b
    return x / x.square().sum(1, keepdim=True).sqrt().clamp(min=EPS) * g


def _norm_grad(x, kind, g, dy):
    """Gradients of x, g and b (None: the norm has none)."""
    if kind == LAYER:
        u = x - x.mean(1, keepdim=True)
        s = (u.square().mean(1, keepdim=True) + EPS).rsqrt()
        u, du = u * s, dy * g
        dx = s * (du - du.mean(1, keepdim=True) - u * (du * u).mean(1, keepdim=True))
        return dx, (dy * u).sum(0), dy.sum(0)
    length = x.square().sum(1, keepdim=True).sqrt()
    u = x / length.clamp(min=EPS)
    along = torch.where(length > EPS, (dy * u).sum(1, keepdim=True), torch.zeros_like(length))
    return (dy - u * along) * g / length.clamp(min=EPS), (dy * u).sum().reshape(1), None


def _checkpoint(st):
    c = st["case"]
    if c["backward"]:
        x = _unpack(st["codes"], st["scales"])
        dx, dg, db = _norm_grad(x, c["norm"], st["g"], st["dn"].float())
        return {"dh": (st["dr"].float() + dx).to(st["dr"].dtype), "dnorm_g": dg, "dnorm_b": db}
    io = st["h"].dtype
    r = st["h"].float() + st["y"].float()
    n = _norm(r, c["norm"], st["g"], st["b"])
    r = r.to(io)
    x = _unpack(*_pack(r))
    return {"r": r, "n": n.to(io), "x": x.to(io),
            "xn": _norm(x, c["norm"], st["g"], st["b"]).to(io)}


def _sample(st):
    """Words in falling order of their logits (equal ones by index).  Each
    filter keeps a beginning of them, the most probable at least: top_k that
    many, top_p those with less than that share of top_k's mass before them,
    min_p those with at least that share of the first one's probability.  The
    token is the first kept one up to whose end more than u of the kept mass
    lies."""
    s, index = st["logits"].float().sort(dim=1, descending=True, stable=True)
    T = st["temperature"].double()[:, None]
    greedy = T == 0
    w = torch.exp((s.double() - s[:, :1].double()) / torch.where(greedy, torch.ones_like(T), T))
    rank = torch.arange(s.shape[1], device=s.device)[None]
    first = rank == 0
    keep = (s > float("-inf")) & (first | ~greedy)
    if st["top_k"] is not None:
        k = st["top_k"][:, None]
        keep &= (rank < k) | (k <= 0)
    if st["top_p"] is not None:
        p = st["top_p"].double()[:, None]
        end = torch.cumsum(w * keep, 1)
        before = torch.nn.functional.pad(end, (1, -1))
        keep &= (before < p * end[:, -1:]) | (p >= 1) | first
    if st["min_p"] is not None:
        m = st["min_p"].double()[:, None]
        keep &= (w >= m) | (m <= 0) | first
    kept = keep.sum(1)
    w = w * keep
    end = torch.cumsum(w, 1)
    total = end[:, -1:]
    place = (end <= st["u"].double()[:, None] * total).sum(1)
    place = torch.minimum(place, kept - 1)[:, None]
    return {"token": index.gather(1, place)[:, 0].int(), "kept": kept.int(),
            "logp": torch.log(w.gather(1, place) / total)[:, 0].float()}


# -------------------------------------------------------------------- run


def run(state):
    st, c = state, state["case"]
    if not own:
        return {"bias": _bias, "checkpoint": _checkpoint, "sample": _sample}[c["op"]](st)
    from efficient_attention_transformer_gb300 import binding as bd
    if c["op"] == "bias":
        relpos = bd.bucket_bias(st["table"], c["C"], c["causal"], max_distance=c["far"])
        dtable = bd.bucket_bias_backward(st["drelpos"], c["buckets"], c["causal"],
                                         max_distance=c["far"])
        return {"relpos": relpos, "dtable": dtable}
    if c["op"] == "sample":
        token, logp, kept = bd.sample(st["logits"], st["u"], temperature=st["temperature"],
                                      top_k=st["top_k"], top_p=st["top_p"], min_p=st["min_p"])
        return {"token": token, "kept": kept, "logp": logp}
    norm = dict(norm=c["norm"], norm_g=st["g"], norm_b=st["b"], eps=EPS)
    if c["backward"]:
        packed = bd.Checkpoint(st["codes"], st["scales"])
        return bd.checkpoint_backward(st["dr"], st["dn"], packed, **norm)
    packed, r, n = bd.checkpoint_pack(st["h"], st["y"], **norm)
    x, xn = bd.checkpoint_restore(packed, st["h"].dtype, **norm)
    return {"r": r, "n": n, "x": x, "xn": xn}


# ------------------------------------------------------------------ exact


def exact(case, seed):
    st, c = prepare(case, seed), case

    def bias():
        """Buckets by whole numbers: distance n is in bucket near + j or above
        when (n / near)^(n_b - near) >= (far / near)^j."""
        n_b = c["buckets"] if c["causal"] else c["buckets"] // 2
        near, bucket, j = n_b // 2, [], 0
        rest = n_b - near
        for n in range(c["C"]):
            while n > near and j + 1 < rest and (
                    n ** rest * near ** (j + 1) >= c["far"] ** (j + 1) * near ** rest):
                j += 1
            bucket.append(n if n < near else near + j)
        past = bucket[::-1]
        ahead = [bucket[0]] * (c["C"] - 1) if c["causal"] else [n_b + x for x in bucket[1:]]
        hot = np.zeros((2 * c["C"] - 1, c["buckets"]))
        hot[np.arange(2 * c["C"] - 1), past + ahead] = 1.0
        hot = torch.from_numpy(hot).cuda()
        return {"relpos": st["table"].double() @ hot.T,
                "dtable": torch.einsum("rhn,nb->hb", st["drelpos"].double(), hot)}

    def checkpoint():
        layer = c["norm"] == LAYER

        def norm(x, g, b):
            if layer:
                return torch.nn.functional.layer_norm(x, (c["d"],), g, b, EPS)
            return g * x / torch.linalg.vector_norm(x, dim=1, keepdim=True).clamp(min=EPS)

        def values(codes, scales):
            return codes.double() * scales.double().repeat_interleave(GROUP, 1)[:, :c["d"]]

        g = st["g"].double().requires_grad_(c["backward"])
        b = st["b"].double().requires_grad_(c["backward"]) if layer else None
        if c["backward"]:
            x = values(st["codes"], st["scales"]).requires_grad_(True)
            (norm(x, g, b) * st["dn"].double()).sum().backward()
            return {"dh": st["dr"].double() + x.grad, "dnorm_g": g.grad,
                    "dnorm_b": b.grad if layer else None}
        r = st["h"].double() + st["y"].double()
        n = norm(r, g, b)
        # the codes are of the stream as it is stored; their scales are fp32 numbers
        stored = r.to(st["h"].dtype).double()
        scales = torch.stack([a.abs().amax(1) for a in stored.split(GROUP, 1)], 1).float() / 127.0
        one = values(torch.ones_like(stored), scales)
        x = values(torch.round(stored / one).nan_to_num(), scales)
        return {"r": r, "n": n, "x": x, "xn": norm(x, g, b)}

    def sample():
        """Row by row, in numpy."""
        get = lambda k: None if st[k] is None else st[k].cpu().numpy()  # noqa: E731
        T, k, p, m, u = (get(x) for x in ("temperature", "top_k", "top_p", "min_p", "u"))
        logits = st["logits"].double().cpu().numpy()
        token, kept, logp = [], [], []
        for i, l in enumerate(logits):
            at = np.flatnonzero(np.isfinite(l))
            at = at[np.argsort(-l[at], kind="stable")]
            n = len(at) if T[i] else 1
            prob = np.exp((l[at] - l[at[0]]) / np.float64(T[i] or 1.0))
            if k is not None and k[i] > 0:
                n = min(n, int(k[i]))
            most = n
            if p is not None and p[i] < 1:
                mass = np.cumsum(prob[:n])
                share = np.float64(p[i]) * mass[-1]
                most = 1 + int(np.searchsorted(mass[:-1], share, side="left"))
            if m is not None and m[i] > 0:
                most = min(most, max(1, int((prob >= np.float64(m[i])).sum())))
            n = min(n, most)
            mass = np.cumsum(prob[:n])
            j = min(int(np.searchsorted(mass, np.float64(u[i]) * mass[-1], side="right")), n - 1)
            token.append(at[j])
            kept.append(n)
            logp.append(np.log(prob[j] / mass[-1]))
        cuda = lambda v, dt: torch.tensor(np.array(v), dtype=dt, device="cuda")  # noqa: E731
        return {"token": cuda(token, torch.int32), "kept": cuda(kept, torch.int32),
                "logp": cuda(logp, torch.float64)}

    return {"bias": bias, "checkpoint": checkpoint, "sample": sample}[c["op"]]()
