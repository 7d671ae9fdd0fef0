"""CPU oracle of the operators around the layer in a training step (TEST
INFRASTRUCTURE ONLY: the same import rule as ``oracle.flash_gau``): the
residual stream with its norms, softmax cross entropy over a vocabulary, and
AdamW.  Float64 numpy, written from the formulas; only the codes of 8-bit
moments are defined by fp32 operations and are therefore followed in fp32,
one rounding at a time.

  r = h + scale * gate * post(y),  n = norm(r)
  loss_i = log sum_v exp(x_i . w_v) - x_i . w_{y_i}
  m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
  p = (1 - lr wd) p - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)
"""

import numpy as np

__all__ = ["norm_rows", "residual_norm", "residual_norm_grad", "xent", "adamw",
           "adamw_codes", "decode_moments", "encode_moments"]


def _f(x):
    return None if x is None else np.asarray(x, dtype=np.float64)


def norm_rows(x, kind, g, b, eps):
    """kind: 'none', 'layer' or 'scale'.  Returns (u, 1 / spread, output), u
    being the normalised rows without the parameters."""
    x = _f(x)
    if kind == "none":
        return x, np.ones((len(x), 1)), x
    if kind == "layer":
        c = x - x.mean(axis=1, keepdims=True)
        inv = 1.0 / np.sqrt((c * c).mean(axis=1, keepdims=True) + eps)
        u = c * inv
        return u, inv, u * _f(g) + (0.0 if b is None else _f(b))
    inv = 1.0 / np.maximum(np.sqrt((x * x).sum(axis=1, keepdims=True)), eps)
    return x * inv, inv, x * inv * _f(g)


def residual_norm(h, y, post, post_g, post_b, gate, scale, norm, norm_g, norm_b, eps):
    r = _f(h).copy()
    if y is not None:
        add = norm_rows(y, post, post_g, post_b, eps)[2]
        add = add if gate is None else add * _f(gate)
        add = add if scale is None else add * _f(scale)
        r = r + add
    return r, norm_rows(r, norm, norm_g, norm_b, eps)[2]


def _norm_grad(x, kind, g, dout, eps):
    """(dx, dg, db): the derivative of sum(dout * norm(x)) row by row."""
    if kind == "none":
        return dout, None, None
    u, inv, _ = norm_rows(x, kind, g, None, eps)
    w = dout * _f(g)
    if kind == "layer":
        dx = inv * (w - w.mean(axis=1, keepdims=True) - u * (w * u).mean(axis=1, keepdims=True))
        return dx, (dout * u).sum(axis=0), dout.sum(axis=0)
    longer = np.sqrt((x * x).sum(axis=1, keepdims=True)) > eps
    dx = inv * (w - np.where(longer, u * (w * u).sum(axis=1, keepdims=True), 0.0))
    return dx, (dout * u).sum().reshape(1), None


def residual_norm_grad(dr, dn, r, y, post, post_g, post_b, gate, scale, norm, norm_g, norm_b,
                       eps):
    """Gradients of sum(dr r) + sum(dn n) at the stored r, as a dict."""
    like = _f(dr) if dr is not None else _f(dn)
    dh = np.zeros_like(like) if dr is None else _f(dr).copy()
    out = dict.fromkeys(("dh", "dy", "dgate", "dscale", "dpost_g", "dpost_b", "dnorm_g",
                         "dnorm_b"))
    if norm != "none":
        dx, out["dnorm_g"], out["dnorm_b"] = _norm_grad(_f(r), norm, norm_g, _f(dn), eps)
        dh = dh + dx
    out["dh"] = dh
    if y is None:
        return out
    k = np.ones(dh.shape[1]) if scale is None else _f(scale)
    g = 1.0 if gate is None else _f(gate)
    p = norm_rows(y, post, post_g, post_b, eps)[2]
    if gate is not None:
        out["dgate"] = dh * p * k
    if scale is not None:
        out["dscale"] = (dh * p * g).sum(axis=0)
    out["dy"], out["dpost_g"], out["dpost_b"] = _norm_grad(_f(y), post, post_g, dh * g * k, eps)
    return out


def xent(X, W, labels, reduction="mean", scale=1.0):
    """loss, lse [N], total and the gradients dX, dW of total; a label outside
    [0, V) leaves its row out of everything (whatever the row holds)."""
    X, W = _f(X).copy(), _f(W)
    labels = np.asarray(labels)
    live = (labels >= 0) & (labels < len(W))
    X[~live] = 0.0
    at = np.arange(len(X))
    y = np.where(live, labels, 0)
    logits = X @ W.T
    top = logits.max(axis=1)
    lse = top + np.log(np.exp(logits - top[:, None]).sum(axis=1))
    # lse - l_y as the logarithm of 1 + the others' share, which keeps the
    # digits of a small loss
    d = logits - logits[at, y][:, None]
    d[at, y] = -np.inf
    m = np.maximum(d.max(axis=1), 0.0)
    r = np.exp(d - m[:, None]).sum(axis=1)
    loss = np.where(live, np.where(m > 0, m + np.log(np.exp(-m) + r), np.log1p(r)), 0.0)
    n = max(int(live.sum()), 1) if reduction == "mean" else 1
    P = np.exp(logits - lse[:, None])
    # p - 1 at the label as minus the others' sum
    P[at, y] = 0.0
    P[at, y] = -P.sum(axis=1)
    P *= (live * scale / n)[:, None]
    return dict(loss=loss, lse=np.where(live, lse, 0.0), total=scale * loss.sum() / n,
                dX=P @ W, dW=P.T @ X)


def adamw(p, g, m, v, lr, beta1, beta2, eps, weight_decay, step, grad_scale=1.0):
    """(p, m, v) after one step, float64."""
    g = _f(g) * grad_scale
    m = beta1 * _f(m) + (1.0 - beta1) * g
    v = beta2 * _f(v) + (1.0 - beta2) * g * g
    den = np.sqrt(v / (1.0 - beta2 ** step)) + eps
    return (1.0 - lr * weight_decay) * _f(p) - lr / (1.0 - beta1 ** step) * m / den, m, v


# ---- 8-bit moments: fp32, one rounding at a time ---------------------------

_F = np.float32


def _blocks(x):
    x = np.asarray(x).reshape(-1)
    return np.pad(x, (0, -x.size % 256)).reshape(-1, 256)


def decode_moments(m, m_scale, v, v_scale):
    """fp32 (m, v) of the codes, flat."""
    out = []
    for c, s in ((m, m_scale), (v, v_scale)):
        n = np.asarray(c).size
        c = _blocks(c).astype(_F)
        out.append((c * np.abs(c) * np.asarray(s, _F)[:, None]).reshape(-1)[:n])
    return out[0], out[1] * out[1]


def encode_moments(x, top):
    """Codes (signed with top 127, at least 1 for what is not zero with top
    255) and scales of m (top 127) or sqrt(v) (top 255)."""
    n = np.asarray(x).size
    a = _blocks(np.asarray(x, _F))
    big = np.abs(a).max(axis=1, keepdims=True)
    live = big >= _F(2.0 ** -60)
    scale = np.where(live, big * _F(1.0 / (top * top)), _F(0))
    inv = np.where(live, (_F(1) / np.where(live, big, _F(1))) * _F(top * top), _F(0))
    c = np.minimum(np.rint(np.sqrt(np.abs(a) * inv)), _F(top))
    if top == 255:
        c = np.where((a > 0) & live & (c == 0), _F(1), c)
    c = (c * np.sign(a)).reshape(-1)[:n]
    return c.astype(np.uint8 if top == 255 else np.int8), scale.reshape(-1)


def adamw_codes(g, m, m_scale, v, v_scale, beta1, beta2, grad_scale=None):
    """(m codes, m scales, v codes, v scales) after one step, and the fresh
    fp32 moments that the update uses."""
    g = np.asarray(g, _F).reshape(-1)
    if grad_scale is not None:
        g = g * _F(grad_scale)
    m0, v0 = decode_moments(m, m_scale, v, v_scale)
    m1 = m0 * _F(beta1) + g * _F(1.0 - beta1)
    v1 = v0 * _F(beta2) + (g * _F(1.0 - beta2)) * g
    return encode_moments(m1, 127) + encode_moments(np.sqrt(v1), 255) + (m1, v1)
