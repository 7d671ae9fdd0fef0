"""CPU oracle of the operators of a language model on the layer (TEST
INFRASTRUCTURE ONLY: the same import rule as ``oracle.flash_gau``): the
relative position table by buckets of distance, 8-bit activation checkpoints,
and sampling.  Whole numbers where a definition turns on a border, float64
elsewhere; written from the formulas.

  bucket(t) = t below near, else min(n - 1, near +
              floor(log(t / near) / log(far / near) (n - near))),  near = n // 2
  scale = max |x| * (1 / 127) of 128 neighbours, fp32; code = x / scale to the nearest
  w_i = exp((l_i - max l) / T), falling, ties by index; top-k, top-p, min-p each
  keep a beginning; the first kept word past u of the kept mass
"""

import numpy as np

__all__ = ["buckets_of_offsets", "bucket_bias", "bucket_bias_grad", "checkpoint_codes",
           "checkpoint_values", "sample_row"]

GROUP = 128


def _bucket(t, n, far):
    """Bucket of distance t among n of a direction, by whole numbers: it is
    near + j or above when t^m near^j >= far^j near^m, m = n - near."""
    near = n // 2
    if t < near:
        return t
    m = n - near
    j = 0
    while j + 1 < m and t ** m * near ** (j + 1) >= far ** (j + 1) * near ** m:
        j += 1
    return near + j


def buckets_of_offsets(C, buckets, far, causal):
    """Buckets of the offsets -(C-1) .. C-1 of a key from its query."""
    n = buckets if causal else buckets // 2
    past = [_bucket(t, n, far) for t in range(C)]
    ahead = [past[0]] * (C - 1) if causal else [n + past[t] for t in range(1, C)]
    return np.array(past[::-1] + ahead)


def bucket_bias(table, C, far, causal):
    """[H, 2C-1] of values [H, buckets]."""
    table = np.asarray(table, dtype=np.float64)
    return table[:, buckets_of_offsets(C, table.shape[1], far, causal)]


def bucket_bias_grad(drelpos, buckets, far, causal):
    """[H, buckets] of gradients [R, H, 2C-1]."""
    d = np.asarray(drelpos, dtype=np.float64).sum(axis=0)
    at = buckets_of_offsets((d.shape[1] + 1) // 2, buckets, far, causal)
    out = np.zeros((len(d), buckets))
    for k, b in enumerate(at):
        out[:, b] += d[:, k]
    return out


def _groups(d):
    return [slice(c, min(c + GROUP, d)) for c in range(0, d, GROUP)]


def checkpoint_codes(x):
    """(codes int8, scales fp32) of rows x whose values fp32 holds.  The
    quotient is taken in float64: of two fp32 numbers, it is off a half by more
    than float64's rounding wherever it is not a half."""
    x = np.asarray(x, dtype=np.float64)
    M, d = x.shape
    codes = np.zeros((M, d), np.int8)
    scales = np.zeros((M, -(-d // GROUP)), np.float32)
    with np.errstate(invalid="ignore"):
        for k, c in enumerate(_groups(d)):
            top = np.abs(x[:, c]).max(axis=1).astype(np.float32)
            s = np.where(top < np.float32(2.0 ** -100), np.float32(0), top * (np.float32(1) / np.float32(127)))
            scales[:, k] = s
            fine = (s > 0) & np.isfinite(s)
            q = x[:, c] / np.where(fine, s, 1).astype(np.float64)[:, None]
            codes[:, c] = np.where(fine[:, None], np.rint(np.where(fine[:, None], q, 0)), 0)
    return codes, scales


def checkpoint_values(codes, scales):
    """code * scale, one rounding to fp32 each."""
    d = np.asarray(codes).shape[1]
    s = np.repeat(np.asarray(scales, np.float32), GROUP, axis=1)[:, :d]
    with np.errstate(invalid="ignore"):
        return (np.asarray(codes).astype(np.float32) * s).astype(np.float64)


def sample_row(l, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logp, kept) of one row of logits."""
    l = np.asarray(l, dtype=np.float64)
    given = np.array([u, temperature, top_p, min_p], dtype=np.float64)
    if (np.isnan(l).any() or (l == np.inf).any() or not np.isfinite(l).any() or
            np.isnan(given).any() or temperature < 0 or u < 0):
        return -1, np.nan, 0
    words = np.argsort(-l, kind="stable")
    words = words[l[words] > -np.inf]
    if temperature < 1e-30:
        return int(words[0]), 0.0, 1
    w = np.exp((l[words] - l[words[0]]) / np.float64(temperature))
    n = len(words)
    if top_k > 0:
        n = min(n, int(top_k))
    kept = n
    if top_p < 1:
        share, before, kept = np.float64(top_p) * w[:n].sum(), 0.0, 0
        while kept < n and (kept == 0 or before < share):
            before += w[kept]
            kept += 1
    if min_p > 0:
        kept = min(kept, max(1, int((w >= np.float64(min_p)).sum())))
    end = np.cumsum(w[:kept])
    j = int((end <= min(np.float64(u), 1 - 2.0 ** -24) * end[-1]).sum())
    j = min(j, kept - 1)
    return int(words[j]), float(np.log(w[j] / end[-1])), kept
