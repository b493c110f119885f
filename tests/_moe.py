"""The routed expert layer's operators in plain 64-bit numpy, and their error bounds.

Bounds.  U32 = 2^-24 is half a step of fp32 (relative), U16 = 2^-8 of bf16, U8 = 2^-4 of E4M3; below
E4M3's normal numbers half a step is 2^-10 in units of the group's scale.

ELEM = 2^-18 bounds the relative error of one elementary fp32 value here (a weight, silu(g) u, ...):
an exponential evaluated as 2^(x log2 e) has an argument off by |x| U32 |log2 e| and 2 steps of its own, so
for |x| <= 24 it is off by at most 24 * 2^-24 * 1.45 + 2^-22 < 2^-18.5; a reciprocal, a sum of
positive terms (pairwise over <= 1024, 10 U32) and the four products around it add less than 20 U32 < 2^-19.
"""
from __future__ import annotations

import math

import numpy as np

import oracle

U32, U16, U8, ELEM = 2.0 ** -24, 2.0 ** -8, 2.0 ** -4, 2.0 ** -18


# -- routing ------------------------------------------------------------------------------------ #

def scores(l, score):
    """Scores of one token's logits in binary64, and which experts are masked by their logit."""
    with np.errstate(invalid="ignore", over="ignore"):
        masked = ~(np.isfinite(l))
        if score == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-l))
        else:
            top = l[~masked].max() if (~masked).any() else 0.0
            s = np.exp(l - top)
            s = s / max(s[~masked].sum(), 1e-300)
    return np.where(masked, 0.0, s), masked


def route(logits, k, bias=None, score="sigmoid", n_group=1, topk_group=1, renormalize=True, scale=1.0):
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    idx, w = np.zeros((T, k), np.int32), np.zeros((T, k))
    per = E // n_group
    for t in range(T):
        l = logits[t]
        s, masked = scores(l, score)
        bad = np.isnan(l).any() or (l == np.inf).any()
        if bias is None:
            key = np.where(masked, -np.inf, l)
        else:
            b = np.asarray(bias, dtype=np.float64)
            bad = bad or np.isnan(b).any() or (b == np.inf).any()
            masked = masked | ~np.isfinite(b)
            key = np.where(masked, -np.inf, s + np.where(np.isfinite(b), b, 0.0))
        group = []
        for g in range(n_group):
            best = sorted((v for v in key[g * per:(g + 1) * per] if v > -np.inf), reverse=True)
            best = best[:2] if bias is not None else best[:1]
            group.append(sum(best) if best else -np.inf)
        kept = set(sorted(range(n_group), key=lambda g: (-group[g], g))[:topk_group])
        order = sorted((e for e in range(E) if e // per in kept), key=lambda e: (-key[e], e))[:k]
        idx[t] = order
        w[t] = weights_of(l, order, masked, s, score, renormalize, scale)
        if bad:
            w[t] = np.nan
    return idx, w


def weights_of(l, order, masked, s, score, renormalize, scale):
    order = np.asarray(order)
    live = ~masked[order]
    if not renormalize:
        return scale * np.where(live, s[order], 0.0)
    if not live.any():
        return np.zeros(len(order))
    x = np.where(live, l[order], -np.inf)
    if score == "softmax":
        p = np.exp(x - x.max())
    else:   # log sigmoid(x) = -log(1 + e^-x), which does not underflow
        ls = -np.logaddexp(0.0, -x)
        p = np.exp(ls - ls.max())
    return scale * p / p.sum()


def route_backward(dw, idx, logits, score="sigmoid", renormalize=True, scale=1.0):
    """dlogits of L = sum dw * w with the choice held fixed, and sum of the magnitudes of its terms."""
    logits = np.asarray(logits, dtype=np.float64)
    out, mag = np.zeros_like(logits), np.zeros_like(logits)
    for t in range(logits.shape[0]):
        l, e, g = logits[t], idx[t], np.asarray(dw[t], dtype=np.float64)
        s, masked = scores(l, score)
        w = weights_of(l, e, masked, s, score, renormalize, scale)
        g = np.where(w == 0, 0.0, g)
        p = w / scale
        a = np.abs(w * g)
        if renormalize:
            d = w * (p[None, :] * (g[:, None] - g[None, :])).sum(1)   # sum p = 1: no cancellation
            a = np.abs(w) * (np.abs(p)[None, :] * np.abs(g[:, None] - g[None, :])).sum(1)
        else:
            d = w * g
        if score == "sigmoid":
            c = np.exp(-np.logaddexp(0.0, np.where(masked[e], 0.0, l[e])))   # 1 - s, which must not be formed by cancellation
            np.add.at(out[t], e, d * c)
            np.add.at(mag[t], e, a * c)
        else:
            np.add.at(out[t], e, d)
            np.add.at(mag[t], e, a)
            if not renormalize:
                out[t] -= s * d.sum()
                mag[t] += s * np.abs(d).sum()
    return out, mag


# -- plan, quantised groups ------------------------------------------------------------------------ #

def plan(idx, E):
    flat = np.asarray(idx).reshape(-1)
    slots = np.argsort(flat, kind="stable").astype(np.int32)
    rows = np.empty_like(slots)
    rows[slots] = np.arange(flat.size, dtype=np.int32)
    offsets = np.searchsorted(flat[slots], np.arange(E + 1)).astype(np.int32)
    return offsets, slots, rows.reshape(np.asarray(idx).shape)


def quant_groups(v):
    """v[..., 128] float32 -> codes and scales, bit by bit as the quantisers' definition."""
    v = np.asarray(v, dtype=np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        a = np.maximum(np.fmax.reduce(np.abs(v), axis=-1), np.float32(2.0 ** -100)).astype(np.float32)
        s = (a / np.float32(448)).astype(np.float32)
        inv = (np.float32(448) / a).astype(np.float32)
        codes = oracle.e4m3_encode((v * inv[..., None]).astype(np.float32).reshape(-1)).reshape(v.shape)
    return codes, s


def quant_rows(v):
    M, C = v.shape
    q, s = quant_groups(v.reshape(M, C // 128, 128))
    return q.reshape(M, C), np.ascontiguousarray(s.T)


def padded_rows(v, offsets):
    """Each expert's rows padded with zeros to whole groups, one after another."""
    parts = [np.zeros((0, v.shape[1]), v.dtype)]
    for lo, hi in zip(offsets[:-1], offsets[1:]):
        parts += [v[lo:hi], np.zeros((-(hi - lo) % 128, v.shape[1]), v.dtype)]
    return np.concatenate(parts)


def quant_cols(v, offsets):
    """Codes [C, 128 P], scales [P, C]."""
    p = padded_rows(v, offsets)
    G = p.shape[0] // 128
    q, s = quant_groups(p.reshape(G, 128, -1).transpose(0, 2, 1))
    return np.ascontiguousarray(q.transpose(1, 0, 2).reshape(v.shape[1], G * 128)), s


def decode_rows(q, s):
    return oracle.e4m3_decode(q.reshape(-1)).reshape(q.shape).astype(np.float64) * \
        np.repeat(s.T.astype(np.float64), 128, axis=1)


def decode_cols(q, s):
    return oracle.e4m3_decode(q.reshape(-1)).reshape(q.shape).astype(np.float64) * \
        np.repeat(s.astype(np.float64), 128, axis=0).T


def check_quantised(q, s, ref, err, rows=True, what=""):
    """Codes and scales of values known to `err` each: `ref` and `err` are [M, C] (rows) or the padded,
    transposed [C, K] (columns), in binary64.  The scale is within the group's largest err of
    amax / 448 (and one rounding), a decoded code within half a step of its value."""
    r = ref.reshape(ref.shape[0], -1, 128)
    e = np.broadcast_to(err, ref.shape).reshape(r.shape)
    amax = np.maximum(np.abs(r).max(-1), 2.0 ** -100)
    want = (amax / 448.0).T                                        # [groups, M]
    slack = (e.max(-1) / 448.0).T + 2 * U32 * want
    off = np.abs(s.astype(np.float64) - want)
    assert (off <= slack).all(), f"{what}: scale off by {off.max()} ({(off > slack).sum()} of {off.size})"
    got = decode_rows(q, s)
    tol = U8 * (1 + 2.0 ** -10) * np.abs(ref) + 2.0 ** -10 * np.repeat(s.T.astype(np.float64), 128, axis=1) + \
        2 * np.broadcast_to(err, ref.shape) + 4 * U32 * np.repeat(amax, 128, axis=1)
    bad = np.abs(got - ref) > tol
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} codes further than half a step off"


# -- SwiGLU ---------------------------------------------------------------------------------------- #

def sigmoid(x):
    return np.exp(-np.logaddexp(0.0, -x))


def swiglu(h):
    I = h.shape[1] // 2
    g, u = h[:, :I].astype(np.float64), h[:, I:].astype(np.float64)
    return g * sigmoid(g) * u


def swiglu_backward(da, g, u):
    """(dg, du, a) and the bounds of their fp32 evaluation."""
    r = sigmoid(g)
    a = g * r
    dg = da * u * (r + a * (1 - r))
    du = da * a
    return (dg, du, a * u), (ELEM * np.abs(da * u) * (r + np.abs(a) * (1 - r)) + 1e-37, ELEM * np.abs(du) + 1e-37,
                             ELEM * np.abs(a * u) + 1e-37)


# -- small helpers ----------------------------------------------------------------------------------- #

def capacity(M, E):
    return 128 * (math.ceil(M / 128) + E)


def distinct(rng, T, k, E):
    return np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32) if T else np.zeros((0, k), np.int32)
