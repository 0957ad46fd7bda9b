"""Plain numpy forms, in 64 bits, of the draft side's operators -- TEST INFRASTRUCTURE ONLY.

Beam selection and state reordering (include/spec_beam.h), distillation from a teacher's top
logits (include/spec_distill.h), row quantisation and the integer product (include/spec_int8.h),
their 4-bit counterparts (include/spec_mxfp4.h), scores of given tokens and their gradient
(include/spec_logprobs.h), written from the definitions in those headers. Only the test suite imports this module.
Pinned in tests/test_oracle_draft_ops.py: the selection by sorting Python tuples, the loss by
torch's log_softmax in float64, the gradient by autograd and by central differences, the
quantisation by exact fractions, the product by Python integers; the 4-bit forms and the scores in
tests/test_oracle_scores.py, by a table's nearest entry, exact fractions, Python sorting, torch's
log_softmax and autograd in float64, and central differences; the gradient at masked entries in
tests/test_oracle_scores_masked.py.
"""
from __future__ import annotations

import numpy as np


def row_parts(x):
    """The largest entry M of the last axis (0 where it is not finite) and log sum exp(x - M)."""
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore", divide="ignore"):
        m = x.max(-1, keepdims=True)
        safe = np.where(np.isfinite(m), m, 0.0)
        return safe[..., 0], np.log(np.exp(x - safe).sum(-1, keepdims=True))[..., 0]


def row_lse(x):
    """log sum exp over the last axis, float64."""
    m, log_s = row_parts(x)
    return m + log_s


def beam_select(logits, score, lse, keep):
    """logits [B, W, V] (float32 values), score [B, W] float32, lse [B, W] float64 or None.
    Returns parent, token [B, K] int32 and value, logq [B, K] float64."""
    z = np.asarray(logits, np.float32)
    B, W, V = z.shape
    top = np.zeros((B, W))
    if lse is None:
        lse = row_lse(z)
        m, log_s = row_parts(z)
        far = np.isfinite(lse) & (np.abs(lse) > 2.0 ** 22)
        top, lse = np.where(far, m, 0.0), np.where(far, log_s, lse)
    parent = np.full((B, keep), -1, np.int32)
    token = np.full((B, keep), -1, np.int32)
    value = np.full((B, keep), -np.inf)
    logq = np.full((B, keep), -np.inf)
    for b in range(B):
        alive = np.isfinite(score[b]) & np.isfinite(lse[b])
        ok = np.isfinite(z[b]) & alive[:, None]
        w, v = np.nonzero(ok)
        q = (z[b, w, v].astype(np.float64) - top[b, w]) - lse[b, w]
        val = score[b, w].astype(np.float64) + q
        order = np.lexsort((v, -z[b, w, v], w, -val))[:keep]
        n = order.size
        parent[b, :n], token[b, :n] = w[order], v[order]
        value[b, :n], logq[b, :n] = val[order], q[order]
    return parent, token, value, logq


def beam_reorder(parent, src, dst):
    """src [L, B, W, ...], dst [L, B, K, ...] (copied), parent [B, K]."""
    out = np.array(dst, copy=True)
    old = np.array(src, copy=True)
    B, K = parent.shape
    for b in range(B):
        for j in range(K):
            if 0 <= parent[b, j] < src.shape[2]:
                out[:, b, j] = old[:, b, parent[b, j]]
    return out


def distill_scaled(x, ids, y, teacher_lse, weight, r):
    """Loss [N], lse [N] and gradient [N, V] of rows with scaled logits x [N, V] and scaled
    teacher logits y [N, K] (float64), r [N] the scale the gradient carries. Valid rows only."""
    x = np.asarray(x, np.float64)
    N, V = x.shape
    lse = row_lse(x)
    top, log_s = row_parts(x)
    loss, grad = np.zeros(N), np.zeros((N, V))
    for n in range(N):
        j = np.nonzero(ids[n] >= 0)[0]
        if j.size == 0 or (teacher_lse is None and np.all(np.isneginf(y[n, j]))):
            lse[n] = np.nan
            continue
        lt = row_lse(y[n, j]) if teacher_lse is None else teacher_lse[n]
        logp = y[n, j].astype(np.float64) - lt
        p = np.exp(logp)
        with np.errstate(invalid="ignore"):
            terms = np.where(p > 0, p * (logp - ((x[n, ids[n, j]] - top[n]) - log_s[n])), 0.0)
        loss[n] = terms.sum()
        g = p.sum() * np.exp((x[n] - top[n]) - log_s[n])
        np.add.at(g, ids[n, j], -p)
        grad[n] = weight[n] * r[n] * g
    return loss, lse, grad


def distill(z, ids, teacher, teacher_lse, temperature, weight):
    """The header's definition, its sentinels included: z [N, V] and teacher [N, K] float32
    values. Returns loss, lse [N] and grad [N, V] in float64."""
    z = np.asarray(z, np.float32)
    N, V = z.shape
    t = np.asarray(temperature, np.float32)
    with np.errstate(all="ignore"):
        r = np.float32(1.0) / t
        ok = (t > 0) & np.isfinite(t) & np.isfinite(r)
        rs = np.where(ok, r, np.float32(1.0)).astype(np.float32)
        x = (z * rs[:, None]).astype(np.float32)
        y = (np.asarray(teacher, np.float32) * rs[:, None]).astype(np.float32)
    used = ids >= 0
    out = (ids >= V).any(1)
    safe = np.where(out[:, None], -1, ids)
    with np.errstate(all="ignore"):
        loss, lse, grad = distill_scaled(x, safe, y, teacher_lse, weight, rs.astype(np.float64))
        lt = row_lse(np.where(used, y, -np.inf)) if teacher_lse is None else teacher_lse
    massless = (teacher_lse is None) & np.all(~used | np.isneginf(y), 1) & ok & ~out
    empty = ~used.any(1) | massless
    bad = ~empty & (~ok | out | ~np.isfinite(lse) | ~np.isfinite(lt))
    loss[empty], lse[empty], grad[empty] = 0.0, np.nan, 0.0
    loss[bad], lse[bad], grad[bad] = np.nan, np.nan, np.nan
    return loss, lse, grad


def quantize_rows(x):
    """x [N, D] float32 values: (q int8, scale float32)."""
    x = np.asarray(x, np.float32)
    wild = ~np.isfinite(x).all(1)
    m = np.where(wild[:, None], np.float32(0), np.abs(x)).max(1).astype(np.float32)
    scale = (m / np.float32(127.0)).astype(np.float32)
    d = np.where(scale > 0, scale, np.float32(1.0)).astype(np.float64)
    # x / scale has at most 24 by 24 bits: the float64 quotient is nearer to the exact one than
    # any tie that is not one itself, and exact ties are representable
    q = np.rint(np.where(wild[:, None], 0.0, x.astype(np.float64)) / d[:, None])
    q = np.clip(q, -127, 127)
    q[~(scale > 0)] = 0
    return q.astype(np.int8), np.where(wild, np.float32(np.nan), scale).astype(np.float32)


def int8_product(a, a_scale, w, w_scale):
    """out [N, V] float32, in the header's order of roundings."""
    # float64 products of 8-bit values are exact far beyond the sums here
    acc = a.astype(np.float64) @ w.astype(np.float64).T
    f = acc.astype(np.float32)
    with np.errstate(all="ignore"):
        return (f * a_scale[:, None].astype(np.float32)) * w_scale[None, :].astype(np.float32)


MXFP4_LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def mxfp4_quantize(x):
    """x [N, D] float32 values: codes [N, D' / 2] uint8, scales [N, D' / 32] uint8, values
    [N, D] float64."""
    x = np.asarray(x, np.float32).astype(np.float64)
    N, D = x.shape
    whole = (D + 127) // 128 * 128
    y = np.zeros((N, whole))
    y[:, :D] = x
    y = y.reshape(N, -1, 32)
    wild = ~np.isfinite(y).all(2)
    y = np.where(wild[..., None], 0.0, y)
    top = np.abs(y).max(2)
    e = np.maximum(np.frexp(top)[1] - 1 - 2, -127)
    e = np.where(top == 0, -127, e)
    mag = np.ldexp(np.abs(y), -e[..., None])
    # the step of the representable values around mag; ties to even of mag / step are ties to the
    # even code (each octave holds two codes, the even one first)
    step = np.where(mag < 2, 0.5, np.where(mag < 4, 1.0, 2.0))
    level = np.minimum(np.rint(mag / step) * step, 6.0)
    code = np.searchsorted(MXFP4_LEVELS, level).astype(np.uint8)
    code = (code + 8 * np.signbit(y)).astype(np.uint8)
    code[wild] = 0
    values = np.where(wild[..., None], np.nan, np.ldexp(np.copysign(level, y), e[..., None]))
    code = code.reshape(N, whole)
    scale = np.where(wild, 255, e + 127).astype(np.uint8)
    return code[:, 0::2] | code[:, 1::2] << 4, scale, values.reshape(N, whole)[:, :D]


def mxfp4_values(q, scale):
    """What codes [N, D' / 2] with scales [N, D' / 32] stand for, float64 [N, D']."""
    code = np.stack((q & 15, q >> 4), 2).reshape(q.shape[0], -1, 32).astype(np.int64)
    v = MXFP4_LEVELS[code & 7] * np.where(code & 8, -1.0, 1.0)
    v = np.ldexp(v, scale.astype(np.int64)[..., None] - 127)
    return np.where((scale == 255)[..., None], np.nan, v).reshape(q.shape[0], -1)


def mxfp4_product(q, scale, wq, w_scale):
    """The exact product rounded to float64, and sum_k |a w|."""
    a, w = mxfp4_values(q, scale), mxfp4_values(wq, w_scale)
    with np.errstate(invalid="ignore"):
        return a @ w.T, np.abs(a) @ np.abs(w).T


def score_scaled(z, temperature):
    """x [N, V] float32 = fl32(z fl32(1/T)) (NaN rows of bad temperatures) and r [N] float32."""
    z = np.asarray(z, np.float32)
    if temperature is None:
        r = np.ones(z.shape[0], np.float32)
    else:
        t = np.asarray(temperature, np.float32)
        with np.errstate(all="ignore"):
            r = (np.float32(1.0) / t).astype(np.float32)
            r = np.where((t > 0) & np.isfinite(t) & np.isfinite(r), r, np.float32(np.nan)).astype(np.float32)
    with np.errstate(all="ignore"):
        return (z * r[:, None]).astype(np.float32), r


def token_scores(z, token, temperature, keep):
    """z [N, V] float32 values, token [N], temperature [N] float32 or None. Returns a dict of
    logprob, entropy [N], norm [N, 2], top_logprob [N, K] float64, rank [N], top_token [N, K] int32."""
    z = np.asarray(z, np.float32)
    x, _ = score_scaled(z, temperature)
    N, V = z.shape
    out = dict(logprob=np.zeros(N), rank=np.full(N, -1, np.int32), entropy=np.zeros(N),
               norm=np.zeros((N, 2)), top_token=np.full((N, keep), -1, np.int32),
               top_logprob=np.full((N, keep), -np.inf))
    for n in range(N):
        xn, t = x[n].astype(np.float64), int(token[n])
        m = xn.max()
        if np.isnan(xn).any() or m == np.inf:
            for k in ("logprob", "entropy", "norm", "top_logprob"):
                out[k][n] = np.nan
            continue
        if m == -np.inf:
            out["norm"][n] = (m, 0.0)
            out["logprob"][n] = 0.0 if t < 0 else np.nan if t >= V else -np.inf
            continue
        d = xn - m
        e = np.exp(d)
        log_s = np.log(e.sum())
        out["norm"][n] = (m, log_s)
        out["entropy"][n] = log_s - (e * np.where(e > 0, d, 0.0)).sum() / e.sum()
        order = np.argsort(-z[n], kind="stable")
        if t >= V:
            out["logprob"][n] = np.nan
        elif t >= 0:
            out["logprob"][n] = d[t] - log_s
            out["rank"][n] = np.nonzero(order == t)[0][0]
        top = order[:keep]
        top = top[xn[top] > -np.inf]
        out["top_token"][n, :top.size] = top
        out["top_logprob"][n, :top.size] = d[top] - log_s
    return out


def score_parts(x):
    """log p [N, V] and entropy [N] of finite-topped rows x [N, V], float64."""
    x = np.asarray(x, np.float64)
    m, log_s = row_parts(x)
    l = (x - m[:, None]) - log_s[:, None]
    p = np.exp(l)
    return l, p, -(p * np.where(p > 0, l, 0.0)).sum(1)


def score_grad_scaled(x, token, a, b, r):
    """Gradient of sum_n (a logprob + b entropy) for z with x = r z: valid rows only."""
    l, p, h = score_parts(x)
    a = np.where(token >= 0, a, 0.0)
    with np.errstate(invalid="ignore"):
        g = -p * (a[:, None] + b[:, None] * (np.where(p > 0, l, 0.0) + h[:, None]))
    g[np.isneginf(x)] = 0.0   # whatever the weights
    at = np.nonzero(token >= 0)[0]
    g[at, token[at]] += a[at]
    return g * r[:, None]


def token_scores_grad(z, token, temperature, a, b):
    """The header's definition, its sentinels included: float64 [N, V]."""
    z = np.asarray(z, np.float32)
    N, V = z.shape
    x, r = score_scaled(z, temperature)
    with np.errstate(all="ignore"):
        m = x.max(1)
        bad = np.isnan(x).any(1) | (m == np.inf) | (token >= V) | ~np.isfinite(r)
        empty = ~bad & (m == -np.inf)
        safe = np.where((bad | empty)[:, None], np.float32(0), x)
        g = score_grad_scaled(safe, np.where(token >= V, -1, token), np.asarray(a, np.float64),
                              np.zeros(N) if b is None else np.asarray(b, np.float64),
                              np.where(np.isfinite(r), r, 1.0).astype(np.float64))
    g[empty] = 0.0
    g[bad] = np.nan
    return g
