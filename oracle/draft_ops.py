"""Plain numpy forms, in 64 bits, of the draft side's operators -- TEST INFRASTRUCTURE ONLY.

Beam selection and state reordering (include/spec_beam.h), distillation from a teacher's top
logits (include/spec_distill.h), row quantisation and the integer product (include/spec_int8.h),
written from the definitions in those headers. Only the test suite imports this module.
Pinned in tests/test_oracle_draft_ops.py: the selection by sorting Python tuples, the loss by
torch's log_softmax in float64, the gradient by autograd and by central differences, the
quantisation by exact fractions, the product by Python integers.
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
