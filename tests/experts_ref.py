"""Plain restatements, in 64 bits on the CPU, of the operators around products
over experts. They hold none of the library's code. The 8-bit quantiser alone
is restated in 32 bits, because its rounding is part of its definition."""

from __future__ import annotations

import numpy as np
import torch

BLOCK = 128
LEAST = 2.0 ** -96


def up(x, m):
    return (x + m - 1) // m * m


def inverse(a):
    """448 / a, rounded once (a number divided by a tensor would be its reciprocal times the number, rounded twice)."""
    return torch.div(torch.full_like(a, 448.0), a)


def quantize(x, axis):
    """x (rows x cols, float32 tensor) with a scale per 128 along `axis` (0 or 1) or per 128 x 128 block (None):
    (float8 tensor, scales [row blocks or rows, column blocks or columns])."""
    rows, cols = x.shape
    br, bc = (BLOCK if axis in (0, None) else 1), (BLOCK if axis in (1, None) else 1)
    q = torch.zeros(rows, cols, dtype=torch.float8_e4m3fn)
    s = torch.zeros(-(-rows // br), -(-cols // bc))
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            b = x[i * br:(i + 1) * br, j * bc:(j + 1) * bc]
            a = torch.clamp(b.abs().max(), min=LEAST)
            s[i, j] = a / 448.0
            q[i * br:(i + 1) * br, j * bc:(j + 1) * bc] = (b * inverse(a)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q, s


def quantize_rows_fast(x):
    rows, cols = x.shape
    full = torch.zeros(rows, up(cols, BLOCK))
    full[:, :cols] = x
    b = full.view(rows, -1, BLOCK)
    a = b.abs().amax(2, keepdim=True).clamp(min=LEAST)
    q = (b * inverse(a)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(rows, -1)[:, :cols]
    return q.contiguous(), (a / 448.0)[:, :, 0].contiguous()


def wide_rows(q, s):
    """float64 values of q (rows x K) with scales s (K blocks x rows)."""
    return q.double() * s.double().t().repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def wide_blocks(q, s):
    return q.double() * s.double().repeat_interleave(BLOCK, 0)[:q.shape[0]].repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def product(a, b):
    """(a . b^T, sum |a b|) of float64 matrices."""
    return a @ b.t(), a.abs() @ b.abs().t()


def product_tolerance(nk):
    """Relative to sum |a b|. Products of two e4m3 values are exact in FP32. Within a block at most 128 additions,
    each allowed a truncation to 24 bits (2^-23); across nk blocks one multiply of the scales, one multiply and one
    addition each, rounded (2^-24)."""
    return BLOCK * 2.0 ** -23 + (nk + 3) * 2.0 ** -24


def scores(l, kind):
    """float64 scores of a row of logits; ineligible ones 0."""
    ok = l > -np.inf
    s = np.zeros(l.shape)
    if kind == "sigmoid":
        s[ok] = 1.0 / (1.0 + np.exp(-l[ok]))
    elif ok.any():
        m = l[ok].max()
        e = np.where(l[ok] == m, 1.0, np.exp(l[ok] - m)) if np.isinf(m) else np.exp(l[ok] - m)
        s[ok] = e / e.sum()
    return s


def route(logits, bias, kind, groups, kept, two, k, renorm, scale):
    """Token by token; the choice by falling keys, ties to the lowest expert."""
    T, E = logits.shape
    W, I = np.zeros((T, k)), np.full((T, k), -1)
    for t in range(T):
        l = logits[t].astype(np.float64)
        s = scores(l, kind)
        key = np.where(l > -np.inf, l, -np.inf)
        if bias is not None or two:
            key = np.where(l > -np.inf, s + (bias if bias is not None else 0.0), -np.inf)
        key = np.where(np.isnan(key), -np.inf, key)
        if kept < groups:
            g = np.sort(key.reshape(groups, -1), 1)[:, ::-1]
            rank = g[:, 0] + g[:, 1] if two else g[:, 0]
            keep = np.argsort(-rank, kind="stable")[:kept]
            mask = np.zeros(groups, bool)
            mask[keep] = True
            key = np.where(np.repeat(mask, E // groups), key, -np.inf)
        order = np.argsort(-key, kind="stable")[:k]
        order = [e for e in order if key[e] > -np.inf]
        w = s[order]
        if renorm:
            w = w / w.sum() if w.sum() > 0 else np.zeros_like(w)
        W[t, :len(order)], I[t, :len(order)] = scale * w, order
    return W, I


def dispatch(indices, E):
    T, k = indices.shape
    flat = indices.reshape(-1)
    ok = (flat >= 0) & (flat < E)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[ok], minlength=E)[:E])])
    order = np.flatnonzero(ok)[np.argsort(flat[ok], kind="stable")]
    row_of, token_of = np.full(T * k, -1), np.full(T * k, -1)
    row_of[order] = np.arange(len(order))
    token_of[:len(order)] = order // k
    return offsets, row_of.reshape(T, k), token_of
