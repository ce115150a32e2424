"""fp64 oracle of the calls that keep state: the paged key/value cache, attention
of new tokens over it, and linear attention with a decay per head.

TEST INFRASTRUCTURE, written from the definitions: a cache position is a table
lookup, attention is a softmax over the visible keys of one row at a time, the
decayed recurrence is stepped token by token.
"""
from __future__ import annotations

import math

import numpy as np

from .sparse_attention import E4M3_MAX, e4m3_round

CACHE_MAX = {"e4m3": E4M3_MAX, "int8": 127.0}


def cache_slot(table_row, page: int, pos: int, n_pages: int):
    """(page, slot) of a position, or None where it has none."""
    if pos < 0 or pos // page >= len(table_row):
        return None
    p = int(table_row[pos // page])
    return (p, pos % page) if 0 <= p < n_pages else None


def cache_encode(x, kind: str):
    """(codes as numbers, scale) of one row x [d]: with a = max(amax, M 2^-126),
    a / M and M / a are fp32 numbers, the product with the latter is rounded to fp32 and then to the kind
    (ties to even)."""
    M = np.float32(CACHE_MAX[kind])
    x32 = np.asarray(x, dtype=np.float32)
    amax = np.float32(np.abs(x32).max())
    if amax == 0:
        return np.zeros(x32.shape), 1.0
    a = max(amax, M * np.float32(2.0 ** -126))
    y = (x32 * np.float32(M / a)).astype(np.float64)
    codes = np.clip(np.rint(y), -127, 127) if kind == "int8" else e4m3_round(y)
    return codes, float(np.float32(a / M))


def cache_attention(q, k, v, n_visible, scale=None):
    """(o [G, d], lse [G]) of one token's query heads q [G, d] that share the keys
    and values k, v [L, d], of which the first n_visible are seen."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    scale = 1.0 / math.sqrt(q.shape[1]) if scale is None else scale
    n = min(max(int(n_visible), 0), k.shape[0])
    if n == 0:
        return np.zeros_like(q), np.full(q.shape[0], -np.inf)
    s = scale * (q @ k[:n].T)
    m = s.max(axis=1, keepdims=True)
    p = np.exp(s - m)
    l = p.sum(axis=1, keepdims=True)
    return (p @ v[:n]) / l, (m + np.log(l))[:, 0]


def decay_attention(q, k, v, log_decay, scale, state=None):
    """(o [N, d], S) with S_t = e^log_decay S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t."""
    N, d = q.shape
    S = np.zeros((d, d)) if state is None else np.array(state, dtype=np.float64)
    w = math.exp(log_decay)
    o = np.zeros((N, d))
    for t in range(N):
        S = w * S + np.outer(k[t], v[t])
        o[t] = scale * (S.T @ q[t])
    return o, S


def decay_attention_bwd(q, k, v, log_decay, scale, dout, state=None, dstate=None):
    """(dq, dk, dv, dstate_in): the chain rule through decay_attention, step by step."""
    N, d = q.shape
    w = math.exp(log_decay)
    S = np.zeros((d, d)) if state is None else np.array(state, dtype=np.float64)
    dq, dk, dv = np.zeros((N, d)), np.zeros((N, d)), np.zeros((N, d))
    for t in range(N):
        S = w * S + np.outer(k[t], v[t])
        dq[t] = scale * (S @ dout[t])
    E = np.zeros((d, d)) if dstate is None else np.array(dstate, dtype=np.float64)   # dL/dS_t
    for t in range(N - 1, -1, -1):
        E = E + scale * np.outer(q[t], dout[t])
        dk[t] = E @ v[t]
        dv[t] = E.T @ k[t]
        E = w * E
    return dq, dk, dv, E
