"""fp64 oracle of the gated delta rule with one decay per token and head (TEST INFRASTRUCTURE ONLY): token by token,
from the definition, with the slot rules of the library's calls. Nothing here is shared with the CUDA path."""
from __future__ import annotations

import numpy as np

ERR_SLOT_RANGE, ERR_LENGTHS = 1, 16


def gate(raw_g, raw_beta, A_log, dt_bias):
    """alpha and beta [N, Hv]."""
    x = raw_g + (0.0 if dt_bias is None else dt_bias)
    return np.exp(-np.exp(A_log) * np.logaddexp(0.0, x)), np.exp(-np.logaddexp(0.0, -raw_beta))


def step(S, q, k, v, alpha, beta, scale, eps):
    """One token of one head: the new state [K, V] and o [V]."""
    q = scale * q / np.sqrt(q @ q + eps)
    k = k / np.sqrt(k @ k + eps)
    S = alpha * S
    S = S + np.outer(k, beta * (v - k @ S))
    return S, q @ S


def run(qkv, raw_g, raw_beta, A_log, dt_bias, pool, slots, bounds, Hk, scale=None, eps=1e-6, null_slot=-1, rows=None):
    """A call over entries with rows [bounds[e][0], bounds[e][1]) and slots[e]; all arguments fp64 arrays, pool [slots, Hv, K, V].
    Returns out [N, Hv * V] (NaN where no entry writes), the pool afterwards and the error bits."""
    n, Hv, K, V = pool.shape
    scale = K ** -0.5 if scale is None else scale
    rows = len(qkv) if rows is None else rows
    out, after, err = np.full((len(qkv), Hv * V), np.nan), pool.copy(), 0
    alpha, beta = gate(raw_g[:, :Hv], raw_beta[:, :Hv], A_log, dt_bias)
    for slot, (r0, r1) in zip(slots, bounds):
        if r0 < 0 or r1 < r0 or r1 > rows:
            err |= ERR_LENGTHS
            r1 = r0
        if slot >= n:
            err |= ERR_SLOT_RANGE
            if r1 > r0:
                out[r0:r1] = 0.0
            continue
        if r1 == r0:
            continue
        for h in range(Hv):
            hk = h // (Hv // Hk)
            S = pool[slot, h].copy() if slot >= 0 else np.zeros((K, V))
            for t in range(r0, r1):
                q, k = qkv[t, hk * K:(hk + 1) * K], qkv[t, (Hk + hk) * K:(Hk + hk + 1) * K]
                v = qkv[t, 2 * Hk * K + h * V:2 * Hk * K + (h + 1) * V]
                S, out[t, h * V:(h + 1) * V] = step(S, q, k, v, alpha[t, h], beta[t, h], scale, eps)
            if slot >= 0 and slot != null_slot:
                after[slot, h] = S
    return out, after, err
