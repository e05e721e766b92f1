"""Eviction by accumulated weight, one sequence and head at a time in plain
Python, from its definition.  Test infrastructure only."""
import math

import numpy as np


def kept_positions(weights, budget, sink, recent):
    """Former position of each position after eviction, for the weights of one
    sequence's tokens (a list) and one head."""
    L = len(weights)
    if L <= budget:
        return list(range(L))
    heavy = budget - recent
    low = [-math.inf if math.isnan(w) else w for w in weights]
    # NaN comes after -inf, and among equal weights the lower position wins
    order = sorted(range(sink, L - recent), key=lambda t: (math.isnan(weights[t]), -low[t], t))
    keep = set(range(sink)) | set(order[:heavy - sink])
    out = [t if t in keep else None for t in range(heavy)]
    behind = sorted(t for t in keep if t >= heavy)
    for j in range(heavy):
        if out[j] is None:
            out[j] = behind.pop(0)
    assert not behind
    return out + list(range(L - recent, L))


def evict(pools, weights, tables, lens, budget, sink, recent, bs, move, new_tables=None):
    """(pools, weights, new lengths, kept) after the call.  pools: arrays
    [NB, bs, Hkv, ...] whose last axes are a row; weights [NB, Hkv, bs]."""
    B, Hkv = len(lens), weights.shape[1]
    before = [p.copy() for p in pools], weights.copy()
    pools, weights = [p.copy() for p in pools], weights.copy()
    kept = np.full((B, Hkv, budget), -1, np.int32)
    dst = tables if new_tables is None else new_tables
    for i, L in enumerate(lens):
        for g in range(Hkv):
            w = [float(before[1][tables[i][t // bs], g, t % bs]) for t in range(L)]
            src = kept_positions(w, budget, sink, recent)
            kept[i, g, :len(src)] = src
            for j, t in enumerate(src):
                sb, db = tables[i][t // bs], dst[i][j // bs]
                for p, old in zip(pools, before[0]):
                    p[db, j % bs, g] = old[sb, t % bs, g]
                weights[db, g, j % bs] = before[1][sb, g, t % bs]
    return pools, weights, np.minimum(lens, budget).astype(np.int32), kept
