"""Oracle of the row dispatch, the combine and their gradients: float64 NumPy, slot by slot.

A slot is s = t * topk + j. Expert e keeps its first min(n_e, capacity) slots (capacity 0: all) in
ascending order; its rows start at a multiple of align and are padded to one.
"""

import numpy as np


def row_count(T, topk, E, align, capacity):
    """Rows of the sorted buffer for T tokens, whatever their routes."""
    S = T * topk
    R = S + min(E, S) * (align - 1)
    if capacity > 0:
        R = min(R, E * (-(-capacity // align) * align))
    return R


def row_maps(ids, E, align=1, capacity=0):
    """ids [T, topk] -> row_slot [R], slot_row [T, topk], row_offsets [E + 1]."""
    ids = np.asarray(ids)
    T, k = ids.shape
    R = row_count(T, k, E, align, capacity)
    row_slot = np.full(R, -1, dtype=np.int64)
    slot_row = np.full(T * k, -1, dtype=np.int64)
    offsets = np.zeros(E + 1, dtype=np.int64)
    start = 0
    for e in range(E):
        mine = [s for s in range(T * k) if ids[s // k, s % k] == e] if T * k < 4096 else np.flatnonzero(ids.reshape(-1) == e)
        mine = list(mine)[:capacity] if capacity else list(mine)
        for i, s in enumerate(mine):
            row_slot[start + i] = s
            slot_row[s] = start + i
        start += -(-len(mine) // align) * align
        offsets[e + 1] = start
    return row_slot, slot_row.reshape(T, k), offsets


def dispatch(x, row_slot, topk, gates=None):
    """rows[r] = (gates[s]) x[s // topk], zero where there is no slot."""
    x = np.asarray(x, dtype=np.float64)
    rows = np.zeros((len(row_slot), x.shape[1]))
    for r, s in enumerate(row_slot):
        if s >= 0:
            g = 1.0 if gates is None else float(np.asarray(gates).reshape(-1)[s])
            rows[r] = g * x[s // topk]
    return rows


def combine(rows, slot_row, gates=None):
    """out[t] = sum_j (gates[t, j]) rows[slot_row[t, j]]."""
    rows = np.asarray(rows, dtype=np.float64)
    T, k = slot_row.shape
    out = np.zeros((T, rows.shape[1]))
    for t in range(T):
        for j in range(k):
            r = slot_row[t, j]
            if r >= 0:
                out[t] += (1.0 if gates is None else float(gates[t, j])) * rows[r]
    return out


def gate_grads(rows, v, slot_row):
    """<rows[slot_row[t, j]], v[t]> and the same with absolute values (an error bound's scale); 0 for dropped slots."""
    T, k = slot_row.shape
    d, a = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            if slot_row[t, j] >= 0:
                p = np.asarray(rows[slot_row[t, j]], dtype=np.float64) * np.asarray(v[t], dtype=np.float64)
                d[t, j], a[t, j] = p.sum(), np.abs(p).sum()
    return d, a


def logit_grads(dgates, gates, ids, E):
    """The gradient of the router logits through gates = softmax over the chosen logits."""
    T, k = ids.shape
    out = np.zeros((T, E))
    for t in range(T):
        for j in range(k):
            out[t, ids[t, j]] = gates[t, j] * (dgates[t, j] - float(np.dot(gates[t], dgates[t])))
    return out
