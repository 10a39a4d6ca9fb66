"""Oracle of the low-rank adapters: out[t] = base[t] + scale_a B_a (A_a x[t]), float64 NumPy, row by row."""

import numpy as np


def forward(x, ids, adapters, base=None, N=None):
    """adapters: {slot: (A [rank, K], B [N, rank], scale)}; an id that is not in it adds nothing."""
    x = np.asarray(x, dtype=np.float64)
    out = np.zeros((x.shape[0], N)) if base is None else np.array(base, dtype=np.float64)
    for t, a in enumerate(ids):
        if int(a) in adapters:
            A, B, scale = adapters[int(a)]
            out[t] += scale * (np.asarray(B, dtype=np.float64) @ (np.asarray(A, dtype=np.float64) @ x[t]))
    return out
