"""Low-rank adapters beside a product, in float64 numpy: y[b] += scaling[a] B_a (A_a x[b])."""

from __future__ import annotations

import numpy as np


def lora_delta(x, a, b, scaling, ids) -> np.ndarray:
    """float64 [rows, out]; rows whose id is outside the adapters get zeros."""
    x, a, b = (np.asarray(t).astype(np.float64) for t in (x, a, b))
    out = np.zeros((x.shape[0], b.shape[1]))
    for i, n in enumerate(ids):
        if 0 <= n < a.shape[0]:
            out[i] = float(scaling[n]) * (b[n] @ (a[n] @ x[i]))
    return out
