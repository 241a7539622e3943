"""The size of the 4-bit decode's logits, from which its tolerances follow."""

from __future__ import annotations

import numpy as np


def logit_size(q, k, lens, scale: float, mode: str) -> float:
    """The largest sum of the products' magnitudes in any logit: sum |q_e k_e| scale, and for the distance score twice
    that and ||k||^2 scale.  q (N, Hq, L, E), k (N, H, C, E), float64; sequence n has lens[n] keys."""
    group = q.shape[1] // k.shape[1]
    most = 0.0
    for n, length in enumerate(lens):
        if length < 1:
            continue
        kk = np.repeat(k[n, :, :length], group, 0)
        size = scale * np.einsum("hle,hse->hls", np.abs(q[n]), np.abs(kk))
        if mode == "rbf":
            size = 2 * size + scale * (kk * kk).sum(-1)[:, None]
        most = max(most, float(size.max()))
    return most
