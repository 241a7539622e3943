"""Inputs and comparisons shared by the tests of the 4-bit cache."""

from __future__ import annotations

import numpy as np
import torch

from oracle import kv4 as orc4

# Tolerances of the decode, from the roundings between the cache's exact values and the output:
#   out  one rounding of the result to bf16 (at most 2^-9 + of the value: half a step is 2^-8 relative to
#        the power of two below it) and one of each probability to fp16 (2^-11 of each term, so at most 2^-11
#        of sum p|v| / sum p <= max|v|); 2^x, log2 and fp32 sums stay below 2^-18.
#   lse  fp32: 2^x to 2^-22 relative, the sum and the logits to 2^-22 of their sizes.
REL_OUT = 2.0 ** -8
P_ROUND = 2.0 ** -11 + 2.0 ** -18


def bf16(x) -> torch.Tensor:
    return torch.as_tensor(np.asarray(x, dtype=np.float32)).to(torch.bfloat16)


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def random_rows(rng, shape, dtype=torch.bfloat16):
    """Normal rows whose dimensions have different sizes."""
    x = rng.standard_normal(shape) * np.exp(0.7 * rng.standard_normal(shape[-1]))
    return torch.as_tensor(x.astype(np.float32)).to(dtype)


def random_cache(rng, N, H, C, E, Ev):
    """(cache tensors on the CPU, k values, v values): whole random rows through the oracle's rounding."""
    k, v = f64(random_rows(rng, (N, H, C, E))), f64(random_rows(rng, (N, H, C, Ev)))
    kc, ks = orc4.quantise(k)
    vc, vs = orc4.quantise(v)
    cache = tuple(torch.from_numpy(a) for a in (kc, ks, vc, vs))
    return cache, orc4.dequantise(kc, ks), orc4.dequantise(vc, vs)


def compare(out, lse, ref_out, ref_lse, v_most: float, scale_of_logits: float = 1.0, what=""):
    """v_most: the largest |v|; scale_of_logits: the largest sum |q_e k_e| * scale, whose fp32 roundings the lse has."""
    out, lse = f64(out), f64(lse)
    dead = ~np.isfinite(ref_lse)
    assert np.array_equal(~np.isfinite(lse), dead), f"{what}: rows without a key differ"
    assert np.all(lse[dead] == -np.inf) and np.all(out[dead] == 0.0), f"{what}: a row without a key"
    live = ~dead
    lse_tol = 2.0 ** -20 * (8 + np.abs(ref_lse[live]) + scale_of_logits)
    # an error d of the logits changes the probabilities by a factor up to e^(2 d)
    tol = REL_OUT * np.abs(ref_out) + (P_ROUND + 2.0 ** -18 * (4 + scale_of_logits)) * v_most
    err = np.abs(out - ref_out)
    assert np.all(err <= tol), f"{what}: out off by {err.max():.3e}, {(err / tol).max():.2f} of the tolerance"
    lerr = np.abs(lse[live] - ref_lse[live])
    assert np.all(lerr <= lse_tol), f"{what}: lse off by {lerr.max():.3e}, {(lerr / lse_tol).max():.2f} of the tolerance"
