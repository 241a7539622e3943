"""The 4-bit decode's tolerances against planted mistakes (on the CPU): with the logits' size taken per sequence, a window
that is off by one, a missing norm term of the distance score, a dropped key and a wrong sink are all outside of them."""

import numpy as np
import pytest
import torch

from oracle import kv4 as orc4

import kv4_util as ku
from kv4_bounds import logit_size

LENS = [0, 1, 2, 5, 16, 63, 64, 65, 200, 511, 512]
SCALE = 64 ** -0.5


def inputs(seed):
    rng = np.random.default_rng(seed)
    _, k, v = ku.random_cache(rng, len(LENS), 4, 512, 64, 64)
    return ku.f64(ku.bf16(rng.standard_normal((len(LENS), 8, 3, 64)))), k, v, rng.standard_normal(8)


def as_outputs(out, lse):
    return torch.from_numpy(out).bfloat16(), torch.from_numpy(lse).float()


@pytest.mark.parametrize("mode", ["dot", "rbf"])
@pytest.mark.parametrize("mask,window,keep", [("none", 0, 0), ("causal", 0, 0), ("window", 100, 0), ("streaming", 100, 4)])
def test_mistakes_are_outside_of_the_tolerances(mask, window, keep, mode):
    q, k, v, sink = inputs(window + keep)
    kw = dict(scale=SCALE, mode=mode, mask_kind=mask, window=window, keep=keep)
    ref = orc4.attention(q, k, v, LENS, sink=sink, **kw)
    size = logit_size(q, k, LENS, SCALE, mode)
    assert size < 120  # not doubled from sequence to sequence

    def compare(got):
        ku.compare(*as_outputs(*got), *ref, v_most=float(np.abs(v).max()), scale_of_logits=size)

    compare(ref)
    wrong = {"sink": orc4.attention(q, k, v, LENS, sink=np.roll(sink, 1), **kw),
             "last key": orc4.attention(q, k, v, [max(0, n - 1) for n in LENS], sink=sink, **kw),
             "value rows": orc4.attention(q, k, np.roll(v, 1, 2), LENS, sink=sink, **kw)}
    if window:
        wrong["window"] = orc4.attention(q, k, v, LENS, sink=sink, **(kw | dict(window=window + 1)))
        wrong["window, narrower"] = orc4.attention(q, k, v, LENS, sink=sink, **(kw | dict(window=window - 1)))
    if keep:
        wrong["kept keys"] = orc4.attention(q, k, v, LENS, sink=sink, **(kw | dict(keep=keep + 1)))
    if mode == "rbf":
        wrong["norms"] = orc4.attention(q, k, v, LENS, sink=sink, **(kw | dict(mode="dot", scale=2 * SCALE)))
    for name, got in wrong.items():
        with pytest.raises(AssertionError):
            compare(got)
            pytest.fail(f"{name}: not noticed", pytrace=False)
        if name in ("sink", "value rows", "window", "kept keys", "norms"):  # by the output alone
            with pytest.raises(AssertionError):
                compare((got[0], ref[1]))
