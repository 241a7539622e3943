"""Scale bytes outside the 4-bit cache's format (227 to 254): what they stand for is not defined, but they stay where
they are: rows that no query sees or no call asks for may hold them."""

import numpy as np
import pytest
import torch

import attention_tiled_attn_b200 as attn
from oracle import kv4 as orc4

import kv4_util as ku
from kv4_bounds import logit_size

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda_ready():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from attention_tiled_attn_b200 import build as b
    b.build()
    yield
    assert attn.device_status() == 0


@pytest.mark.parametrize("mode", ["dot", "rbf"])
@pytest.mark.parametrize("E,Ev,group,L", [(128, 128, 4, 1), (64, 64, 2, 4), (64, 128, 3, 5)])
@pytest.mark.parametrize("mask,window,keep", [("none", 0, 0), ("window", 75, 0), ("streaming", 75, 20)])
def test_hidden_rows_may_hold_any_bytes(mask, window, keep, E, Ev, group, L, mode):
    rng = np.random.default_rng(E + Ev + L)
    H, C, lens = 2, 400, [333, 200, 7]
    cpu, k, v = ku.random_cache(rng, len(lens), H, C, E, Ev)
    for n, length in enumerate(lens):
        j = np.arange(C)
        seen = j < length
        if mask != "none":  # by some row: the first row's window starts at length - L - window + 1
            seen &= (j > length - L - window) | (j < keep)
        hidden = torch.from_numpy(np.flatnonzero(~seen))
        for scales in (cpu[1], cpu[3]):
            w = scales.shape[-1]
            scales[n][:, hidden] = torch.from_numpy(rng.integers(227, 256, (H, len(hidden), w)).astype(np.uint8))
    q = ku.bf16(rng.standard_normal((len(lens), group * H, L, E)))
    cache = attn.KV4Cache(*(t.cuda() for t in cpu))
    scale = 0.5 * E ** -0.5
    out, lse = attn.attn_decode_kv4(q.cuda(), cache, scale=scale, length=max(lens), kv_len=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                    mode=mode, mask_kind=mask, window=window, keep_first=keep)
    ref, ref_lse = orc4.attention(ku.f64(q), k, v, lens, scale=scale, mode=mode, mask_kind=mask, window=window, keep=keep)
    ku.compare(out, lse, ref, ref_lse, v_most=float(np.abs(v).max()),
               scale_of_logits=logit_size(ku.f64(q), k, lens, scale, mode))


@pytest.mark.parametrize("which", ["k", "v"])
def test_a_row_that_does_not_see_the_key_is_untouched(which):
    """Of four query rows under the causal mask, only those at or after the key may differ."""
    rng = np.random.default_rng(9)
    S, L = 150, 4
    cpu, k, v = ku.random_cache(rng, 1, 1, 160, 128, 128)
    scales = cpu[1] if which == "k" else cpu[3]
    scales[0, 0, S - 2] = torch.arange(247, 255, dtype=torch.uint8)  # seen by the last two rows
    q = ku.bf16(rng.standard_normal((1, 2, L, 128)))
    out, lse = attn.attn_decode_kv4(q.cuda(), attn.KV4Cache(*(t.cuda() for t in cpu)), scale=0.09, length=S, mask_kind="causal")
    ref, ref_lse = orc4.attention(ku.f64(q), k, v, [S], scale=0.09, mask_kind="causal")
    first = slice(0, L - 2)
    ku.compare(out[:, :, first], lse[:, :, first], ref[:, :, first], ref_lse[:, :, first], v_most=float(np.abs(v).max()), scale_of_logits=logit_size(ku.f64(q), k, [S], 0.09, "dot"))


def test_reading_other_rows():
    rng = np.random.default_rng(10)
    cpu, k, v = ku.random_cache(rng, 2, 2, 64, 64, 128)
    for scales in (cpu[1], cpu[3]):
        scales[:, :, :20] = 250
        scales[:, :, 50:] = 228
    kb, vb = attn.attn_kv4_read(attn.KV4Cache(*(t.cuda() for t in cpu)), 40, start=20, kv_len=torch.tensor([50, 33], dtype=torch.int32, device="cuda"))
    for got, want in ((kb, k), (vb, v)):
        for n, end in enumerate((50, 33)):
            assert np.array_equal(ku.f64(got[n, :, :end - 20]), want[n, :, 20:end]) and not got[n, :, end - 20:].any()
