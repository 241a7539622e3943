"""The distance score of the 4-bit decode, with tolerances from each sequence's own logits."""

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


def run(N, Hq, H, L, C, E, Ev, lens, *, sink=False, mask="none", window=0, keep=0, seed=0):
    rng = np.random.default_rng(seed)
    cpu, k, v = ku.random_cache(rng, N, H, C, E, Ev)
    q = ku.bf16(rng.standard_normal((N, Hq, L, E)))
    s = rng.standard_normal(Hq).astype(np.float32) if sink else None
    out, lse = attn.attn_decode_kv4(q.cuda(), attn.KV4Cache(*(t.cuda() for t in cpu)), scale=E ** -0.5, length=max(lens),
                                    kv_len=torch.tensor(lens, dtype=torch.int32, device="cuda"), mode="rbf",
                                    sink=None if s is None else torch.from_numpy(s).cuda(), mask_kind=mask, window=window,
                                    keep_first=keep if mask == "streaming" else 0)
    ref = orc4.attention(ku.f64(q), k, v, lens, scale=E ** -0.5, mode="rbf", sink=None if s is None else s.astype(np.float64),
                         mask_kind=mask, window=window, keep=keep)
    ku.compare(out, lse, *ref, v_most=float(np.abs(v).max()), scale_of_logits=logit_size(ku.f64(q), k, lens, E ** -0.5, "rbf"))


@pytest.mark.parametrize("mask,window,keep", [("none", 0, 0), ("causal", 0, 0), ("window", 1, 0), ("window", 100, 0),
                                             ("window", 2**31 - 1, 0), ("streaming", 1, 1), ("streaming", 100, 4),
                                             ("streaming", 64, 65), ("streaming", 130, 500), ("streaming", 7, 2**31 - 1)])
@pytest.mark.parametrize("sink", [False, True])
def test_ragged_lengths(mask, window, keep, sink):
    lens = [0, 1, 2, 5, 16, 63, 64, 65, 200, 511, 512]
    run(len(lens), 8, 4, 3, 512, 64, 64, lens, mask=mask, window=window, keep=keep, sink=sink, seed=window % 97 + keep % 89)


@pytest.mark.parametrize("E,Ev", [(64, 64), (128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("S", [1, 2, 15, 16, 17, 63, 64, 65, 127, 300, 777])
def test_lengths(S, E, Ev):
    run(2, 6, 2, 1, -(-S // 16) * 16, E, Ev, [S, max(1, S // 2)], sink=S % 2 == 0, seed=S)


@pytest.mark.parametrize("E,Ev", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("group,L", [(4, 1), (9, 1), (4, 4)])
def test_head_widths(group, L, E, Ev):
    run(2, 2 * group, 2, L, 1296, E, Ev, [1290, 530], mask="streaming", window=600, keep=130, sink=True, seed=E + Ev + L)
